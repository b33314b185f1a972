// Group norm with an activation, channels last: the output norm of a gated
// delta rule layer ("Research Sprint Day 2 - Rooflines", GDN layer pseudocode:
// RMSNorm of the operator's output times SiLU of a gate) and of a state space
// mixer.  Per row and group of Cg channels, act one of none, SiLU, sigmoid:
//   x' = x act(gate) if the gate comes first, else x
//   m  = mean(x') if centered, else 0;   r = (mean((x' - m)^2) + eps)^-1/2
//   n  = r (x' - m),   v = n weight + bias
//   y  = v act(gate) (gate after), v (gate first), act(v) (no gate).
// Reverse mode, with dv the gradient of v and dn = dv weight:
//   dx' = r (dn - n mean(dn n) - [mean(dn) if centered]),
//   dweight = sum_rows dv n,   dbias = sum_rows dv,
// and the product and activation rules around it; n is recomputed.
// Bound by HBM (3 accesses per element gated forward, 5 backward): a team of
// lanes holds its group's row in registers, so every input is read once; the
// mean is subtracted before squaring.  In the forward a team takes a few rows
// with all their loads in flight.  In the reverse mode it keeps one group and
// walks rows, the next row's loads under way, so the weight gradients
// accumulate in its registers and leave as one partial row per team, summed
// afterwards in a fixed order.  Arithmetic runs on pairs of channels.
// Measured, bf16 and gated: forward 16384 rows of 16 groups of 128 35 us, 5.8
// TB/s; 64 rows 2.0 us, one access after another; gradients 16384 rows of one
// group of 2048 66 us, 5.1 TB/s.
#include "gdn.h"
#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

// act(x) of H pairs in place, and act'(x) into d: the kind is asked for once.
template <int H>
__device__ __forceinline__ void activate(Two (&x)[H], int kind) {
    if (kind == GDN_ACT_SILU) {
#pragma unroll
        for (int h = 0; h < H; ++h) x[h] = mul2(x[h], sigmoid_2(x[h]));
    } else if (kind == GDN_ACT_SIGMOID) {
#pragma unroll
        for (int h = 0; h < H; ++h) x[h] = sigmoid_2(x[h]);
    }
}
template <int H>
__device__ __forceinline__ void activate(Two (&x)[H], Two (&d)[H], int kind) {
    const Two one = two(1.f, 1.f), neg = two(-1.f, -1.f);
    if (kind == GDN_ACT_NONE) {
#pragma unroll
        for (int h = 0; h < H; ++h) d[h] = one;
    } else if (kind == GDN_ACT_SILU) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const Two s = sigmoid_2(x[h]), y = mul2(x[h], s);
            d[h] = fma2(y, fma2(s, neg, one), s);  // s + x s (1 - s)
            x[h] = y;
        }
    } else {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const Two s = sigmoid_2(x[h]);
            d[h] = mul2(s, fma2(s, neg, one));
            x[h] = s;
        }
    }
}

// Where the activation stands: on the result, on a gate after the norm, on a
// gate before it.
enum Mode { kPlain, kAfter, kFirst };

// A team: 16 or 32 lanes of a warp, or a whole block of 64 or more.  Its row of
// a group is V vectors of E elements per lane, vector i at lane + i LANES, held
// as H pairs of consecutive elements (of vectors 2 h and 2 h + 1 for E = 1).
template <typename T, int E, int LANES, int V>
struct Team {
    static constexpr int kBlock = LANES < 64 ? 128 : LANES;
    static constexpr int kTeams = kBlock / LANES;  // per block
    static constexpr int H = V * E / 2;
    int lane, nv;
    float* red;  // shared, 2 x kBlock / 32 floats, for teams of several warps

    __device__ __forceinline__ bool on(int i) const { return lane + i * LANES < nv; }
    template <typename S>
    __device__ __forceinline__ void load(const S* p, bool live, Raw<S, E> (&r)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i)
            r[i] = load_raw<S, E>(p + static_cast<long long>(lane + i * LANES) * E, live && on(i) ? E : 0);
    }
    template <typename S>
    __device__ __forceinline__ void pairs(const Raw<S, E> (&r)[V], Two (&x)[H]) const {
#pragma unroll
        for (int h = 0; h < H; ++h)
            x[h] = E == 1 ? two(r[2 * h % V].get(0), r[(2 * h + 1) % V].get(0)) : two(r[2 * h / E].get(2 * h % E), r[2 * h / E].get(2 * h % E + (E > 1)));
    }
    __device__ __forceinline__ void store(T* p, bool live, const Two (&x)[H]) const {
        float f[2 * H];
#pragma unroll
        for (int h = 0; h < H; ++h) split(x[h], f[2 * h], f[2 * h + 1]);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (live && on(i)) store_raw<T, E>(p + static_cast<long long>(lane + i * LANES) * E, pack<T, E>(f + i * E), E);
    }
    // a per-channel parameter, or `missing` everywhere
    __device__ __forceinline__ void param(const float* p, float missing, Two (&w)[H]) const {
        if (p) {
            Raw<float, E> r[V];
            load(p, true, r);
            pairs(r, w);
        } else {
#pragma unroll
            for (int h = 0; h < H; ++h) w[h] = two(missing, missing);
        }
    }
    // zero where the row has no element
    __device__ __forceinline__ void clip(Two (&x)[H]) const {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float lo = on(E == 1 ? 2 * h : 2 * h / E) ? 1.f : 0.f, hi = on(E == 1 ? 2 * h + 1 : 2 * h / E) ? 1.f : 0.f;
            x[h] = mul2(x[h], two(lo, hi));
        }
    }
    // sums over the team of both arguments
    __device__ __forceinline__ void sums(Two a, Two b, float& sa, float& sb) const {
        float lo, hi;
        split(a, lo, hi);
        sa = lo + hi;
        split(b, lo, hi);
        sb = lo + hi;
        constexpr int M = LANES < 32 ? LANES : 32;
#pragma unroll
        for (int m = M / 2; m > 0; m /= 2) {
            sa += __shfl_xor_sync(0xffffffffu, sa, m);
            sb += __shfl_xor_sync(0xffffffffu, sb, m);
        }
        if constexpr (LANES > 32) {
            constexpr int WARPS = LANES / 32;
            __syncthreads();  // the previous sums have been read
            if ((threadIdx.x & 31) == 0) {
                red[threadIdx.x >> 5] = sa;
                red[WARPS + (threadIdx.x >> 5)] = sb;
            }
            __syncthreads();
            sa = red[0];
            sb = red[WARPS];
#pragma unroll
            for (int i = 1; i < WARPS; ++i) {
                sa += red[i];
                sb += red[WARPS + i];
            }
        }
    }
    __device__ __forceinline__ float sum(Two a) const {
        float lo, hi;
        split(a, lo, hi);
        lo += hi;
        constexpr int M = LANES < 32 ? LANES : 32;
#pragma unroll
        for (int m = M / 2; m > 0; m /= 2) lo += __shfl_xor_sync(0xffffffffu, lo, m);
        if constexpr (LANES > 32) {
            __syncthreads();  // the previous sums have been read
            if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = lo;
            __syncthreads();
            lo = red[0];
#pragma unroll
            for (int i = 1; i < LANES / 32; ++i) lo += red[i];
        }
        return lo;
    }
    // x' -> x' - mean (where centered)
    __device__ __forceinline__ void center(Two (&x)[H], float inv) const {
        Two a = two(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < H; ++h) a = add2(a, x[h]);
        const float m = -sum(a) * inv;
#pragma unroll
        for (int h = 0; h < H; ++h) x[h] = add2(x[h], two(m, m));
        clip(x);
    }
};

// A team takes R rows of one group.
template <typename T, int E, int LANES, int V, int R, int M>
__global__ void __launch_bounds__(Team<T, E, LANES, V>::kBlock) norm_fwd_kernel(const NormArgs p) {
    using Tm = Team<T, E, LANES, V>;
    constexpr int H = Tm::H;
    __shared__ float red[LANES > 32 ? 2 * LANES / 32 : 1];
    const int size = p.C / p.groups;
    const Tm tm{static_cast<int>(threadIdx.x) % LANES, size / E, red};
    const long long unit = static_cast<long long>(blockIdx.x) * Tm::kTeams + threadIdx.x / LANES;
    const long long row0 = unit / p.groups * R;  // a team past the last row still meets the others' shuffles
    const int c0 = static_cast<int>(unit % p.groups) * size;
    Raw<T, E> xr[R][V], gr[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool live = row0 + r < p.rows;
        const long long row = live ? row0 + r : 0;
        tm.load(static_cast<const T*>(p.x) + row * p.x_stride + c0, live, xr[r]);
        if (M != kPlain) tm.load(static_cast<const T*>(p.gate) + row * p.gate_stride + c0, live, gr[r]);
    }
    Two w[H];
    tm.param(p.weight ? p.weight + c0 : nullptr, 1.f, w);
    const float inv = 1.f / size;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        Two x[H], g[H];
        tm.pairs(xr[r], x);
        if (M != kPlain) {
            tm.pairs(gr[r], g);
            activate(g, p.activation);
        }
        if (M == kFirst) {
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = mul2(x[h], g[h]);
        }
        if (p.center) tm.center(x, inv);
        Two a = two(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < H; ++h) a = fma2(x[h], x[h], a);
        const float rs = 1.f / sqrtf(fmaf(tm.sum(a), inv, p.eps));
        const Two r2 = two(rs, rs);
#pragma unroll
        for (int h = 0; h < H; ++h) x[h] = mul2(mul2(x[h], r2), w[h]);
        if (p.bias) {
            Two b[H];
            tm.param(p.bias + c0, 0.f, b);
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = add2(x[h], b[h]);
        }
        if (M == kPlain) activate(x, p.activation);
        if (M == kAfter) {
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = mul2(x[h], g[h]);
        }
        tm.store(static_cast<T*>(p.y) + (row0 + r) * p.C + c0, row0 + r < p.rows, x);
    }
}

// Threads per SM in the reverse mode: eight channels per lane keep to the 128
// registers of 512 threads, sixteen want 168 (16384 x 2048 in one group: 66 us
// with 384 threads, 111 us with 512).
template <int E, int LANES, int V>
constexpr int kBwdThreads = V * E > 8 && LANES <= 128 ? 384 : 512;

// Team `unit` keeps group unit % groups and takes rows unit / groups, + teams, ...
template <typename T, int E, int LANES, int V, int M>
__global__ void __launch_bounds__(Team<T, E, LANES, V>::kBlock, kBwdThreads<E, LANES, V> / Team<T, E, LANES, V>::kBlock) norm_bwd_kernel(const NormArgs p, int teams) {
    using Tm = Team<T, E, LANES, V>;
    constexpr int H = Tm::H;
    __shared__ float red[LANES > 32 ? 2 * LANES / 32 : 1];
    const int size = p.C / p.groups;
    const float inv = 1.f / size;
    const Tm tm{static_cast<int>(threadIdx.x) % LANES, size / E, red};
    const long long unit = static_cast<long long>(blockIdx.x) * Tm::kTeams + threadIdx.x / LANES;
    const bool live = unit < static_cast<long long>(teams) * p.groups;
    const int team = live ? static_cast<int>(unit / p.groups) : 0;
    const int c0 = live ? static_cast<int>(unit % p.groups) * size : 0;
    const Two zero = two(0.f, 0.f);
    Two w[H], dw[H], db[H];
    tm.param(p.weight ? p.weight + c0 : nullptr, 1.f, w);
#pragma unroll
    for (int h = 0; h < H; ++h) dw[h] = db[h] = zero;
    Raw<T, E> xr[V], gr[V], dr[V];
    auto load = [&](long long row) {
        const bool on = live && row < p.rows;
        if (!on) row = 0;
        tm.load(static_cast<const T*>(p.x) + row * p.x_stride + c0, on, xr);
        tm.load(static_cast<const T*>(p.d_out) + row * p.C + c0, on, dr);
        if (M != kPlain) tm.load(static_cast<const T*>(p.gate) + row * p.gate_stride + c0, on, gr);
    };
    load(team);
    const long long steps = (p.rows + teams - 1) / teams;
    for (long long s = 0; s < steps; ++s) {
        const long long row = team + s * teams;
        const bool on = live && row < p.rows;  // a row that is not there is all zeros
        Two x[H], ga[H], gd[H], dy[H], n[H];
        tm.pairs(xr, x);
        tm.pairs(dr, dy);
        if (M != kPlain) tm.pairs(gr, ga);
        load(row + teams);
        if (M != kPlain) activate(ga, gd, p.activation);
#pragma unroll
        for (int h = 0; h < H; ++h) n[h] = M == kFirst ? mul2(x[h], ga[h]) : x[h];
        if (p.center) tm.center(n, inv);
        // With a gate dv does not need the norm, and one exchange gives both sums.
        Two a = zero, c = zero;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            a = fma2(n[h], n[h], a);
            if (M == kAfter) {  // the gate's own gradient is dy act'(gate) v: v below
                gd[h] = mul2(dy[h], gd[h]);
                dy[h] = mul2(dy[h], ga[h]);
            }
            if (M != kPlain) c = fma2(mul2(dy[h], w[h]), n[h], c);
        }
        float ss, sn;
        tm.sums(a, c, ss, sn);
        const float rs = on ? 1.f / sqrtf(fmaf(ss, inv, p.eps)) : 0.f;
        const Two r2 = two(rs, rs);
        sn *= rs * inv;
#pragma unroll
        for (int h = 0; h < H; ++h) n[h] = mul2(n[h], r2);
        if (M != kFirst) {
            Two v[H];
#pragma unroll
            for (int h = 0; h < H; ++h) v[h] = mul2(n[h], w[h]);
            if (p.bias) {
                Two b[H];
                tm.param(p.bias + c0, 0.f, b);
#pragma unroll
                for (int h = 0; h < H; ++h) v[h] = add2(v[h], b[h]);
            }
            if (M == kAfter) {
#pragma unroll
                for (int h = 0; h < H; ++h) gd[h] = mul2(gd[h], v[h]);
            } else {
                activate(v, gd, p.activation);
                c = zero;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    dy[h] = mul2(dy[h], gd[h]);
                    c = fma2(mul2(dy[h], w[h]), n[h], c);
                }
                sn = tm.sum(c) * inv;
            }
        }
        Two m1 = zero;
        if (p.center) {
            c = zero;
#pragma unroll
            for (int h = 0; h < H; ++h) c = fma2(dy[h], w[h], c);
            const float s1 = -tm.sum(c) * inv;
            m1 = two(s1, s1);
        }
        const Two sn2 = two(-sn, -sn);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            dw[h] = fma2(dy[h], n[h], dw[h]);
            db[h] = add2(db[h], dy[h]);
            const Two d = mul2(r2, fma2(n[h], sn2, fma2(dy[h], w[h], m1)));
            if (M == kFirst) {
                gd[h] = mul2(mul2(d, x[h]), gd[h]);
                x[h] = mul2(d, ga[h]);
            } else {
                x[h] = d;
            }
        }
        tm.store(static_cast<T*>(p.dx) + row * p.C + c0, on, x);
        if (M != kPlain) tm.store(static_cast<T*>(p.dgate) + row * p.C + c0, on, gd);
    }
    if (!p.partial || !live) return;
    float* pw = p.partial + static_cast<long long>(team) * (p.bias ? 2 : 1) * p.C + c0;
    float fw[2 * H], fb[2 * H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        split(dw[h], fw[2 * h], fw[2 * h + 1]);
        split(db[h], fb[2 * h], fb[2 * h + 1]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (!tm.on(i)) continue;
        const int at = (tm.lane + i * LANES) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            pw[at + e] = fw[i * E + e];
            if (p.bias) pw[p.C + at + e] = fb[i * E + e];
        }
    }
}

template <typename T, int E, int LANES, int V, int R>
cudaError_t norm_fwd_r(const NormArgs& a, cudaStream_t stream) {
    using Tm = Team<T, E, LANES, V>;
    const long long units = (a.rows + R - 1) / R * a.groups;
    const unsigned grid = static_cast<unsigned>((units + Tm::kTeams - 1) / Tm::kTeams);
    if (!a.gate)
        norm_fwd_kernel<T, E, LANES, V, R, kPlain><<<grid, Tm::kBlock, 0, stream>>>(a);
    else if (a.gate_first)
        norm_fwd_kernel<T, E, LANES, V, R, kFirst><<<grid, Tm::kBlock, 0, stream>>>(a);
    else
        norm_fwd_kernel<T, E, LANES, V, R, kAfter><<<grid, Tm::kBlock, 0, stream>>>(a);
    return cudaGetLastError();
}
// Several rows per team once one row each gives the GPU more teams than it
// holds at a time; before that they would only leave SMs without work (16
// groups of 128: 16384 rows 33 us by four, 41 by one; 2048 rows 5.0 and 5.7; 256
// rows 3.1 and 2.5).
template <typename T, int E, int LANES, int V>
cudaError_t norm_fwd_v(const NormArgs& a, cudaStream_t stream) {
    constexpr int R = V == 1 && E > 1 ? 4 : 1;
    if (R > 1 && a.rows * a.groups * LANES >= 152LL * 2048) return norm_fwd_r<T, E, LANES, V, R>(a, stream);
    return norm_fwd_r<T, E, LANES, V, 1>(a, stream);
}
template <typename T, int E, int LANES, int V>
cudaError_t norm_bwd_v(const NormArgs& a, cudaStream_t stream) {
    using Tm = Team<T, E, LANES, V>;
    const int teams = norm_partial_rows(a.rows, a.C, a.groups, a.dtype);
    const long long units = static_cast<long long>(teams) * a.groups;
    const unsigned grid = static_cast<unsigned>((units + Tm::kTeams - 1) / Tm::kTeams);
    if (!a.gate)
        norm_bwd_kernel<T, E, LANES, V, kPlain><<<grid, Tm::kBlock, 0, stream>>>(a, teams);
    else if (a.gate_first)
        norm_bwd_kernel<T, E, LANES, V, kFirst><<<grid, Tm::kBlock, 0, stream>>>(a, teams);
    else
        norm_bwd_kernel<T, E, LANES, V, kAfter><<<grid, Tm::kBlock, 0, stream>>>(a, teams);
    return cudaGetLastError();
}

// Whether rows can be accessed E elements at a time.
template <typename T, int E>
bool rows_take(const NormArgs& a) {
    auto ok = [](const void* p, long long stride) { return reinterpret_cast<uintptr_t>(p) % (E * sizeof(T)) == 0 && stride % E == 0; };
    return (a.C / a.groups) % E == 0 && ok(a.x, a.x_stride) && (!a.gate || ok(a.gate, a.gate_stride));
}

// Lanes and registers per group: a half warp or a warp where the group fits
// its registers, else a block.  Rows that 16-byte accesses cannot take (odd
// sizes, strides or addresses) go 4 bytes or one element at a time,
// neighbouring lanes on neighbouring elements.  8192 x 4096 bf16 takes 40 us
// with 256 lanes forward (512: 65 us), 74 us with 512 lanes in reverse (256: 77
// to 115 us): L512 and V512.
#define GDN_NORM_SIZES(fn, T, L512, V512)                               \
    const int size = a.C / a.groups;                                    \
    constexpr int E = 16 / sizeof(T);                                   \
    if (rows_take<T, E>(a)) {                                           \
        const int nv = size / E;                                        \
        if (nv <= 16) return fn<T, E, 16, 1>(a, stream);                \
        if (nv <= 32) return fn<T, E, 32, 1>(a, stream);                \
        if (nv <= 64) return fn<T, E, 32, 2>(a, stream);                \
        if (nv <= 128) return fn<T, E, 128, 1>(a, stream);              \
        if (nv <= 256) return fn<T, E, 128, 2>(a, stream);              \
        if (nv <= 512) return fn<T, E, L512, V512>(a, stream);          \
        if (nv <= 1024) return fn<T, E, 512, 2>(a, stream);             \
        if constexpr (sizeof(T) == 4) return fn<T, E, 512, 4>(a, stream); \
    }                                                                   \
    if constexpr (sizeof(T) == 2) {                                     \
        if (rows_take<T, 2>(a)) {                                       \
            const int nv = size / 2;                                    \
            if (nv <= 128) return fn<T, 2, 32, 4>(a, stream);           \
            if (nv <= 256) return fn<T, 2, 32, 8>(a, stream);           \
            if (nv <= 512) return fn<T, 2, 128, 4>(a, stream);          \
            if (nv <= 2048) return fn<T, 2, 512, 4>(a, stream);         \
            return fn<T, 2, 512, 8>(a, stream);                         \
        }                                                               \
    }                                                                   \
    if (size <= 128) return fn<T, 1, 32, 4>(a, stream);                 \
    if (size <= 512) return fn<T, 1, 128, 4>(a, stream);                \
    if (size <= 1024) return fn<T, 1, 128, 8>(a, stream);               \
    if (size <= 4096) return fn<T, 1, 512, 8>(a, stream);               \
    return fn<T, 1, 512, 16>(a, stream)

template <typename T>
cudaError_t norm_fwd_t(const NormArgs& a, cudaStream_t stream) {
    GDN_NORM_SIZES(norm_fwd_v, T, 256, 2);
}
template <typename T>
cudaError_t norm_bwd_t(const NormArgs& a, cudaStream_t stream) {
    GDN_NORM_SIZES(norm_bwd_v, T, 512, 1);
}

}  // namespace

// Teams per group in the reverse mode, one partial row each: one wave of the
// threads that an SM holds at a time, few enough that the partial rows cost
// little beside the inputs.
int norm_partial_rows(long long rows, int C, int groups, int dtype) {
    const int nv = C / groups / (dtype == 0 ? 8 : 4);
    const int lanes = nv <= 16 ? 16 : nv <= 64 ? 32 : nv <= 256 ? 128 : 512;
    const bool wide = dtype == 0 && ((nv > 32 && nv <= 64) || (nv > 128 && nv <= 256));  // sixteen channels per lane
    long long teams = 152LL * (wide ? 384 : 512) / lanes / groups;
    if (teams < 1) teams = 1;
    return static_cast<int>(rows < teams ? rows : teams);
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream) {
    return a.dtype == 0 ? norm_fwd_t<uint16_t>(a, stream) : norm_fwd_t<float>(a, stream);
}
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t stream) {
    return a.dtype == 0 ? norm_bwd_t<uint16_t>(a, stream) : norm_bwd_t<float>(a, stream);
}

}  // namespace gdn
