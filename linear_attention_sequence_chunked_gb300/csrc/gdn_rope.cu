// Norm of every query's and key's head with the rotation by position in the
// same pass, and its reverse mode.
//
//   n = x (mean(x^2) + eps)^-1/2 weight;   pair (u, v) of n at position p and
//   frequency f:  (u cos(p f) - v sin(p f), v cos(p f) + u sin(p f))
//
// A head of d channels lies across d / 8 lanes, each with two pieces of four
// channels that hold both halves of its four pairs, so a row needs no exchange
// but its sum of squares, and a lane needs no angles but four.  Such a team of
// lanes takes a token, forms its angles and walks its heads; where tokens are
// few, several teams share a token's heads.  Each row is read once and written
// once: 4 x 4096 tokens of 20 heads of 128 bf16 take 36 us, 4.7 TB/s or 70 % of a
// copy, and the gradients of 8191 tokens of 12 heads of 64 fp32 18, 4.2 TB/s.  What
// bounds it is latency: 15 warps an SM (128 registers) use 53 % of the issue slots
// (126 instructions per two rows) and 39 % of HBM's rate.  Angles kept in shared
// memory for a block's teams took 43 us.
//
// The angle p f is formed in turns, in fixed point: f / 2 pi as a 64-bit
// fraction (24 bits of f times 64 bits of 1 / 2 pi), multiplied by the integer
// position modulo 2^64.  Whole turns drop out of the product by themselves and
// the fraction keeps 2^-33 turns at a position of 2^31, where a product in fp32
// would have lost every bit of it.
#include <algorithm>

#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kThreads = 256;

// f / 2 pi modulo 1, in units of 2^-64.
__device__ __forceinline__ unsigned long long turns_of(float f) {
    const uint32_t bits = __float_as_uint(f);
    const int exp = static_cast<int>((bits >> 23) & 255u);
    const unsigned long long mant = exp ? (bits & 0x7fffffu) | 0x800000u : 0;  // |f| = mant 2^(exp - 150)
    constexpr unsigned long long kInv2Pi = 0x28be60db9391054aULL;  // 2^64 / 2 pi
    const unsigned long long lo = mant * kInv2Pi, hi = __umul64hi(mant, kInv2Pi);
    const int shift = 150 - exp;  // the 128-bit product, this many places to the right
    unsigned long long r;
    if (shift >= 128)
        r = 0;
    else if (shift >= 64)
        r = hi >> (shift - 64);
    else if (shift > 0)
        r = (hi << (64 - shift)) | (lo >> shift);
    else
        r = shift > -64 ? lo << -shift : 0;
    return bits >> 31 ? 0 - r : r;
}

// cos and sin of an angle in units of 2^-64 turns.  For bf16 outputs, whose
// rounding is 2^-9 of them, by the hardware's functions on [-pi, pi] (an absolute
// error of about 2^-21, a third of the instructions).  For fp32 the nearest
// quarter turn, then the Taylor series on [-pi/4, pi/4] up to x^9 and x^10 (remainders below
// 2^-28).
template <bool FAST>
__device__ __forceinline__ float2 cos_sin(unsigned long long phase) {
    if constexpr (FAST) {
        const float x = static_cast<float>(static_cast<int>(phase >> 32)) * (6.283185307179586f * 2.3283064365386963e-10f);
        return make_float2(__cosf(x), __sinf(x));
    }
    const uint32_t q = static_cast<uint32_t>((phase + (1ull << 61)) >> 62);
    const long long rest = static_cast<long long>(phase - (static_cast<unsigned long long>(q) << 62));
    const float x = static_cast<float>(static_cast<int>(rest >> 30)) * (6.283185307179586f * 5.8207660913467407e-11f);
    const float x2 = x * x;
    float s = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(x2, s, 1.f / 120.f);
    s = fmaf(x2, s, -1.f / 6.f);
    s = fmaf(x2 * s, x, x);
    float c = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(x2, c, -1.f / 720.f);
    c = fmaf(x2, c, 1.f / 24.f);
    c = fmaf(x2, c, -0.5f);
    c = fmaf(x2, c, 1.f);
    const float cs = q & 1 ? s : c, sn = q & 1 ? c : s;
    return make_float2(q == 1 || q == 2 ? -cs : cs, q >= 2 ? -sn : sn);
}

__device__ __forceinline__ int position(const RopeArgs& p, long long tok) {
    if (p.positions) return p.positions[tok];
    if (p.cu_seqlens == nullptr) return static_cast<int>(tok % p.T);
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[mid] <= tok)
            lo = mid;
        else
            hi = mid - 1;
    }
    return static_cast<int>(tok - p.cu_seqlens[lo]);
}

// Where lane j's two pieces of four channels begin, and the pairs they hold
// (first: its first frequency, or -1 where the lane's channels do not turn).
struct Pieces {
    int c0, c1, first;
};
template <bool NEXT>
__device__ __forceinline__ Pieces pieces(int j, int pairs) {
    if (8 * j >= 2 * pairs) return Pieces{8 * j, 8 * j + 4, -1};
    return NEXT ? Pieces{8 * j, 8 * j + 4, 4 * j} : Pieces{4 * j, pairs + 4 * j, 4 * j};
}

template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = LANES / 2; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}
__device__ __forceinline__ Two same(float c) { return two(c, c); }
__device__ __forceinline__ float sum_2(Two a) {
    float x, y;
    split(a, x, y);
    return x + y;
}

// A lane's eight channels as pairs: u0 u1, u2 u3, v0 v1, v2 v3 of its four pairs
// (u, v) where the halves turn with each other; as they lie where neighbours do.
struct Eight {
    Two v[4];
};
template <typename T>
__device__ __forceinline__ Eight eight(const Raw<T, 4>& a, const Raw<T, 4>& b) {
    Eight r;
    unpack_2<T, 4>(a, r.v);
    unpack_2<T, 4>(b, r.v + 2);
    return r;
}

// What a lane holds through the kernel: its pieces and its frequencies.
template <int LANES, bool NEXT>
struct Lane {
    static constexpr int d = 8 * LANES, TEAMS = 32 / LANES;  // teams of a warp
    Pieces at;
    unsigned long long f[4];
    bool bad[4];
    float cosine[4], sine[4];
    __device__ __forceinline__ explicit Lane(const RopeArgs& p) {
        at = pieces<NEXT>(threadIdx.x % LANES, p.pairs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w = at.first >= 0 ? p.inv_freq[at.first + i] : 0.f;
            f[i] = turns_of(w);
            bad[i] = (__float_as_uint(w) & 0x7f800000u) == 0x7f800000u;
        }
    }
    template <bool FAST>
    __device__ __forceinline__ void angles(int pos) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = cos_sin<FAST>(static_cast<unsigned long long>(static_cast<long long>(pos)) * f[i]);
            cosine[i] = bad[i] ? __int_as_float(0x7fffffff) : v.x;
            sine[i] = bad[i] ? __int_as_float(0x7fffffff) : v.y;
        }
    }
    // by +angle, or by -angle
    template <bool BACK>
    __device__ __forceinline__ void turn(Eight& x) const {
        if (at.first < 0) return;
        if constexpr (NEXT) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float u, v;
                split(x.v[i], u, v);
                const float s = BACK ? -sine[i] : sine[i];
                x.v[i] = two(fmaf(u, cosine[i], -v * s), fmaf(v, cosine[i], u * s));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const Two c = two(cosine[2 * i], cosine[2 * i + 1]);
                const Two s = BACK ? two(-sine[2 * i], -sine[2 * i + 1]) : two(sine[2 * i], sine[2 * i + 1]);
                const Two u = x.v[i], v = x.v[2 + i];
                x.v[i] = fma2(u, c, mul2(mul2(v, same(-1.f)), s));
                x.v[2 + i] = fma2(v, c, mul2(u, s));
            }
        }
    }
    __device__ __forceinline__ Eight weight(const float* w) const {
        Eight r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            r.v[i] = w ? two(w[at.c0 + 2 * i], w[at.c0 + 2 * i + 1]) : same(1.f);
            r.v[2 + i] = w ? two(w[at.c1 + 2 * i], w[at.c1 + 2 * i + 1]) : same(1.f);
        }
        return r;
    }
};
template <typename T>
__device__ __forceinline__ void store_eight(T* y, const Pieces& at, const Eight& x) {
    store_raw<T, 4>(y + at.c0, pack_2<T, 4>(x.v), 4);
    store_raw<T, 4>(y + at.c1, pack_2<T, 4>(x.v + 2), 4);
}

// Rows that a lane works on together: their loads are in flight at once.
template <typename T>
constexpr int kRows = sizeof(T) == 2 ? 4 : 2;

template <typename T>
struct Batch {
    Raw<T, 4> a[kRows<T>], b[kRows<T>];
};
// The heads h0 + first, + share, ... of one token's q or k
template <bool VEC, typename T, int LANES, bool NEXT>
__device__ __forceinline__ void load_heads(Batch<T>& x, const Lane<LANES, NEXT>& ln, const T* src, int h0, int first, int heads, int share,
                                           bool on) {
#pragma unroll
    for (int u = 0; u < kRows<T>; ++u) {
        const int h = h0 + first + u * share, n = on && h < heads ? 4 : 0;
        x.a[u] = load_raw<T, 4, VEC>(src + h * (8 * LANES) + ln.at.c0, n);
        x.b[u] = load_raw<T, 4, VEC>(src + h * (8 * LANES) + ln.at.c1, n);
    }
}

// All of one token's q or k heads that are this team's; `next` holds the first of them.
template <typename T, int LANES, bool NEXT, bool VEC>
__device__ __forceinline__ void forward_heads(const Lane<LANES, NEXT>& ln, Batch<T>& next, const T* src, T* dst, int first, int heads,
                                              int share, bool on, float eps, const float* weight) {
    constexpr int d = 8 * LANES, R = kRows<T>;
    const Eight w = ln.weight(weight);
    for (int h0 = 0; h0 < heads; h0 += R * share) {  // as many turns for every team
        const Batch<T> now = next;
        if (h0 + R * share < heads) load_heads<VEC>(next, ln, src, h0 + R * share, first, heads, share, on);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (h0 + u * share >= heads) break;  // no team has a head left
            const int h = h0 + first + u * share;
            Eight x = eight<T>(now.a[u], now.b[u]);
            Two sq = mul2(x.v[0], x.v[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) sq = fma2(x.v[i], x.v[i], sq);
            const float rs = rsqrtf(row_sum<LANES>(sum_2(sq)) * (1.f / d) + eps);
#pragma unroll
            for (int i = 0; i < 4; ++i) x.v[i] = mul2(mul2(x.v[i], same(rs)), w.v[i]);
            ln.template turn<false>(x);
            if (on && h < heads) store_eight<T>(dst + h * d, ln.at, x);
        }
    }
}

template <typename T, int LANES, bool NEXT, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) rope_fwd_kernel(const RopeArgs p) {
    constexpr int d = 8 * LANES, TEAMS = 32 / LANES;
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    Lane<LANES, NEXT> ln(p);
    const long long units = p.tokens * p.share, warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
    const int team = threadIdx.x % 32 / LANES;
    for (long long w = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; w * TEAMS < units; w += warps) {
        const long long unit = w * TEAMS + team;
        const bool on = unit < units;
        const long long tok = on ? unit / p.share : 0;
        const int first = on ? static_cast<int>(unit % p.share) : 0;
        const T* q = static_cast<const T*>(p.q) + tok * p.q_stride;
        const T* k = static_cast<const T*>(p.k) + tok * p.k_stride;
        Batch<T> bq, bk;
        load_heads<VEC>(bq, ln, q, 0, first, p.H, p.share, on);
        load_heads<VEC>(bk, ln, k, 0, first, p.Hk, p.share, on);
        if (p.pairs > 0) ln.template angles<sizeof(T) == 2>(position(p, tok));
        forward_heads<T, LANES, NEXT, VEC>(ln, bq, q, static_cast<T*>(p.q_out) + tok * p.H * d, first, p.H, p.share, on, p.eps, p.q_weight);
        forward_heads<T, LANES, NEXT, VEC>(ln, bk, k, static_cast<T*>(p.k_out) + tok * p.Hk * d, first, p.Hk, p.share, on, p.eps,
                                           p.k_weight);
    }
}

// With g the output's gradient turned back and n = x r:
//   dx = r (g w - n mean(g w n)),  dweight = sum over rows of g n
// Each lane keeps its sums of dweight; the blocks' partial sums are added in
// order by a second kernel.
template <typename T, int LANES, bool NEXT, bool VEC>
__device__ __forceinline__ void backward_heads(const Lane<LANES, NEXT>& ln, const T* src, const T* grad, T* dst, int first, int heads,
                                               int share, bool on, float eps, const Eight& w, Eight& dw) {
    constexpr int d = 8 * LANES, R = 2;
    for (int h0 = 0; h0 < heads; h0 += R * share) {
        Raw<T, 4> a[R], b[R], ga[R], gb[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const int h = h0 + first + u * share, n = on && h < heads ? 4 : 0;
            a[u] = load_raw<T, 4, VEC>(src + h * d + ln.at.c0, n);
            b[u] = load_raw<T, 4, VEC>(src + h * d + ln.at.c1, n);
            ga[u] = load_raw<T, 4>(grad + h * d + ln.at.c0, n);
            gb[u] = load_raw<T, 4>(grad + h * d + ln.at.c1, n);
        }
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (h0 + u * share >= heads) break;
            const int h = h0 + first + u * share;
            const Eight x = eight<T>(a[u], b[u]);
            Eight g = eight<T>(ga[u], gb[u]);
            ln.template turn<true>(g);
            Eight gw;
            Two sq = mul2(x.v[0], x.v[0]);
            gw.v[0] = mul2(g.v[0], w.v[0]);
            Two dot = mul2(gw.v[0], x.v[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                gw.v[i] = mul2(g.v[i], w.v[i]);
                sq = fma2(x.v[i], x.v[i], sq);
                dot = fma2(gw.v[i], x.v[i], dot);
            }
            const float rs = rsqrtf(row_sum<LANES>(sum_2(sq)) * (1.f / d) + eps);
            const float mean = row_sum<LANES>(sum_2(dot)) * (rs * (1.f / d));
            if (on && h < heads) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const Two n = mul2(x.v[i], same(rs));
                    dw.v[i] = fma2(g.v[i], n, dw.v[i]);
                    gw.v[i] = mul2(same(rs), fma2(n, same(-mean), gw.v[i]));
                }
                store_eight<T>(dst + h * d, ln.at, gw);
            }
        }
    }
}

template <typename T, int LANES, bool NEXT, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) rope_bwd_kernel(const RopeArgs p) {
    constexpr int d = 8 * LANES, TEAMS = 32 / LANES;
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    Lane<LANES, NEXT> ln(p);
    const Eight wq = ln.weight(p.q_weight), wk = ln.weight(p.k_weight);
    Eight dq, dk;
#pragma unroll
    for (int i = 0; i < 4; ++i) dq.v[i] = dk.v[i] = same(0.f);
    const long long units = p.tokens * p.share, warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
    const int team = threadIdx.x % 32 / LANES;
    for (long long w = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; w * TEAMS < units; w += warps) {
        const long long unit = w * TEAMS + team;
        const bool on = unit < units;
        const long long tok = on ? unit / p.share : 0;
        const int first = on ? static_cast<int>(unit % p.share) : 0;
        if (p.pairs > 0) ln.template angles<sizeof(T) == 2>(position(p, tok));
        const long long oq = tok * p.H * d, ok = tok * p.Hk * d;
        backward_heads<T, LANES, NEXT, VEC>(ln, static_cast<const T*>(p.q) + tok * p.q_stride, static_cast<const T*>(p.dq_out) + oq,
                                            static_cast<T*>(p.dq) + oq, first, p.H, p.share, on, p.eps, wq, dq);
        backward_heads<T, LANES, NEXT, VEC>(ln, static_cast<const T*>(p.k) + tok * p.k_stride, static_cast<const T*>(p.dk_out) + ok,
                                            static_cast<T*>(p.dk) + ok, first, p.Hk, p.share, on, p.eps, wk, dk);
    }
    if (!p.partial) return;
    __shared__ float sum[kThreads][9];  // nine: no two lanes of a warp on one bank
#pragma unroll
    for (int key = 0; key < 2; ++key) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) split(key ? dk.v[i] : dq.v[i], sum[threadIdx.x][2 * i], sum[threadIdx.x][2 * i + 1]);
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += kThreads) {
            const int jj = c / 8, i = c % 8;
            float s = 0.f;
            for (int t = 0; t < kThreads / LANES; ++t) s += sum[t * LANES + jj][i];
            const Pieces q = pieces<NEXT>(jj, p.pairs);
            p.partial[(2ll * blockIdx.x + key) * d + (i < 4 ? q.c0 + i : q.c1 + i - 4)] = s;
        }
    }
}

template <typename T, int LANES, bool NEXT, bool VEC>
cudaError_t launch_one(const RopeArgs& a, bool backward, cudaStream_t stream) {
    if (backward)
        rope_bwd_kernel<T, LANES, NEXT, VEC><<<a.blocks, kThreads, 0, stream>>>(a);
    else
        rope_fwd_kernel<T, LANES, NEXT, VEC><<<a.blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}
template <typename T, int LANES>
cudaError_t launch_lanes(const RopeArgs& a, bool backward, cudaStream_t stream) {
    const auto off = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % (4 * sizeof(T)) != 0; };
    const bool vec = !off(a.q) && !off(a.k) && a.q_stride % 4 == 0 && a.k_stride % 4 == 0;
    if (vec) return a.interleaved ? launch_one<T, LANES, true, true>(a, backward, stream) : launch_one<T, LANES, false, true>(a, backward, stream);
    return a.interleaved ? launch_one<T, LANES, true, false>(a, backward, stream) : launch_one<T, LANES, false, false>(a, backward, stream);
}
template <typename T>
cudaError_t launch(const RopeArgs& a, bool backward, cudaStream_t stream) {
    switch (a.d) {
        case 32: return launch_lanes<T, 4>(a, backward, stream);
        case 64: return launch_lanes<T, 8>(a, backward, stream);
        case 128: return launch_lanes<T, 16>(a, backward, stream);
        case 256: return launch_lanes<T, 32>(a, backward, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// Teams that share a token's heads, each of which forms the token's angles: one,
// until that leaves lanes of the GPU idle (4 x 4096 tokens of 20 heads of 128: 35.5
// us, two teams 38.1, four 46.0).
int rope_share(long long tokens, int heads, int d) {
    const long long teams = 152ll * 2 * kThreads / (d / 8);
    int s = 1;
    while (2 * s <= heads && tokens * s * 2 <= teams) s *= 2;
    return s;
}
// No more blocks than are resident together: a team goes on to its next token.
long long rope_blocks(long long tokens, int heads, int d) {
    const long long per = kThreads / (d / 8), units = tokens * rope_share(tokens, heads, d);
    return std::min((units + per - 1) / per, 152ll * 2);
}

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch<float>(a, false, stream) : launch<uint16_t>(a, false, stream);
}
cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch<float>(a, true, stream) : launch<uint16_t>(a, true, stream);
}

}  // namespace gdn
