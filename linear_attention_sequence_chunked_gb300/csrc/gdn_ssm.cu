// Selective state space scan: forward, and the single-token step for decode.
// The layout is described in gdn_ssm_common.cuh; gdn_ssm_bwd.cu holds the
// reverse mode.
#include <algorithm>
#include <cmath>

#include "gdn_ssm_common.cuh"

namespace gdn {

namespace {

using namespace ssm;

// A warp's tiles: what is on its way from global memory, and B and C as fp32.
template <typename T, int N, bool kOut>
struct alignas(16) FwdStage {
    static constexpr int CH = Lanes<N>::CH;
    T u[kTile][CH], dt[kTile][CH];
    T B[kTile][N];
    T z[kOut ? kTile : 0][CH];
    T C[kOut ? kTile : 0][N];
};
template <typename T, int N, bool kOut>
struct alignas(16) FwdShared {
    FwdStage<T, N, kOut> stage[kStages];
    float B[kTile][N];
    float C[kOut ? kTile : 0][N];
    // dt and x = dt u, where several lanes share a channel
    float2 dx[Lanes<N>::LPC > 1 ? kTile : 0][Lanes<N>::CH];
};

// kOut: the whole forward.  Without it, only the segment's end state from a
// zero start and the sum of its dt (the first pass of a split scan).  Twelve
// warps per SM of 168 registers: 4 x 4096 x 2048 took 275 us, sixteen of 128
// registers 300, twenty of 96 329.
template <typename T, int N, bool kOut, int PB>
__global__ void __launch_bounds__(32 * kWarps, 3) ssm_fwd_kernel(const SsmArgs p, int blocks) {
    using L = Lanes<N>;
    constexpr int LPC = L::LPC, CH = L::CH, NL = L::NL;
    extern __shared__ __align__(16) unsigned char smem[];
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    FwdShared<T, N, kOut>& sm = reinterpret_cast<FwdShared<T, N, kOut>*>(smem)[warp];
    const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
    const int nblk = blocks * p.G;
    if (unit >= p.slots * nblk) return;
    Place w;
    if (!find_place<CH>(p, unit / nblk, static_cast<int>(unit % nblk), p.seg, blocks, w)) return;
    if (!kOut && w.last) return;  // nothing starts after it

    const int ch = lane / LPC, q = lane % LPC;
    const bool mine = ch < w.nd;
    const int d = w.d0 + (mine ? ch : 0);
    const long long so = (static_cast<long long>(w.n) * p.D + d) * N;
    const long long co = (w.slot * p.D + d) * N;
    Two A2[NL / 2], h[NL / 2];
    load_states<N>(p.A + static_cast<long long>(d) * N, q, A2);
#pragma unroll
    for (int i = 0; i < NL / 2; ++i) {
        A2[i] = mul2(A2[i], two(kLog2e, kLog2e));
        h[i] = two(0.f, 0.f);
    }
    if (kOut && !w.first && p.joined) {
        load_states<N>(p.carry + co, q, h);
    } else if (kOut) {
        if (p.initial_state) load_states<N>(p.initial_state + so, q, h);
        for (int i = w.before; i > 0; --i) {  // h <- exp(A sum dt) h + own end state, segment by segment
            const long long sl = (w.slot - i) * p.D + d;
            const float s = p.carry_dt[sl];
            Two e[NL / 2];
            load_states<N>(p.carry + sl * N, q, e);
#pragma unroll
            for (int k = 0; k < NL / 2; ++k) h[k] = fma2(ex2_2(mul2(A2[k], two(s, s))), h[k], e[k]);
        }
    }
    const float dskip = kOut && p.D_skip ? p.D_skip[d] : 0.f;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    float sum = 0.f;
    const long long row0 = static_cast<long long>(w.b) * p.T + w.s0;
    const T* u = static_cast<const T*>(p.u) + row0 * p.u_stride + w.d0;
    const T* dt = static_cast<const T*>(p.dt) + row0 * p.dt_stride + w.d0;
    const T* z = kOut && p.z ? static_cast<const T*>(p.z) + row0 * p.z_stride + w.d0 : nullptr;
    const T* Bm = static_cast<const T*>(p.Bm) + row0 * p.B_stride + w.g * N;
    const T* Cm = static_cast<const T*>(p.Cm) + row0 * p.C_stride + w.g * N;
    T* out = kOut ? static_cast<T*>(p.out) + row0 * p.D + d : nullptr;
    const int len = w.s1 - w.s0;
    auto fetch = [&](int t) {  // the tile at token t, if there is one
        if (t < len) {
            FwdStage<T, N, kOut>& st = sm.stage[t / kTile % kStages];
            fill_tile<T, CH, PB>(&st.u[0][0], u + t * p.u_stride, p.u_stride, len - t, w.nd, lane);
            fill_tile<T, CH, PB>(&st.dt[0][0], dt + t * p.dt_stride, p.dt_stride, len - t, w.nd, lane);
            fill_tile<T, N, PB>(&st.B[0][0], Bm + t * p.B_stride, p.B_stride, len - t, N, lane);
            if constexpr (kOut) {
                if (z) fill_tile<T, CH, PB>(&st.z[0][0], z + t * p.z_stride, p.z_stride, len - t, w.nd, lane);
                fill_tile<T, N, PB>(&st.C[0][0], Cm + t * p.C_stride, p.C_stride, len - t, N, lane);
            }
        }
        commit_copies();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i * kTile);
    for (int t = 0; t < len; t += kTile) {
        if (kOut && p.saved && mine) store_states<N>(p.saved + ((w.chunk0 + t / kTile) * p.D + d) * N, q, h);
        wait_copies<kStages - 2>();
        __syncwarp();  // the tile is there, and everyone is through with the one before
        fetch(t + (kStages - 1) * kTile);
        const FwdStage<T, N, kOut>& st = sm.stage[t / kTile % kStages];
        widen_rows<T, N>(&st.B[0][0], &sm.B[0][0], lane);
        if constexpr (kOut) widen_rows<T, N>(&st.C[0][0], &sm.C[0][0], lane);
        const int left = len - t;
        Two d2[kTile], x2[kTile], y2[kTile];
        if constexpr (LPC == 1) {
            // two tokens at a time: dt and x = dt u of each, in both halves of a pair
#pragma unroll
            for (int k = 0; k < kTile; k += 2) {
                const Two u2 = two(to_f32(st.u[k][ch]), to_f32(st.u[k + 1][ch]));
                Two v = add2(two(to_f32(st.dt[k][ch]), to_f32(st.dt[k + 1][ch])), two(bias, bias));
                if (p.softplus) v = softplus_2(v);
                float v0, v1, x0, x1;
                if (left < kTile) {
                    split(v, v0, v1);
                    v = two(k < left ? v0 : 0.f, k + 1 < left ? v1 : 0.f);
                }
                split(v, v0, v1);
                split(mul2(v, u2), x0, x1);
                if (!kOut) sum += v0 + v1;
                d2[k] = two(v0, v0);
                d2[k + 1] = two(v1, v1);
                x2[k] = two(x0, x0);
                x2[k + 1] = two(x1, x1);
                if (kOut) {
                    split(mul2(u2, two(dskip, dskip)), x0, x1);
                    y2[k] = two(x0, 0.f);
                    y2[k + 1] = two(x1, 0.f);
                }
            }
        } else {
            // each of a channel's lanes forms its share of the tokens
#pragma unroll
            for (int i = 0; i < kTile / LPC; ++i) {
                const int k = i * LPC + q;
                float v = to_f32(st.dt[k][ch]) + bias;
                if (p.softplus) v = softplus(v);
                v = k < left ? v : 0.f;
                if (!kOut) sum += v;
                sm.dx[k][ch] = make_float2(v, v * to_f32(st.u[k][ch]));
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kTile; ++k) {
                const float2 v = sm.dx[k][ch];
                d2[k] = two(v.x, v.x);
                x2[k] = two(v.y, v.y);
                if (kOut) y2[k] = two(0.f, 0.f);
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < L::GR; ++j) {
#pragma unroll
            for (int k = 0; k < kTile; ++k) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&sm.B[k][4 * (j * LPC + q)]);
                h[2 * j] = fma2(ex2_2(mul2(d2[k], A2[2 * j])), h[2 * j], mul2(x2[k], Two{b.x}));
                h[2 * j + 1] = fma2(ex2_2(mul2(d2[k], A2[2 * j + 1])), h[2 * j + 1], mul2(x2[k], Two{b.y}));
                if constexpr (kOut) {
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&sm.C[k][4 * (j * LPC + q)]);
                    y2[k] = fma2(h[2 * j], Two{c.x}, y2[k]);
                    y2[k] = fma2(h[2 * j + 1], Two{c.y}, y2[k]);
                }
            }
        }
        if constexpr (kOut) {
            float y[kTile];
#pragma unroll
            for (int k = 0; k < kTile; ++k) {
                float hi;
                split(y2[k], y[k], hi);
                y[k] += hi;
            }
            if constexpr (LPC == 1) {
                if (z) {
#pragma unroll
                    for (int k = 0; k < kTile; k += 2) {
                        const Two z2 = two(to_f32(st.z[k][ch]), to_f32(st.z[k + 1][ch]));
                        split(mul2(two(y[k], y[k + 1]), mul2(z2, sigmoid_2(z2))), y[k], y[k + 1]);
                    }
                }
                if (mine) {
#pragma unroll
                    for (int k = 0; k < kTile; ++k)
                        if (k < left) out[k * static_cast<long long>(p.D)] = from_f32<T>(y[k]);
                }
            } else {
                share_sums<LPC>(y, q);
#pragma unroll
                for (int i = 0; i < kTile / LPC; ++i) {
                    const int k = i * LPC + q;
                    float v = fmaf(dskip, to_f32(st.u[k][ch]), y[i]);
                    if (z) {
                        const float zk = to_f32(st.z[k][ch]);
                        v *= zk * sigmoid(zk);
                    }
                    if (mine && k < left) out[k * static_cast<long long>(p.D)] = from_f32<T>(v);
                }
            }
            out += kTile * static_cast<long long>(p.D);
        }
    }
    if constexpr (!kOut) {
#pragma unroll
        for (int m = 1; m < LPC; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    }
    if (!mine) return;
    if constexpr (kOut) {
        if (w.last && p.final_state) store_states<N>(p.final_state + so, q, h);
    } else {
        store_states<N>(p.carry + co, q, h);
        if (q == 0) p.carry_dt[w.slot * p.D + d] = sum;
    }
}

// One token: lane q of a channel updates four of its states where they lie, for
// R batch rows whose states are all on their way together.  Bound by HBM: the
// state is read and written once (256 x 2048, N = 16: 16 us, 4.4 TB/s, in more
// than three waves of short threads, each with one round of loads and the stores
// that wait for it).
template <typename T, int N, int R, bool VEC>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmStepArgs p) {
    constexpr int LPC = N / 4;
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int q = static_cast<int>(id % LPC);
    const long long bd = id / LPC;
    const long long b0 = bd / p.D * R;
    const int d = static_cast<int>(bd % p.D);
    const int g = d / (p.D / p.G);
    float4 s[R];
    Raw<T, 4> br[R], cr[R];
    uint32_t ur[R], dr[R], zr[R];
    long long so[R];
    bool live[R], on[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        live[r] = on[r] = b0 + r < p.B;  // whole channels: a channel's lanes agree
        long long slot = b0 + r;
        if (p.slots && live[r]) {
            slot = p.slots[b0 + r];
            if (slot >= p.S) record_error(p.err, kErrBadSlot);
            on[r] = slot >= 0 && slot < p.S;
        }
        so[r] = (slot * p.D + d) * N + 4 * q;
        s[r] = on[r] ? *reinterpret_cast<const float4*>(p.state + so[r]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long b = on[r] ? b0 + r : 0;
        br[r] = load_raw<T, 4, VEC>(static_cast<const T*>(p.Bm) + b * p.B_stride + g * N + 4 * q, on[r] ? 4 : 0);
        cr[r] = load_raw<T, 4, VEC>(static_cast<const T*>(p.Cm) + b * p.C_stride + g * N + 4 * q, on[r] ? 4 : 0);
        ur[r] = load_one(static_cast<const T*>(p.u) + b * p.u_stride + d, on[r]);
        dr[r] = load_one(static_cast<const T*>(p.dt) + b * p.dt_stride + d, on[r]);
        zr[r] = p.z ? load_one(static_cast<const T*>(p.z) + b * p.z_stride + d, on[r]) : 0;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.A + static_cast<long long>(d) * N + 4 * q));
    const float bias = p.dt_bias ? __ldg(p.dt_bias + d) : 0.f, dskip = p.D_skip ? __ldg(p.D_skip + d) : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float bv[4], cv[4], h[4];
        unpack<T, 4>(br[r], bv);
        unpack<T, 4>(cr[r], cv);
        const float uu = one_f32<T>(ur[r]), z = one_f32<T>(zr[r]);
        float dt = one_f32<T>(dr[r]) + bias;
        if (p.softplus) dt = softplus(dt);
        const float x = dt * uu, d2 = dt * kLog2e;
        h[0] = fmaf(ex2(d2 * a.x), s[r].x, x * bv[0]);
        h[1] = fmaf(ex2(d2 * a.y), s[r].y, x * bv[1]);
        h[2] = fmaf(ex2(d2 * a.z), s[r].z, x * bv[2]);
        h[3] = fmaf(ex2(d2 * a.w), s[r].w, x * bv[3]);
        if (on[r]) *reinterpret_cast<float4*>(p.out_state + so[r]) = make_float4(h[0], h[1], h[2], h[3]);
        float y = fmaf(cv[0], h[0], cv[1] * h[1]) + fmaf(cv[2], h[2], cv[3] * h[3]);
#pragma unroll
        for (int m = LPC / 2; m > 0; m /= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (live[r] && q == 0) {
            y = fmaf(dskip, uu, y);
            if (p.z) y *= z * sigmoid(z);
            static_cast<T*>(p.out)[(b0 + r) * p.D + d] = from_f32<T>(on[r] ? y : 0.f);
        }
    }
}

// The states between the segments of a split scan: carry holds every segment's
// own contribution and receives the state it starts from (reverse: the
// gradient that reaches its end), four states per thread, segment after segment
// with the loads of 32 in flight.
__global__ void __launch_bounds__(256) ssm_compose_kernel(const SsmArgs p, int reverse) {
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long per = static_cast<long long>(p.D) * p.N / 4;
    if (id >= per * p.nseq) return;
    const int n = static_cast<int>(id / per);
    const long long i4 = id % per;  // float4 of a state
    const long long d = i4 * 4 / p.N;
    int b, t0, t1;
    if (!token_range(p.cu_seqlens, n, p.nseq, p.T, p.err, b, t0, t1)) return;
    const int segs = max(1, (t1 - t0 + p.seg - 1) / p.seg);
    const long long base = p.cu_seqlens ? static_cast<long long>(t0 / p.seg) + n
                                        : static_cast<long long>(n) * max(1, (p.T + p.seg - 1) / p.seg);
    const float* start = reverse ? p.d_final_state : p.initial_state;
    float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
    if (start) h = *reinterpret_cast<const float4*>(start + (n * per + i4) * 4);
    float4 a = *reinterpret_cast<const float4*>(p.A + i4 * 4);
    a.x *= kLog2e; a.y *= kLog2e; a.z *= kLog2e; a.w *= kLog2e;
    constexpr int U = 32;
    for (int c = 0; c < segs; c += U) {
        float4 e[U];
        float s[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int j = c + k;
            // the last segment in walking order contributes to nothing
            if (j < segs - 1) {
                const long long slot = base + (reverse ? segs - 1 - j : j);
                e[k] = *reinterpret_cast<const float4*>(p.carry + (slot * per + i4) * 4);
                s[k] = p.carry_dt[slot * p.D + d];
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int j = c + k;
            if (j < segs) {
                const long long slot = base + (reverse ? segs - 1 - j : j);
                *reinterpret_cast<float4*>(p.carry + (slot * per + i4) * 4) = h;
                if (j < segs - 1) {
                    h.x = fmaf(ex2(a.x * s[k]), h.x, e[k].x);
                    h.y = fmaf(ex2(a.y * s[k]), h.y, e[k].y);
                    h.z = fmaf(ex2(a.z * s[k]), h.z, e[k].z);
                    h.w = fmaf(ex2(a.w * s[k]), h.w, e[k].w);
                }
            }
        }
    }
}

cudaError_t launch_compose(const SsmArgs& a, bool reverse, cudaStream_t stream) {
    const long long threads = static_cast<long long>(a.nseq) * a.D * a.N / 4;
    ssm_compose_kernel<<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(a, reverse);
    return cudaGetLastError();
}

template <typename T, int N, int PB>
cudaError_t fwd_v(const SsmArgs& a, cudaStream_t stream) {
    const int blocks = (a.D / a.G + Lanes<N>::CH - 1) / Lanes<N>::CH;
    const long long units = a.slots * blocks * a.G;
    if (a.carry) {
        cudaError_t e = launch_warps<kWarps>(ssm_fwd_kernel<T, N, false, PB>, units, sizeof(FwdShared<T, N, false>), a, blocks, stream);
        if (e == cudaSuccess && a.joined) e = launch_compose(a, false, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_warps<kWarps>(ssm_fwd_kernel<T, N, true, PB>, units, sizeof(FwdShared<T, N, true>), a, blocks, stream);
}

template <typename T, int N>
cudaError_t fwd_n(const SsmArgs& a, cudaStream_t stream) {
    switch (scan_pieces<T, N>(a)) {
        case 16: return fwd_v<T, N, 16>(a, stream);
        case 4: return fwd_v<T, N, 4>(a, stream);
    }
    if constexpr (sizeof(T) == 2) return fwd_v<T, N, 0>(a, stream);
    return cudaErrorMisalignedAddress;  // fp32 is 4-byte aligned
}

template <typename T, int N, int R>
cudaError_t step_r(const SsmStepArgs& a, cudaStream_t stream) {
    const long long threads = (a.B + R - 1) / R * static_cast<long long>(a.D) * (N / 4);
    const unsigned grid = static_cast<unsigned>((threads + 255) / 256);
    auto ok = [](const void* p, long long stride) { return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && stride % 4 == 0; };
    if (ok(a.Bm, a.B_stride) && ok(a.Cm, a.C_stride))
        ssm_step_kernel<T, N, R, true><<<grid, 256, 0, stream>>>(a);
    else
        ssm_step_kernel<T, N, R, false><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}
// Two rows per thread once that still leaves the GPU full of threads (256 rows
// of 2048 channels, N = 16: 16 us of GPU time, one row 20 us, four 21 us).
template <typename T, int N>
cudaError_t step_n(const SsmStepArgs& a, cudaStream_t stream) {
    if (static_cast<long long>(a.B) * a.D * (N / 4) >= 152LL * 2048 * 2) return step_r<T, N, 2>(a, stream);
    return step_r<T, N, 1>(a, stream);
}

}  // namespace

#define GDN_SSM_N(fn, T)                          \
    switch (a.N) {                                \
        case 8: return fn<T, 8>(a, stream);       \
        case 16: return fn<T, 16>(a, stream);     \
        case 32: return fn<T, 32>(a, stream);     \
        case 64: return fn<T, 64>(a, stream);     \
        default: return fn<T, 128>(a, stream);    \
    }
#define GDN_SSM_DISPATCH(fn)              \
    if (a.dtype == 0) {                   \
        GDN_SSM_N(fn, uint16_t)           \
    }                                     \
    GDN_SSM_N(fn, float)

// Segments, none where the channels alone fill the GPU or the sequence is short.
// At least 16 tokens each, and sqrt(T) in the forward of one sequence, half that
// otherwise: what joins a segment to those before it grows with their number
// (16384 x 64: 49 us, 103 us with 16 tokens each; reverse mode 97 and 134 us; 256
// x 2048: 14 and 41 us, 20 and 70 us with 64 each).
// Forward: as many as give one wave of twelve warps per SM.  Splitting costs a
// second pass, 0.7 of the first, so it stays whole from 456 warps (512 warps: 266
// us whole, 269 us in segments of the same work) and below 64 tokens (1 x 64 x
// 2048: 9.8 us split, 10.8 whole; 32 tokens: 9.0 and 6.8), 96 of packed sequences,
// which are shorter.
// Reverse mode: a second pass costs 0.2, and the time of n warps is about that of
// their whole waves and f^0.4 of one for the part f of a wave that is left (512
// warps: 1479 us whole, 967 in three segments each, 834 in seven).  Whole below
// 24 tokens (32 tokens: 29 us split, 35 whole).  Packed sequences end inside a
// segment, half of one too many each (1 x 16384 x 2048, 12 sequences: 908 us so,
// 1065 without; the forward loses by it, 331 and 303 us).
int ssm_segment(int nseq, int T, int D, int G, int N, bool varlen, bool backward) {
    const int ch = N <= 16 ? 32 : 512 / N;
    const long long warps = static_cast<long long>(varlen ? 1 : nseq) * G * ((D / G + ch - 1) / ch);
    const int whole = 1 << 30;
    auto tokens = [&](long long segs) {  // of each of `segs` segments
        if (backward && varlen) segs = std::max(segs - nseq / 2, 1LL);  // sequences end inside one
        const long long least = static_cast<long long>((backward || varlen ? 0.5 : 1.) * std::sqrt(static_cast<double>(T)));
        const long long len = std::max((T + segs - 1) / segs, least);
        return std::max(16, static_cast<int>((len + kSsmChunk - 1) / kSsmChunk * kSsmChunk));
    };
    if (!backward) return warps >= 456 || T < (varlen ? 96 : 64) ? whole : tokens(152 * 12 / warps);
    if (T < 24) return whole;
    const double wave = 152. * (N <= 16 ? 12 : N == 32 ? 10 : N == 64 ? 8 : 6);  // by shared memory
    auto cost = [&](long long n) {  // per unit of work
        const double w = n * warps / wave, f = w - std::floor(w);
        return (std::floor(w) + std::pow(f, 0.4)) / w;
    };
    double best = cost(1);
    int seg = whole;
    for (int k = 1; k <= 4; ++k) {  // as many segments as k waves hold
        const long long n = static_cast<long long>(k * wave / warps);
        if (n < 2) continue;
        const int len = tokens(n);
        const long long segs = (T + len - 1) / len;
        const double c = 1.2 * cost(segs) + 0.0015 * segs;  // and what joins them
        if (segs > 1 && c < best) {
            best = c;
            seg = len;
        }
    }
    return seg;
}

cudaError_t launch_ssm_compose(const SsmArgs& a, bool reverse, cudaStream_t stream) {
    return launch_compose(a, reverse, stream);
}
cudaError_t launch_ssm_fwd(const SsmArgs& a, cudaStream_t stream) { GDN_SSM_DISPATCH(fwd_n) }
cudaError_t launch_ssm_step(const SsmStepArgs& a, cudaStream_t stream) { GDN_SSM_DISPATCH(step_n) }

}  // namespace gdn
