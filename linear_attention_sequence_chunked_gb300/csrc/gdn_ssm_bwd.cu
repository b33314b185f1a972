// Reverse mode of the selective state space scan (gdn_ssm_common.cuh has the
// forward's formulas and the layout).  With dy = d_out silu(z) and e_t the
// gradient of h_t,
//   e_t  = C_t dy_t + a_{t+1} e_{t+1},   a_t = exp(dt_t A)   (from d_final_state)
//   dC_t = sum_d dy_t h_t,   dB_t = sum_d e_t x_t,   dx_t = sum_n e_t B_t
//   q_t  = a_t e_t h_{t-1}:  ddt_t = u_t dx_t + sum_n A q_t,   dA = sum_t dt_t q_t
//   du_t = dt_t dx_t + D dy_t,   dD = sum_t dy_t u_t,   dz_t = d_out_t y_t silu'(z_t)
//   ddt_raw = ddt sigmoid(dt_raw + bias),   ddt_bias = sum_t ddt_raw.
// A warp walks its tokens from the last tile to the first.  Four states at a
// time it takes the state before the tile, which the forward kept, runs the
// tile forward once more with the decays and states in registers, then back.
// The eight sums over channels per token (dB and dC of four states) halve with
// each of the first three shuffles; a warp's sums for its 32 channels go out as
// partial rows, dA, dD and ddt_bias as one partial row per segment, and two
// small kernels add those up in a fixed order.  A long scan over few channels
// runs in segments: a pass that only carries the state gradient back, the
// composition, then this.  Bound by instruction issue: about 16 paired
// operations, 4 exponentials and 32 instructions of the sums over channels per
// token and four states.  Measured, 2 x 4096 x 2048 with N = 16: 434 us (the pass
// that carries 62, this one 344, the sums over blocks and segments 24).
#include "gdn_ssm_common.cuh"

namespace gdn {

namespace {

using namespace ssm;

// Sums of v[0..7] over the CH channels of a warp (lanes LPC apart): value i of
// channel lane ch is then the sum of v[i * min(CH, 8) + ch mod 8].
template <int LPC, int CH>
__device__ __forceinline__ void across_channels(float (&v)[8], int ch) {
#pragma unroll
    for (int m = 1; m < CH; m *= 2) {
        if (m < 8) {
            const bool hi = (ch & m) != 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < 4 / m) {
                    const float send = hi ? v[2 * i] : v[2 * i + 1];
                    const float keep = hi ? v[2 * i + 1] : v[2 * i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m * LPC);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m * LPC);
        }
    }
}

// A tile goes back in two halves: decays and states of four tokens fit the
// registers of twelve warps per SM, those of eight only those of eight warps.
constexpr int kHalf = kTile / 2;

// Warps per block: from N = 32 on shared memory holds fewer than twelve warps per
// SM, and more of them in smaller blocks (1 x 2048 x 1024, N = 32: 150 us by two
// warps, 189 by four; N = 128: 612 and 657, 646 by one).
template <int N>
constexpr int kBwdWarps = N >= 32 ? 2 : 4;

// kFull: the whole reverse mode.  Without it, only the state gradient that a
// segment sends to the one before it, from a zero one at its end, and the sum
// of its dt.

template <typename T, int N, bool kFull>
struct alignas(16) BwdStage {
    static constexpr int CH = Lanes<N>::CH;
    T dt[kTile][CH], z[kTile][CH], d_out[kTile][CH];
    T C[kTile][N];
    T u[kFull ? kTile : 0][CH];
    T B[kFull ? kTile : 0][N];
    float saved[kFull ? CH : 0][N];
};
template <typename T, int N, bool kFull>
struct alignas(16) BwdShared {
    static constexpr int GR = Lanes<N>::GR;
    BwdStage<T, N, kFull> stage[2];
    float C[kTile][N];
    float B[kFull ? kTile : 0][N];
    // a lane's own: A log2(e), the state gradient, the sum for dA
    float4 A2[GR][32], g[GR][32];
    float4 dA[kFull ? GR : 0][32];
    float4 mid[kFull ? GR : 0][32];  // its states in the middle of the tile
    float bc[kFull ? kHalf : 0][2 * N];
    float4 tok[Lanes<N>::LPC > 1 ? kTile : 0][Lanes<N>::CH];  // dt, x and dy of a token, where lanes share a channel
};

struct Four {
    Two lo, hi;
};
__device__ __forceinline__ Four get4(const float* p) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(p);
    return Four{Two{x.x}, Two{x.y}};
}
__device__ __forceinline__ Four get4(const float4& p) { return get4(&p.x); }
__device__ __forceinline__ void put4(float4& p, Four v) {
    *reinterpret_cast<ulonglong2*>(&p) = make_ulonglong2(v.lo.v, v.hi.v);
}
__device__ __forceinline__ Four mul4(Four a, Two b) { return Four{mul2(a.lo, b), mul2(a.hi, b)}; }
__device__ __forceinline__ Four mul4(Four a, Four b) { return Four{mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ Four fma4(Four a, Two b, Four c) { return Four{fma2(a.lo, b, c.lo), fma2(a.hi, b, c.hi)}; }
__device__ __forceinline__ Four fma4(Four a, Four b, Four c) { return Four{fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)}; }
__device__ __forceinline__ Two dot4(Four a, Four b, Two c) { return fma2(a.hi, b.hi, fma2(a.lo, b.lo, c)); }
__device__ __forceinline__ Four ex2_4(Four a) { return Four{ex2_2(a.lo), ex2_2(a.hi)}; }
// the sum of both halves
__device__ __forceinline__ float both(Two v) {
    float lo, hi;
    split(v, lo, hi);
    return lo + hi;
}

template <typename T, int N, bool kFull, int PB>
__global__ void __launch_bounds__(32 * kBwdWarps<N>, 12 / kBwdWarps<N>) ssm_bwd_kernel(const SsmArgs p, int blocks) {
    using L = Lanes<N>;
    constexpr int CH = L::CH, LPC = L::LPC, GR = L::GR;
    constexpr int M8 = CH < 8 ? CH : 8;
    extern __shared__ __align__(16) unsigned char smem[];
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    BwdShared<T, N, kFull>& sm = reinterpret_cast<BwdShared<T, N, kFull>*>(smem)[warp];
    const long long unit = static_cast<long long>(blockIdx.x) * kBwdWarps<N> + warp;
    const int nblk = blocks * p.G;
    if (unit >= p.slots * nblk) return;
    const long long slot = unit / nblk;
    const int block = static_cast<int>(unit % nblk);
    const int ch = lane / LPC, q = lane % LPC;
    Place w;
    const bool found = find_place<CH>(p, slot, block, p.seg, blocks, w);
    if (!kFull && (!found || w.first)) return;  // nothing comes before it
    if (!found) {  // its row of the parameters' partial sums is read all the same
        const int per = p.D / p.G, off = block % blocks * CH;
        if (kFull && ch < min(CH, per - off)) {
            const int d = block / blocks * per + off + ch;
            float* par = p.par_part + slot * ssm_par_stride(p.D, N);
            for (int j = 0; j < GR; ++j)
                *reinterpret_cast<float4*>(par + static_cast<long long>(d) * N + 4 * (j * LPC + q)) = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q == 0) par[static_cast<long long>(p.D) * N + d] = par[static_cast<long long>(p.D) * N + p.D + d] = 0.f;
        }
        return;
    }
    const bool mine = ch < w.nd;
    const int d = w.d0 + (mine ? ch : 0);
    const bool composed = kFull && p.carry && p.joined;
    const float* start = !kFull ? nullptr : composed ? p.carry + (slot * p.D + d) * N
                         : p.d_final_state ? p.d_final_state + (static_cast<long long>(w.n) * p.D + d) * N : nullptr;
#pragma unroll
    for (int j = 0; j < GR; ++j) {
        const int at = 4 * (j * LPC + q);
        float4 a = *reinterpret_cast<const float4*>(p.A + static_cast<long long>(d) * N + at);
        a.x *= kLog2e; a.y *= kLog2e; a.z *= kLog2e; a.w *= kLog2e;
        sm.A2[j][lane] = a;
        float4 g = start && mine ? *reinterpret_cast<const float4*>(start + at) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (kFull && p.carry && !composed && mine) {
            for (int i = w.after; i > 0; --i) {  // g <- exp(A sum dt) g + own gradient, from the last segment
                const long long sl = (slot + i) * p.D + d;
                const float s = p.carry_dt[sl];
                const float4 e = *reinterpret_cast<const float4*>(p.carry + sl * N + at);
                g.x = fmaf(ex2(a.x * s), g.x, e.x);
                g.y = fmaf(ex2(a.y * s), g.y, e.y);
                g.z = fmaf(ex2(a.z * s), g.z, e.z);
                g.w = fmaf(ex2(a.w * s), g.w, e.w);
            }
        }
        sm.g[j][lane] = g;
        if constexpr (kFull) sm.dA[j][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float dskip = kFull && p.D_skip ? p.D_skip[d] : 0.f;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    float s_dD = 0.f, s_db = 0.f;
    const long long row0 = static_cast<long long>(w.b) * p.T + w.s0;
    const T* u = static_cast<const T*>(p.u) + row0 * p.u_stride + w.d0;
    const T* dt = static_cast<const T*>(p.dt) + row0 * p.dt_stride + w.d0;
    const T* z = p.z ? static_cast<const T*>(p.z) + row0 * p.z_stride + w.d0 : nullptr;
    const T* d_out = static_cast<const T*>(p.d_out) + row0 * p.D + w.d0;
    const T* Bm = static_cast<const T*>(p.Bm) + row0 * p.B_stride + w.g * N;
    const T* Cm = static_cast<const T*>(p.Cm) + row0 * p.C_stride + w.g * N;
    const long long dense = row0 * p.D + d;
    const long long rows = p.cu_seqlens ? p.T : static_cast<long long>(p.nseq) * p.T;
    float* bc = kFull ? p.bc_part + (block * rows + row0) * 2 * N : nullptr;
    const int len = w.s1 - w.s0;
    const int tiles = (len + kTile - 1) / kTile;
    auto fetch = [&](int it) {  // tile `it`, if there is one
        if (it >= 0) {
            BwdStage<T, N, kFull>& st = sm.stage[it & 1];
            const int t = it * kTile, nt = len - t;
            fill_tile<T, CH, PB>(&st.dt[0][0], dt + t * p.dt_stride, p.dt_stride, nt, w.nd, lane);
            if (z) fill_tile<T, CH, PB>(&st.z[0][0], z + t * p.z_stride, p.z_stride, nt, w.nd, lane);
            fill_tile<T, CH, PB>(&st.d_out[0][0], d_out + t * static_cast<long long>(p.D), p.D, nt, w.nd, lane);
            fill_tile<T, N, PB>(&st.C[0][0], Cm + t * p.C_stride, p.C_stride, nt, N, lane);
            if constexpr (kFull) {
                fill_tile<T, CH, PB>(&st.u[0][0], u + t * p.u_stride, p.u_stride, nt, w.nd, lane);
                fill_tile<T, N, PB>(&st.B[0][0], Bm + t * p.B_stride, p.B_stride, nt, N, lane);
                // the channels' states before the tile, 16 bytes at a time
                const float* from = p.saved + ((w.chunk0 + it) * p.D + w.d0) * N;
#pragma unroll
                for (int i = 0; i < (CH * N / 4 + 31) / 32; ++i) {
                    const int id = i * 32 + lane;
                    const bool ok = id * 4 < w.nd * N;
                    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&st.saved[0][0] + id * 4));
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(ok ? from + id * 4 : from),
                                 "r"(ok ? 16 : 0)
                                 : "memory");
                }
            }
        }
        commit_copies();
    };
    fetch(tiles - 1);
    for (int it = tiles - 1; it >= 0; --it) {
        __syncwarp();  // everyone is through with the tile before
        fetch(it - 1);
        wait_copies<1>();
        __syncwarp();
        const BwdStage<T, N, kFull>& st = sm.stage[it & 1];
        widen_rows<T, N>(&st.C[0][0], &sm.C[0][0], lane);
        if constexpr (kFull) widen_rows<T, N>(&st.B[0][0], &sm.B[0][0], lane);
        const int t = it * kTile, left = len - t;
        // dt, x = dt u and dy of token k
        auto form = [&](int k, float& dk, float& xk, float& yk) {
            float v = to_f32(st.dt[k][ch]) + bias;
            if (p.softplus) v = softplus(v);
            dk = k < left ? v : 0.f;
            yk = to_f32(st.d_out[k][ch]);
            if (z) {
                const float zk = to_f32(st.z[k][ch]);
                yk *= zk * sigmoid(zk);
            }
            if constexpr (kFull) xk = dk * to_f32(st.u[k][ch]);
        };
        if constexpr (LPC > 1) {
#pragma unroll
            for (int i = 0; i < kTile / LPC; ++i) {
                float dk, xk = 0.f, yk;
                form(i * LPC + q, dk, xk, yk);
                sm.tok[i * LPC + q][ch] = make_float4(dk, xk, yk, 0.f);
            }
        }
        auto token = [&](int k, float& dk, float& xk, float& yk) {
            if constexpr (LPC > 1) {
                const float4 v = sm.tok[k][ch];
                dk = v.x;
                xk = v.y;
                yk = v.z;
            } else {
                form(k, dk, xk, yk);
            }
        };
        __syncwarp();
        if constexpr (!kFull) {
            float dk[kTile], yk[kTile], unused;
#pragma unroll
            for (int k = 0; k < kTile; ++k) {
                token(k, dk[k], unused, yk[k]);
                s_db += dk[k];
            }
#pragma unroll
            for (int j = 0; j < GR; ++j) {
                const Four A2 = get4(sm.A2[j][lane]);
                Four g = get4(sm.g[j][lane]);
#pragma unroll
                for (int k = kTile - 1; k >= 0; --k)
                    g = mul4(ex2_4(mul4(A2, two(dk[k], dk[k]))), fma4(get4(&sm.C[k][4 * (j * LPC + q)]), two(yk[k], yk[k]), g));
                put4(sm.g[j][lane], g);
            }
        } else {
            float dts[kHalf], xs[kHalf], dys[kHalf];
#pragma unroll
            for (int k = 0; k < kHalf; ++k) token(k, dts[k], xs[k], dys[k]);
            if (left > kHalf) {  // the states in the middle of the tile
#pragma unroll
                for (int j = 0; j < GR; ++j) {
                    const int at = 4 * (j * LPC + q);
                    const Four A2 = get4(sm.A2[j][lane]);
                    Four h = get4(&st.saved[ch][at]);
#pragma unroll
                    for (int k = 0; k < kHalf; ++k)
                        h = fma4(ex2_4(mul4(A2, two(dts[k], dts[k]))), h, mul4(get4(&sm.B[k][at]), two(xs[k], xs[k])));
                    put4(sm.mid[j][lane], h);
                }
            }
#pragma unroll
            for (int half = 1; half >= 0; --half) {
                if (half == 1 && left <= kHalf) continue;
                const int k0 = half * kHalf;
#pragma unroll
                for (int k = 0; k < kHalf; ++k) token(k0 + k, dts[k], xs[k], dys[k]);
                Two sx[kHalf], sa[kHalf], sy[kHalf];
#pragma unroll
                for (int k = 0; k < kHalf; ++k) sx[k] = sa[k] = sy[k] = two(0.f, 0.f);
#pragma unroll 1
                for (int j = 0; j < GR; ++j) {
                    const int at = 4 * (j * LPC + q);
                    const Four A2 = get4(sm.A2[j][lane]);
                    Four g = get4(sm.g[j][lane]), dA = get4(sm.dA[j][lane]);
                    // forward again: decays, and the state before and after every token
                    Four a[kHalf], h[kHalf + 1];
                    h[0] = half ? get4(sm.mid[j][lane]) : get4(&st.saved[ch][at]);
#pragma unroll
                    for (int k = 0; k < kHalf; ++k) {
                        a[k] = ex2_4(mul4(A2, two(dts[k], dts[k])));
                        h[k + 1] = fma4(a[k], h[k], mul4(get4(&sm.B[k0 + k][at]), two(xs[k], xs[k])));
                        sy[k] = dot4(h[k + 1], get4(&sm.C[k0 + k][at]), sy[k]);
                    }
                    // and back
#pragma unroll
                    for (int k = kHalf - 1; k >= 0; --k) {
                        const Two y2 = two(dys[k], dys[k]);
                        const Four e = fma4(get4(&sm.C[k0 + k][at]), y2, g);
                        float v[8];
                        {
                            const Four vb = mul4(e, two(xs[k], xs[k])), vc = mul4(h[k + 1], y2);
                            split(vb.lo, v[0], v[1]);
                            split(vb.hi, v[2], v[3]);
                            split(vc.lo, v[4], v[5]);
                            split(vc.hi, v[6], v[7]);
                        }
                        sx[k] = dot4(e, get4(&sm.B[k0 + k][at]), sx[k]);
                        g = mul4(a[k], e);
                        const Four qq = mul4(g, h[k]);
                        sa[k] = dot4(A2, qq, sa[k]);
                        dA = fma4(qq, two(dts[k], dts[k]), dA);
                        across_channels<LPC, CH>(v, ch);
                        if (ch < 8) {
#pragma unroll
                            for (int i = 0; i < 8 / M8; ++i) {
                                const int idx = i * M8 + ch;
                                sm.bc[k][(idx >> 2) * N + at + (idx & 3)] = v[i];
                            }
                        }
                    }
                    put4(sm.g[j][lane], g);
                    put4(sm.dA[j][lane], dA);
                }
                __syncwarp();
                // the warp's share of dB and dC
                {
                    float4* to = reinterpret_cast<float4*>(bc + (t + k0) * static_cast<long long>(2 * N));
                    const float4* from = reinterpret_cast<const float4*>(&sm.bc[0][0]);
                    const int n4 = min(kHalf, left - k0) * (N / 2);
#pragma unroll
                    for (int i = 0; i < (kHalf * N / 2 + 31) / 32; ++i)
                        if (i * 32 + lane < n4) to[i * 32 + lane] = from[i * 32 + lane];
                }
                const long long at = dense + (t + k0) * static_cast<long long>(p.D);
                // the outputs of token k0 + k
                auto finish = [&](int k, float dk, float yk, float y, float dx, float da) {
                    const float uk = to_f32(st.u[k0 + k][ch]);
                    float dr = fmaf(uk, dx, da * (1.f / kLog2e));
                    if (p.softplus) dr *= sigmoid(to_f32(st.dt[k0 + k][ch]) + bias);
                    if (k0 + k < left) {
                        s_dD = fmaf(yk, uk, s_dD);
                        s_db += dr;
                        if (mine) {
                            const long long to = at + k * static_cast<long long>(p.D);
                            static_cast<T*>(p.du)[to] = from_f32<T>(fmaf(dk, dx, dskip * yk));
                            static_cast<T*>(p.ddt)[to] = from_f32<T>(dr);
                            if (z) {
                                const float zk = to_f32(st.z[k0 + k][ch]);
                                static_cast<T*>(p.dz)[to] =
                                    from_f32<T>(to_f32(st.d_out[k0 + k][ch]) * fmaf(dskip, uk, y) * dsilu(zk, sigmoid(zk)));
                            }
                        }
                    }
                };
                if constexpr (LPC == 1) {
#pragma unroll
                    for (int k = 0; k < kHalf; ++k) finish(k, dts[k], dys[k], both(sy[k]), both(sx[k]), both(sa[k]));
                } else {  // a lane takes the tokens whose sums it ends up with
                    float y[kHalf], dx[kHalf], da[kHalf];
#pragma unroll
                    for (int k = 0; k < kHalf; ++k) {
                        y[k] = both(sy[k]);
                        dx[k] = both(sx[k]);
                        da[k] = both(sa[k]);
                    }
                    share_sums<LPC>(y, q);
                    share_sums<LPC>(dx, q);
                    share_sums<LPC>(da, q);
                    if (LPC <= kHalf || q < kHalf) {
#pragma unroll
                        for (int i = 0; i < (kHalf + LPC - 1) / LPC; ++i) {
                            const float4 v = sm.tok[k0 + i * LPC + q][ch];
                            finish(i * LPC + q, v.x, v.z, y[i], dx[i], da[i]);
                        }
                    }
                }
                __syncwarp();  // before the other half's sums go where these were
            }
        }
    }
    if constexpr (kFull) {  // a channel's lanes took different tokens
#pragma unroll
        for (int m = 1; m < LPC; m *= 2) {
            s_dD += __shfl_xor_sync(0xffffffffu, s_dD, m);
            s_db += __shfl_xor_sync(0xffffffffu, s_db, m);
        }
    }
    if (!mine) return;
    if constexpr (!kFull) {
#pragma unroll
        for (int j = 0; j < GR; ++j)
            *reinterpret_cast<float4*>(p.carry + (slot * p.D + d) * N + 4 * (j * LPC + q)) = sm.g[j][lane];
        if (q == 0) p.carry_dt[slot * p.D + d] = s_db;
    } else {
        float* par = p.par_part + slot * ssm_par_stride(p.D, N);
#pragma unroll
        for (int j = 0; j < GR; ++j) {
            const long long at = static_cast<long long>(d) * N + 4 * (j * LPC + q);
            *reinterpret_cast<float4*>(par + at) = sm.dA[j][lane];
            if (w.first && p.d_initial_state)
                *reinterpret_cast<float4*>(p.d_initial_state + static_cast<long long>(w.n) * p.D * N + at) = sm.g[j][lane];
        }
        if (q == 0) {
            par[static_cast<long long>(p.D) * N + d] = s_dD;
            par[static_cast<long long>(p.D) * N + p.D + d] = s_db;
        }
    }
}

// dB and dC: the partial rows of a group's channel blocks, added in order (2 x
// 4096 tokens, 64 blocks of 2 x 16 columns: 15 us, 4.5 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) ssm_bc_kernel(const SsmBcArgs p) {
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int w2 = 2 * p.N;
    const long long per = p.rows * w2;
    if (id >= per * p.G) return;
    const int g = static_cast<int>(id / per);
    const long long row = id % per / w2;
    const int col = static_cast<int>(id % w2);
    const float* src = p.bc_part + static_cast<long long>(g) * p.blocks * per + id % per;
    float s = 0.f;
#pragma unroll 8
    for (int i = 0; i < p.blocks; ++i) s += __ldg(src + i * per);
    T* out = static_cast<T*>(col < p.N ? p.dB : p.dC);
    out[(row * p.G + g) * p.N + (col < p.N ? col : col - p.N)] = from_f32<T>(s);
}

template <typename T, int N, int PB>
cudaError_t bwd_v(const SsmArgs& a, cudaStream_t stream) {
    const int blocks = ssm_group_blocks(a.D, a.G, N);
    const long long units = a.slots * blocks * a.G;
    if (a.carry) {
        cudaError_t e = launch_warps<kBwdWarps<N>>(ssm_bwd_kernel<T, N, false, PB>, units, sizeof(BwdShared<T, N, false>), a, blocks, stream);
        if (e == cudaSuccess && a.joined) e = launch_ssm_compose(a, true, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_warps<kBwdWarps<N>>(ssm_bwd_kernel<T, N, true, PB>, units, sizeof(BwdShared<T, N, true>), a, blocks, stream);
}

template <typename T, int N>
cudaError_t bwd_n(const SsmArgs& a, cudaStream_t stream) {
    switch (scan_pieces<T, N>(a)) {
        case 16: return bwd_v<T, N, 16>(a, stream);
        case 4: return bwd_v<T, N, 4>(a, stream);
    }
    if constexpr (sizeof(T) == 2) return bwd_v<T, N, 0>(a, stream);
    return cudaErrorMisalignedAddress;  // fp32 is 4-byte aligned
}

}  // namespace

int ssm_group_blocks(int D, int G, int N) {
    const int ch = N <= 16 ? 32 : 512 / N;
    return (D / G + ch - 1) / ch;
}

cudaError_t launch_ssm_bwd(const SsmArgs& a, cudaStream_t stream) {
#define GDN_SSM_N(T)                                 \
    switch (a.N) {                                   \
        case 8: return bwd_n<T, 8>(a, stream);       \
        case 16: return bwd_n<T, 16>(a, stream);     \
        case 32: return bwd_n<T, 32>(a, stream);     \
        case 64: return bwd_n<T, 64>(a, stream);     \
        default: return bwd_n<T, 128>(a, stream);    \
    }
    if (a.dtype == 0) {
        GDN_SSM_N(uint16_t)
    }
    GDN_SSM_N(float)
#undef GDN_SSM_N
}

cudaError_t launch_ssm_bc(const SsmBcArgs& a, cudaStream_t stream) {
    const long long n = a.rows * 2 * a.N * a.G;
    if (n == 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>((n + 255) / 256);
    if (a.dtype == 0)
        ssm_bc_kernel<uint16_t><<<grid, 256, 0, stream>>>(a);
    else
        ssm_bc_kernel<float><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
