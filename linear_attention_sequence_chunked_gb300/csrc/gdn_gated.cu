// Gated linear recurrence: forward, reverse mode and the single-token step.
//
//   L_t = -rate softplus(lam) sigmoid(r_t),  a_t = exp(L_t),  m_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t
//
// per channel.  A token's map h -> a h + b composes with its neighbours', so a
// row of T tokens is cut into strips of kStrip tokens, one warp to a strip with
// its channels across the lanes.  A strip's tokens are loaded and its (a, b)
// formed once, in registers; the warp composes them from a zero state, the
// strips' products (P, H) meet in shared memory, and each warp then walks its
// tokens again from the state it really starts from.  Every input is read once
// and every output written once.  A block is kWarps consecutive strips; where
// the channels alone do not fill the GPU a cluster of blocks works side by side
// on consecutive stretches and exchanges one (P, H) per block and channel
// through distributed shared memory.  The cluster then takes the next stretch,
// with the state it ended in.  All compositions run in a fixed order.
//
// Packed sequences are one row: a sequence's first token starts from its own
// initial state, and a strip that holds such a token ignores what comes in.
#include <algorithm>

#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kWarps = 8;
constexpr int kStrip = kGatedStrip;

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A store to the same shared variable of block `rank` of the cluster.
__device__ __forceinline__ void store_remote(float2* p, uint32_t rank, float2 v) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v.x), "f"(v.y) : "memory");
}

// ---------------------------------------------------------------- the gates

// 1 - exp(y) for y <= 0: the exponential series up to y^9 / 9! for y >= -1/2
// (relative error below 2^-24), else from the exponential itself (which has lost
// at most a bit and a half there).
__device__ __forceinline__ float one_minus_exp(float y, float e) {
    float s = fmaf(y, 1.f / 362880.f, 1.f / 40320.f);
    s = fmaf(y, s, 1.f / 5040.f);
    s = fmaf(y, s, 1.f / 720.f);
    s = fmaf(y, s, 1.f / 120.f);
    s = fmaf(y, s, 1.f / 24.f);
    s = fmaf(y, s, 1.f / 6.f);
    s = fmaf(y, s, 0.5f);
    s = fmaf(y, s, 1.f);
    return y >= -0.5f ? -y * s : 1.f - e;
}
__device__ __forceinline__ float root(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// a and m of a token from L (in natural logarithms)
__device__ __forceinline__ void decay(float L, float& a, float& m) {
    a = ex2(kLog2e * L);
    m = root(one_minus_exp(2.f * L, a * a));
}

// ---------------------------------------------------------------- sequences

// The sequence that holds a token of the row, and its ends.
struct Seq {
    int n, s0, s1;
};
__device__ __forceinline__ Seq find_seq(const GatedArgs& p, int row, int t) {
    if (p.cu_seqlens == nullptr) return Seq{row, 0, p.T};
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return Seq{lo, p.cu_seqlens[lo], p.cu_seqlens[lo + 1]};
}

// The composition of the strips before this warp's: `mine` receives the value
// that reaches the warp's strip, the return value what leaves the cluster's
// whole stretch.  P.x is NaN-safe: a strip that ignores what comes in says so
// by `cut`.
template <int E>
struct Exchange {
    float2 strip[2][kWarps][E][32];   // (P, H) of this block's strips
    float2 block[2][kGatedMaxCluster][E][32];
    int cut[2][kWarps];
    float2 block_cut[2][kGatedMaxCluster];
};

__device__ __forceinline__ float pass(float2 ph, int cut, float h) { return cut ? ph.y : fmaf(ph.x, h, ph.y); }

template <int E>
__device__ __forceinline__ void exchange(Exchange<E>& sm, int parity, int warp, int lane, uint32_t rank, int C,
                                         const float* P, const float* H, int cut, float* carry, float* mine) {
#pragma unroll
    for (int e = 0; e < E; ++e) sm.strip[parity][warp][e][lane] = make_float2(P[e], H[e]);
    if (lane == 0) sm.cut[parity][warp] = cut;
    __syncthreads();
    if (C > 1) {
        if (warp < E) {  // the whole block's map, one row of channels per warp
            float2 s = make_float2(1.f, 0.f);
            int any = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ph = sm.strip[parity][w][warp][lane];
                const int c = sm.cut[parity][w];
                s.y = pass(ph, c, s.y);
                s.x *= ph.x;
                any |= c;
            }
            for (int c = 0; c < C; ++c) {
                store_remote(&sm.block[parity][rank][warp][lane], c, s);
                if (warp == 0 && lane == 0) store_remote(&sm.block_cut[parity][rank], c, make_float2(any ? 1.f : 0.f, 0.f));
            }
        }
        cluster_sync();
#pragma unroll
        for (int e = 0; e < E; ++e) mine[e] = carry[e];
        for (int c = 0; c < C; ++c) {
            const int ct = sm.block_cut[parity][c].x != 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (c == static_cast<int>(rank)) mine[e] = carry[e];
                carry[e] = pass(sm.block[parity][c][e][lane], ct, carry[e]);
            }
        }
        for (int w = 0; w < warp; ++w) {
            const int ct = sm.cut[parity][w];
#pragma unroll
            for (int e = 0; e < E; ++e) mine[e] = pass(sm.strip[parity][w][e][lane], ct, mine[e]);
        }
    } else {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int ct = sm.cut[parity][w];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (w == warp) mine[e] = carry[e];
                carry[e] = pass(sm.strip[parity][w][e][lane], ct, carry[e]);
            }
        }
    }
}

template <int E>
__device__ __forceinline__ void load_state(const float* p, int nd, float* h) {
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] = p && e < nd ? p[e] : 0.f;
}
template <int E>
__device__ __forceinline__ void store_state(float* p, int nd, const float* h) {
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e < nd) p[e] = h[e];
}

// ---------------------------------------------------------------- forward

template <typename T, int E>
__global__ void __launch_bounds__(32 * kWarps, 2) gated_fwd_kernel(const GatedArgs p) {
    __shared__ Exchange<E> sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = p.cluster, row = blockIdx.y;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int d = (blockIdx.x / C) * (32 * E) + lane * E;
    const int nd = max(0, min(E, p.D - d));  // this lane's channels
    if (blockIdx.x == 0 && row == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    float scale[E];  // -rate softplus(lam)
#pragma unroll
    for (int e = 0; e < E; ++e) scale[e] = e < nd ? -p.rate * softplus(p.lam[d + e]) : 0.f;
    const long long row0 = static_cast<long long>(row) * p.T;
    const T* x = static_cast<const T*>(p.x) + row0 * p.x_stride + d;
    const T* r = static_cast<const T*>(p.r) + row0 * p.r_stride + d;
    const T* gi = static_cast<const T*>(p.i) + row0 * p.i_stride + d;
    T* y = static_cast<T*>(p.y) + row0 * p.D + d;
    const int strips = (p.T + kStrip - 1) / kStrip;
    if (p.final_state && rank == 0) {  // sequences without tokens
        const int first = p.cu_seqlens ? 0 : row, last = p.cu_seqlens ? p.nseq : row + 1;
        for (int n = first + warp; n < last; n += kWarps) {
            if (p.cu_seqlens ? p.cu_seqlens[n] < p.cu_seqlens[n + 1] : p.T > 0) continue;
            float h[E];
            load_state<E>(p.initial_state ? p.initial_state + static_cast<long long>(n) * p.D + d : nullptr, nd, h);
            store_state<E>(p.final_state + static_cast<long long>(n) * p.D + d, nd, h);
        }
    }
    if (C > 1) cluster_sync();  // every block of the cluster is there
    float carry[E] = {};
    for (int s0 = 0, round = 0; s0 < strips; s0 += C * kWarps, ++round) {
        const int s = s0 + rank * kWarps + warp;
        const int t0 = s * kStrip;  // s < strips + 64: below 2^30 + 2^10
        const int nk = max(0, min(kStrip, p.T - t0));
        Raw<T, E> rx[kStrip], rr[kStrip], ri[kStrip];
#pragma unroll
        for (int k = 0; k < kStrip; ++k) {
            const long long t = t0 + k;
            const int n = k < nk ? nd : 0;
            rr[k] = load_raw<T, E>(r + t * p.r_stride, n);
            ri[k] = load_raw<T, E>(gi + t * p.i_stride, n);
            rx[k] = load_raw<T, E>(x + t * p.x_stride, n);
        }
        Seq q = nk > 0 ? find_seq(p, row, t0) : Seq{0, -1, 1 << 30};
        const bool ends = q.s0 == t0 || q.s1 <= t0 + nk;  // a sequence starts or ends here
        float a[kStrip][E], b[kStrip][E];
#pragma unroll
        for (int k = 0; k < kStrip; ++k) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float m;
                decay(scale[e] * sigmoid(rr[k].get(e)), a[k][e], m);
                b[k][e] = m * (sigmoid(ri[k].get(e)) * rx[k].get(e));
            }
        }
        float P[E], H[E];
        int cut = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            P[e] = 1.f;
            H[e] = 0.f;
        }
        if (!ends) {
#pragma unroll
            for (int k = 0; k < kStrip; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    H[e] = fmaf(a[k][e], H[e], b[k][e]);
                    P[e] *= a[k][e];
                }
        } else {
            Seq w = q;
#pragma unroll
            for (int k = 0; k < kStrip; ++k) {
                if (k < nk) {
                    if (t0 + k >= w.s1) w = find_seq(p, row, t0 + k);
                    if (t0 + k == w.s0) {
                        cut = 1;
                        load_state<E>(p.initial_state ? p.initial_state + static_cast<long long>(w.n) * p.D + d : nullptr, nd, H);
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e) H[e] = fmaf(a[k][e], H[e], b[k][e]);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) P[e] *= a[k][e];
            }
        }
        float h[E];
        exchange<E>(sm, round & 1, warp, lane, rank, C, P, H, cut, carry, h);
        if (p.saved && nk > 0) store_state<E>(p.saved + (static_cast<long long>(row) * strips + s) * p.D + d, nd, h);
#pragma unroll
        for (int k = 0; k < kStrip; ++k) {
            if (ends && k < nk) {
                if (t0 + k >= q.s1) q = find_seq(p, row, t0 + k);
                if (t0 + k == q.s0)
                    load_state<E>(p.initial_state ? p.initial_state + static_cast<long long>(q.n) * p.D + d : nullptr, nd, h);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = fmaf(a[k][e], h[e], b[k][e]);
            if (k < nk) store_raw<T, E>(y + static_cast<long long>(t0 + k) * p.D, pack<T, E>(h), nd);
            if (ends && k < nk && t0 + k == q.s1 - 1 && p.final_state)
                store_state<E>(p.final_state + static_cast<long long>(q.n) * p.D + d, nd, h);
        }
    }
    if (C > 1) cluster_sync();  // the others may still write here
}

// ---------------------------------------------------------------- reverse mode

// With c_t = a_t dh_t, the gradient that reaches h_{t-1}, dh_t = dout_t + c_{t+1}:
// c composes backwards as h does forwards, from the last strip to the first.
// The states before each token come from the strip's saved start.
//   dL = dh (a h_{t-1} - a^2 / m sigmoid(i) x);  dr = dL L (1 - sigmoid(r));
//   d(sigmoid(i) x) = dh m;  dlam = -rate sigmoid(lam) sum dL sigmoid(r)
// Where m = 0 (a rounds to 1) a^2 / m L has the limit 0, and the term is left out.
template <typename T, int E>
__global__ void __launch_bounds__(32 * kWarps, 2) gated_bwd_kernel(const GatedArgs p) {
    __shared__ Exchange<E> sm;
    __shared__ float part[kWarps][E][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = p.cluster, row = blockIdx.y;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int d = (blockIdx.x / C) * (32 * E) + lane * E;
    const int nd = max(0, min(E, p.D - d));
    if (blockIdx.x == 0 && row == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    float scale[E];
#pragma unroll
    for (int e = 0; e < E; ++e) scale[e] = e < nd ? -p.rate * softplus(p.lam[d + e]) : 0.f;
    const long long row0 = static_cast<long long>(row) * p.T;
    const T* x = static_cast<const T*>(p.x) + row0 * p.x_stride + d;
    const T* r = static_cast<const T*>(p.r) + row0 * p.r_stride + d;
    const T* gi = static_cast<const T*>(p.i) + row0 * p.i_stride + d;
    const T* go = static_cast<const T*>(p.d_out) + row0 * p.D + d;
    T* dx = static_cast<T*>(p.dx) + row0 * p.D + d;
    T* dr = static_cast<T*>(p.dr) + row0 * p.D + d;
    T* di = static_cast<T*>(p.di) + row0 * p.D + d;
    const int strips = (p.T + kStrip - 1) / kStrip;
    const auto state_of = [&](const float* s, int n) { return s ? s + static_cast<long long>(n) * p.D + d : nullptr; };
    if (p.d_initial_state && rank == 0) {  // sequences without tokens pass the final state's gradient on
        const int first = p.cu_seqlens ? 0 : row, last = p.cu_seqlens ? p.nseq : row + 1;
        for (int n = first + warp; n < last; n += kWarps) {
            if (p.cu_seqlens ? p.cu_seqlens[n] < p.cu_seqlens[n + 1] : p.T > 0) continue;
            float h[E];
            load_state<E>(state_of(p.d_final_state, n), nd, h);
            store_state<E>(p.d_initial_state + static_cast<long long>(n) * p.D + d, nd, h);
        }
    }
    if (C > 1) cluster_sync();  // every block of the cluster is there
    float carry[E] = {}, dlam[E] = {};
    for (int j0 = 0, round = 0; j0 < strips; j0 += C * kWarps, ++round) {
        const int s = strips - 1 - (j0 + static_cast<int>(rank) * kWarps + warp);  // from the last strip on
        const int t0 = s * kStrip;
        const int nk = s < 0 ? 0 : min(kStrip, p.T - t0);
        Raw<T, E> rx[kStrip], rr[kStrip], ri[kStrip], rg[kStrip];
#pragma unroll
        for (int k = 0; k < kStrip; ++k) {
            const long long t = t0 + k;
            const int n = k < nk ? nd : 0;
            rr[k] = load_raw<T, E>(r + t * p.r_stride, n);
            ri[k] = load_raw<T, E>(gi + t * p.i_stride, n);
            rx[k] = load_raw<T, E>(x + t * p.x_stride, n);
            rg[k] = load_raw<T, E>(go + t * p.D, n);
        }
        float h[E];
        load_state<E>(nk > 0 ? p.saved + (static_cast<long long>(row) * strips + s) * p.D + d : nullptr, nd, h);
        const Seq q0 = nk > 0 ? find_seq(p, row, t0) : Seq{0, -1, 1 << 30};
        const bool ends = q0.s0 == t0 || q0.s1 <= t0 + nk;
        // per token: a, sigmoid(r), sigmoid(i) and the state before it
        float a[kStrip][E], sr[kStrip][E], si[kStrip][E], hp[kStrip][E];
        Seq q = q0;
#pragma unroll
        for (int k = 0; k < kStrip; ++k) {
            if (ends && k < nk) {
                if (t0 + k >= q.s1) q = find_seq(p, row, t0 + k);
                if (t0 + k == q.s0) load_state<E>(state_of(p.initial_state, q.n), nd, h);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float m;
                sr[k][e] = sigmoid(rr[k].get(e));
                si[k][e] = sigmoid(ri[k].get(e));
                decay(scale[e] * sr[k][e], a[k][e], m);
                hp[k][e] = h[e];
                h[e] = fmaf(a[k][e], h[e], m * (si[k][e] * rx[k].get(e)));
            }
        }
        float P[E], Q[E];
        int cut = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            P[e] = 1.f;
            Q[e] = 0.f;
        }
        Seq w = q;
#pragma unroll
        for (int k = kStrip - 1; k >= 0; --k) {
            if (ends && k < nk) {
                if (t0 + k < w.s0) w = find_seq(p, row, t0 + k);
                if (t0 + k == w.s1 - 1) {  // nothing comes from the next sequence
                    cut = 1;
                    load_state<E>(state_of(p.d_final_state, w.n), nd, Q);
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (k < nk) {  // the row's last strip may be short: its other tokens are not there
                    Q[e] = a[k][e] * (rg[k].get(e) + Q[e]);
                    P[e] *= a[k][e];
                }
            }
        }
        float c[E];
        exchange<E>(sm, round & 1, warp, lane, rank, C, P, Q, cut, carry, c);
        w = q;
#pragma unroll
        for (int k = kStrip - 1; k >= 0; --k) {
            if (k >= nk) continue;
            if (ends) {
                if (t0 + k < w.s0) w = find_seq(p, row, t0 + k);
                if (t0 + k == w.s1 - 1) load_state<E>(state_of(p.d_final_state, w.n), nd, c);
            }
            float ox[E], orr[E], oi[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float dh = rg[k].get(e) + c[e], xk = rx[k].get(e), ak = a[k][e];
                const float L = scale[e] * sr[k][e];
                const float a2 = ak * ak;
                const float m = root(one_minus_exp(2.f * L, a2));
                const float through = m > 0.f ? a2 * rcp(m) : 0.f;
                const float gx = si[k][e] * xk;
                const float dL = dh * fmaf(ak, hp[k][e], -through * gx);
                const float dg = dh * m;
                ox[e] = dg * si[k][e];
                oi[e] = dg * gx * (1.f - si[k][e]);
                orr[e] = dL * L * (1.f - sr[k][e]);
                dlam[e] = fmaf(dL, sr[k][e], dlam[e]);
                c[e] = ak * dh;
            }
            const long long o = static_cast<long long>(t0 + k) * p.D;
            store_raw<T, E>(dx + o, pack<T, E>(ox), nd);
            store_raw<T, E>(dr + o, pack<T, E>(orr), nd);
            store_raw<T, E>(di + o, pack<T, E>(oi), nd);
            if (ends && t0 + k == w.s0 && p.d_initial_state)
                store_state<E>(p.d_initial_state + static_cast<long long>(w.n) * p.D + d, nd, c);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][e][lane] = dlam[e];
    __syncthreads();
    if (warp < E) {  // one row of channels per warp
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += part[w][warp][lane];
        const int dd = d + warp;
        if (dd < p.D)
            p.partial[(static_cast<long long>(row) * C + rank) * p.D + dd] = -p.rate * sigmoid(p.lam[dd]) * sum;
    }
    if (C > 1) cluster_sync();
}

// ---------------------------------------------------------------- one token

template <typename T, int E, bool VEC>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedStepArgs p) {
    const int per = (p.D + E - 1) / E;
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long b = id / per;
    if (b >= p.B) return;
    const int d = static_cast<int>(id % per) * E;
    const int nd = min(E, p.D - d);
    long long slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot >= p.S) record_error(p.err, kErrBadSlot);
    }
    const bool on = slot >= 0 && slot < p.S;
    const int n = on ? nd : 0;
    const Raw<float, E> rl = load_raw<float, E, VEC>(p.lam + d, nd);
    const Raw<T, E> rr = load_raw<T, E, VEC>(static_cast<const T*>(p.r) + b * p.r_stride + d, n);
    const Raw<T, E> ri = load_raw<T, E, VEC>(static_cast<const T*>(p.i) + b * p.i_stride + d, n);
    const Raw<T, E> rx = load_raw<T, E, VEC>(static_cast<const T*>(p.x) + b * p.x_stride + d, n);
    Raw<float, E> h;  // not load_raw: the cache may be written in place
    const long long so = (on ? slot : 0) * p.D + d;
#pragma unroll
    for (int e = 0; e < E; ++e) h.w[e] = 0;
    if (on) {
        if constexpr (VEC && E == 4) {
            const float4 v = *reinterpret_cast<const float4*>(p.state + so);
            h.w[0] = __float_as_uint(v.x); h.w[1] = __float_as_uint(v.y);
            h.w[2] = __float_as_uint(v.z); h.w[3] = __float_as_uint(v.w);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < nd) h.w[e] = __float_as_uint(p.state[so + e]);
        }
    }
    float out[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float a, m;
        decay(-p.rate * softplus(rl.get(e)) * sigmoid(rr.get(e)), a, m);
        out[e] = on ? fmaf(a, h.get(e), m * (sigmoid(ri.get(e)) * rx.get(e))) : 0.f;
    }
    if (on) store_raw<float, E, VEC>(p.out_state + so, pack<float, E>(out), nd);
    store_raw<T, E, VEC>(static_cast<T*>(p.y) + b * p.D + d, pack<T, E>(out), nd);
}

// ---------------------------------------------------------------- launches

// E elements per access: every row starts at a multiple of their size
template <typename T>
bool fits(int E, int D, std::initializer_list<const void*> ptrs, std::initializer_list<long long> strides) {
    if (D % E != 0) return false;
    for (const void* q : ptrs)
        if (q && reinterpret_cast<uintptr_t>(q) % (sizeof(T) * E) != 0) return false;
    for (long long s : strides)
        if (s % E != 0) return false;
    return true;
}

template <typename K>
cudaError_t launch_clusters(K kernel, dim3 grid, int cluster, const GatedArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T>
cudaError_t launch(const GatedArgs& a, bool backward, cudaStream_t stream) {
    const bool pair = fits<T>(2, a.D, {a.x, a.r, a.i}, {a.x_stride, a.r_stride, a.i_stride});
    const dim3 grid(static_cast<unsigned>((a.D + (pair ? 63 : 31)) / (pair ? 64 : 32) * a.cluster), a.rows);
    if (backward)
        return pair ? launch_clusters(gated_bwd_kernel<T, 2>, grid, a.cluster, a, stream)
                    : launch_clusters(gated_bwd_kernel<T, 1>, grid, a.cluster, a, stream);
    return pair ? launch_clusters(gated_fwd_kernel<T, 2>, grid, a.cluster, a, stream)
                : launch_clusters(gated_fwd_kernel<T, 1>, grid, a.cluster, a, stream);
}

}  // namespace

int gated_cluster(int rows, int T, int D) {
    const long long units = static_cast<long long>(rows) * ((D + 63) / 64);
    int c = 1;
    while (c < kGatedMaxCluster && units * c < 3 * 152 && static_cast<long long>(T) > static_cast<long long>(c) * kWarps * kStrip) c *= 2;
    return c;
}

cudaError_t launch_gated_fwd(const GatedArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch<float>(a, false, stream) : launch<uint16_t>(a, false, stream);
}
cudaError_t launch_gated_bwd(const GatedArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch<float>(a, true, stream) : launch<uint16_t>(a, true, stream);
}

namespace {
template <typename T>
cudaError_t launch_step(const GatedStepArgs& a, cudaStream_t stream) {
    const bool vec = fits<T>(4, a.D, {a.x, a.r, a.i}, {a.x_stride, a.r_stride, a.i_stride});
    const long long n = static_cast<long long>(a.B) * (vec ? a.D / 4 : a.D);
    const unsigned blocks = static_cast<unsigned>((n + 255) / 256);
    if (vec)
        gated_step_kernel<T, 4, true><<<blocks, 256, 0, stream>>>(a);
    else
        gated_step_kernel<T, 1, true><<<blocks, 256, 0, stream>>>(a);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_gated_step(const GatedStepArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch_step<float>(a, stream) : launch_step<uint16_t>(a, stream);
}

}  // namespace gdn
