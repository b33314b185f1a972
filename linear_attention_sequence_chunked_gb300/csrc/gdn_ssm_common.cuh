// Geometry and tile staging shared by the selective state space scan kernels.
//
// Per sequence and channel d (group g of B and C), with N states:
//   dt_t = softplus(dt_raw_t + dt_bias_d)          (or without the softplus)
//   h_t  = exp(dt_t A_dn) h_{t-1} + dt_t u_t B_tn,   y_t = sum_n C_tn h_tn + D_d u_t,
//   out_t = y_t silu(z_t)                           (or y_t without a gate).
// One warp walks a run of tokens for CH = 32 NS / N channels: lane
// ch * LPC + q holds states NS q .. NS q + NS - 1 of channel ch in registers, so
// a token costs NS exponentials and about 4 NS fp32 operations per lane.  Tokens
// come in tiles of kSsmChunk = 16: lane l first takes the l-th share of the
// tile's (token, channel) elements, forms dt and x = dt u once per element and
// puts them, B and C into the warp's shared memory as fp32; the 16 tokens then
// run from there without a branch (a token after the end has dt = x = 0, which
// leaves the state as it is).
#pragma once

#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {
namespace ssm {

using namespace mix;

constexpr int K = kSsmChunk;

// K tokens x CH channels over 32 lanes: token lane / PARTS, EPL channels from
// (lane % PARTS) * EPL.
template <int N, int NS>
struct Geo {
    static constexpr int LPC = N / NS;
    static constexpr int CH = 32 / LPC;
    static constexpr int EPL = CH >= 2 ? CH / 2 : 1;
    static constexpr int PARTS = CH >= 2 ? 2 : 1;
};

// B or C rows of a tile: K x N elements in pieces of PE, NP pieces per lane.
template <typename T, int N, bool VEC>
struct RowTile {
    static constexpr int PE = (N / 2 < 16 / static_cast<int>(sizeof(T))) ? N / 2 : 16 / static_cast<int>(sizeof(T));
    static constexpr int NP = N / 2 / PE;
    Raw<T, PE> v[NP];

    // rows: the tile's first row at this group's column 0; nt rows are valid
    __device__ __forceinline__ void load(const T* rows, long long stride, int nt, int lane) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int id = p * 32 + lane;
            const int tok = id / (N / PE), n0 = id % (N / PE) * PE;
            v[p] = load_raw<T, PE, VEC>(rows + tok * stride + n0, tok < nt ? PE : 0);
        }
    }
    __device__ __forceinline__ void store(float* dst, int lane) const {  // [K][N]
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            float x[PE];
            unpack<T, PE>(v[p], x);
            float4* d = reinterpret_cast<float4*>(dst + (p * 32 + lane) * PE);
#pragma unroll
            for (int i = 0; i < PE / 4; ++i) d[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
    }
};

// Whether every activation of the scan can be accessed in the vectors of this
// geometry (decided on the host: the kernels have no branch on it).
template <typename T, int N, int NS>
bool all_vec(const SsmArgs& a) {
    constexpr int EPL = Geo<N, NS>::EPL, PE = RowTile<T, N, true>::PE;
    auto ok = [](const void* p, long long stride, int e) {
        const int bytes = e * static_cast<int>(sizeof(T)) < 16 ? e * static_cast<int>(sizeof(T)) : 16;
        return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * static_cast<long long>(sizeof(T)) % bytes == 0;
    };
    return a.D / a.G % EPL == 0 && ok(a.u, a.u_stride, EPL) && ok(a.dt, a.dt_stride, EPL) &&
           (!a.z || ok(a.z, a.z_stride, EPL)) && ok(a.out, a.D, EPL) && ok(a.Bm, a.B_stride, PE) &&
           ok(a.Cm, a.C_stride, PE);
}

// Sums over the LPC lanes of a channel of v[t], t < K: value i of lane q is
// then the sum of token i * min(LPC, K) + (q mod K).
template <int LPC>
__device__ __forceinline__ void channel_sums(float (&v)[K], int q) {
#pragma unroll
    for (int s = 0, m = 1; m < LPC; ++s, m *= 2) {
        if (m < K) {
            const bool hi = (q & m) != 0;
#pragma unroll
            for (int i = 0; i < K / 2; ++i) {
                if (i < K / (2 * m)) {
                    const float send = hi ? v[2 * i] : v[2 * i + 1];
                    const float keep = hi ? v[2 * i + 1] : v[2 * i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
        }
    }
}

// This lane's channel_sums into out[token][CH].
template <int LPC, int CH>
__device__ __forceinline__ void put_channel_sums(float (&v)[K], int q, int ch, float* out) {
    channel_sums<LPC>(v, q);
    constexpr int M = LPC < K ? LPC : K;
#pragma unroll
    for (int i = 0; i < K / M; ++i) out[(i * M + q % M) * CH + ch] = v[i];
}

// Sum over the token lanes that share a channel share (same lane % PARTS).
template <int PARTS>
__device__ __forceinline__ float over_tokens(float x) {
#pragma unroll
    for (int m = PARTS; m < 32; m *= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Where a warp works: segment `slot` of the tokens, one block of CH channels.
struct Place {
    int n, b, t0, t1;         // sequence, batch row, its token range
    int s0, s1;               // the segment's tokens
    bool first, last;         // segment of its sequence
    int g, d0, nd;            // group, first channel, channels (<= CH)
    long long chunk0;         // the segment's first slot of the saved chunk states
    long long slot;           // the segment itself
};

template <int CH>
__device__ __forceinline__ bool find_place(const SsmArgs& p, long long slot, int block, int seg, int blocks, Place& w) {
    long long c;
    if (!find_block(p.cu_seqlens, p.nseq, p.T, seg, slot, p.err, w.n, c)) return false;
    if (!token_range(p.cu_seqlens, w.n, p.nseq, p.T, p.err, w.b, w.t0, w.t1)) return false;
    const long long begin = w.t0 + c * seg;
    w.first = c == 0;
    w.slot = slot;
    if (begin >= w.t1 && !w.first) return false;  // no such segment
    w.s0 = static_cast<int>(begin);
    w.s1 = static_cast<int>(min(begin + seg, static_cast<long long>(w.t1)));
    w.last = w.s1 == w.t1;
    const int per = p.D / p.G;
    w.g = block / blocks;
    const int off = block % blocks * CH;
    w.d0 = w.g * per + off;
    w.nd = min(CH, per - off);
    const long long base = p.cu_seqlens ? static_cast<long long>(w.t0 / K) + w.n
                                        : static_cast<long long>(w.n) * ((p.T + K - 1) / K);
    w.chunk0 = base + (w.s0 - w.t0) / K;
    return true;
}

}  // namespace ssm
}  // namespace gdn
