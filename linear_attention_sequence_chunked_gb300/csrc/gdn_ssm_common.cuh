// Geometry and tile staging shared by the selective state space scan kernels.
//
// Per sequence and channel d (group g of B and C), with N states:
//   dt_t = softplus(dt_raw_t + dt_bias_d)          (or without the softplus)
//   h_t  = exp(dt_t A_dn) h_{t-1} + dt_t u_t B_tn,   y_t = sum_n C_tn h_tn + D_d u_t,
//   out_t = y_t silu(z_t)                           (or y_t without a gate).
// A warp walks a run of tokens for 32 channels (fewer for N > 16), a lane per
// channel with its states in registers, so that a row of every activation is
// one 64-byte access and nothing is exchanged between lanes.  Tokens come in
// tiles of kTile: copied to shared memory a tile ahead, B and C widened
// to fp32 once, dt and x = dt u formed once per element, and then four states
// at a time over the tile without a branch (a token after the end has
// dt = x = 0, which leaves the state as it is).  Arithmetic runs on pairs of
// states in register pairs.  Per token and channel that is N exponentials, 2 N
// paired operations and about 40 others: bound by instruction issue, not by HBM.
// Measured, 4 x 4096 x 2048 with N = 16: 266 us, 1.0 TB/s, 156 of them in the
// pass with the outputs and 110 in the one before it, which joins the segments.
// 156 us are 43 cycles per token and four states of a warp: 24 in the loop over
// states (by the 92 us that one group of four instead of four takes; 20 are
// register reads, since three different pairs cost an operation 3 cycles, next to
// 16 of the exponentials), the rest work per token and channel (softplus and SiLU
// 24 us, copies 8, and widening, dt u, the sums' ends and the stores).
#pragma once

#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {
namespace ssm {

using namespace mix;

constexpr int kWarps = 4;
// Tokens worked on at a time (4 x 4096 x 2048: 275 us by eight, 324 by four, 323
// by sixteen).
constexpr int kTile = kSsmChunk;
// Tiles of the forward in shared memory or on their way to it.  A third gains
// nothing (4 x 4096 x 2048: 263 us against 260) and from N = 128 on would leave
// room for eight warps per SM only (1 x 2048 x 1024: 224 us against 175).
constexpr int kStages = 2;

// Where a warp works: segment `slot` of the tokens, one block of CH channels.
struct Place {
    int n, b, t0, t1;         // sequence, batch row, its token range
    int s0, s1;               // the segment's tokens
    bool first, last;         // segment of its sequence
    int g, d0, nd;            // group, first channel, channels (<= CH)
    long long chunk0;         // the segment's first slot of the saved chunk states
    long long slot;           // the segment itself
    int before, after;        // segments of its sequence before and after it
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
    w.before = static_cast<int>(c);
    w.after = (w.t1 - w.s1 + seg - 1) / seg;
    const int per = p.D / p.G;
    w.g = block / blocks;
    const int off = block % blocks * CH;
    w.d0 = w.g * per + off;
    w.nd = min(CH, per - off);
    const long long base = p.cu_seqlens ? static_cast<long long>(w.t0 / kTile) + w.n
                                        : static_cast<long long>(w.n) * ((p.T + kTile - 1) / kTile);
    w.chunk0 = base + (w.s0 - w.t0) / kTile;
    return true;
}

// ---------------------------------------------------------------------------
// Lanes as channels: the geometry of the forward.
// ---------------------------------------------------------------------------


// A lane holds NL = min(N, 16) states of one channel, four at a time: group j
// of lane q of a channel's LPC = N / NL lanes is states 4 (j LPC + q) .. + 3, so
// that those lanes read neighbouring 16 bytes of a row of B.  CH channels per
// warp; with N <= 16 a lane is a channel, and a row of 32 channels is 64 bytes.
template <int N>
struct Lanes {
    static constexpr int NL = N < 16 ? N : 16;
    static constexpr int LPC = N / NL;
    static constexpr int CH = 32 / LPC;
    static constexpr int GR = NL / 4;
};

// Copies rows [0, nt) and columns [0, nc) of a kTile x ROW tile to shared
// memory, zeros elsewhere, asynchronously in pieces of up to PB bytes (every
// row's pieces aligned, nc a multiple of a piece).  PB = 0: element by element
// and at once, for 2-byte elements at odd places.
template <typename T, int ROW, int PB>
__device__ __forceinline__ void fill_tile(T* dst, const T* src, long long stride, int nt, int nc, int lane) {
    constexpr int row_bytes = ROW * static_cast<int>(sizeof(T));
    constexpr int CB = row_bytes < PB ? row_bytes : PB, CE = PB ? CB / static_cast<int>(sizeof(T)) : 1;
    constexpr int PER = ROW / CE, TOTAL = kTile * PER;
#pragma unroll
    for (int i = 0; i < (TOTAL + 31) / 32; ++i) {
        const int id = i * 32 + lane, row = id / PER, c = id % PER * CE;
        if (TOTAL % 32 != 0 && id >= TOTAL) continue;
        const bool ok = row < nt && c < nc;
        if constexpr (PB != 0) {
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + id * CE));
            const T* from = ok ? src + row * stride + c : src;
            const int bytes = ok ? CB : 0;
            if constexpr (CB == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(CB), "r"(bytes) : "memory");
        } else {
            dst[id] = ok ? __ldg(src + row * stride + c) : T(0);
        }
    }
}
// Whether fill_tile can take pieces of up to `piece` bytes of ROW elements from
// rows at p.
template <typename T, int ROW>
bool takes_pieces(const void* p, long long stride, int piece) {
    const int b = ROW * static_cast<int>(sizeof(T)) < piece ? ROW * static_cast<int>(sizeof(T)) : piece;
    return reinterpret_cast<uintptr_t>(p) % b == 0 && stride * static_cast<long long>(sizeof(T)) % b == 0;
}
// The widest pieces that every activation of a scan takes: 16 bytes, 4, or
// (bf16 at odd places) none.  4 x 4096 x 2048: 264, 286, 410 us.
template <typename T, int N>
int scan_pieces(const SsmArgs& a) {
    constexpr int CH = Lanes<N>::CH;
    for (const int b : {16, 4}) {
        const int w = CH * static_cast<int>(sizeof(T)) < b ? CH * static_cast<int>(sizeof(T)) : b;
        if (a.D / a.G * static_cast<long long>(sizeof(T)) % w == 0 && takes_pieces<T, CH>(a.u, a.u_stride, b) &&
            takes_pieces<T, CH>(a.dt, a.dt_stride, b) && (!a.z || takes_pieces<T, CH>(a.z, a.z_stride, b)) &&
            takes_pieces<T, N>(a.Bm, a.B_stride, b) && takes_pieces<T, N>(a.Cm, a.C_stride, b))
            return b;
    }
    return 0;
}

// kTile x N elements of B or C, as fp32.
template <typename T, int N>
__device__ __forceinline__ void widen_rows(const T* src, float* dst, int lane) {
    constexpr int PE = N * kTile / 32 < 16 / static_cast<int>(sizeof(T)) ? N * kTile / 32 : 16 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int i = 0; i < N * kTile / 32 / PE; ++i) {
        const int at = (i * 32 + lane) * PE;
        Raw<T, PE> r;
        if constexpr (sizeof(T) * PE == 16)
            *reinterpret_cast<uint4*>(r.w) = *reinterpret_cast<const uint4*>(src + at);
        else if constexpr (sizeof(T) * PE == 8)
            *reinterpret_cast<uint2*>(r.w) = *reinterpret_cast<const uint2*>(src + at);
        else
            r.w[0] = *reinterpret_cast<const uint32_t*>(src + at);
        float x[PE];
        unpack<T, PE>(r, x);
        if constexpr (PE >= 4) {
#pragma unroll
            for (int e = 0; e < PE; e += 4)
                *reinterpret_cast<float4*>(dst + at + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        } else {
            *reinterpret_cast<float2*>(dst + at) = make_float2(x[0], x[1]);
        }
    }
}

// Sums over the LPC lanes of a channel of v[t], t < W: value i of lane q is then
// the sum of token i LPC + q (of token q mod W where LPC > W).  Half as many
// values after each exchange.
template <int LPC, int W>
__device__ __forceinline__ void share_sums(float (&v)[W], int q) {
#pragma unroll
    for (int m = 1; m < LPC; m *= 2) {
        if (m < W) {
            const bool hi = (q & m) != 0;
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                if (i < W / (2 * m)) {
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

// The states of a lane, as register pairs, from or to a channel's N floats.
template <int N>
__device__ __forceinline__ void load_states(const float* p, int q, Two (&v)[Lanes<N>::NL / 2]) {
#pragma unroll
    for (int j = 0; j < Lanes<N>::GR; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(p + 4 * (j * Lanes<N>::LPC + q));
        v[2 * j] = two(x.x, x.y);
        v[2 * j + 1] = two(x.z, x.w);
    }
}
template <int N>
__device__ __forceinline__ void store_states(float* p, int q, const Two (&v)[Lanes<N>::NL / 2]) {
#pragma unroll
    for (int j = 0; j < Lanes<N>::GR; ++j) {
        float4 x;
        split(v[2 * j], x.x, x.y);
        split(v[2 * j + 1], x.z, x.w);
        *reinterpret_cast<float4*>(p + 4 * (j * Lanes<N>::LPC + q)) = x;
    }
}

// One launch; shared memory beyond 48 KB has to be asked for.
template <int WARPS, typename F>
cudaError_t launch_warps(F kernel, long long units, int bytes_per_warp, const SsmArgs& a, int blocks, cudaStream_t stream) {
    const int bytes = WARPS * bytes_per_warp;
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    kernel<<<static_cast<unsigned>((units + WARPS - 1) / WARPS), 32 * WARPS, bytes, stream>>>(a, blocks);
    return cudaGetLastError();
}

}  // namespace ssm
}  // namespace gdn
