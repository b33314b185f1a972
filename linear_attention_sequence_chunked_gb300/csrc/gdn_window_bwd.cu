// Attention with a sliding window and first tokens that stay visible: reverse
// mode.  With delta_i = dout_i . out_i (a kernel of its own),
//
//   P = exp(S - lse),  dP = dout V^T,  dS = P (dP - delta)
//   dV = P^T dout,  dK = scale dS^T Q,  dQ = scale dS K
//
// in two kernels, one that owns a tile of keys and one that owns a tile of
// queries, each of which forms S and dP for itself: two products more, but every
// gradient is summed by one block in one order, without atomics.
// All products run on the tensor cores, with operands that stay in tensor memory,
// written over the S and dP that they come from.  P is rounded to bf16 for dV, as
// in the forward.  dS goes in as two bf16 parts, what it rounds to and what is
// left: it is a difference that carries delta's error already, and one part alone
// left dQ and dK at 2.5e-3 to 2.7e-3 of L2, 1.6 times the rounding of the outputs
// themselves (2.0e-3 so, for two more products of nine).
//
// 16384 tokens, 16 / 4 heads of 128, window 2048 take 496 us for dK and dV, 357 for
// dQ, 25 for delta and 4 for the join.  A tile of dK and dV is 2560 clocks of
// products in some 3300: dS, dK over it, dP in its place and dS again are a chain
// (tensor memory holds S, dP and two accumulators, no second dP), and 544 blocks, the
// last tiles' of less work, in 3.6 rounds leave a fifth of the SMs' time idle: the
// tensor pipe is active in 76 % of the cycles in which an SM is, in 61 % of the
// kernel's.  A tile of dQ is 2048 in some
// 2950: dP has two places and K three, so that nothing waits but the elementwise
// work's own chain.  With eight warps for that work, one that issues all products
// and two places of K the two kernels took 519 and 439 us.
//
// The first tokens that stay visible are seen by every later query.  Their
// share beyond the reach of their own tile's window is cut into stretches of
// queries, one block each, whose fp32 sums a last kernel adds in order.  So are
// the shares of a key head's query heads where the keys alone leave SMs idle.
#include <algorithm>
#include <cmath>

#include "gdn_launch.h"
#include "gdn_window_common.cuh"

namespace gdn {

namespace {

using namespace win;

// Warps 0-15: elementwise work, 32 rows and a quarter of the columns each; 16:
// copies; 17 and 18: products.  Two warps issue them, so that what waits for one
// operand does not hold up the others.
constexpr int kElem = 16, kCopies = kElem, kProducts = kElem + 1, kThreads = 32 * (kElem + 3);

// A warp's 32 rows of W columns of an accumulator, times `mul`, as bf16 rows of
// `out`, rows `stride` elements apart, rows [first, rows) of them; through `mine`,
// the warp's own shared memory, in 16-byte chunks permuted so that neither side
// meets a bank twice.
template <int W>
__device__ __forceinline__ void store_rows(uint32_t t, float mul, uint8_t* mine, uint16_t* out, long long stride, int first,
                                           int rows, int lane) {
    constexpr int kChunks = W / 8, kMask = kChunks < 8 ? kChunks - 1 : 7;
#pragma unroll
    for (int g = 0; g < W; g += 32) {
        uint32_t o[32];
        tmem_ld32(t + g, o);
        tmem_ld_wait();
        after_wait32(o);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = cvt_bf16x2(__uint_as_float(o[8 * q + 2 * e]) * mul, __uint_as_float(o[8 * q + 2 * e + 1]) * mul);
            *reinterpret_cast<uint4*>(mine + lane * (W * 2) + (((g / 8 + q) ^ (lane & kMask)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __syncwarp();
#pragma unroll 4
    for (int k = 0; k < kChunks; ++k) {
        const int r = (k * 32 + lane) / kChunks, ch = (k * 32 + lane) % kChunks;
        const uint4 w = *reinterpret_cast<const uint4*>(mine + r * (W * 2) + ((ch ^ (r & kMask)) * 16));
        if (r >= first && r < rows) *reinterpret_cast<uint4*>(out + r * stride + ch * 8) = w;
    }
}

// A row's 32 values as bf16 pairs: 16 columns of the rounded values and 16 of what
// rounding left over.
__device__ __forceinline__ void store_split(uint32_t t, const float* x) {
    uint32_t w[32];
#pragma unroll
    for (int e = 0; e < 16; ++e) tc::split_bf16x2(x[2 * e], x[2 * e + 1], w[e], w[16 + e]);
    tmem_st32(t, w);
}

// ------------------------------------------------------------------ delta

// delta[b][h][t] = dout . out, D / 8 lanes to a row.
template <int D>
__global__ void __launch_bounds__(256) window_delta_kernel(const WindowArgs p) {
    constexpr int LANES = D / 8;
    const long long row = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / LANES;  // (token, head)
    const long long rows = p.tokens * p.H;
    const bool on = row < rows;
    const long long o = row * D + (threadIdx.x % LANES) * 8;
    const mix::Raw<uint16_t, 8> a = mix::load_raw<uint16_t, 8>(p.out + o, on ? 8 : 0), b = mix::load_raw<uint16_t, 8>(p.d_out + o, on ? 8 : 0);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(a.get(e), b.get(e), s);
#pragma unroll
    for (int m = LANES / 2; m > 0; m /= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (on && threadIdx.x % LANES == 0) {
        const long long tok = row / p.H, h = row % p.H;
        p.delta[(tok / p.T * p.H + h) * p.T + tok % p.T] = s;
    }
}

// ------------------------------------------------------------------ dK, dV

enum { kvIn = 0, kvQ = 1, kvQFree = 3, kvG = 5, kvGFree = 7, kvS = 9, kvP = 10, kvDP = 11, kvDS = 12, kvDone = 13, kvTail = 14, kvBars = 15 };

template <int D>
struct KvSmem {
    static constexpr int kTileBytes = kSlab * (D / 64);
    static constexpr int k = 0, v = kTileBytes, q = 2 * kTileBytes, g = 4 * kTileBytes, stats = 6 * kTileBytes;
    static constexpr int bars = stats + 2 * 2 * kTile * 4;
    static constexpr int misc = bars + kvBars * 8;
    static constexpr int total = misc + 32 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_g, const WindowArgs p) {
    using L = KvSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + smem_align_pad(smem_raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::misc);
    volatile int* stop = reinterpret_cast<volatile int*>(sm + L::misc + 4);
    float* stats = reinterpret_cast<float*>(sm + L::stats);  // [2][lse, delta][kTile]
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0) mix::check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);

    if (threadIdx.x == 32 * kCopies) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
        tma_prefetch_desc(&map_g);
    }
    // a tile of keys and the tiles of queries [qa, qb) that its block looks at:
    // those in reach of the tile's own window, or a stretch that sees only the
    // first tokens of block 0
    const int hk = blockIdx.x % p.Hk, piece = blockIdx.x / p.Hk % p.pieces;
    const int H0 = p.H / p.Hk * hk;  // the first of the key head's query heads
    const int g0 = p.H / p.Hk * piece / p.pieces, G = p.H / p.Hk * (piece + 1) / p.pieces - g0;  // this block's, from there
    long long slot = blockIdx.x / p.Hk / p.pieces;
    const int reach = (kTile - 1 + p.window - 1) / kTile + 1;  // tiles that a tile's keys reach, its own included
    const bool far = slot >= p.slots;
    int n, b, t0, t1;
    long long c;
    if (!mix::find_block(p.cu_seqlens, p.nseq, p.T, far ? p.far_tokens : kTile, far ? slot - p.slots : slot, p.err, n, c)) return;
    if (!mix::token_range(p.cu_seqlens, n, p.nseq, p.T, p.err, b, t0, t1)) return;
    const int len = t1 - t0, tiles = (len + kTile - 1) / kTile;
    if (c * (far ? p.far_tokens : kTile) >= len || (far && c == 0)) return;
    const int j0 = far ? 0 : static_cast<int>(c) * kTile;
    const int qa = far ? static_cast<int>(c) * reach : j0 / kTile;
    const int qb = min(tiles, qa + reach), nq = qb - qa;
    const int steps = nq * G;
    const long long row0 = static_cast<long long>(b) * p.T + t0;
    // rows whose sums are joined by a later kernel, and where they go (row j at j
    // times `pitch`, dV before dK `apart`): all where the heads are in pieces, else
    // the first tokens' of block 0
    int joined = 0;
    long long pitch = D, apart = static_cast<long long>(p.sinks) * D;
    float* part = nullptr;
    if (!far && p.pieces > 1) {
        joined = min(len, j0 + kTile);
        pitch = static_cast<long long>(p.Hk) * 2 * D;
        apart = D;
        part = p.head_part + ((piece * p.tokens + row0) * p.Hk + hk) * 2 * D;
    } else if (j0 == 0 && p.sinks > 0) {
        joined = min(p.sinks, len);
        const long long base = p.cu_seqlens ? static_cast<long long>(t0 / p.far_tokens) + n
                                            : static_cast<long long>(n) * (p.T > p.far_tokens ? (p.T + p.far_tokens - 1) / p.far_tokens : 1);
        part = p.far_part + (((base + (far ? c : 0)) * p.pieces + piece) * p.Hk + hk) * 2 * p.sinks * D;
    }

    if (warp == kProducts) {
        __syncwarp();  // (the checks before may have parted its lanes)
        tmem_alloc(smem_u32(tslot), 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kvBars; ++i) mbar_init(bar(i), i == kvP || i == kvDS ? kElem : i == kvGFree || i == kvGFree + 1 || i == kvDone ? 2 : 1);
        fence_mbar_init();
        *stop = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    constexpr uint32_t cS = 0, cDP = 128, cDV = 256, cDK = 384;
    const auto wait = [&](int i, int parity) { return warp_wait(bar(i), parity, stop); };

    if (warp == kCopies) {
        int tails = 0, lq = 0, lg = 0;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar(kvIn), 2 * L::kTileBytes);
            for (int s = 0; s < D / 64; ++s) {
                tma_load_3d(smem_u32(sm + L::k + s * kSlab), &map_k, 64 * s, hk, static_cast<int>(row0 + j0), bar(kvIn));
                tma_load_3d(smem_u32(sm + L::v + s * kSlab), &map_v, 64 * s, hk, static_cast<int>(row0 + j0), bar(kvIn));
            }
        }
        bool ok = true;
        for (int i = 0; i < steps && ok; ++i) {
            const int h = H0 + g0 + i / nq, i0 = (qa + i % nq) * kTile, st = i & 1, ph = ((i >> 1) & 1) ^ 1;
            const int row = static_cast<int>(row0 + i0), valid = min(kTile, len - i0);
            // (dout before Q, whose place is free later)
            ok = i < 2 || wait(kvGFree + st, ph);
            if (ok) ok = load_tile<D>(sm + L::g + st * L::kTileBytes, &map_g, h, row, valid, bar(kvG + st), bar(kvTail), tails, lane);
            if (!ok) break;
            lg = i + 1;
            ok = i < 2 || wait(kvQFree + st, ph);
            if (ok) ok = load_tile<D>(sm + L::q + st * L::kTileBytes, &map_q, h, row, valid, bar(kvQ + st), bar(kvTail), tails, lane);
            if (!ok) break;
            lq = i + 1;
        }
        if (!ok) *stop = 1;
        // every copy has landed before the block may leave
        mbar_wait(bar(kvIn), 0);
        for (int i = max(0, lq - 2); i < lq; ++i) mbar_wait(bar(kvQ + (i & 1)), (i >> 1) & 1);
        for (int i = max(0, lg - 2); i < lg; ++i) mbar_wait(bar(kvG + (i & 1)), (i >> 1) & 1);
        __syncwarp();
    } else if (warp >= kProducts) {
        const Issuer issue;
        const uint32_t base = uniform(smem_u32(sm)), tm = uniform(tmem), bar0 = base + L::bars;
        const int ns = uniform(steps);
        constexpr uint32_t id_s = idesc(kFmtBf16, 0, 0, 128, kTile), id_o = idesc(kFmtBf16, 0, 1, 128, D);
        // D[tmem] = rows (K-major) of `a` times rows of `b`
        const auto outer = [&](uint32_t d, uint32_t a, uint32_t b) {
            const uint64_t da = desc_sw128(base + a, 0, 1024), db = desc_sw128(base + b, 0, 1024);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint32_t o = ((s >> 2) * kSlab + (s & 3) * 32) >> 4;
                issue.ss(tm + d, da + o, db + o, id_s, s > 0);
            }
        };
        // D[tmem] += bf16 pairs at `a` (four times 16 columns, 32 apart) times rows of `b`
        const auto inner = [&](uint32_t d, uint32_t a, uint32_t b, bool more) {
            const uint64_t db = desc_sw128(base + b, kSlab, 1024);
#pragma unroll
            for (int s = 0; s < kTile / 16; ++s) issue.ts(tm + d, tm + a + (s >> 1) * 32 + (s & 1) * 8, db + s * 128, id_o, more || s > 0);
        };
        bool ok = wait(kvIn, 0);
        if (warp == kProducts) {  // S, and dV from P, which lies over it
            for (int i = 0; i < ns && ok; ++i) {
                const int st = i & 1, ph = (i >> 1) & 1;
                ok = wait(kvQ + st, ph);
                if (!ok) break;
                tc_fence_after();
                outer(cS, L::k, L::q + st * L::kTileBytes);
                issue.commit(bar0 + 8 * kvS);
                ok = wait(kvG + st, ph) && wait(kvP, i & 1);
                if (!ok) break;
                tc_fence_after();
                inner(cDV, cS, L::g + st * L::kTileBytes, i > 0);
                issue.commit(bar0 + 8 * (kvGFree + st));
            }
        } else {  // dP, and dK from dS, which lies over it
            const auto forms = [&](int i) {
                tc_fence_after();
                outer(cDP, L::v, L::g + (i & 1) * L::kTileBytes);
                issue.commit(bar0 + 8 * kvDP);
                issue.commit(bar0 + 8 * (kvGFree + (i & 1)));
            };
            ok = ok && wait(kvG, 0);
            if (ok) forms(0);
            for (int i = 0; i < ns && ok; ++i) {
                const int st = i & 1, nx = i + 1;
                ok = (nx == ns || wait(kvG + (nx & 1), (nx >> 1) & 1)) && wait(kvDS, i & 1);
                if (!ok) break;
                tc_fence_after();
                inner(cDK, cDP, L::q + st * L::kTileBytes, i > 0);
                inner(cDK, cDP + 16, L::q + st * L::kTileBytes, true);
                issue.commit(bar0 + 8 * (kvQFree + st));
                if (nx < ns) forms(nx);
            }
        }
        // every product has completed before the tensor memory is read or freed
        issue.commit(bar0 + 8 * kvDone);
        mbar_wait(bar(kvDone), 0);
        __syncwarp();
    } else {
        const int quarter = warp >> 2;  // which 32 queries of the tile
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + cS + 32 * quarter, tDP = tmem + lanes + cDP + 32 * quarter;
        const int j = j0 + 32 * (warp & 3) + lane;  // this thread's key
        const float c2 = p.scale * mix::kLog2e;
        const mix::Two cc = mix::two(c2, c2);
        // the tile's lse, in powers of two, and delta: a value each of 256 threads
        const auto stat = [&](int g, int x) {
            const int t = (qa + x) * kTile + static_cast<int>(threadIdx.x & (kTile - 1));
            if (g >= G || t >= len || quarter > 1) return 0.f;
            const long long o = (static_cast<long long>(b) * p.H + H0 + g0 + g) * p.T + t0 + t;
            return quarter ? p.delta[o] : p.lse[o] * mix::kLog2e;
        };
        int g = 0, x = 0;  // this step's head and tile
        float next = stat(0, 0);
        if (quarter < 2) stats[threadIdx.x] = next;
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            const float* ls = stats + (i & 1) * 2 * kTile;
            const int i0 = (qa + x) * kTile;  // the tile's first query
            if (++x == nq) x = 0, ++g;
            __syncwarp();  // (one lane arrived on the last step's barrier)
            tc::named_bar(1, 32 * kElem);
            next = stat(g, x);
            const float4* lse4 = reinterpret_cast<const float4*>(ls + 32 * quarter);
            const float4* del4 = reinterpret_cast<const float4*>(ls + kTile + 32 * quarter);
            // queries that see the key: from it on, up to its window's end or, a first token, the sequence's
            uint32_t see = 0xffffffffu;
            const bool masked = i0 < j0 + kTile || (i0 + kTile - 1 - j0 >= p.window) || i0 + kTile > len;
            if (masked) {
                const int from = j - i0 - 32 * quarter;
                const int to = (j < p.sinks ? len : static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(j) + p.window))) - i0 - 32 * quarter;
                const auto below = [](int k) { return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u; };
                see = below(to) & ~below(from);
            }
            ok = ok && wait(kvS, i & 1);
            if (!ok) continue;  // (the named barrier above stays in step)
            tc_fence_after();
            uint32_t s[32], pk[16];
            float pr[32];
            tmem_ld32(tS, s);
            tmem_ld_wait();
            after_wait32(s);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 l4 = lse4[e / 4];
                mix::split(mix::ex2_2(mix::fma2(mix::two(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), cc, mix::two(-l4.x, -l4.y))),
                           pr[e], pr[e + 1]);
                mix::split(mix::ex2_2(mix::fma2(mix::two(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), cc, mix::two(-l4.z, -l4.w))),
                           pr[e + 2], pr[e + 3]);
            }
            if (masked) {
#pragma unroll
                for (int e = 0; e < 32; ++e) pr[e] = (see >> e) & 1 ? pr[e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = cvt_bf16x2(pr[2 * e], pr[2 * e + 1]);
            tmem_st16(tS, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kvP));
            if (quarter < 2) stats[((i + 1) & 1) * 2 * kTile + threadIdx.x] = next;
            ok = wait(kvDP, i & 1);
            if (!ok) continue;
            tc_fence_after();
            tmem_ld32(tDP, s);
            tmem_ld_wait();
            after_wait32(s);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 d4 = del4[e / 4];
                const mix::Two a = mix::mul2(mix::two(pr[e], pr[e + 1]),
                                             mix::add2(mix::two(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), mix::two(-d4.x, -d4.y)));
                const mix::Two bb = mix::mul2(mix::two(pr[e + 2], pr[e + 3]),
                                              mix::add2(mix::two(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), mix::two(-d4.z, -d4.w)));
                mix::split(a, pr[e], pr[e + 1]);
                mix::split(bb, pr[e + 2], pr[e + 3]);
            }
            if (masked) {
#pragma unroll
                for (int e = 0; e < 32; ++e) pr[e] = (see >> e) & 1 ? pr[e] : 0.f;
            }
            store_split(tDP, pr);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kvDS));
        }
        if (ok && wait(kvDone, 0)) {
            tc_fence_after();
            // the first eight warps store dV, half of the channels each, the others dK
            constexpr int W = D / 2;
            const int to_k = quarter >> 1, ch = (quarter & 1) * W;
            const uint32_t t = tmem + lanes + (to_k ? cDK : cDV) + ch;
            const float mul = to_k ? p.scale : 1.f;
            const int r0 = 32 * (warp & 3);
            uint8_t* mine = sm + L::q + warp * 32 * (W * 2);
            if (part && j0 + r0 < joined) {
                float* to = part + to_k * apart + j * pitch + ch;
#pragma unroll
                for (int g = 0; g < W; g += 32) {
                    uint32_t o[32];
                    tmem_ld32(t + g, o);
                    tmem_ld_wait();
                    after_wait32(o);
                    if (j < joined) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(to + g + e) = make_float4(__uint_as_float(o[e]) * mul, __uint_as_float(o[e + 1]) * mul,
                                                                                 __uint_as_float(o[e + 2]) * mul, __uint_as_float(o[e + 3]) * mul);
                    }
                    __syncwarp();  // (the next loads take the whole warp)
                }
            }
            if (!far && joined < j0 + kTile)
                store_rows<W>(t, mul, mine, (to_k ? p.dk : p.dv) + ((row0 + j0 + r0) * p.Hk + hk) * D + ch, static_cast<long long>(p.Hk) * D,
                              joined - j0 - r0, min(32, len - j0 - r0), lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*stop && threadIdx.x == 0) record_error(p.err, kErrTimeout);
    if (warp == kProducts) tmem_dealloc(tmem, 512);
}

// The first tokens' dK and dV: the sums of their stretches, in order.
__global__ void __launch_bounds__(256) window_join_kernel(const WindowArgs p) {
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int d = static_cast<int>(id % p.d);
    long long rest = id / p.d;
    const int j = static_cast<int>(rest % p.sinks);
    rest /= p.sinks;
    const int which = static_cast<int>(rest % 2);
    rest /= 2;
    const int hk = static_cast<int>(rest % p.Hk);
    const long long n = rest / p.Hk;
    if (n >= p.nseq) return;
    int b, t0, t1;
    if (!mix::token_range(p.cu_seqlens, static_cast<int>(n), p.nseq, p.T, p.err, b, t0, t1)) return;
    if (j >= t1 - t0) return;
    const long long base = p.cu_seqlens ? static_cast<long long>(t0 / p.far_tokens) + n
                                        : n * (p.T > p.far_tokens ? (p.T + p.far_tokens - 1) / p.far_tokens : 1);
    const int parts = (t1 - t0 + p.far_tokens - 1) / p.far_tokens;
    float s = 0.f;
    const long long step = static_cast<long long>(p.Hk) * 2 * p.sinks * p.d;
    const float* from = p.far_part + base * step + ((static_cast<long long>(hk) * 2 + which) * p.sinks + j) * p.d + d;
    for (int c = 0; c < parts; c += 8) {  // eight on their way together, added in order
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = c + k < parts ? from[(c + k) * step] : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k];
    }
    (which ? p.dk : p.dv)[((static_cast<long long>(b) * p.T + t0 + j) * p.Hk + hk) * p.d + d] = f32_to_bf16(s);
}

// Every row's dK and dV where the heads are in pieces: the sums of the pieces and,
// for a first token, of its stretches, in order.  Four channels per thread.
__global__ void __launch_bounds__(256) window_sum_kernel(const WindowArgs p) {
    const long long id = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 4;
    const long long row = static_cast<long long>(p.Hk) * 2 * p.d;
    const long long tok = id / row;
    if (tok >= p.tokens) return;
    const int rest = static_cast<int>(id % row), d = rest % p.d, which = rest / p.d % 2, hk = rest / p.d / 2;
    int n = static_cast<int>(tok / p.T), b, t0, t1;
    if (p.cu_seqlens) {  // the last sequence that starts at or before the token
        int end = p.nseq - 1;
        n = 0;
        while (n < end) {
            const int mid = (n + end + 1) >> 1;
            if (p.cu_seqlens[mid] <= tok)
                n = mid;
            else
                end = mid - 1;
        }
    }
    if (!mix::token_range(p.cu_seqlens, n, p.nseq, p.T, p.err, b, t0, t1)) return;
    const long long j = tok - static_cast<long long>(b) * p.T - t0;
    if (j < 0 || j >= t1 - t0) return;  // a row of no sequence
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](const float* from) {
        const float4 v = *reinterpret_cast<const float4*>(from);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    };
    for (int k = 0; k < p.pieces; ++k) add(p.head_part + k * p.tokens * row + id);
    if (j < p.sinks) {
        const long long base = p.cu_seqlens ? static_cast<long long>(t0 / p.far_tokens) + n
                                            : static_cast<long long>(n) * (p.T > p.far_tokens ? (p.T + p.far_tokens - 1) / p.far_tokens : 1);
        const int parts = (t1 - t0 + p.far_tokens - 1) / p.far_tokens;
        for (int c = 1; c < parts; ++c)
            for (int k = 0; k < p.pieces; ++k) add(p.far_part + (((((base + c) * p.pieces + k) * p.Hk + hk) * 2 + which) * p.sinks + j) * p.d + d);
    }
    *reinterpret_cast<uint2*>((which ? p.dk : p.dv) + (tok * p.Hk + hk) * p.d + d) = make_uint2(cvt_bf16x2(s.x, s.y), cvt_bf16x2(s.z, s.w));
}

// ------------------------------------------------------------------ dQ

// K has three places: the next block's is loaded while dQ still reads the last one's.
enum { qIn = 0, qK = 1, qKFree = 4, qV = 7, qVFree = 9, qS = 11, qRead = 12, qDP = 13, qDS = 15, qDone = 17, qTail = 18, qBars = 19 };

template <int D>
struct QSmem {
    static constexpr int kTileBytes = kSlab * (D / 64);
    static constexpr int q = 0, g = kTileBytes, k = 2 * kTileBytes, v = 5 * kTileBytes, bars = 7 * kTileBytes;
    static constexpr int misc = bars + qBars * 8;
    static constexpr int total = misc + 32 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_k_first,
                     const WindowArgs p) {
    using L = QSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + smem_align_pad(smem_raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::misc);
    volatile int* stop = reinterpret_cast<volatile int*>(sm + L::misc + 4);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 32 * kCopies) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
        tma_prefetch_desc(&map_g);
        tma_prefetch_desc(&map_k_first);
    }
    const int h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
    const long long slot = p.slots - 1 - blockIdx.x / p.H;  // late tiles, with the most keys, first
    int n, b, t0, t1;
    long long c;
    if (!mix::find_block(p.cu_seqlens, p.nseq, p.T, kTile, slot, p.err, n, c)) return;
    if (!mix::token_range(p.cu_seqlens, n, p.nseq, p.T, p.err, b, t0, t1)) return;
    const int len = t1 - t0;
    if (c * kTile >= len) return;
    const int q0 = static_cast<int>(c) * kTile;
    const Blocks blk = blocks_of(q0, kTile, len, p.window, p.sinks);
    const int nblk = blk.count();
    const long long row0 = static_cast<long long>(b) * p.T + t0;

    if (warp == kProducts) {
        __syncwarp();  // (the checks before may have parted its lanes)
        tmem_alloc(smem_u32(tslot), 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < qBars; ++i) mbar_init(bar(i), i == qRead || i == qDS || i == qDS + 1 ? kElem : i == qDone ? 2 : 1);
        fence_mbar_init();
        *stop = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    constexpr uint32_t cS = 0, cDP = 128, cDQ = 384;  // dP alternates between 128 and 256
    const auto wait = [&](int i, int parity) { return warp_wait(bar(i), parity, stop); };

    if (warp == kCopies) {
        int tails = 0, lk = 0, lv = 0;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar(qIn), 2 * L::kTileBytes);
            for (int s = 0; s < D / 64; ++s) {
                tma_load_3d(smem_u32(sm + L::q + s * kSlab), &map_q, 64 * s, h, static_cast<int>(row0 + q0), bar(qIn));
                tma_load_3d(smem_u32(sm + L::g + s * kSlab), &map_g, 64 * s, h, static_cast<int>(row0 + q0), bar(qIn));
            }
        }
        bool ok = true;
        for (int j = 0; j < nblk && ok; ++j) {
            const int j0 = blk.start(j), st = j & 1, ph = ((j >> 1) & 1) ^ 1;
            const int row = static_cast<int>(row0 + j0);
            ok = j < 3 || wait(qKFree + j % 3, (j / 3 & 1) ^ 1);
            if (ok && blk.first > 0 && j == 0)  // of the first tokens' block they alone
                load_first<D>(sm + L::k, &map_k_first, hk, row, p.sinks, blk.first, bar(qK), lane);
            else if (ok)
                ok = load_tile<D>(sm + L::k + j % 3 * L::kTileBytes, &map_k, hk, row, min(kTile, len - j0), bar(qK + j % 3), bar(qTail), tails, lane);
            if (!ok) break;
            lk = j + 1;
            ok = j < 2 || wait(qVFree + st, ph);
            if (ok) ok = load_tile<D>(sm + L::v + st * L::kTileBytes, &map_v, hk, row, kTile, bar(qV + st), bar(qTail), tails, lane);
            if (!ok) break;
            lv = j + 1;
        }
        if (!ok) *stop = 1;
        mbar_wait(bar(qIn), 0);
        for (int j = max(0, lk - 3); j < lk; ++j) mbar_wait(bar(qK + j % 3), j / 3 & 1);
        for (int j = max(0, lv - 2); j < lv; ++j) mbar_wait(bar(qV + (j & 1)), (j >> 1) & 1);
        __syncwarp();
    } else if (warp >= kProducts) {
        const Issuer issue;
        const uint32_t base = uniform(smem_u32(sm)), tm = uniform(tmem), bar0 = base + L::bars;
        Blocks ub;
        ub.first = uniform(blk.first);
        ub.lo = uniform(blk.lo);
        ub.hi = uniform(blk.hi);
        const int nb = ub.count();
                constexpr uint32_t id_o = idesc(kFmtBf16, 0, 1, 128, D);
        const auto outer = [&](uint32_t d, uint32_t a, uint32_t b, int width) {
            const uint64_t da = desc_sw128(base + a, 0, 1024), db = desc_sw128(base + b, 0, 1024);
            const uint32_t id = idesc(kFmtBf16, 0, 0, 128, width);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint32_t o = ((s >> 2) * kSlab + (s & 3) * 32) >> 4;
                issue.ss(tm + d, da + o, db + o, id, s > 0);
            }
        };
        bool ok = wait(qIn, 0);
        if (warp == kProducts) {
            // S and dP: while one block's are turned into dS, the next block's are on their way
            for (int j = 0; j < nb && ok; ++j) {
                const int st = j & 1, ph = (j >> 1) & 1;
                ok = wait(qK + j % 3, j / 3 & 1) && wait(qV + st, ph) && (j == 0 || wait(qRead, (j - 1) & 1));
                if (!ok) break;
                tc_fence_after();
                outer(cS, L::q, L::k + j % 3 * L::kTileBytes, ub.width(j));
                issue.commit(bar0 + 8 * qS);
                // (dP goes over dS of the last block but one)
                ok = j < 2 || wait(qKFree + (j - 2) % 3, (j - 2) / 3 & 1);
                if (!ok) break;
                tc_fence_after();
                outer(cDP + 128 * st, L::g, L::v + st * L::kTileBytes, ub.width(j));
                issue.commit(bar0 + 8 * (qDP + st));  // (a barrier per buffer, for dS too: the next block's may follow before this one is looked at)
                issue.commit(bar0 + 8 * (qVFree + st));
            }
        } else {
            for (int j = 0; j < nb && ok; ++j) {
                const int st = j & 1;
                ok = wait(qDS + st, (j >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t k = desc_sw128(base + L::k + j % 3 * L::kTileBytes, kSlab, 1024);
                const int steps = ub.width(j) / 16;
#pragma unroll
                for (int s = 0; s < kTile / 16; ++s)
                    if (s < steps) issue.ts(tm + cDQ, tm + cDP + 128 * st + (s >> 1) * 32 + (s & 1) * 8, k + s * 128, id_o, (j | s) != 0);
#pragma unroll
                for (int s = 0; s < kTile / 16; ++s)
                    if (s < steps) issue.ts(tm + cDQ, tm + cDP + 128 * st + (s >> 1) * 32 + 16 + (s & 1) * 8, k + s * 128, id_o, true);
                issue.commit(bar0 + 8 * (qKFree + j % 3));
            }
        }
        issue.commit(bar0 + 8 * qDone);
        mbar_wait(bar(qDone), 0);
        __syncwarp();
    } else {
        const int quarter = warp >> 2;  // which 32 keys of the block
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + cS + 32 * quarter;
        const int i = q0 + 32 * (warp & 3) + lane;  // this thread's query
        const float c2 = p.scale * mix::kLog2e;
        float lse = 0.f, delta = 0.f;
        if (i < len) {
            const long long o = (static_cast<long long>(b) * p.H + h) * p.T + t0 + i;
            lse = p.lse[o] * mix::kLog2e;
            delta = p.delta[o];
        }
        const mix::Two cc = mix::two(c2, c2), ll = mix::two(-lse, -lse), dd = mix::two(-delta, -delta);
        bool ok = true;
        for (int j = 0; j < nblk; ++j) {
            ok = wait(qS, j & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tDP = tmem + lanes + cDP + 128 * (j & 1) + 32 * quarter;
            const int j0 = blk.start(j) + 32 * quarter;
            const bool any = blk.width(j) > 32 * quarter;  // a block of first tokens may be narrower
            uint32_t s[32];
            float pr[32];
            if (any) tmem_ld32(tS, s);
            tmem_ld_wait();
            after_wait32(s);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(qRead));
            const bool masked = blk.width(j) < kTile || !all_seen(q0, kTile, blk.start(j), kTile, p.window, p.sinks);
            const uint32_t see = masked && any ? seen_bits(i, j0, p.window, p.sinks) : 0xffffffffu;
#pragma unroll
            for (int e = 0; e < 32; e += 2)
                mix::split(mix::ex2_2(mix::fma2(mix::two(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), cc, ll)), pr[e], pr[e + 1]);
            ok = wait(qDP + (j & 1), (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (any) tmem_ld32(tDP, s);
            tmem_ld_wait();
            after_wait32(s);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const mix::Two a = mix::mul2(mix::two(pr[e], pr[e + 1]),
                                             mix::add2(mix::two(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), dd));
                mix::split(a, pr[e], pr[e + 1]);
            }
            if (masked) {
#pragma unroll
                for (int e = 0; e < 32; ++e) pr[e] = (see >> e) & 1 ? pr[e] : 0.f;
            }
            if (any) store_split(tDP, pr);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(qDS + (j & 1)));
        }
        if (ok && quarter < 2 && wait(qDone, 0)) {
            tc_fence_after();
            constexpr int W = D / 2;
            const int r0 = 32 * (warp & 3), ch = quarter * W;
            store_rows<W>(tmem + lanes + cDQ + ch, p.scale, sm + L::q + warp * 32 * (W * 2), p.dq + ((row0 + q0 + r0) * p.H + h) * D + ch,
                          static_cast<long long>(p.H) * D, 0, min(32, len - q0 - r0), lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*stop && threadIdx.x == 0) record_error(p.err, kErrTimeout);
    if (warp == kProducts) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const WindowArgs& a, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mg, mf;
    if (!make_heads_map(&mq, a.q, a.tokens, a.q_stride, a.H, D, kTile) ||
        !make_heads_map(&mk, a.k, a.tokens, a.k_stride, a.Hk, D, kTile) ||
        !make_heads_map(&mv, a.v, a.tokens, a.v_stride, a.Hk, D, kTile) ||
        !make_heads_map(&mg, a.d_out, a.tokens, static_cast<long long>(a.H) * D, a.H, D, kTile) ||
        !make_heads_map(&mf, a.k, a.tokens, a.k_stride, a.Hk, D, a.sinks > 0 ? a.sinks : kTile))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done_kv{0}, done_q{0};
    cudaError_t e = allow_once(window_dkv_kernel<D>, KvSmem<D>::total, false, done_kv);
    if (e != cudaSuccess) return e;
    e = allow_once(window_dq_kernel<D>, QSmem<D>::total, false, done_q);
    if (e != cudaSuccess) return e;
    const long long rows = a.tokens * a.H * (D / 8);
    window_delta_kernel<D><<<static_cast<unsigned>((rows + 255) / 256), 256, 0, stream>>>(a);
    window_dkv_kernel<D><<<static_cast<unsigned>((a.slots + a.far_slots) * a.Hk * a.pieces), kThreads, KvSmem<D>::total, stream>>>(mq, mk, mv, mg, a);
    if (a.pieces > 1) {
        const long long ids = a.tokens * a.Hk * 2 * D / 4;
        window_sum_kernel<<<static_cast<unsigned>((ids + 255) / 256), 256, 0, stream>>>(a);
    } else if (a.sinks > 0) {
        const long long ids = static_cast<long long>(a.nseq) * a.Hk * 2 * a.sinks * D;
        window_join_kernel<<<static_cast<unsigned>((ids + 255) / 256), 256, 0, stream>>>(a);
    }
    window_dq_kernel<D><<<static_cast<unsigned>(a.slots * a.H), kThreads, QSmem<D>::total, stream>>>(mq, mk, mv, mg, mf, a);
    return cudaGetLastError();
}

}  // namespace

// Pieces of a key head's query heads, each a block of its own: as many as find an
// SM.  More than one costs a pass over fp32 sums and reads the keys once a piece.
// Gradients in us, one piece and as the rule has it, of 16 query heads of 128:
// 1 x 512 tokens, 4 key heads (16 blocks in one piece) 44 and 34; 1 x 2048, 2 key
// heads (32) 237 and 99; 1 x 4096, 2 key heads, window 1024 (64) 195 and 144, where
// four pieces take 155.  With more blocks than half of the SMs it is one: 1 x 4096, 4
// key heads (128 blocks) take 136 in one, 161 in two.  (The rule does not look at how a
// last round of several fills: no other size beyond one round was measured.)  What
// pieces cost where there is little to share: 1 x 128 tokens, 4 key heads 21.6 and 24.
int window_pieces(long long slots, int H, int Hk) {
    const long long blocks = slots * Hk;
    return static_cast<int>(std::min<long long>(H / Hk, std::max(1ll, 152 / std::max(blocks, 1ll))));
}

cudaError_t launch_window_bwd(const WindowArgs& a, cudaStream_t stream) {
    return a.d == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace gdn
