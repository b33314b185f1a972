// Attention with a sliding window and first tokens that stay visible: forward.
//
//   out_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  s_ij = scale q_i . k_j
//
// A block of threads holds two tiles of 128 queries that share their keys: two
// heads of a group, or (groups of odd size) two consecutive tiles of a head.
// Per 128 keys and tile, S = Q K^T and O += P V are tensor-core products with
// their accumulators in tensor memory; each tile has a warpgroup, one thread per
// row, that turns S into P = 2^(S c - m) with a running maximum m and sum, and
// writes it over S as the bf16 operand of the second product.  P is rounded to
// bf16 (half a step of 2^-8, in random directions over a row's keys) because
// that is what the tensor cores multiply; the sum is of the unrounded values.
// While one tile's warpgroup works, the tensor cores run the other's products.
// O is rescaled only when a row's maximum has grown by more than 2^8, so most
// blocks leave it where it is; until then P is at most 2^8.
//
// 4 x 4096 tokens, 16 / 4 heads of 128, window 1024 take 136 us, 890 TFLOP/s.  What
// bounds it is one tile's chain: 128 keys of both tiles take 3300 clocks, in which
// the products need 2048 and a warpgroup some 1700 from the scores' arrival to P's.
// The chain cannot start on the next scores before P V is done, since P lies over
// them: tensor memory holds two tiles' S and O and no third.
//
// A masked place has P = 0, and 0 times a NaN or an infinity in V would not be
// zero: rows behind the sequence and behind the first tokens are cleared in V's tiles,
// and queries that end up non-finite by a value that they do not see are formed again.
#include <cmath>

#include "gdn_launch.h"
#include "gdn_mma.cuh"
#include "gdn_window_common.cuh"

namespace gdn {

namespace {

using namespace win;

constexpr int kThreads = 384;  // warps 0-3 and 4-7: a tile's rows each; 8: copies; 9: products
// The rows' warps hold 128 scores a thread: the registers that the third
// warpgroup does not need go to them.  The shares add up to what the block is
// launched with, which the launch checks.
constexpr int kRegsLaunch = 168, kRegsRows = 224, kRegsOther = 56;
static_assert(2 * kRegsRows + kRegsOther == 3 * kRegsLaunch, "register shares");
constexpr float kGrow = 8.f;

// mbarriers
enum { bQ = 0, bK = 2, bKFree = 4, bV = 6, bVFree = 8, bS = 10, bP = 12, bO = 14, bTail = 16, bDrain = 17, kBars = 18 };

template <int D>
struct Smem {
    static constexpr int kTileBytes = kSlab * (D / 64);
    static constexpr int q = 0, k = 2 * kTileBytes, v = 4 * kTileBytes, bars = 6 * kTileBytes;
    static constexpr int misc = bars + kBars * 8;
    static constexpr int total = misc + 32 + 1024;
};

__device__ __forceinline__ bool is_finite(uint32_t bf16) { return (bf16 & 0x7f80u) != 0x7f80u; }

// The rows of a warp (i0 + its lanes, those of `again`) whose outputs are not finite
// though their sums are: formed again from the keys that they see where it was a value
// that they do not see, in the blocks of keys [j0, end) of their tile.  What such a
// value can reach is looked up once for the warp.  Sixteen rows and sixteen keys at a
// time by products of registers, the newest keys first; where some row does not see
// some key, key by key, so that nothing is multiplied by a weight that is not there.
// Rows that see a NaN themselves in all of the channels in question stay as they are.
// So a NaN that is seen costs its readers little, and one that is not the rows of its
// tiles: 8192 tokens of 16 / 4 heads of 128 that see everything before them take 0.22
// ms, 0.25 where the first value is a NaN and 0.83 where one in the middle is (209 and
// 168 where every reader walked over its keys one by one).
template <int D>
__device__ __noinline__ void form_again(const WindowArgs& p, long long row0, int i0, int h, int j0, int end, uint32_t again) {
    constexpr int E = D / 32, CH = D / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, hk = h / (p.H / p.Hk), W = p.window, S = p.sinks;
    const uint16_t* const k0 = p.k + row0 * p.k_stride + hk * D;
    const uint16_t* const v0 = p.v + row0 * p.v_stride + hk * D;
    // of channels lane E + e: the last and the first place, of those that some row of
    // the warp does not see, with a value that is not finite
    int late[E], early[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        late[e] = -1;
        early[e] = 0x7fffffff;
    }
    const auto note = [&](int j, int* at) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const uint32_t x = mix::load_4(v0 + j * p.v_stride + lane * E + e, true);
            at[e] = is_finite(x) ? at[e] : j;
            at[e + 1] = is_finite(x >> 16) ? at[e + 1] : j;
        }
    };
#pragma unroll 8
    for (int j = i0 + 1; j < end; ++j) note(j, late);
#pragma unroll 8
    for (int j = min(i0 + 31, end - 1) - W; j >= max(j0, S); --j) note(j, early);

#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const uint32_t rows = again >> (16 * half) & 0xffffu;
        if (rows == 0) continue;
        // this lane's rows, and their outputs: bit 16 c + 8 e + k is channel 64 c + 8 (2 t + e) + k
        const int ia = i0 + 16 * half + g;
        const bool on[2] = {(rows >> g & 1) != 0, (rows >> (g + 8) & 1) != 0};
        uint16_t* const out = p.out + (row0 + ia) * (static_cast<long long>(p.H) * D) + h * D + 16 * t;
        const long long eight = 8ll * p.H * D;  // to the second row
        uint32_t reached[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint4 was[2];
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    was[x] = on[x] ? *reinterpret_cast<const uint4*>(out + x * eight + c * 64 + e * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int from = (64 * c + 8 * (2 * t + e) + k) / E;  // (its place there: k modulo E)
                    const int last = __shfl_sync(0xffffffffu, late[k % E], from), first = __shfl_sync(0xffffffffu, early[k % E], from);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int i = ia + 8 * x;
                        const uint32_t w = mma::word(was[x], k / 2);
                        if (!is_finite(k & 1 ? w >> 16 : w) && (last > i || first <= i - W)) reached[x] |= 1u << (16 * c + 8 * e + k);
                    }
                }
            }
        uint32_t todo = 0;
        const uint32_t any0 = __ballot_sync(0xffffffffu, reached[0] != 0), any1 = __ballot_sync(0xffffffffu, reached[1] != 0);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (any0 >> (4 * r) & 15u) todo |= 1u << r;
            if (any1 >> (4 * r) & 15u) todo |= 256u << r;
        }
        if (todo == 0) continue;
        const int imin = i0 + 16 * half + __ffs(todo) - 1, imax = i0 + 16 * half + 31 - __clz(todo);

        uint32_t q[CH][2][4];
        const uint16_t* const q0 = p.q + (row0 + ia) * p.q_stride + h * D;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint4 lo = mix::load_16(q0 + (c * 4 + t) * 8, on[0]), hi = mix::load_16(q0 + 8 * p.q_stride + (c * 4 + t) * 8, on[1]);
            q[c][0][0] = lo.x; q[c][0][1] = hi.x; q[c][0][2] = lo.y; q[c][0][3] = hi.y;
            q[c][1][0] = lo.z; q[c][1][1] = hi.z; q[c][1][2] = lo.w; q[c][1][3] = hi.w;
        }
        float o[D / 8][4];  // o[8 c + k][2 x + e]
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        const float c2 = p.scale * mix::kLog2e;
        // keys [lowest, imax] in strips from the last one on, then the first tokens before them
        const int lowest = max(0, imin - W + 1), firsts = min(S, lowest);
        const int near = (imax - lowest + 16) / 16, strips = near + (firsts + 15) / 16;
        bool same = false;
#pragma unroll 1
        for (int s = 0; s < strips && !same; ++s) {
            const int jb = s < near ? imax - 16 * s - 15 : 16 * (s - near);
            const int ja = s < near ? lowest : 0, jz = s < near ? imax + 1 : firsts;  // the strip's keys are among these
            const bool full = jb >= ja && jb + 16 <= min(jz, imin + 1) && (imax - jb < W || jb + 15 < S);
            float sc[2][4] = {};
            {
                uint4 kr[2][CH];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int j = jb + 8 * n + g;
#pragma unroll
                    for (int c = 0; c < CH; ++c) kr[n][c] = mix::load_16(k0 + j * p.k_stride + (c * 4 + t) * 8, j >= ja && j < jz);
                }
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma::bf16_16x8x16(sc[n], q[c][0], kr[n][c].x, kr[n][c].y);
                        mma::bf16_16x8x16(sc[n], q[c][1], kr[n][c].z, kr[n][c].w);
                    }
            }
            uint4 vr[4][CH / 2];  // (on their way while the scores become weights)
#pragma unroll
            for (int n = 0; n < 4; ++n) {  // keys 2 t, + 1, + 8, + 9
                const uint16_t* const v = v0 + (jb + 2 * t + (n & 1) + (n >> 1) * 8) * p.v_stride + g * 8;
#pragma unroll
                for (int c = 0; c < CH / 2; ++c) vr[n][c] = mix::load_16(v + c * 64, full);
            }
            const auto sees = [&](int x, int j) {
                const int i = ia + 8 * x;
                return j >= ja && j < jz && j <= i && (i - j < W || j < S);
            };
            float w[2][4];  // of rows g + 8 x and keys jb + 8 n + 2 t + e at 2 n + e
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        w[x][2 * n + e] = sees(x, jb + 8 * n + 2 * t + e) ? sc[n][2 * x + e] * c2 : -INFINITY;
                        top = fmaxf(top, w[x][2 * n + e]);
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = fmaxf(m[x], top), ms = mn == -INFINITY ? 0.f : mn;
                const float f = m[x] == mn ? 1.f : mix::ex2(m[x] - ms);
                m[x] = mn;
                l[x] *= f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[x][e] = mix::ex2(w[x][e] - ms);
                    l[x] += w[x][e];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][2 * x] *= f;
                    o[i][2 * x + 1] *= f;
                }
            }
            if (full) {
                uint32_t pa[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) pa[e >> 1][x + 2 * (e & 1)] = mma::tf32(w[x][e]);
#pragma unroll
                for (int c = 0; c < CH / 2; ++c)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // column g is channel 64 c + 8 g + k
                        const auto channel = [&](int n) { return mma::widen(mma::word(vr[n][c], k / 2), k & 1); };
                        mma::tf32_16x8x8(o[8 * c + k], pa[0], channel(0), channel(1));
                        mma::tf32_16x8x8(o[8 * c + k], pa[1], channel(2), channel(3));
                    }
            } else {
#pragma unroll
                for (int kk = 0; kk < 16; ++kk) {
                    const int j = jb + kk, from = (lane & 28) | (kk % 8) / 2, e4 = kk / 8 * 2 + (kk & 1);
                    const float w0 = __shfl_sync(0xffffffffu, w[0][e4], from), w1 = __shfl_sync(0xffffffffu, w[1][e4], from);
                    const bool see0 = sees(0, j), see1 = sees(1, j);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint4 v = mix::load_16(v0 + j * p.v_stride + c * 64 + 16 * t + 8 * e, see0 || see1);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float y = __uint_as_float(mma::widen(mma::word(v, k / 2), k & 1));
                                float* const to = o[8 * c + k];
                                to[e] = see0 ? fmaf(w0, y, to[e]) : to[e];
                                to[2 + e] = see1 ? fmaf(w1, y, to[2 + e]) : to[2 + e];
                            }
                        }
                }
            }
            if (s % 16 > 1) continue;  // (a look at all sums costs as much as a strip)
            same = true;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            same = same && (!(reached[x] >> (16 * c + 8 * e + k) & 1) || isnan(o[8 * c + k][2 * x + e]));
            same = __all_sync(0xffffffffu, same);
        }
        if (same) continue;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            const float r = 1.f / l[x];
            if (!(todo >> (g + 8 * x) & 1)) continue;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[k] = cvt_bf16x2(o[8 * c + 2 * k][2 * x + e] * r, o[8 * c + 2 * k + 1][2 * x + e] * r);
                    *reinterpret_cast<uint4*>(out + x * eight + c * 64 + e * 8) = make_uint4(y[0], y[1], y[2], y[3]);
                }
        }
        __syncwarp();
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_v_first, const WindowArgs p) {
    using L = Smem<D>;
    constexpr int kSlabs = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + smem_align_pad(smem_raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::misc);
    volatile int* stop = reinterpret_cast<volatile int*>(sm + L::misc + 4);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0) mix::check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);

    if (threadIdx.x == 256) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
        tma_prefetch_desc(&map_v_first);
    }

    // the two tiles: heads h and h + 1 of one tile, or two tiles of head h
    const int G = p.H / p.Hk, two_heads = G % 2 == 0;
    const int units = two_heads ? p.H / 2 : p.H;
    const long long slot = p.slots - 1 - blockIdx.x / units;  // late tiles, with the most keys, first
    const int unit = blockIdx.x % units;
    int n;
    long long c;
    int b, t0, t1;
    // every thread takes the same way out
    if (!mix::find_block(p.cu_seqlens, p.nseq, p.T, two_heads ? kTile : 2 * kTile, slot, p.err, n, c)) return;
    if (!mix::token_range(p.cu_seqlens, n, p.nseq, p.T, p.err, b, t0, t1)) return;
    const int len = t1 - t0;
    const long long at = c * (two_heads ? kTile : 2 * kTile);
    if (at >= len) return;
    const int q0 = static_cast<int>(at);
    const int h0 = two_heads ? 2 * unit : unit, hk = h0 / G;
    const int rows = two_heads ? kTile : 2 * kTile;
    const bool second = two_heads || q0 + kTile < len;
    const Blocks blk = blocks_of(q0, rows, len, p.window, p.sinks);
    const int nblk = blk.count();
    const long long row0 = static_cast<long long>(b) * p.T + t0;  // the sequence's first row

    if (warp == 9) {
        __syncwarp();  // (the checks before may have parted its lanes)
        tmem_alloc(smem_u32(tslot), 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i >= bP && i < bO ? 4 : 1);
        fence_mbar_init();
        *stop = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    // S (then P) of tile x at column 128 x, O at 256 + 128 x
    const auto wait = [&](int i, int parity) { return warp_wait(bar(i), parity, stop); };

    if (warp >= 8) {
        registers_down<kRegsOther>();
        if (warp == 8) {
            if (lane == 0) {
                for (int x = 0; x < (second ? 2 : 1); ++x) {
                    mbar_arrive_expect_tx(bar(bQ + x), L::kTileBytes);
                    for (int s = 0; s < kSlabs; ++s)
                        tma_load_3d(smem_u32(sm + L::q + x * L::kTileBytes + s * kSlab), &map_q, 64 * s, h0 + (two_heads ? x : 0),
                                    static_cast<int>(row0 + q0 + (two_heads ? 0 : x * kTile)), bar(bQ + x));
                }
            }
            int loaded_k = 0, loaded_v = 0, tails = 0;
            bool ok = true;
            for (int j = 0; j < nblk; ++j) {
                const int st = j & 1, ph = ((j >> 1) & 1) ^ 1;
                const int row = static_cast<int>(row0 + blk.start(j));
                ok = j < 2 || wait(bKFree + st, ph);
                // K's rows behind the sequence are masked, V's have to be zeros
                if (ok) ok = load_tile<D>(sm + L::k + st * L::kTileBytes, &map_k, hk, row, kTile, bar(bK + st), bar(bTail), tails, lane);
                if (!ok) break;
                loaded_k = j + 1;
                ok = j < 2 || wait(bVFree + st, ph);
                if (ok && blk.first > 0 && j == 0)  // of the first tokens' block they alone
                    load_first<D>(sm + L::v + st * L::kTileBytes, &map_v_first, hk, row, p.sinks, blk.first, bar(bV + st), lane);
                else if (ok)
                    ok = load_tile<D>(sm + L::v + st * L::kTileBytes, &map_v, hk, row, min(kTile, len - blk.start(j)), bar(bV + st),
                                      bar(bTail), tails, lane);
                if (!ok) break;
                loaded_v = j + 1;
            }
            if (!ok) *stop = 1;
            // every copy has landed before the block may leave
            for (int x = 0; x < (second ? 2 : 1); ++x) mbar_wait(bar(bQ + x), 0);
            for (int j = max(0, loaded_k - 2); j < loaded_k; ++j) mbar_wait(bar(bK + (j & 1)), (j >> 1) & 1);
            for (int j = max(0, loaded_v - 2); j < loaded_v; ++j) mbar_wait(bar(bV + (j & 1)), (j >> 1) & 1);
            __syncwarp();
        } else if (warp == 9) {
            const Issuer issue;
            const uint32_t base = uniform(smem_u32(sm)), tm = uniform(tmem), bar0 = base + L::bars;
            Blocks ub;
            ub.first = uniform(blk.first);
            ub.lo = uniform(blk.lo);
            ub.hi = uniform(blk.hi);
            const int nb = ub.count(), tiles = uniform(second ? 2 : 1);
            const auto scores = [&](int j, int x) {  // S of tile x with block j
                const uint64_t q = desc_sw128(base + L::q + x * L::kTileBytes, 0, 1024), k = desc_sw128(base + L::k + (j & 1) * L::kTileBytes, 0, 1024);
                const uint32_t id = idesc(kFmtBf16, 0, 0, 128, ub.width(j));
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t o = ((s >> 2) * kSlab + (s & 3) * 32) >> 4;
                    issue.ss(tm + 128 * x, q + o, k + o, id, s > 0);
                }
                issue.commit(bar0 + 8 * (bS + x));
            };
            bool ok = true;
            for (int x = 0; x < tiles && ok; ++x) {
                ok = wait(bQ + x, 0) && wait(bK, 0);
                if (!ok) break;
                tc_fence_after();
                scores(0, x);
            }
            if (ok) issue.commit(bar0 + 8 * bKFree);
            constexpr uint32_t id_o = idesc(kFmtBf16, 0, 1, 128, D);
            for (int j = 0; j < nb && ok; ++j) {
                const int steps = ub.width(j) / 16;
                // the copies first: they were there before P
                ok = wait(bV + (j & 1), (j >> 1) & 1) && (j + 1 == nb || wait(bK + ((j + 1) & 1), ((j + 1) >> 1) & 1));
                for (int x = 0; x < tiles && ok; ++x) {
                    ok = wait(bP + x, j & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v = desc_sw128(base + L::v + (j & 1) * L::kTileBytes, kSlab, 1024);
#pragma unroll
                    for (int s = 0; s < kTile / 16; ++s)
                        if (s < steps) issue.ts(tm + 256 + 128 * x, tm + 128 * x + 8 * s, v + s * 128, id_o, (j | s) != 0);
                    if (j + 1 == nb) issue.commit(bar0 + 8 * (bO + x));
                    if (j + 1 < nb) {
                        scores(j + 1, x);
                        if (x == tiles - 1) issue.commit(bar0 + 8 * (bKFree + ((j + 1) & 1)));
                    }
                    if (x == tiles - 1) issue.commit(bar0 + 8 * (bVFree + (j & 1)));
                }
            }
            // every product has completed before the tensor memory is freed
            issue.commit(bar0 + 8 * bDrain);
            mbar_wait(bar(bDrain), 0);
            __syncwarp();
        }
    } else {
        registers_up<kRegsRows>();
        if (warp < 4 || second) {
            const int x = warp >> 2;
            const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
            const uint32_t tS = tmem + lanes + 128 * x, tO = tmem + lanes + 256 + 128 * x;
            const int qx = q0 + (two_heads ? 0 : x * kTile);  // this tile's first query
            const int i = qx + 32 * (warp & 3) + lane;        // this thread's
            const float c2 = p.scale * mix::kLog2e;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < nblk; ++j) {
                ok = wait(bS + x, j & 1);
                if (!ok) break;
                tc_fence_after();
                const int j0 = blk.start(j), width = blk.width(j);
                uint32_t s[kTile];
#pragma unroll
                for (int g = 0; g < kTile; g += 32)
                    if (g < width) tmem_ld32(tS + g, s + g);
                tmem_ld_wait();
#pragma unroll
                for (int g = 0; g < kTile; g += 32) after_wait32(s + g);
                if (width < kTile || !all_seen(qx, kTile, j0, width, p.window, p.sinks)) {
#pragma unroll
                    for (int g = 0; g < kTile; g += 32) {
                        const uint32_t see = g < width ? seen_bits(i, j0 + g, p.window, p.sinks) : 0;
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[g + e] = (see >> e) & 1 ? s[g + e] : 0xff800000u;
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < kTile; e += 8)
#pragma unroll
                    for (int g = 0; g < 4; ++g) top[g] = max3(top[g], __uint_as_float(s[e + 2 * g]), __uint_as_float(s[e + 2 * g + 1]));
                const float mb = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c2;
                if (__any_sync(0xffffffffu, mb > m + kGrow && i < len)) {  // (rows behind the sequence move nobody's maximum)
                    const float mn = fmaxf(m, mb);
                    const float f = m == -INFINITY ? 0.f : mix::ex2(m - mn);
                    m = mn;
                    l *= f;
                    if (j > 0) {  // the scores came behind the last product into O
#pragma unroll
                        for (int g = 0; g < D; g += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + g, o);
                            tmem_ld_wait();
                            after_wait32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(tO + g, o);
                        }
                    }
                }
                const float ms = m == -INFINITY ? 0.f : -m;
                const mix::Two cc = mix::two(c2, c2), mm = mix::two(ms, ms);
                mix::Two sum[2] = {mix::two(0.f, 0.f), mix::two(0.f, 0.f)};
#pragma unroll
                for (int g = 0; g < kTile; g += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a, bb;
                        const mix::Two y =
                            mix::ex2_2(mix::fma2(mix::two(__uint_as_float(s[g + e]), __uint_as_float(s[g + e + 1])), cc, mm));
                        sum[(e >> 1) & 1] = mix::add2(sum[(e >> 1) & 1], y);
                        mix::split(y, a, bb);
                        pk[e / 2] = cvt_bf16x2(a, bb);
                    }
                    if (g < width) tmem_st16(tS + g / 2, pk);
                }
                float a, bb;
                mix::split(mix::add2(sum[0], sum[1]), a, bb);
                l += a + bb;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bP + x));
            }
            if (ok && wait(bO + x, 0)) {
                tc_fence_after();
                const int h = h0 + (two_heads ? x : 0);
                const float r = 1.f / l;
                const float lse = (m + log2f(l)) * 0.6931471805599453f;
                // through this warp's own 32 rows of Q's buffer (its products are done):
                // 16-byte chunks, permuted so that neither side meets a bank twice
                uint8_t* mine = sm + L::q + x * L::kTileBytes + (warp & 3) * 32 * (D * 2);
                float bad = 0.f;
#pragma unroll
                for (int g = 0; g < D; g += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + g, o);
                    tmem_ld_wait();
                    after_wait32(o);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float u = __uint_as_float(o[8 * q + 2 * e]) * r, v = __uint_as_float(o[8 * q + 2 * e + 1]) * r;
                            bad = fmaf(u, 0.f, fmaf(v, 0.f, bad));
                            w[e] = cvt_bf16x2(u, v);
                        }
                        *reinterpret_cast<uint4*>(mine + lane * (D * 2) + (((g / 8 + q) ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
                constexpr int kChunks = D / 8;  // of 16 bytes in a row
#pragma unroll 4
                for (int k = 0; k < kChunks; ++k) {
                    const int r2 = (k * 32 + lane) / kChunks, ch = (k * 32 + lane) % kChunks;
                    const int t = qx + 32 * (warp & 3) + r2;
                    const uint4 w = *reinterpret_cast<const uint4*>(mine + r2 * (D * 2) + ((ch ^ (r2 & 7)) * 16));
                    if (t < len)
                        *reinterpret_cast<uint4*>(p.out + (row0 + t) * (static_cast<long long>(p.H) * D) + h * D + ch * 8) = w;
                }
                __syncwarp();
                // (a sum that is not finite: its own scores)
                const uint32_t again = __ballot_sync(0xffffffffu, bad != 0.f && l < INFINITY && i < len);
                if (again) form_again<D>(p, row0, qx + 32 * (warp & 3), h, blk.lo * kTile, min(len, (blk.hi + 1) * kTile), again);
                if (p.lse && i < len)  // (row of the batch, head, token)
                    p.lse[(static_cast<long long>(b) * p.H + h) * p.T + t0 + i] = lse;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*stop && threadIdx.x == 0) record_error(p.err, kErrTimeout);
    if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const WindowArgs& a, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mf;
    const long long tokens = a.cu_seqlens ? a.T : static_cast<long long>(a.nseq) * a.T;
    if (!make_heads_map(&mq, a.q, tokens, a.q_stride, a.H, D, kTile) ||
        !make_heads_map(&mk, a.k, tokens, a.k_stride, a.Hk, D, kTile) ||
        !make_heads_map(&mv, a.v, tokens, a.v_stride, a.Hk, D, kTile) ||
        !make_heads_map(&mf, a.v, tokens, a.v_stride, a.Hk, D, a.sinks > 0 ? a.sinks : kTile))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    if (!done.load(std::memory_order_acquire)) {
        cudaFuncAttributes at;
        const cudaError_t e = cudaFuncGetAttributes(&at, window_fwd_kernel<D>);
        if (e != cudaSuccess) return e;
        if (at.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the shares would wait for registers that are not there
    }
    const cudaError_t e = allow_once(window_fwd_kernel<D>, Smem<D>::total, false, done);
    if (e != cudaSuccess) return e;
    const int units = (a.H / a.Hk) % 2 == 0 ? a.H / 2 : a.H;
    window_fwd_kernel<D><<<static_cast<unsigned>(a.slots * units), kThreads, Smem<D>::total, stream>>>(mq, mk, mv, mf, a);
    return cudaGetLastError();
}

}  // namespace

// Two heads read their keys once for both and end at the same one.  In us against
// two tiles of a head: 4 x 4096 tokens, 16 / 4 heads, window 1024 134 and 148; 8 x
// 512, 16 / 2 heads 23 and 26; one tile of 16 / 4 heads 8.2 and 7.2, where twice the
// blocks run.  One warp issues the products of both: two that do make every product
// of one tile wait for half of the other's (177 us instead of 138).
int window_fwd_rows(int H, int Hk) { return (H / Hk) % 2 == 0 ? win::kTile : 2 * win::kTile; }

cudaError_t launch_window_fwd(const WindowArgs& a, cudaStream_t stream) {
    return a.d == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace gdn
