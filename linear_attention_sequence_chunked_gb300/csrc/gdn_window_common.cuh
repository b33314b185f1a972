// What the kernels of window attention share: which keys a tile of queries
// looks at, tensor maps, and the tensor-memory accesses that the other
// tensor-core kernels do not need.
//
// Token i of a sequence sees j <= i with i - j < window or j < sinks.  Tiles
// are 128 tokens of one sequence; a tile of queries meets the blocks of 128
// keys from its first query's window to its last query, and before them, where
// those leave it out, the first few keys of block 0.
#pragma once

#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"
#include "gdn_tc_common.cuh"

namespace gdn {
namespace win {

using namespace sm100;
using tc::cvt_bf16x2;
using tc::smem_align_pad;

constexpr int kTile = 128;
constexpr int kSlab = kTile * 128;  // bytes of 128 rows of 64 channels, swizzled

// Products are issued by one lane (`on`) of a warp whose other lanes run along:
// what an instruction names (descriptors, columns) then stays in uniform registers
// from the start.  In a branch that only one lane takes every operand is moved
// there first, which took longer than the product (100 clocks for 128 x 128 x 16).
struct Issuer {
    uint32_t on;
    __device__ __forceinline__ Issuer() : on(elect_one() ? 1u : 0u) {}
    // D[tmem] (+)= A[smem] * B[smem]
    __device__ __forceinline__ void ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool more) const {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(more)), "r"(on)
            : "memory");
    }
    // D[tmem] (+)= A[tmem] * B[smem]: A holds two bf16 of a row per column
    __device__ __forceinline__ void ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool more) const {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(more)), "r"(on)
            : "memory");
    }
    // arrives on `bar` when everything issued so far has completed
    __device__ __forceinline__ void commit(uint32_t bar) const {
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
            "r"(on)
            : "memory");
    }
};
// The warp's value of x, which all its lanes have
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }
__device__ __forceinline__ int uniform(int x) { return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x))); }

// 32 lanes x 32 bits, 32 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Holds every use of r behind the wait before it (a load's registers are only
// there after tcgen05.wait::ld, which names none).
__device__ __forceinline__ void after_wait32(uint32_t* r) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]));
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Registers per thread of this warpgroup from here on.
template <int N>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The tile of queries [q0, q0 + kTile) of a sequence of n tokens: its blocks of
// keys are block 0 cut to the first keys if `first`, then lo .. hi.
struct Blocks {
    int first;     // columns of the block of first keys (a multiple of 32), or 0
    int lo, hi;
    __device__ __forceinline__ int count() const { return hi - lo + 1 + (first > 0); }
    __device__ __forceinline__ int start(int j) const { return first > 0 ? (j == 0 ? 0 : (lo + j - 1) * kTile) : (lo + j) * kTile; }
    __device__ __forceinline__ int width(int j) const { return first > 0 && j == 0 ? first : kTile; }
};
// `rows`: the queries from q0 on that count (two tiles share their blocks)
__device__ __forceinline__ Blocks blocks_of(int q0, int rows, int n, int window, int sinks) {
    Blocks b;
    const int last = min(q0 + rows, n) - 1;
    b.lo = q0 >= window ? (q0 - window + 1) / kTile : 0;
    b.hi = last / kTile;
    b.first = b.lo > 0 && sinks > 0 ? (sinks + 31) / 32 * 32 : 0;
    return b;
}

// Bit e of the result: row i sees key j0 + e (e < 32).
__device__ __forceinline__ uint32_t seen_bits(int i, int j0, int window, int sinks) {
    // keys up to i, from i - window + 1 on, or before `sinks`
    const auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
    return below(i + 1 - j0) & (~below(i - window + 1 - j0) | below(sinks - j0));
}

// Whether every row of the tile sees every key of [j0, j0 + width).
__device__ __forceinline__ bool all_seen(int q0, int rows, int j0, int width, int window, int sinks) {
    return j0 + width - 1 <= q0 && (q0 + rows - 1 - j0 < window || j0 + width <= sinks);
}

// A warp's wait, false where it ran out here or in another warp of the block.  Every
// branch hangs on a vote: what follows is uniform to the compiler, as the products'
// operands and the instructions that a whole warp issues need it, and a phase that
// is over costs 65 clocks (200 with each lane in a loop of its own).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
    for (uint32_t k = 0; k < 4000000u; ++k) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *stop != 0)) return false;
    }
    *stop = 1;
    return false;
}

// Zeros in the rows [from, to) of a swizzled tile: they belong to another sequence
// (or to nobody), and 0 times what they hold need not be zero.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from, int to, int lane) {
#pragma unroll
    for (int s = 0; s < D / 64; ++s)
        for (int o = from * 128 + lane * 16; o < to * 128; o += 512) *reinterpret_cast<uint4*>(tile + s * kSlab + o) = make_uint4(0, 0, 0, 0);
}

// A tile of one head by TMA, onto barrier `full`; one that ends behind its
// sequence (valid < kTile) goes through `tail` and is cleared from there on.
// Whole warp.  False: the wait ran out.
template <int D>
__device__ __forceinline__ bool load_tile(uint8_t* tile, const CUtensorMap* map, int head, int row, int valid, uint32_t full,
                                          uint32_t tail, int& tails, int lane) {
    const uint32_t on = valid < kTile ? tail : full;
    if (lane == 0) {
        mbar_arrive_expect_tx(on, kSlab * (D / 64));
#pragma unroll
        for (int s = 0; s < D / 64; ++s) tma_load_3d(smem_u32(tile + s * kSlab), map, 64 * s, head, row, on);
    }
    __syncwarp();
    if (valid < kTile) {
        if (!__all_sync(0xffffffffu, mbar_wait(tail, tails & 1))) return false;
        ++tails;
        clear_rows<D>(tile, valid, kTile, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
    }
    return true;
}

// The first tokens alone (`map` has boxes of that many), zeros behind them up to the
// block's width: nobody who looks at this block sees what lies there.  Into a place that
// nothing has used yet.  Whole warp.
template <int D>
__device__ __forceinline__ void load_first(uint8_t* tile, const CUtensorMap* map, int head, int row, int sinks, int width, uint32_t full,
                                           int lane) {
    clear_rows<D>(tile, sinks, width, lane);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        mbar_arrive_expect_tx(full, sinks * 128 * (D / 64));
#pragma unroll
        for (int s = 0; s < D / 64; ++s) tma_load_3d(smem_u32(tile + s * kSlab), map, 64 * s, head, row, full);
    }
    __syncwarp();
}

// {64 channels, 1 head, `box` tokens} of (tokens, heads, d) bf16, tokens `stride`
// elements apart: 128-byte swizzled rows.
inline bool make_heads_map(CUtensorMap* m, const void* base, long long tokens, long long stride, int heads, int d, int box_rows) {
    tc::EncodeTiledFn fn = tc::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace win
}  // namespace gdn
