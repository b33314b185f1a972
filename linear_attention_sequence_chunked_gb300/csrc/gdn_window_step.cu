// Attention with a sliding window, one token per row on a cache of sinks +
// window rows, and the filling of such a cache from prompts.
//
// The cache keeps token p in row p while p < sinks and in row sinks + (p -
// sinks) % window from there on, so after the token at position p its first
// min(p + 1, rows) rows are exactly the keys that the token sees, in an order
// that a softmax does not care about.
//
// The step is bound by reading the cache once.  A warp takes 16 rows at a time
// for up to 16 query heads of a group: S = Q K^T and O += P V are 16 x 8 x 16
// register products (mma.sync: one query per head leaves the 128 rows of a
// tensor-memory product empty, and nothing here waits for arithmetic).  The
// channels are numbered so that both operands are what 16-byte loads of the
// rows bring, without shared memory: in the first product a channel's place
// does not matter as long as Q and K agree, in the second a lane's 16 bytes of V
// are its column in eight products.  The warps of a block, and the blocks of a
// cluster where the rows alone leave SMs idle, join their (maximum, sum, O) in a
// fixed order through (distributed) shared memory.
#include <algorithm>
#include <cmath>

#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kWarps = 4;
constexpr int kKeys = 16;  // of a warp's step

__device__ __forceinline__ void mma_16x8x16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pair_of(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float load_remote(const float* p, uint32_t rank) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t from;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from) : "memory");
    return v;
}

template <int D>
struct Joined {
    float o[kWarps][16][D + 4];
    float m[kWarps][16], l[kWarps][16];
    float jo[16][D], jm[16], jl[16];  // the block's
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps) window_step_kernel(const WindowStepArgs p) {
    constexpr int CH = D / 32;  // 16-byte chunks of a row per lane
    extern __shared__ __align__(16) unsigned char smem[];
    Joined<D>& sm = *reinterpret_cast<Joined<D>*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int C = p.cluster;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int G = p.H / p.Hk, sets = (G + 15) / 16;
    long long unit = blockIdx.x / C;
    const int set = static_cast<int>(unit % sets);
    unit /= sets;
    const int hk = static_cast<int>(unit % p.Hk);
    const long long b = unit / p.Hk;
    const int h0 = hk * G + set * 16, heads = min(16, G - set * 16);
    long long slot = p.slots ? p.slots[b] : b;
    if (p.slots && slot >= p.S) record_error(p.err, kErrBadSlot);
    const int pos = p.lengths[b];
    const bool on = slot >= 0 && slot < p.S && pos >= 0;
    if (!on) slot = 0;
    const int at = !on || pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.window;
    const int rows = !on ? 0 : pos >= p.rows ? p.rows : pos + 1;

    const long long stride = static_cast<long long>(p.Hk) * D;
    uint16_t* kc = p.k_cache + slot * p.rows * stride + hk * D;
    uint16_t* vc = p.v_cache + slot * p.rows * stride + hk * D;
    const uint16_t* kn = p.k + b * p.k_stride + hk * D;
    const uint16_t* vn = p.v + b * p.v_stride + hk * D;
    if (on && set == 0 && rank == 0 && threadIdx.x < D / 4) {  // the token's own row (read from k and v below)
        const int c = threadIdx.x % (D / 8);
        if (threadIdx.x < D / 8)
            *reinterpret_cast<uint4*>(kc + at * stride + 8 * c) = *reinterpret_cast<const uint4*>(kn + 8 * c);
        else
            *reinterpret_cast<uint4*>(vc + at * stride + 8 * c) = *reinterpret_cast<const uint4*>(vn + 8 * c);
    }

    // Q: rows g and g + 8 of the product, this lane's chunks t, t + 4, ...
    uint32_t q[2 * CH][4];
    const uint16_t* qp = p.q + b * p.q_stride + static_cast<long long>(h0) * D;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const uint4 lo = load_16(qp + g * D + (c * 4 + t) * 8, g < heads), hi = load_16(qp + (g + 8) * D + (c * 4 + t) * 8, g + 8 < heads);
        q[2 * c][0] = lo.x; q[2 * c][1] = hi.x; q[2 * c][2] = lo.y; q[2 * c][3] = hi.y;
        q[2 * c + 1][0] = lo.z; q[2 * c + 1][1] = hi.z; q[2 * c + 1][2] = lo.w; q[2 * c + 1][3] = hi.w;
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const float c2 = p.scale * kLog2e;

    const int strips = (rows + kKeys - 1) / kKeys, per = (strips + C - 1) / C;
    const int s1 = min(strips, static_cast<int>(rank + 1) * per);
    for (int s = static_cast<int>(rank) * per + warp; s < s1; s += kWarps) {
        const int r0 = s * kKeys;
        uint4 kr[2][CH], vr[4][CH / 2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {  // keys r0 + 8 n + g
            const int r = r0 + 8 * n + g;
            const uint16_t* k = r == at ? kn : kc + r * stride;
#pragma unroll
            for (int c = 0; c < CH; ++c) kr[n][c] = load_16(k + (c * 4 + t) * 8, r < rows);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {  // keys r0 + 2 t, + 1, + 8, + 9
            const int r = r0 + 2 * t + (n & 1) + (n >> 1) * 8;
            const uint16_t* v = r == at ? vn : vc + r * stride;
#pragma unroll
            for (int c = 0; c < CH / 2; ++c) vr[n][c] = load_16(v + c * 64 + g * 8, r < rows);
        }
        float sc[2][4] = {};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                mma_16x8x16(sc[n], q[2 * c], kr[n][c].x, kr[n][c].y);
                mma_16x8x16(sc[n], q[2 * c + 1], kr[n][c].z, kr[n][c].w);
            }
        // sc[n][e]: query row g + 8 (e / 2), key r0 + 8 n + 2 t + e % 2
        uint32_t pa[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float v[4], top = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    v[2 * n + e] = r0 + 8 * n + 2 * t + e < rows ? sc[n][2 * x + e] * c2 : -INFINITY;
                    top = fmaxf(top, v[2 * n + e]);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float mn = fmaxf(m[x], top), ms = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(m[x] - ms);
            m[x] = mn;
            l[x] *= f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = ex2(v[e] - ms);
                l[x] += v[e];
            }
            pa[x] = pair_of(v[0], v[1]);
            pa[x + 2] = pair_of(v[2], v[3]);
            if (f != 1.f) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][2 * x] *= f;
                    o[i][2 * x + 1] *= f;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CH / 2; ++c) {
            const uint32_t w[4][4] = {{vr[0][c].x, vr[0][c].y, vr[0][c].z, vr[0][c].w}, {vr[1][c].x, vr[1][c].y, vr[1][c].z, vr[1][c].w},
                                      {vr[2][c].x, vr[2][c].y, vr[2][c].z, vr[2][c].w}, {vr[3][c].x, vr[3][c].y, vr[3][c].z, vr[3][c].w}};
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // column g is channel 64 c + 8 g + j
                const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                mma_16x8x16(o[8 * c + j], pa, __byte_perm(w[0][j / 2], w[1][j / 2], sel), __byte_perm(w[2][j / 2], w[3][j / 2], sel));
            }
        }
    }
    // a row's sum lies across its four lanes
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (t == 0) {
            sm.m[warp][g + 8 * x] = m[x];
            sm.l[warp][g + 8 * x] = l[x];
        }
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sm.o[warp][g + 8 * (e >> 1)][(i / 8) * 64 + (2 * t + (e & 1)) * 8 + i % 8] = o[i][e];
    __syncthreads();
    // the block's warps
    for (int i = threadIdx.x; i < heads * D; i += 32 * kWarps) {
        const int r = i / D, d = i % D;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][r]);
        const float ms = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(sm.m[w][r] - ms);
            sum = fmaf(sm.l[w][r], f, sum);
            acc = fmaf(sm.o[w][r][d], f, acc);
        }
        if (C > 1) {
            sm.jo[r][d] = acc;
            if (d == 0) {
                sm.jm[r] = mx;
                sm.jl[r] = sum;
            }
        } else {
            p.out[(b * p.H + h0 + r) * D + d] = f32_to_bf16(on ? acc / sum : 0.f);
        }
    }
    if (C == 1) return;
    cluster_sync();
    const int share = (heads * D + C - 1) / C, last = min(heads * D, static_cast<int>(rank + 1) * share);
    for (int i = static_cast<int>(rank) * share + threadIdx.x; i < last; i += 32 * kWarps) {
        const int r = i / D, d = i % D;
        float mx = -INFINITY;
        for (int c = 0; c < C; ++c) mx = fmaxf(mx, load_remote(&sm.jm[r], c));
        const float ms = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f, acc = 0.f;
        for (int c = 0; c < C; ++c) {
            const float f = ex2(load_remote(&sm.jm[r], c) - ms);
            sum = fmaf(load_remote(&sm.jl[r], c), f, sum);
            acc = fmaf(load_remote(&sm.jo[r][d], c), f, acc);
        }
        p.out[(b * p.H + h0 + r) * D + d] = f32_to_bf16(on ? acc / sum : 0.f);
    }
    cluster_sync();  // the others may still read here
}

// The rows of a cache that a prompt leaves behind, 16 bytes per thread.
__global__ void __launch_bounds__(256) window_fill_kernel(const WindowFillArgs p) {
    const int chunks = p.Hk * p.d / 8, rows = p.sinks + p.window;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const int n = blockIdx.y;
    int b, t0, t1;
    if (!token_range(p.cu_seqlens, n, p.nseq, p.T, p.err, b, t0, t1)) return;
    long long slot = p.slots ? p.slots[n] : n;
    if (slot >= p.S) {
        record_error(p.err, kErrBadSlot);
        return;
    }
    if (slot < 0) return;
    const int len = t1 - t0;
    const long long ids = static_cast<long long>(min(len, rows)) * chunks;
    for (long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; id < ids; id += static_cast<long long>(gridDim.x) * 256) {
        const int r = static_cast<int>(id / chunks), c = static_cast<int>(id % chunks);
        // the last token that row r holds
        const int tok = r < p.sinks ? r : r + (len - 1 - r) / p.window * p.window;
        const long long from = static_cast<long long>(b) * p.T + t0 + tok, to = (slot * rows + r) * (static_cast<long long>(chunks) * 8) + 8 * c;
        *reinterpret_cast<uint4*>(p.k_cache + to) = load_16(p.k + from * p.k_stride + 8 * c, true);
        *reinterpret_cast<uint4*>(p.v_cache + to) = load_16(p.v + from * p.v_stride + 8 * c, true);
    }
}

template <int D>
cudaError_t launch(const WindowStepArgs& a, cudaStream_t stream) {
    const int sets = (a.H / a.Hk + 15) / 16;
    cudaError_t e = cudaFuncSetAttribute(window_step_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Joined<D>));
    if (e != cudaSuccess) return e;
    if (a.cluster > 8) {
        e = cudaFuncSetAttribute(window_step_kernel<D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.B) * a.Hk * sets * a.cluster));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = sizeof(Joined<D>);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.cluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, window_step_kernel<D>, a);
}

}  // namespace

// Blocks per row, group and set of heads: enough of them for the GPU, none
// with less than a step per warp.
int window_step_cluster(int B, int Hk, int sets, int rows) {
    int c = 1;
    while (c < 16 && static_cast<long long>(B) * Hk * sets * c < 3 * 152 && rows > c * kWarps * kKeys) c *= 2;
    return c;
}

cudaError_t launch_window_step(const WindowStepArgs& a, cudaStream_t stream) {
    return a.d == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

cudaError_t launch_window_fill(const WindowFillArgs& a, cudaStream_t stream) {
    const long long ids = static_cast<long long>(std::min(a.T, a.sinks + a.window)) * (a.Hk * a.d / 8);
    const unsigned blocks = static_cast<unsigned>(std::min<long long>((ids + 255) / 256, 1024));
    window_fill_kernel<<<dim3(blocks, a.nseq), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
