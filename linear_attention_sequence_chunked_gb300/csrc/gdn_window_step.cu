// Attention with a sliding window, one token per row on a cache of sinks +
// window rows, and the filling of such a cache from prompts.
//
// The cache keeps token p in row p while p < sinks and in row sinks + (p -
// sinks) % window from there on, so after the token at position p its first
// min(p + 1, rows) rows are exactly the keys that the token sees, in an order
// that a softmax does not care about.
//
// The step is bound by reading the cache once.  A warp takes 16 rows at a time
// for up to 16 query heads of a group: S = Q K^T (bf16, 16 x 8 x 16) and O += P V
// (tf32, 16 x 8 x 8) are register products (mma.sync: one query per head leaves the
// 128 rows of a tensor-memory product empty, and nothing here waits for arithmetic).
// P keeps eleven bits there: as bf16 its rounding was as large as the output's own
// (2.0e-3 of L2 together, 1.7e-3 so), and a second bf16 part, which may be zero,
// would make a NaN of an infinite value.  The
// channels are numbered so that both operands are what 16-byte loads of the
// rows bring, without shared memory: in the first product a channel's place
// does not matter as long as Q and K agree, in the second a lane's 16 bytes of V
// are its column in eight products.  The warps of a block, and the blocks of a
// cluster where the rows alone leave SMs idle, join their (maximum, sum, O) in a
// fixed order through (distributed) shared memory.  64 rows of 1028 keys, 16 / 4
// heads of 128, take 26 us, 4.6 TB/s: the latency of HBM with as many loads on
// their way as the registers hold, 69 % of a copy (the tensor pipe is active in 20 %
// of the cycles).  One row of 16388 keys takes 14 on the sixteen blocks that a cluster
// may have.
#include <algorithm>
#include <cmath>

#include "gdn_cluster.cuh"
#include "gdn_kernels.h"
#include "gdn_launch.h"
#include "gdn_mix_common.cuh"
#include "gdn_mma.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kKeys = 16;  // of a warp's step
// Warps of a block: six, two blocks to an SM (64 rows of 1028 keys, 4 key heads, with
// P in bf16: 25 us; four warps and three blocks 29, twelve and one 31), or twelve where
// the rows and heads of a call are too few for that.
constexpr int kFew = 6, kMany = 12;

__device__ __forceinline__ uint32_t pair_of(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
constexpr int kMaxCluster = 16;

template <int D, int kWarps>
struct Joined {
    uint4 q[D / 32][2][32];  // Q as the first product's operand, a lane's four registers together
    float o[kWarps][16][D + 4];
    float m[kWarps][16], l[kWarps][16], f[kWarps][16];
    float2 ml[16];                         // the block's maximum and sum
    // what the blocks of the cluster send: everyone's maxima and sums, and their
    // sums of the part of the output that is this block's
    float2 sent_ml[kMaxCluster][16];
    float4 sent[16 * D / 4 + kMaxCluster];
};

template <int D, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 12 / kWarps) window_step_kernel(const WindowStepArgs p) {
    constexpr int CH = D / 32;  // 16-byte chunks of a row per lane
    extern __shared__ __align__(16) unsigned char smem[];
    Joined<D, kWarps>& sm = *reinterpret_cast<Joined<D, kWarps>*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int C = p.cluster;
    const uint32_t rank = C > 1 ? cluster::rank() : 0;
    if (C > 1) cluster::arrive();
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
    const uint16_t* qp = p.q + b * p.q_stride + static_cast<long long>(h0) * D;
    if (warp == 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint4 lo = load_16(qp + g * D + (c * 4 + t) * 8, g < heads), hi = load_16(qp + (g + 8) * D + (c * 4 + t) * 8, g + 8 < heads);
            sm.q[c][0][lane] = make_uint4(lo.x, hi.x, lo.y, hi.y);
            sm.q[c][1][lane] = make_uint4(lo.z, hi.z, lo.w, hi.w);
        }
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
    // the next strip's keys are on their way from the first product on, its
    // values from the second on
    uint4 kr[2][CH], vr[4][CH / 2];
    const auto load_keys = [&](int s) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {  // keys 8 n + g of the strip
            const int r = s * kKeys + 8 * n + g;
            const uint16_t* k = r == at ? kn : kc + r * stride;
#pragma unroll
            for (int c = 0; c < CH; ++c) kr[n][c] = load_16(k + (c * 4 + t) * 8, s < s1 && r < rows);
        }
    };
    const auto load_values = [&](int s) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {  // keys 2 t, + 1, + 8, + 9
            const int r = s * kKeys + 2 * t + (n & 1) + (n >> 1) * 8;
            const uint16_t* v = r == at ? vn : vc + r * stride;
#pragma unroll
            for (int c = 0; c < CH / 2; ++c) vr[n][c] = load_16(v + c * 64 + g * 8, s < s1 && r < rows);
        }
    };
    int s = static_cast<int>(rank) * per + warp;
    load_keys(s);
    load_values(s);
    __syncthreads();  // Q is there
    for (; s < s1; s += kWarps) {
        const int r0 = s * kKeys;
        float sc[2][4] = {};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint4 q0 = sm.q[c][0][lane], q1 = sm.q[c][1][lane];
            const uint32_t a0[4] = {q0.x, q0.y, q0.z, q0.w}, a1[4] = {q1.x, q1.y, q1.z, q1.w};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                mma::bf16_16x8x16(sc[n], a0, kr[n][c].x, kr[n][c].y);
                mma::bf16_16x8x16(sc[n], a1, kr[n][c].z, kr[n][c].w);
            }
        }
        load_keys(s + kWarps);
        // sc[n][e]: query row g + 8 (e / 2), key r0 + 8 n + 2 t + e % 2
        uint32_t pa[2][4];  // P of keys 2 t and 2 t + 1, and of 8 and 9 + 2 t, as the second product's operand
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
#pragma unroll
            for (int e = 0; e < 4; ++e) pa[e >> 1][x + 2 * (e & 1)] = mma::tf32(v[e]);
            if (__any_sync(0xffffffffu, f != 1.f)) {  // (the products behind it take the whole warp)
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][2 * x] *= f;
                    o[i][2 * x + 1] *= f;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CH / 2; ++c) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // column g is channel 64 c + 8 g + j
                const auto channel = [&](int n) { return mma::widen(mma::word(vr[n][c], j / 2), j & 1); };
                mma::tf32_16x8x8(o[8 * c + j], pa[0], channel(0), channel(1));
                mma::tf32_16x8x8(o[8 * c + j], pa[1], channel(2), channel(3));
            }
        }
        load_values(s + kWarps);
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
    // the block's warps: each one's weight against the largest maximum
    if (threadIdx.x < 16 * kWarps) {
        const int w = threadIdx.x / 16, r = threadIdx.x % 16;
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, sm.m[i][r]);
        const float ms = mx == -INFINITY ? 0.f : mx;
        sm.f[w][r] = ex2(sm.m[w][r] - ms);
        if (w == 0) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) sum = fmaf(sm.l[i][r], ex2(sm.m[i][r] - ms), sum);
            sm.ml[r] = make_float2(mx, sum);
        }
    }
    __syncthreads();
    const auto write = [&](int r, int d, const float4& o, float sum) {
        const float inv = on ? 1.f / sum : 0.f;
        *reinterpret_cast<uint2*>(p.out + (b * p.H + h0 + r) * D + d) =
            on ? make_uint2(pair_of(o.x * inv, o.y * inv), pair_of(o.z * inv, o.w * inv)) : make_uint2(0, 0);
    };
    const int quads = heads * D / 4, share = (quads + C - 1) / C;  // of the output's 4 channels each
    if (C > 1) cluster::wait();  // every block of the cluster is there
    for (int i = threadIdx.x; i < quads; i += 32 * kWarps) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm.f[w][r];
            const float4 v = *reinterpret_cast<const float4*>(&sm.o[w][r][d]);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        if (C == 1)
            write(r, d, acc, sm.ml[r].y);
        else
            cluster::store(&sm.sent[rank * share + i % share], i / share, acc);
    }
    if (C == 1) return;
    for (int i = threadIdx.x; i < 16 * C; i += 32 * kWarps) cluster::store(&sm.sent_ml[rank][i % 16], i / 16, sm.ml[i % 16]);
    cluster::arrive();
    cluster::wait();
    for (int i = threadIdx.x; i < share && static_cast<int>(rank) * share + i < quads; i += 32 * kWarps) {
        const int at4 = static_cast<int>(rank) * share + i, r = at4 / (D / 4), d = at4 % (D / 4) * 4;
        float mx = -INFINITY;
        for (int c = 0; c < C; ++c) mx = fmaxf(mx, sm.sent_ml[c][r].x);
        const float ms = mx == -INFINITY ? 0.f : mx;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
        for (int c = 0; c < C; ++c) {
            const float2 ml = sm.sent_ml[c][r];
            const float f = ex2(ml.x - ms);
            const float4 v = sm.sent[c * share + i];
            sum = fmaf(ml.y, f, sum);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        write(r, d, acc, sum);
    }
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

template <int D, int kWarps>
cudaError_t launch(const WindowStepArgs& a, cudaStream_t stream) {
    const int sets = (a.H / a.Hk + 15) / 16;
    constexpr size_t smem = sizeof(Joined<D, kWarps>);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_once(window_step_kernel<D, kWarps>, smem, true, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.B) * a.Hk * sets * a.cluster));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.cluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, window_step_kernel<D, kWarps>, a);
}
template <int D>
cudaError_t launch_warps(const WindowStepArgs& a, cudaStream_t stream) {
    return a.warps == kMany ? launch<D, kMany>(a, stream) : launch<D, kFew>(a, stream);
}

}  // namespace

// Blocks per row, group and set of heads, and their warps: enough for the GPU,
// none with less than a step per warp.
void window_step_shape(WindowStepArgs& a) {
    const long long units = static_cast<long long>(a.B) * a.Hk * ((a.H / a.Hk + 15) / 16);
    a.warps = units * 16 < 2 * 152 && a.rows > 16 * kFew * kKeys ? kMany : kFew;
    a.cluster = 1;
    while (a.cluster < kMaxCluster && units * a.cluster * a.warps < 12 * 152 / 2 && a.rows > a.cluster * a.warps * kKeys) a.cluster *= 2;
}

cudaError_t launch_window_step(const WindowStepArgs& a, cudaStream_t stream) {
    return a.d == 64 ? launch_warps<64>(a, stream) : launch_warps<128>(a, stream);
}

cudaError_t launch_window_fill(const WindowFillArgs& a, cudaStream_t stream) {
    const long long ids = static_cast<long long>(std::min(a.T, a.sinks + a.window)) * (a.Hk * a.d / 8);
    const unsigned blocks = static_cast<unsigned>(std::min<long long>((ids + 255) / 256, 1024));
    window_fill_kernel<<<dim3(blocks, a.nseq), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
