// Group norm with an activation, channels last: the output norm of a gated
// delta rule layer ("Research Sprint Day 2 - Rooflines", GDN layer pseudocode:
// RMSNorm of the operator's output times SiLU of a gate) and of a state space
// mixer.  Per row and group of Cg channels, act one of none, SiLU, sigmoid:
//   x' = x act(gate) if the gate comes first, else x
//   m  = mean(x') if centered, else 0;   r = (mean((x' - m)^2) + eps)^-1/2
//   n  = r (x' - m),   v = n weight + bias
//   y  = v act(gate) (gate after), v (gate first), act(v) (no gate).
// Reverse mode, with dv the gradient of v and dn = dv weight:
//   dx' = r (dn - n mean(dn n) - [mean(dn) if centered]),
//   dweight = sum_rows dv n,   dbias = sum_rows dv,
// and the product and activation rules around it; n is recomputed.
// Bound by HBM (3 accesses per element gated forward, 5 backward): a team of
// lanes holds its group's row in registers, so every input is read once; the
// mean is subtracted before squaring.  In the reverse mode a team keeps one
// group and walks rows, so the weight gradients accumulate in its registers
// and leave as one partial row per team, summed afterwards in a fixed order.
#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kThreads = 256;

__device__ __forceinline__ float act(float x, int kind) {
    return kind == 0 ? x : kind == 1 ? x * sigmoid(x) : sigmoid(x);
}
__device__ __forceinline__ float dact(float x, int kind) {
    if (kind == 0) return 1.f;
    const float s = sigmoid(x);
    return kind == 1 ? dsilu(x, s) : s * (1.f - s);
}

// Sum over the LANES lanes of a team (16 or 32: within a warp; 256: the block).
template <int LANES>
__device__ __forceinline__ float team_sum(float x, float* red) {
    constexpr int M = LANES < 32 ? LANES : 32;
#pragma unroll
    for (int m = M / 2; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
    if constexpr (LANES > 32) {
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int i = 1; i < LANES / 32; ++i) x += red[i];
    }
    return x;
}

// Row of a group: V vectors of E elements per lane, vector v at lane + v LANES.
template <typename T, int E, int LANES, int V>
struct Row {
    float v[V][E];
    __device__ __forceinline__ void load(const T* p, int lane, int nv, bool on) {
        Raw<T, E> r[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = lane + i * LANES;
            r[i] = load_raw<T, E>(p + static_cast<long long>(j) * E, on && j < nv ? E : 0);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) unpack<T, E>(r[i], v[i]);
    }
    __device__ __forceinline__ void store(T* p, int lane, int nv, bool on) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = lane + i * LANES;
            if (on && j < nv) store_raw<T, E>(p + static_cast<long long>(j) * E, pack<T, E>(v[i]), E);
        }
    }
};

// x' -> n in place; returns r
template <int E, int LANES, int V>
__device__ __forceinline__ float normalise(float (&x)[V][E], int lane, int nv, float inv, float eps, int center,
                                           float* red) {
    if (center) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) s += x[i][e];
        const float m = team_sum<LANES>(s, red) * inv;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) x[i][e] = lane + i * LANES < nv ? x[i][e] - m : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(x[i][e], x[i][e], s);
    const float r = 1.f / sqrtf(fmaf(team_sum<LANES>(s, red), inv, eps));
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] *= r;
    return r;
}

template <int E, int LANES, int V>
__device__ __forceinline__ void load_param(const float* p, float missing, int lane, int nv, float (&w)[V][E]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = lane + i * LANES;
#pragma unroll
        for (int e = 0; e < E; ++e) w[i][e] = missing;
        if (p && j < nv) unpack<float, E>(load_raw<float, E>(p + static_cast<long long>(j) * E, E), w[i]);
    }
}

template <typename T, int E, int LANES, int V>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormArgs p) {
    __shared__ float red[kThreads / 32];
    const int size = p.C / p.groups, nv = size / E;
    const int lane = threadIdx.x % LANES;
    const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
    const bool on = unit < p.rows * p.groups;  // whole teams; an idle one still meets the others' shuffles
    const long long row = on ? unit / p.groups : 0;
    const int c0 = on ? static_cast<int>(unit % p.groups) * size : 0;
    Row<T, E, LANES, V> x, gt;
    x.load(static_cast<const T*>(p.x) + row * p.x_stride + c0, lane, nv, on);
    if (p.gate) {
        gt.load(static_cast<const T*>(p.gate) + row * p.gate_stride + c0, lane, nv, on);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                gt.v[i][e] = act(gt.v[i][e], p.activation);
                if (p.gate_first) x.v[i][e] = lane + i * LANES < nv ? x.v[i][e] * gt.v[i][e] : 0.f;
            }
    }
    normalise<E, LANES, V>(x.v, lane, nv, 1.f / size, p.eps, p.center, red);
    float w[V][E], b[V][E];
    load_param<E, LANES, V>(p.weight ? p.weight + c0 : nullptr, 1.f, lane, nv, w);
    load_param<E, LANES, V>(p.bias ? p.bias + c0 : nullptr, 0.f, lane, nv, b);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float v = fmaf(x.v[i][e], w[i][e], b[i][e]);
            x.v[i][e] = p.gate ? (p.gate_first ? v : v * gt.v[i][e]) : act(v, p.activation);
        }
    x.store(static_cast<T*>(p.y) + row * p.C + c0, lane, nv, on);
}

// Team `unit` keeps group unit % groups and takes rows unit / groups, + teams, ...
template <typename T, int E, int LANES, int V>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormArgs p, int teams) {
    __shared__ float red[kThreads / 32];
    const int size = p.C / p.groups, nv = size / E;
    const float inv = 1.f / size;
    const int lane = threadIdx.x % LANES;
    const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
    const bool live = unit < static_cast<long long>(teams) * p.groups;
    const int team = live ? static_cast<int>(unit / p.groups) : 0;
    const int c0 = live ? static_cast<int>(unit % p.groups) * size : 0;
    float w[V][E], b[V][E], dw[V][E], db[V][E];
    load_param<E, LANES, V>(p.weight ? p.weight + c0 : nullptr, 1.f, lane, nv, w);
    load_param<E, LANES, V>(p.bias ? p.bias + c0 : nullptr, 0.f, lane, nv, b);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[i][e] = db[i][e] = 0.f;
    const long long steps = (p.rows + teams - 1) / teams;
    for (long long s = 0; s < steps; ++s) {
        const long long row = team + s * teams;
        const bool on = live && row < p.rows;
        Row<T, E, LANES, V> x, gt, dy;
        float n[V][E];
        x.load(static_cast<const T*>(p.x) + (on ? row : 0) * p.x_stride + c0, lane, nv, on);
        dy.load(static_cast<const T*>(p.d_out) + (on ? row : 0) * p.C + c0, lane, nv, on);
        if (p.gate) gt.load(static_cast<const T*>(p.gate) + (on ? row : 0) * p.gate_stride + c0, lane, nv, on);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e)
                n[i][e] = p.gate && p.gate_first && lane + i * LANES < nv ? x.v[i][e] * act(gt.v[i][e], p.activation) : x.v[i][e];
        const float r = normalise<E, LANES, V>(n, lane, nv, inv, p.eps, p.center, red);
        // dv into dy; with the gate after the norm, its own gradient at once
        float sn = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float v = fmaf(n[i][e], w[i][e], b[i][e]);
                float dv = dy.v[i][e];
                if (!p.gate) {
                    dv *= dact(v, p.activation);
                } else if (!p.gate_first) {
                    const float ga = gt.v[i][e];
                    gt.v[i][e] = dv * v * dact(ga, p.activation);
                    dv *= act(ga, p.activation);
                }
                if (on && lane + i * LANES < nv) {
                    dw[i][e] = fmaf(dv, n[i][e], dw[i][e]);
                    db[i][e] += dv;
                } else {
                    dv = 0.f;
                }
                const float dn = dv * w[i][e];
                dy.v[i][e] = dn;
                sn = fmaf(dn, n[i][e], sn);
                s1 += dn;
            }
        sn = team_sum<LANES>(sn, red) * inv;
        s1 = p.center ? team_sum<LANES>(s1, red) * inv : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = r * (dy.v[i][e] - s1 - n[i][e] * sn);
                if (p.gate && p.gate_first) {
                    const float ga = gt.v[i][e];
                    gt.v[i][e] = d * x.v[i][e] * dact(ga, p.activation);
                    x.v[i][e] = d * act(ga, p.activation);
                } else {
                    x.v[i][e] = d;
                }
            }
        x.store(static_cast<T*>(p.dx) + row * p.C + c0, lane, nv, on);
        if (p.gate) gt.store(static_cast<T*>(p.dgate) + row * p.C + c0, lane, nv, on);
    }
    if (!p.partial || !live) return;
    float* pw = p.partial + static_cast<long long>(team) * (p.bias ? 2 : 1) * p.C + c0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = lane + i * LANES;
        if (j >= nv) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            pw[j * E + e] = dw[i][e];
            if (p.bias) pw[p.C + j * E + e] = db[i][e];
        }
    }
}

template <typename T, int E, int LANES, int V>
cudaError_t norm_fwd_v(const NormArgs& a, cudaStream_t stream) {
    const long long units = a.rows * a.groups, per = kThreads / LANES;
    norm_fwd_kernel<T, E, LANES, V><<<static_cast<unsigned>((units + per - 1) / per), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}
template <typename T, int E, int LANES, int V>
cudaError_t norm_bwd_v(const NormArgs& a, cudaStream_t stream) {
    const int teams = norm_partial_rows(a.rows, a.C, a.groups, a.dtype);
    const long long units = static_cast<long long>(teams) * a.groups, per = kThreads / LANES;
    norm_bwd_kernel<T, E, LANES, V><<<static_cast<unsigned>((units + per - 1) / per), kThreads, 0, stream>>>(a, teams);
    return cudaGetLastError();
}

template <typename T>
bool wide_rows(const NormArgs& a) {
    constexpr int E = 16 / sizeof(T);
    auto ok = [](const void* p, long long stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % E == 0; };
    return (a.C / a.groups) % E == 0 && ok(a.x, a.x_stride) && (!a.gate || ok(a.gate, a.gate_stride));
}

// Lanes and registers per group: a half warp or a warp where the group fits
// its registers, else the block.  Rows that 16-byte accesses cannot take (odd
// sizes, strides or addresses) go element by element, neighbouring lanes on
// neighbouring elements.
#define GDN_NORM_SIZES(fn, T)                                       \
    const int size = a.C / a.groups;                                \
    constexpr int E = 16 / sizeof(T);                               \
    if (wide_rows<T>(a)) {                                          \
        const int nv = size / E;                                    \
        if (nv <= 16) return fn<T, E, 16, 1>(a, stream);            \
        if (nv <= 32) return fn<T, E, 32, 1>(a, stream);            \
        if (nv <= 64) return fn<T, E, 32, 2>(a, stream);            \
        if (nv <= 256) return fn<T, E, 256, 1>(a, stream);          \
        if (nv <= 512) return fn<T, E, 256, 2>(a, stream);          \
        if (nv <= 1024) return fn<T, E, 256, 4>(a, stream);         \
        if constexpr (sizeof(T) == 4) return fn<T, E, 256, 8>(a, stream); \
    }                                                               \
    if (size <= 128) return fn<T, 1, 32, 4>(a, stream);             \
    if (size <= 512) return fn<T, 1, 32, 16>(a, stream);            \
    if (size <= 2048) return fn<T, 1, 256, 8>(a, stream);           \
    return fn<T, 1, 256, 32>(a, stream)

template <typename T>
cudaError_t norm_fwd_t(const NormArgs& a, cudaStream_t stream) {
    GDN_NORM_SIZES(norm_fwd_v, T);
}
template <typename T>
cudaError_t norm_bwd_t(const NormArgs& a, cudaStream_t stream) {
    GDN_NORM_SIZES(norm_bwd_v, T);
}

}  // namespace

// Teams per group in the reverse mode, one partial row each: enough to fill
// the GPU, few enough that the partial rows cost little beside the inputs.
int norm_partial_rows(long long rows, int C, int groups, int dtype) {
    const int size = C / groups;
    const int lanes = size <= (dtype == 0 ? 512 : 256) ? 16 : 256;
    long long teams = 152LL * 8 * kThreads / lanes / 2 / groups;
    if (teams < 1) teams = 1;
    return static_cast<int>(rows < teams ? rows : teams);
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream) {
    return a.dtype == 0 ? norm_fwd_t<uint16_t>(a, stream) : norm_fwd_t<float>(a, stream);
}
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t stream) {
    return a.dtype == 0 ? norm_bwd_t<uint16_t>(a, stream) : norm_bwd_t<float>(a, stream);
}

}  // namespace gdn
