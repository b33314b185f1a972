// Short causal convolution, channels last, with an optional SiLU: the
// convolution that feeds q, k and v of a gated delta rule layer ("Research
// Sprint Day 2 - Rooflines", GDN layer pseudocode) and the input of a state
// space scan.  Per channel c and token t of a sequence,
//   p_t = bias_c + sum_{j < W} w_cj x_{t - (W-1) + j},   y_t = act(p_t),
// with x before the sequence's start from the W-1 rows of its initial state
// (zeros without one).  The final state is the last W-1 inputs, so a sequence
// can be continued, token by token too (the step kernel).
// Reverse mode, dp = dy act'(p) with p recomputed:
//   dx_s = sum_j w_cj dp_{s + (W-1) - j},  dw_cj = sum_t dp_t x_{t-(W-1)+j},
//   dbias_c = sum_t dp_t,
// and the initial state's gradient is dx at s < 0.
//
// All of it is bound by HBM: 2 (forward) or 3 (backward) accesses per element
// against 2W to 6W operations.  A thread takes E neighbouring channels (16
// bytes where rows allow it) over a block of consecutive tokens with the
// window in registers, so every input is read once but for W-1 rows per block.
#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kThreads = 256;

template <int W, int E>
__device__ __forceinline__ void load_weights(const float* weight, const float* bias, long long d0, float (*w)[E],
                                             float* bs) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = __ldg(weight + (d0 + e) * W + j);
        bs[e] = bias ? __ldg(bias + d0 + e) : 0.f;
    }
}

// Row r of the W-1 inputs before a sequence's start (r = 0 the oldest).
template <typename T, int W, int E>
__device__ __forceinline__ void load_state_row(const T* state, long long seq, int r, long long D, long long d0,
                                               float* x) {
    if (state) {
        unpack<T, E>(load_raw<T, E>(state + (seq * (W - 1) + r) * D + d0, E), x);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
    }
}

template <typename T, int W, int E>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(const ConvArgs p) {
    constexpr int U = 4;  // tokens whose loads are in flight together
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.N, p.T, p.err);
    const long long cv = p.D / E;
    const long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (id >= p.slots * cv) return;
    const long long d0 = id % cv * E;
    int n, b, t0, t1;
    long long c;
    if (!find_block(p.cu_seqlens, p.N, p.T, p.tb, id / cv, p.err, n, c)) return;
    if (!token_range(p.cu_seqlens, n, p.N, p.T, p.err, b, t0, t1)) return;
    const T* x = static_cast<const T*>(p.x) + static_cast<long long>(b) * p.T * p.x_stride + d0;
    T* y = static_cast<T*>(p.y) + static_cast<long long>(b) * p.T * p.D + d0;
    const T* s0 = static_cast<const T*>(p.initial_state);
    const long long begin = t0 + c * p.tb;
    const int tb = static_cast<int>(min(begin, static_cast<long long>(t1)));
    const int te = static_cast<int>(min(begin + p.tb, static_cast<long long>(t1)));
    if (p.final_state && te == t1 && (tb < te || c == 0)) {
        T* fs = static_cast<T*>(p.final_state);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            const int t = t1 - (W - 1) + r;
            float v[E];
            if (t >= t0)
                unpack<T, E>(load_raw<T, E>(x + t * p.x_stride, E), v);
            else
                load_state_row<T, W, E>(s0, n, t - t0 + (W - 1), p.D, d0, v);
            store_raw<T, E>(fs + (static_cast<long long>(n) * (W - 1) + r) * p.D + d0, pack<T, E>(v), E);
        }
    }
    if (tb >= te) return;
    float w[W][E], bs[E], win[W][E];
    load_weights<W, E>(p.weight, p.bias, d0, w, bs);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int t = tb - (W - 1) + r;
        if (t >= t0)
            unpack<T, E>(load_raw<T, E>(x + t * p.x_stride, E), win[r]);
        else
            load_state_row<T, W, E>(s0, n, t - t0 + (W - 1), p.D, d0, win[r]);
    }
    for (int t = tb; t < te; t += U) {
        Raw<T, E> in[U];
#pragma unroll
        for (int k = 0; k < U; ++k) in[k] = load_raw<T, E>(x + (t + k) * p.x_stride, t + k < te ? E : 0);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (t + k >= te) break;
            unpack<T, E>(in[k], win[W - 1]);
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float acc = bs[e];
#pragma unroll
                for (int j = 0; j < W; ++j) acc = fmaf(w[j][e], win[j][e], acc);
                o[e] = p.activation ? acc * sigmoid(acc) : acc;
            }
            store_raw<T, E>(y + (t + k) * static_cast<long long>(p.D), pack<T, E>(o), E);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) win[j][e] = win[j + 1][e];
        }
    }
}

// One block: kLanes channel vectors x kRows time blocks; each thread walks its
// time block (and the W-1 tokens after it, whose dp reach back into it), then
// the block's partial weight gradients are summed over its rows in order.
constexpr int kLanes = 32;
constexpr int kRows = kThreads / kLanes;

template <typename T, int W, int E>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(const ConvArgs p) {
    __shared__ float red[kRows][kLanes][E + 1];
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.cu_seqlens, p.N, p.T, p.err);
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const long long d0 = (static_cast<long long>(blockIdx.y) * kLanes + lane) * E;
    const long long slot = static_cast<long long>(blockIdx.x) * kRows + row;
    float dw[W + 1][E];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[j][e] = 0.f;
    int n, b, t0, t1;
    long long c;
    if (d0 < p.D && slot < p.slots && find_block(p.cu_seqlens, p.N, p.T, p.tb, slot, p.err, n, c) &&
        token_range(p.cu_seqlens, n, p.N, p.T, p.err, b, t0, t1)) {
        const T* x = static_cast<const T*>(p.x) + static_cast<long long>(b) * p.T * p.x_stride + d0;
        const T* dy = static_cast<const T*>(p.d_out) + static_cast<long long>(b) * p.T * p.D + d0;
        T* dx = static_cast<T*>(p.dx) + static_cast<long long>(b) * p.T * p.D + d0;
        const T* s0 = static_cast<const T*>(p.initial_state);
        const T* dfs = static_cast<const T*>(p.d_final_state);
        T* ds0 = static_cast<T*>(p.d_initial_state);
        const long long begin = t0 + c * p.tb;
        const int tb = static_cast<int>(min(begin, static_cast<long long>(t1)));
        const int te = static_cast<int>(min(begin + p.tb, static_cast<long long>(t1)));
        if (tb < te || c == 0) {
            float w[W][E], bs[E], win[W][E], dp[W][E];
            load_weights<W, E>(p.weight, p.bias, d0, w, bs);
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) dp[j][e] = 0.f;
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
                const int t = tb - (W - 1) + r;
                if (t >= t0)
                    unpack<T, E>(load_raw<T, E>(x + t * p.x_stride, E), win[r]);
                else
                    load_state_row<T, W, E>(s0, n, t - t0 + (W - 1), p.D, d0, win[r]);
            }
            for (int t = tb; t < te + W - 1; ++t) {
                const bool in = t < t1;
                float g[E];
                unpack<T, E>(load_raw<T, E>(x + t * p.x_stride, in ? E : 0), win[W - 1]);
                unpack<T, E>(load_raw<T, E>(dy + t * static_cast<long long>(p.D), in ? E : 0), g);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float acc = bs[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) acc = fmaf(w[j][e], win[j][e], acc);
                    const float d = !in ? 0.f : p.activation ? g[e] * dsilu(acc, sigmoid(acc)) : g[e];
                    dp[W - 1][e] = d;
                    if (t < te) {
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][e] = fmaf(d, win[j][e], dw[j][e]);
                        dw[W][e] += d;
                    }
                }
                // input s has now seen every token it feeds
                const int s = t - (W - 1);
                if (s >= tb || (tb == t0 && ds0)) {
                    float o[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        o[e] = 0.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) o[e] = fmaf(w[j][e], dp[W - 1 - j][e], o[e]);
                    }
                    if (dfs && s >= t1 - (W - 1)) {  // one of the rows the final state holds
                        float v[E];
                        unpack<T, E>(load_raw<T, E>(dfs + (static_cast<long long>(n) * (W - 1) + s - t1 + (W - 1)) * p.D + d0, E), v);
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] += v[e];
                    }
                    T* to = s >= tb ? dx + s * static_cast<long long>(p.D)
                                    : ds0 + (static_cast<long long>(n) * (W - 1) + s - t0 + (W - 1)) * p.D + d0;
                    store_raw<T, E>(to, pack<T, E>(o), E);
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        win[j][e] = win[j + 1][e];
                        dp[j][e] = dp[j + 1][e];
                    }
            }
        }
    }
    // partial [block row][W + 1][D]: the weights' gradients, then the bias's
#pragma unroll
    for (int j = 0; j <= W; ++j) {
#pragma unroll
        for (int e = 0; e < E; ++e) red[row][lane][e] = dw[j][e];
        __syncthreads();
        for (int i = threadIdx.x; i < kLanes * E; i += kThreads) {
            const long long d = static_cast<long long>(blockIdx.y) * kLanes * E + i;
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) s += red[r][i / E][i % E];
            if (d < p.D) p.partial[(static_cast<long long>(blockIdx.x) * (W + 1) + j) * p.D + d] = s;
        }
        __syncthreads();
    }
}

template <typename T, int W, int E>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvStepArgs p) {
    const long long cv = p.D / E;
    const long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (id >= p.B * cv) return;
    const long long b = id / cv, d0 = id % cv * E;
    T* y = static_cast<T*>(p.y) + b * p.D + d0;
    long long slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.S) {  // an idle row, or one outside the cache
            if (slot >= p.S) record_error(p.err, kErrBadSlot);
            const float zero[E] = {};
            store_raw<T, E>(y, pack<T, E>(zero), E);
            return;
        }
    }
    const T* st = static_cast<const T*>(p.state) + slot * (W - 1) * p.D + d0;
    T* so = static_cast<T*>(p.out_state) + slot * (W - 1) * p.D + d0;
    Raw<T, E> in[W];
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {  // not the read-only path: out_state may be the same memory
        const T* row = st + r * static_cast<long long>(p.D);
        if constexpr (E * sizeof(T) >= 4)
            in[r] = *reinterpret_cast<const Raw<T, E>*>(row);
        else
            in[r].w[0] = *row;
    }
    in[W - 1] = load_raw<T, E>(static_cast<const T*>(p.x) + b * p.x_stride + d0, E);
    float w[W][E], o[E];
    load_weights<W, E>(p.weight, p.bias, d0, w, o);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float v[E];
        unpack<T, E>(in[j], v);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w[j][e], v[e], o[e]);
        if (j > 0) store_raw<T, E>(so + (j - 1) * static_cast<long long>(p.D), in[j], E);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = p.activation ? o[e] * sigmoid(o[e]) : o[e];
    store_raw<T, E>(y, pack<T, E>(o), E);
}

// Sums of a [rows][cols] partial array over its rows, in a fixed order.
// Columns land in up to three outputs of c0, c1 and the rest (null: dropped);
// with W > 0 the array is [rows][W + 1][D] and the first output (D, W).
__global__ void __launch_bounds__(kThreads) column_sum_kernel(const ColumnSumArgs p) {
    __shared__ float red[kRows][kLanes + 1];
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const long long col = static_cast<long long>(blockIdx.x) * kLanes + lane;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < p.cols) {
        const float* src = p.partial + col;
        for (int r = row; r < p.rows; r += 4 * kRows) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r + k * kRows < p.rows) s[k] += __ldg(src + (r + k * kRows) * p.stride);
        }
    }
    red[row][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (row != 0 || col >= p.cols) return;
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) v += red[r][lane];
    if (p.W > 0) {
        const long long j = col / p.c1, d = col % p.c1;  // c1 = D
        if (j < p.W)
            p.out[0][d * p.W + j] = v;
        else if (p.out[1])
            p.out[1][d] = v;
        return;
    }
    const long long c01 = p.c0 + p.c1;
    float* out = col < p.c0 ? p.out[0] : col < c01 ? p.out[1] : p.out[2];
    if (out) out[col < p.c0 ? col : col < c01 ? col - p.c0 : col - c01] = v;
}

// Whether rows of D channels at p, `stride` elements apart, can be accessed E
// elements at a time.
template <typename T>
bool rows_take(const void* p, long long stride, int D, int E) {
    return D % E == 0 && reinterpret_cast<uintptr_t>(p) % (E * sizeof(T)) == 0 && stride % E == 0;
}

template <typename T, int W, int E>
cudaError_t conv_fwd_e(const ConvArgs& a, cudaStream_t stream) {
    const long long threads = a.slots * (a.D / E);
    conv_fwd_kernel<T, W, E><<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

// 16 bytes of a row per thread where its width, stride and address allow it,
// else 4 bytes (bf16), else one element: neighbouring threads then still read
// neighbouring elements.
template <typename T, int W>
cudaError_t conv_fwd_w(const ConvArgs& a, cudaStream_t stream) {
    constexpr int E = 16 / sizeof(T);
    if (rows_take<T>(a.x, a.x_stride, a.D, E)) return conv_fwd_e<T, W, E>(a, stream);
    if constexpr (sizeof(T) == 2)
        if (rows_take<T>(a.x, a.x_stride, a.D, 2)) return conv_fwd_e<T, W, 2>(a, stream);
    return conv_fwd_e<T, W, 1>(a, stream);
}

template <typename T, int W, int E>
cudaError_t conv_bwd_e(const ConvArgs& a, cudaStream_t stream) {
    dim3 grid(static_cast<unsigned>((a.slots + kRows - 1) / kRows),
              static_cast<unsigned>((a.D + kLanes * E - 1) / (kLanes * E)));
    conv_bwd_kernel<T, W, E><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}
template <typename T, int W>
cudaError_t conv_bwd_w(const ConvArgs& a, cudaStream_t stream) {
    return rows_take<T>(a.x, a.x_stride, a.D, 4) ? conv_bwd_e<T, W, 4>(a, stream) : conv_bwd_e<T, W, 1>(a, stream);
}

template <typename T, int W, int E>
cudaError_t conv_step_e(const ConvStepArgs& a, cudaStream_t stream) {
    const long long threads = static_cast<long long>(a.B) * (a.D / E);
    conv_step_kernel<T, W, E><<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}
template <typename T, int W>
cudaError_t conv_step_w(const ConvStepArgs& a, cudaStream_t stream) {
    return rows_take<T>(a.x, a.x_stride, a.D, 4) ? conv_step_e<T, W, 4>(a, stream) : conv_step_e<T, W, 1>(a, stream);
}

}  // namespace

// Tokens per thread: long blocks re-read fewer rows at their edges (W-1 per
// block), short ones give small inputs enough threads.
int conv_block_tokens(int B, int T, int D, int backward) {
    const long long per_thread = backward ? 4 : 8;
    const long long work = static_cast<long long>(B) * T * ((D + per_thread - 1) / per_thread);
    int tb = 64;
    while (tb > 4 && work / tb < 200000) tb /= 2;
    return tb;
}

#define GDN_CONV_DISPATCH(fn)                                         \
    if (a.dtype == 0) {                                               \
        if (a.W == 2) return fn<uint16_t, 2>(a, stream);              \
        if (a.W == 3) return fn<uint16_t, 3>(a, stream);              \
        return fn<uint16_t, 4>(a, stream);                            \
    }                                                                 \
    if (a.W == 2) return fn<float, 2>(a, stream);                     \
    if (a.W == 3) return fn<float, 3>(a, stream);                     \
    return fn<float, 4>(a, stream)

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t stream) { GDN_CONV_DISPATCH(conv_fwd_w); }
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t stream) { GDN_CONV_DISPATCH(conv_bwd_w); }
cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t stream) { GDN_CONV_DISPATCH(conv_step_w); }

long long conv_partial_rows(long long slots) { return (slots + kRows - 1) / kRows; }

cudaError_t launch_column_sum(const ColumnSumArgs& a, cudaStream_t stream) {
    if (a.cols == 0) return cudaSuccess;
    column_sum_kernel<<<static_cast<unsigned>((a.cols + kLanes - 1) / kLanes), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
