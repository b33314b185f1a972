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
// 2 (forward) or 3 (reverse) accesses per element against 2W to 6W operations, an
// exponential and a reciprocal.  A thread takes E neighbouring channels over a
// block of consecutive tokens with the window in registers, so every input is
// read once but for W-1 rows per block; the next tokens' loads are in flight
// while these are computed, and the arithmetic runs on pairs of channels.
// Measured, bf16 and W = 4: forward 4 x 4096 x 6144 70 us, 5.8 TB/s, bound by
// HBM; gradients 16384 x 2048 57 us, 3.5 TB/s, 50 of them in the kernel, bound by
// instruction latencies (93 instructions per token of four channels, 13 warps per
// SM by 128 registers each; fewer registers or channels per thread are slower);
// step 64 x 6144 3.0 us, the latency of one access after another.
#include <type_traits>

#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kThreads = 256;

template <int W, int E>
__device__ __forceinline__ void load_weights(const float* weight, const float* bias, long long d0, Two (*w)[(E + 1) / 2],
                                             Two* bs) {
    float v[W][E + 1], b[E + 1];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float* row = weight + (d0 + e) * W;
        if constexpr (W == 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(row));
            v[0][e] = x.x; v[1][e] = x.y; v[2][e] = x.z; v[3][e] = x.w;
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) v[j][e] = __ldg(row + j);
        }
        b[e] = bias ? __ldg(bias + d0 + e) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < (E + 1) / 2; ++i) {
        const bool both = 2 * i + 1 < E;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = two(v[j][2 * i], both ? v[j][2 * i + 1] : 0.f);
        bs[i] = two(b[2 * i], both ? b[2 * i + 1] : 0.f);
    }
}

// The input at token t of a sequence that starts at t0: before it, a row of the
// W-1 inputs in its initial state (zeros without one).
template <typename T, int W, int E>
__device__ __forceinline__ Raw<T, E> input_at(const T* x, long long x_stride, const T* state, long long seq, int t, int t0,
                                              long long D) {
    if (t >= t0) return load_raw<T, E>(x + t * x_stride, E);
    return load_raw<T, E>(state ? state + (seq * (W - 1) + t - t0 + (W - 1)) * D : x, state ? E : 0);
}

// The next tokens of A arrays, U at a time, on their way to a thread's own part
// of shared memory, kAhead batches ahead (two, or one of 16-byte items);
// elements too small to copy (one bf16) wait in registers.
template <typename T, int E, int U, int A, int THREADS>
struct Ahead {
    static constexpr bool kCopies = sizeof(T) * E >= 4;
    static constexpr int kAhead = sizeof(T) * E == 4 || sizeof(T) * E == 8 ? 2 : 1;
    static constexpr int kStages = kAhead + 1;
    using Item = Raw<T, E>;
    Item (*buf)[U][A][THREADS];
    Item reg[U][A];
    int at = 0;  // stage of the batch that get() looks at

    // from(k, a): where item (k, a) of the next batch lies; on(k): whether it does
    template <typename F, typename G>
    __device__ __forceinline__ void issue(int ahead, F from, G on) {  // `ahead` batches after that
        const int st = (at + ahead) % kStages;
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int a = 0; a < A; ++a) {
                if constexpr (kCopies)
                    copy_async<T, E>(&buf[st][k][a][threadIdx.x], from(k, a), on(k));
                else
                    reg[k][a] = load_raw<T, E>(from(k, a), on(k) ? E : 0);
            }
        if constexpr (kCopies) commit_copies();
    }
    __device__ __forceinline__ void wait() {
        if constexpr (kCopies) wait_copies<kAhead - 1>();
    }
    __device__ __forceinline__ Item get(int k, int a) const {
        if constexpr (kCopies)
            return buf[at][k][a][threadIdx.x];
        else
            return reg[k][a];
    }
    __device__ __forceinline__ void next() { at = (at + 1) % kStages; }
};

template <typename T, int W, int E>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(const ConvArgs p) {
    constexpr int U = 4, P = (E + 1) / 2;  // tokens whose loads are in flight together, pairs of channels
    using In = Ahead<T, E, U, 1, kThreads>;
    __shared__ typename In::Item buf[In::kCopies ? In::kStages : 1][U][1][kThreads];
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
    const T* s0 = p.initial_state ? static_cast<const T*>(p.initial_state) + d0 : nullptr;
    const long long begin = t0 + c * p.tb;
    const int tb = static_cast<int>(min(begin, static_cast<long long>(t1)));
    const int te = static_cast<int>(min(begin + p.tb, static_cast<long long>(t1)));
    if (p.final_state && te == t1 && (tb < te || c == 0)) {
        T* fs = static_cast<T*>(p.final_state) + d0;
#pragma unroll
        for (int r = 0; r < W - 1; ++r)
            store_raw<T, E>(fs + (static_cast<long long>(n) * (W - 1) + r) * p.D,
                            input_at<T, W, E>(x, p.x_stride, s0, n, t1 - (W - 1) + r, t0, p.D), E);
    }
    if (tb >= te) return;
    Two w[W][P], bs[P], win[W - 1 + U][P];
    load_weights<W, E>(p.weight, p.bias, d0, w, bs);
#pragma unroll
    for (int r = 0; r < W - 1; ++r)
        unpack_2<T, E>(input_at<T, W, E>(x, p.x_stride, s0, n, tb - (W - 1) + r, t0, p.D), win[r]);
    x += tb * p.x_stride;
    T* y = static_cast<T*>(p.y) + (static_cast<long long>(b) * p.T + tb) * p.D + d0;
    In in{buf};
    auto load = [&](int ahead, int left) {
        in.issue(ahead, [&](int k, int) { return x + (k < left ? k : 0) * p.x_stride; }, [&](int k) { return k < left; });
        if (left > U) x += U * p.x_stride;  // the last batch stays inside the row
    };
    int asked = te - tb;  // tokens not yet asked for
#pragma unroll
    for (int i = 0; i < In::kAhead; ++i, asked -= U) load(i, asked);
    for (int left = te - tb; left > 0; left -= U, asked -= U) {
        in.wait();
#pragma unroll
        for (int k = 0; k < U; ++k) unpack_2<T, E>(in.get(k, 0), win[W - 1 + k]);
        load(In::kAhead, asked);
        in.next();
#pragma unroll
        for (int k = 0; k < U; ++k) {
            Two o[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                o[i] = bs[i];
#pragma unroll
                for (int j = 0; j < W; ++j) o[i] = fma2(w[j][i], win[k + j][i], o[i]);
                if (p.activation) o[i] = mul2(o[i], sigmoid_2(o[i]));
            }
            if (k < left) store_raw<T, E>(y + k * static_cast<long long>(p.D), pack_2<T, E>(o), E);
        }
        y += U * static_cast<long long>(p.D);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < P; ++i) win[j][i] = win[j + U][i];
    }
}

// One block: kLanes channel vectors x kRows time blocks; each thread walks its
// time block (and the W-1 tokens after it, whose dp reach back into it), then
// the block's partial weight gradients are summed over its rows in order.
constexpr int kLanes = 32;
constexpr int kRows = 4;

template <typename T, int W, int E>
__global__ void __launch_bounds__(kLanes * kRows, 4) conv_bwd_kernel(const ConvArgs p) {
    constexpr int U = 4, P = (E + 1) / 2;
    using In = Ahead<T, E, U, 2, kLanes * kRows>;
    __shared__ typename In::Item buf[In::kCopies ? In::kStages : 1][U][2][kLanes * kRows];
    __shared__ float red[kRows][kLanes][E + 1];
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.cu_seqlens, p.N, p.T, p.err);
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const long long d0 = (static_cast<long long>(blockIdx.y) * kLanes + lane) * E;
    const long long slot = static_cast<long long>(blockIdx.x) * kRows + row;
    const Two zero = two(0.f, 0.f);
    Two dw[W + 1][P];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) dw[j][i] = zero;
    int n, b, t0, t1;
    long long c;
    if (d0 < p.D && slot < p.slots && find_block(p.cu_seqlens, p.N, p.T, p.tb, slot, p.err, n, c) &&
        token_range(p.cu_seqlens, n, p.N, p.T, p.err, b, t0, t1)) {
        const T* x = static_cast<const T*>(p.x) + static_cast<long long>(b) * p.T * p.x_stride + d0;
        const T* s0 = p.initial_state ? static_cast<const T*>(p.initial_state) + d0 : nullptr;
        const T* dfs = p.d_final_state ? static_cast<const T*>(p.d_final_state) + d0 : nullptr;
        const long long begin = t0 + c * p.tb;
        const int tb = static_cast<int>(min(begin, static_cast<long long>(t1)));
        const int te = static_cast<int>(min(begin + p.tb, static_cast<long long>(t1)));
        if (tb < te || c == 0) {
            Two w[W][P], bs[P], win[W - 1 + U][P], dp[W - 1 + U][P];
            load_weights<W, E>(p.weight, p.bias, d0, w, bs);
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
                unpack_2<T, E>(input_at<T, W, E>(x, p.x_stride, s0, n, tb - (W - 1) + r, t0, p.D), win[r]);
#pragma unroll
                for (int i = 0; i < P; ++i) dp[r][i] = zero;
            }
            const long long base = (static_cast<long long>(b) * p.T + tb) * p.D + d0;
            const T* dy = static_cast<const T*>(p.d_out) + base;
            T* dx = static_cast<T*>(p.dx) + base - (W - 1) * static_cast<long long>(p.D);
            T* ds0 = p.d_initial_state && tb == t0
                         ? static_cast<T*>(p.d_initial_state) + static_cast<long long>(n) * (W - 1) * p.D + d0 : nullptr;
            x += tb * p.x_stride;
            In in{buf};
            const int end = min(t1, te + W - 1);
            int asked = tb;  // the next token to ask for
            auto load = [&](int ahead) {
                in.issue(ahead,
                         [&](int k, int a) {
                             const int kk = asked + k < end ? k : 0;
                             return a ? dy + kk * static_cast<long long>(p.D) : x + kk * p.x_stride;
                         },
                         [&](int k) { return asked + k < end; });
                asked += U;
                if (asked < end) {  // else: nothing is read there any more
                    x += U * p.x_stride;
                    dy += U * static_cast<long long>(p.D);
                }
            };
            // U tokens from t.  kInner: all of them and the inputs whose gradients
            // they complete lie inside the block, away from the sequence's ends.
            auto step = [&](int t, auto inner) {
                constexpr bool kInner = decltype(inner)::value;
                Two g[U][P];
                in.wait();
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    unpack_2<T, E>(in.get(k, 0), win[W - 1 + k]);
                    unpack_2<T, E>(in.get(k, 1), g[k]);
                }
                load(In::kAhead);
                in.next();
#pragma unroll
                for (int k = 0; k < U; ++k) {
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        Two d = g[k][i];
                        if (p.activation) {
                            Two acc = bs[i];
#pragma unroll
                            for (int j = 0; j < W; ++j) acc = fma2(w[j][i], win[k + j][i], acc);
                            const Two s = sigmoid_2(acc), one = two(1.f, 1.f), neg = two(-1.f, -1.f);
                            // silu' = s (1 + p (1 - s))
                            d = mul2(d, mul2(s, fma2(acc, fma2(s, neg, one), one)));
                        }
                        if (!kInner && t + k >= t1) d = zero;
                        dp[W - 1 + k][i] = d;
                        if (!kInner && t + k >= te) d = zero;  // the next block's
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][i] = fma2(d, win[k + j][i], dw[j][i]);
                        dw[W][i] = add2(dw[W][i], d);
                    }
                    // input s has now seen every token it feeds
                    const int s = t + k - (W - 1);
                    if (kInner || (s < te && (s >= tb || ds0))) {
                        Two o[P];
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            o[i] = zero;
#pragma unroll
                            for (int j = 0; j < W; ++j) o[i] = fma2(w[j][i], dp[W - 1 + k - j][i], o[i]);
                        }
                        T* to = dx + k * static_cast<long long>(p.D);
                        if constexpr (!kInner) {
                            if (dfs && s >= t1 - (W - 1)) {  // one of the rows the final state holds
                                Two v[P];
                                unpack_2<T, E>(load_raw<T, E>(dfs + (static_cast<long long>(n) * (W - 1) + s - t1 + (W - 1)) * p.D, E), v);
#pragma unroll
                                for (int i = 0; i < P; ++i) o[i] = add2(o[i], v[i]);
                            }
                            if (s < tb) to = ds0 + (s - t0 + (W - 1)) * static_cast<long long>(p.D);
                        }
                        store_raw<T, E>(to, pack_2<T, E>(o), E);
                    }
                }
                dx += U * static_cast<long long>(p.D);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        win[j][i] = win[j + U][i];
                        dp[j][i] = dp[j + U][i];
                    }
            };
#pragma unroll
            for (int i = 0; i < In::kAhead; ++i) load(i);
            int t = tb;
            step(t, std::false_type{});
            for (t += U; t + U <= te; t += U) step(t, std::true_type{});
            for (; t < te + W - 1; t += U) step(t, std::false_type{});
        }
    }
    // partial [block row][W + 1][D]: the weights' gradients, then the bias's
#pragma unroll
    for (int j = 0; j <= W; ++j) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float lo, hi;
            split(dw[j][i], lo, hi);
            red[row][lane][2 * i] = lo;
            if (2 * i + 1 < E) red[row][lane][2 * i + 1] = hi;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kLanes * E; i += kLanes * kRows) {
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
    constexpr int P = (E + 1) / 2;
    Two w[W][P], o[P];
    load_weights<W, E>(p.weight, p.bias, d0, w, o);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        Two v[P];
        unpack_2<T, E>(in[j], v);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = fma2(w[j][i], v[i], o[i]);
        if (j > 0) store_raw<T, E>(so + (j - 1) * static_cast<long long>(p.D), in[j], E);
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (p.activation) o[i] = mul2(o[i], sigmoid_2(o[i]));
    store_raw<T, E>(y, pack_2<T, E>(o), E);
}

// Sums of a [rows][cols] partial array over its rows, in a fixed order: 32
// columns per block, 32 threads down each (35 x 10240: 5 us, mostly latency).  Columns land in up to three outputs
// of c0, c1 and the rest (null: dropped); with W > 0 the array is
// [rows][W + 1][D] and the first output (D, W).
constexpr int kDown = 32;
__global__ void __launch_bounds__(32 * kDown) column_sum_kernel(const ColumnSumArgs p) {
    __shared__ float red[kDown][33];
    const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
    const long long col = static_cast<long long>(blockIdx.x) * 32 + lane;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < p.cols) {
        const float* src = p.partial + col;
        for (int r = row; r < p.rows; r += 4 * kDown) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r + k * kDown < p.rows) s[k] += __ldg(src + (r + k * kDown) * p.stride);
        }
    }
    red[row][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (row != 0 || col >= p.cols) return;
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kDown; ++r) v += red[r][lane];
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

// Four channels per thread where a row's width, stride and address allow it,
// else two (bf16), else one: neighbouring threads then still read neighbouring
// elements (4 x 4096 x 6144 forward: 68 us by four, 78 by two; 16384 x 2048
// reverse: 57 by four, 66 by two, 99 by one; 1024 x 6142 step: 17 by two, 27 by
// one).
template <typename T, int W>
cudaError_t conv_fwd_w(const ConvArgs& a, cudaStream_t stream) {
    constexpr int E = 4;
    if (rows_take<T>(a.x, a.x_stride, a.D, E)) return conv_fwd_e<T, W, E>(a, stream);
    if constexpr (sizeof(T) == 2)
        if (rows_take<T>(a.x, a.x_stride, a.D, 2)) return conv_fwd_e<T, W, 2>(a, stream);
    return conv_fwd_e<T, W, 1>(a, stream);
}

template <typename T, int W, int E>
cudaError_t conv_bwd_e(const ConvArgs& a, cudaStream_t stream) {
    dim3 grid(static_cast<unsigned>((a.slots + kRows - 1) / kRows),
              static_cast<unsigned>((a.D + kLanes * E - 1) / (kLanes * E)));
    conv_bwd_kernel<T, W, E><<<grid, kLanes * kRows, 0, stream>>>(a);
    return cudaGetLastError();
}
template <typename T, int W>
cudaError_t conv_bwd_w(const ConvArgs& a, cudaStream_t stream) {
    if (rows_take<T>(a.x, a.x_stride, a.D, 4)) return conv_bwd_e<T, W, 4>(a, stream);
    if constexpr (sizeof(T) == 2)
        if (rows_take<T>(a.x, a.x_stride, a.D, 2)) return conv_bwd_e<T, W, 2>(a, stream);
    return conv_bwd_e<T, W, 1>(a, stream);
}

template <typename T, int W, int E>
cudaError_t conv_step_e(const ConvStepArgs& a, cudaStream_t stream) {
    const long long threads = static_cast<long long>(a.B) * (a.D / E);
    conv_step_kernel<T, W, E><<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}
template <typename T, int W>
cudaError_t conv_step_w(const ConvStepArgs& a, cudaStream_t stream) {
    if (rows_take<T>(a.x, a.x_stride, a.D, 4)) return conv_step_e<T, W, 4>(a, stream);
    if constexpr (sizeof(T) == 2)
        if (rows_take<T>(a.x, a.x_stride, a.D, 2)) return conv_step_e<T, W, 2>(a, stream);
    return conv_step_e<T, W, 1>(a, stream);
}

}  // namespace

// Tokens per thread: long blocks re-read fewer rows at their edges (W-1 per
// block) and leave fewer partial rows, short ones give small inputs enough
// threads (16384 x 2048 backward: 128 tokens 57 us, 64 tokens 59 us; 16384 x
// 6144 forward: 64 tokens 68 us, 32 tokens 70 us).  How many are enough: in
// reverse 60 thousand (4 x 1024 x 4096 fp32 34 us, 41 with half, 38 with twice as
// many), forward 50 thousand (2048 x 6144 bf16 11.4 us, 14.6 with 200), 200 where
// a thread's items of 16 bytes leave room for one batch ahead only (4 x 1024 x
// 4096 fp32 23.5 us, 25.3 with 50).
int conv_block_tokens(int B, int T, int D, int backward, int dtype) {
    const int channels = D % 4 == 0 ? 4 : D % 2 == 0 ? 2 : 1;  // of a thread, if it is aligned
    const long long work = static_cast<long long>(B) * T * (D / channels);
    const long long enough = backward ? 60000 : dtype == 1 && channels == 4 ? 200000 : 50000;
    int tb = backward ? 128 : 64;
    while (tb > 4 && work / tb < enough) tb /= 2;
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
    column_sum_kernel<<<static_cast<unsigned>((a.cols + 31) / 32), 32 * kDown, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
