// Norm of every query's and key's head with the rotation by position in the
// same pass, and its reverse mode.
//
//   n = x (mean(x^2) + eps)^-1/2 weight;   pair (u, v) of n at position p and
//   frequency f:  (u cos(p f) - v sin(p f), v cos(p f) + u sin(p f))
//
// A head of d channels lies across d / 8 lanes, each with two pieces of four
// channels that hold both halves of its four pairs, so a row needs no exchange
// but its sum of squares.  Bound by HBM: each row is read once and written once.
// A block takes a few tokens with all their heads and forms their cosines and
// sines once, in shared memory.
//
// The angle p f is formed in turns, in fixed point: f / 2 pi as a 64-bit
// fraction (24 bits of f times 64 bits of 1 / 2 pi), multiplied by the integer
// position modulo 2^64.  Whole turns drop out of the product by themselves and
// the fraction keeps 2^-33 turns at a position of 2^31, where a product in fp32
// would have lost every bit of it.
#include <algorithm>

#include "gdn_kernels.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kThreads = 256;

// f / 2 pi modulo 1, in units of 2^-64.
__device__ __forceinline__ unsigned long long turns_of(float f) {
    const uint32_t bits = __float_as_uint(f);
    const int exp = static_cast<int>((bits >> 23) & 255u);
    const unsigned long long mant = exp ? (bits & 0x7fffffu) | 0x800000u : 0;  // |f| = mant 2^(exp - 150)
    constexpr unsigned long long kInv2Pi = 0x28be60db9391054aULL;  // 2^64 / 2 pi
    const unsigned long long lo = mant * kInv2Pi, hi = __umul64hi(mant, kInv2Pi);
    const int shift = 150 - exp;  // the 128-bit product, this many places to the right
    unsigned long long r;
    if (shift >= 128)
        r = 0;
    else if (shift >= 64)
        r = hi >> (shift - 64);
    else if (shift > 0)
        r = (hi << (64 - shift)) | (lo >> shift);
    else
        r = shift > -64 ? lo << -shift : 0;
    return bits >> 31 ? 0 - r : r;
}

// cos and sin of an angle in units of 2^-64 turns: the nearest quarter turn,
// then the Taylor series on [-pi/4, pi/4] up to x^9 and x^10 (remainders below
// 2^-28).
__device__ __forceinline__ float2 cos_sin(unsigned long long phase) {
    const uint32_t q = static_cast<uint32_t>((phase + (1ull << 61)) >> 62);
    const long long rest = static_cast<long long>(phase - (static_cast<unsigned long long>(q) << 62));
    const float x = static_cast<float>(static_cast<int>(rest >> 30)) * (6.283185307179586f * 5.8207660913467407e-11f);
    const float x2 = x * x;
    float s = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(x2, s, 1.f / 120.f);
    s = fmaf(x2, s, -1.f / 6.f);
    s = fmaf(x2 * s, x, x);
    float c = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(x2, c, -1.f / 720.f);
    c = fmaf(x2, c, 1.f / 24.f);
    c = fmaf(x2, c, -0.5f);
    c = fmaf(x2, c, 1.f);
    const float cs = q & 1 ? s : c, sn = q & 1 ? c : s;
    return make_float2(q == 1 || q == 2 ? -cs : cs, q >= 2 ? -sn : sn);
}

__device__ __forceinline__ int position(const RopeArgs& p, long long tok) {
    if (p.positions) return p.positions[tok];
    if (p.cu_seqlens == nullptr) return static_cast<int>(tok % p.T);
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[mid] <= tok)
            lo = mid;
        else
            hi = mid - 1;
    }
    return static_cast<int>(tok - p.cu_seqlens[lo]);
}

// cos and sin of the tile's tokens: cs[token][pair] and, `pairs` further, sines
__device__ __forceinline__ void fill_angles(const RopeArgs& p, long long tok0, int nt, float* cs, int* pos) {
    const int nf = p.pairs;
    for (int i = threadIdx.x; i < nt; i += kThreads) pos[i] = position(p, tok0 + i);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * nf; i += kThreads) {
        const int t = i / nf, f = i - t * nf;
        const float w = p.inv_freq[f];
        float2 v = cos_sin(static_cast<unsigned long long>(static_cast<long long>(pos[t])) * turns_of(w));
        if ((__float_as_uint(w) & 0x7f800000u) == 0x7f800000u) v = make_float2(w - w, w - w);  // NaN
        cs[2 * t * nf + f] = v.x;
        cs[(2 * t + 1) * nf + f] = v.y;
    }
    __syncthreads();
}

// Where lane j's two pieces of four channels begin, and the pairs they hold
// (first: its first frequency, or -1 where the lane's channels do not turn).
struct Pieces {
    int c0, c1, first;
};
template <bool NEXT>
__device__ __forceinline__ Pieces pieces(int j, int pairs) {
    if (8 * j >= 2 * pairs) return Pieces{8 * j, 8 * j + 4, -1};
    return NEXT ? Pieces{8 * j, 8 * j + 4, 4 * j} : Pieces{4 * j, pairs + 4 * j, 4 * j};
}

// Turns a lane's eight channels by +angle, or by -angle.
template <bool NEXT, bool BACK>
__device__ __forceinline__ void turn(float* n, const float* cs, int pairs, int first) {
    const float4 c4 = *reinterpret_cast<const float4*>(cs + first);
    const float4 s4 = *reinterpret_cast<const float4*>(cs + pairs + first);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w};
    const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float& u = n[NEXT ? 2 * i : i];
        float& v = n[NEXT ? 2 * i + 1 : 4 + i];
        const float sn = BACK ? -s[i] : s[i];
        const float a = fmaf(u, c[i], -v * sn), b = fmaf(v, c[i], u * sn);
        u = a;
        v = b;
    }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = LANES / 2; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

__device__ __forceinline__ void load_weight(const float* w, const Pieces& at, float* out) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        out[i] = w ? w[at.c0 + i] : 1.f;
        out[4 + i] = w ? w[at.c1 + i] : 1.f;
    }
}

// Rows of a tile: the q heads of all its tokens, then the k heads.
struct Row {
    const void* x;
    long long in, out;  // element offsets
    int tok, key;
};

constexpr int kRows = 4;  // rows whose loads a lane has in flight together

template <typename T, int LANES, bool NEXT, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const RopeArgs p) {
    extern __shared__ __align__(16) float cs[];
    int* pos = reinterpret_cast<int*>(cs + 2 * p.tile * p.pairs);
    constexpr int d = 8 * LANES, TEAMS = kThreads / LANES;
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tile;
    const int nt = static_cast<int>(min(static_cast<long long>(p.tile), p.tokens - tok0));
    const int j = threadIdx.x % LANES, team = threadIdx.x / LANES;
    const Pieces at = pieces<NEXT>(j, p.pairs);
    fill_angles(p, tok0, nt, cs, pos);
#pragma unroll
    for (int key = 0; key < 2; ++key) {
        const T* src = static_cast<const T*>(key ? p.k : p.q) + tok0 * (key ? p.k_stride : p.q_stride);
        const long long stride = key ? p.k_stride : p.q_stride;
        const int heads = key ? p.Hk : p.H;
        T* dst = static_cast<T*>(key ? p.k_out : p.q_out) + tok0 * heads * d;
        float w[8];
        load_weight(key ? p.k_weight : p.q_weight, at, w);
        const int rows = nt * heads;
        for (int r0 = team; r0 < (rows + TEAMS - 1) / TEAMS * TEAMS; r0 += kRows * TEAMS) {
            Raw<T, 4> a[kRows], b[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int r = r0 + u * TEAMS;
                const int t = r / heads, h = r - t * heads;
                const T* x = src + t * stride + h * d;
                a[u] = load_raw<T, 4, VEC>(x + at.c0, r < rows ? 4 : 0);
                b[u] = load_raw<T, 4, VEC>(x + at.c1, r < rows ? 4 : 0);
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int r = r0 + u * TEAMS;
                float x[8];
                unpack<T, 4>(a[u], x);
                unpack<T, 4>(b[u], x + 4);
                float sq = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
                const float rs = rsqrtf(row_sum<LANES>(sq) * (1.f / d) + p.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= rs * w[i];
                if (r < rows) {
                    const int t = r / heads;
                    if (at.first >= 0) turn<NEXT, false>(x, cs + 2 * t * p.pairs, p.pairs, at.first);
                    T* y = dst + static_cast<long long>(r) * d;
                    store_raw<T, 4>(y + at.c0, pack<T, 4>(x), 4);
                    store_raw<T, 4>(y + at.c1, pack<T, 4>(x + 4), 4);
                }
            }
        }
    }
}

// With g the output's gradient turned back and n = x r:
//   dx = r (g w - n mean(g w n)),  dweight = sum over rows of g n
// A block walks every gridDim.x-th tile and keeps its sums of dweight; the
// blocks' partial sums are added in order by a second kernel.
template <typename T, int LANES, bool NEXT, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const RopeArgs p) {
    extern __shared__ __align__(16) float cs[];
    constexpr int d = 8 * LANES, TEAMS = kThreads / LANES;
    int* pos = reinterpret_cast<int*>(cs + 2 * p.tile * p.pairs);
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const int j = threadIdx.x % LANES, team = threadIdx.x / LANES;
    const Pieces at = pieces<NEXT>(j, p.pairs);
    float dw[2][8] = {};
    for (long long tok0 = static_cast<long long>(blockIdx.x) * p.tile; tok0 < p.tokens;
         tok0 += static_cast<long long>(gridDim.x) * p.tile) {
        const int nt = static_cast<int>(min(static_cast<long long>(p.tile), p.tokens - tok0));
        __syncthreads();  // the angles of the tile before are through
        fill_angles(p, tok0, nt, cs, pos);
#pragma unroll
        for (int key = 0; key < 2; ++key) {
            const long long stride = key ? p.k_stride : p.q_stride;
            const int heads = key ? p.Hk : p.H;
            const T* src = static_cast<const T*>(key ? p.k : p.q) + tok0 * stride;
            const T* grad = static_cast<const T*>(key ? p.dk_out : p.dq_out) + tok0 * heads * d;
            T* dst = static_cast<T*>(key ? p.dk : p.dq) + tok0 * heads * d;
            float w[8];
            load_weight(key ? p.k_weight : p.q_weight, at, w);
            const int rows = nt * heads;
            constexpr int R = kRows / 2;
            for (int r0 = team; r0 < (rows + TEAMS - 1) / TEAMS * TEAMS; r0 += R * TEAMS) {
                Raw<T, 4> a[R], b[R], ga[R], gb[R];
#pragma unroll
                for (int u = 0; u < R; ++u) {
                    const int r = r0 + u * TEAMS, n = r < rows ? 4 : 0;
                    const int t = r / heads, h = r - t * heads;
                    const T* x = src + t * stride + h * d;
                    const T* g = grad + static_cast<long long>(r) * d;
                    a[u] = load_raw<T, 4, VEC>(x + at.c0, n);
                    b[u] = load_raw<T, 4, VEC>(x + at.c1, n);
                    ga[u] = load_raw<T, 4>(g + at.c0, n);
                    gb[u] = load_raw<T, 4>(g + at.c1, n);
                }
#pragma unroll
                for (int u = 0; u < R; ++u) {
                    const int r = r0 + u * TEAMS;
                    float x[8], g[8];
                    unpack<T, 4>(a[u], x);
                    unpack<T, 4>(b[u], x + 4);
                    unpack<T, 4>(ga[u], g);
                    unpack<T, 4>(gb[u], g + 4);
                    if (at.first >= 0 && r < rows)
                        turn<NEXT, true>(g, cs + 2 * (r / heads) * p.pairs, p.pairs, at.first);
                    float sq = 0.f, dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sq = fmaf(x[i], x[i], sq);
                        dot = fmaf(g[i] * w[i], x[i], dot);
                    }
                    const float rs = rsqrtf(row_sum<LANES>(sq) * (1.f / d) + p.eps);
                    const float mean = row_sum<LANES>(dot) * (rs * (1.f / d));
                    if (r < rows) {
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float n = x[i] * rs;
                            dw[key][i] = fmaf(g[i], n, dw[key][i]);
                            o[i] = rs * fmaf(-n, mean, g[i] * w[i]);
                        }
                        T* y = dst + static_cast<long long>(r) * d;
                        store_raw<T, 4>(y + at.c0, pack<T, 4>(o), 4);
                        store_raw<T, 4>(y + at.c1, pack<T, 4>(o + 4), 4);
                    }
                }
            }
        }
    }
    if (!p.partial) return;
    __shared__ float sum[kThreads][9];  // nine: no two lanes of a warp on one bank
#pragma unroll
    for (int key = 0; key < 2; ++key) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[threadIdx.x][i] = dw[key][i];
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += kThreads) {
            const int jj = c / 8, i = c % 8;
            float s = 0.f;
            for (int t = 0; t < TEAMS; ++t) s += sum[t * LANES + jj][i];
            const Pieces q = pieces<NEXT>(jj, p.pairs);
            p.partial[(2ll * blockIdx.x + key) * d + (i < 4 ? q.c0 + i : q.c1 + i - 4)] = s;
        }
    }
}

template <typename T, int LANES, bool NEXT, bool VEC>
cudaError_t launch_one(const RopeArgs& a, bool backward, cudaStream_t stream) {
    const size_t smem = sizeof(float) * 2 * a.tile * a.pairs + sizeof(int) * a.tile;
    if (backward)
        rope_bwd_kernel<T, LANES, NEXT, VEC><<<a.blocks, kThreads, smem, stream>>>(a);
    else
        rope_fwd_kernel<T, LANES, NEXT, VEC><<<a.blocks, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}
template <typename T, int LANES>
cudaError_t launch_lanes(const RopeArgs& a, bool backward, cudaStream_t stream) {
    const auto off = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % (4 * sizeof(T)) != 0; };
    const bool vec = !off(a.q) && !off(a.k) && a.q_stride % 4 == 0 && a.k_stride % 4 == 0;
    if (vec) return a.interleaved ? launch_one<T, LANES, true, true>(a, backward, stream) : launch_one<T, LANES, false, true>(a, backward, stream);
    return a.interleaved ? launch_one<T, LANES, true, false>(a, backward, stream) : launch_one<T, LANES, false, false>(a, backward, stream);
}
template <typename T>
cudaError_t launch(const RopeArgs& a, bool backward, cudaStream_t stream) {
    switch (a.d) {
        case 32: return launch_lanes<T, 4>(a, backward, stream);
        case 64: return launch_lanes<T, 8>(a, backward, stream);
        case 128: return launch_lanes<T, 16>(a, backward, stream);
        case 256: return launch_lanes<T, 32>(a, backward, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// Tokens per block: some 96 rows, fewer where that leaves SMs without a block.
int rope_tile(long long tokens, int heads) {
    long long t = std::max(1, std::min(32, 96 / heads));
    t = std::min(t, std::max(1ll, tokens / (4 * 152)));
    return static_cast<int>(t);
}
long long rope_blocks(long long tokens, int heads, bool backward) {
    const long long tile = rope_tile(tokens, heads), n = (tokens + tile - 1) / tile;
    return backward ? std::min(n, 4ll * 152) : n;
}

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch<float>(a, false, stream) : launch<uint16_t>(a, false, stream);
}
cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch<float>(a, true, stream) : launch<uint16_t>(a, true, stream);
}

}  // namespace gdn
