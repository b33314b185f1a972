// Shared device helpers of the mixer operators around the delta rule: the
// short causal convolution, the selective state space scan and the group norm.
// Activations are bf16 (uint16_t bit patterns) or fp32 in memory and fp32 in
// registers; everything is rounded once, when it is stored.
#pragma once

#include "gdn_common.cuh"

namespace gdn {
namespace mix {

__device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
    if constexpr (sizeof(T) == 2)
        return f32_to_bf16(x);
    else
        return x;
}

// E consecutive elements as they lie in memory.  Alignment lets load_raw and
// store_raw move them in accesses of up to 16 bytes.
template <typename T, int E>
struct alignas(sizeof(T) * E >= 16 ? 16 : sizeof(T) * E) Raw {
    T v[E];
};

// Elements [0, n) of the E at p (n < E at the right edge of a row; 0: none).
// `vec`: p is aligned to the vector, so a full one moves in wide accesses.
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_raw(const T* p, bool vec, int n) {
    Raw<T, E> r;
    if (vec && n >= E) {
        if constexpr (sizeof(r) % 16 == 0) {
            uint4* d = reinterpret_cast<uint4*>(&r);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) d[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
        } else if constexpr (sizeof(r) == 8) {
            *reinterpret_cast<uint2*>(&r) = __ldg(reinterpret_cast<const uint2*>(p));
        } else if constexpr (sizeof(r) == 4) {
            *reinterpret_cast<uint32_t*>(&r) = __ldg(reinterpret_cast<const uint32_t*>(p));
        } else {
            r.v[0] = __ldg(p);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) r.v[i] = i < n ? __ldg(p + i) : from_f32<T>(0.f);
    }
    return r;
}

template <typename T, int E>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, E>& r, bool vec, int n) {
    if (vec && n >= E) {
        if constexpr (sizeof(r) % 16 == 0) {
            const uint4* s = reinterpret_cast<const uint4*>(&r);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = s[i];
        } else if constexpr (sizeof(r) == 8) {
            *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(&r);
        } else if constexpr (sizeof(r) == 4) {
            *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(&r);
        } else {
            p[0] = r.v[0];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < n) p[i] = r.v[i];
    }
}

template <typename T, int E>
__device__ __forceinline__ void unpack(const Raw<T, E>& r, float* x) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = to_f32(r.v[i]);
}
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> pack(const float* x) {
    Raw<T, E> r;
#pragma unroll
    for (int i = 0; i < E; ++i) r.v[i] = from_f32<T>(x[i]);
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// 2^x in one instruction (relative error about 2^-22, results below the
// normal range become zero)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// softplus without overflow and with a relative error of a few ulp where it
// is small: log1p(e), e = exp(-|x|) in (0, 1]
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(__expf(-fabsf(x))); }

// d silu(x) / dx with s = sigmoid(x)
__device__ __forceinline__ float dsilu(float x, float s) { return s * (1.f + x * (1.f - s)); }

// Token range [t0, t1) of sequence n in its batch row b, as seq_range, for
// callers whose threads look at different sequences.
__device__ __forceinline__ bool token_range(const int32_t* cu, int n, int N, int T, int* err, int& b, int& t0, int& t1) {
    if (cu == nullptr) {
        b = n;
        t0 = 0;
        t1 = T;
        return true;
    }
    b = 0;
    t0 = cu[n];
    t1 = cu[n + 1];
    const bool ok = t0 >= 0 && t1 >= t0 && t1 <= T && (n > 0 || t0 == 0) && (n < N - 1 || t1 == T);
    if (!ok) record_error(err, kErrBadSeqlens);
    return ok;
}

// Time blocks of `tb` tokens never straddle sequences.  Dense: every sequence
// has max(1, ceil(T / tb)) of them.  Packed: sequence n's start at
// cu[n] / tb + n, so T / tb + N slots hold them all and each sequence, an
// empty one too, has at least one.
__device__ __forceinline__ bool find_block(const int32_t* cu, int N, int T, int tb, long long slot, int* err, int& n,
                                           long long& c) {
    if (cu == nullptr) {
        const long long per = T > tb ? (T + tb - 1) / tb : 1;
        n = static_cast<int>(slot / per);
        c = slot % per;
        return true;
    }
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<long long>(cu[mid] / tb) + mid <= slot)
            lo = mid;
        else
            hi = mid - 1;
    }
    n = lo;
    c = slot - (static_cast<long long>(cu[n] / tb) + n);
    if (c < 0) record_error(err, kErrBadSeqlens);
    return c >= 0;
}

// Every offset, by the threads of one block: find_block may pass over a
// malformed one.
__device__ __forceinline__ void check_offsets(const int32_t* cu, int N, int T, int* err) {
    if (cu == nullptr) return;
    for (int n = threadIdx.x; n < N; n += blockDim.x) {
        int b, t0, t1;
        token_range(cu, n, N, T, err, b, t0, t1);
    }
}

}  // namespace mix
}  // namespace gdn
