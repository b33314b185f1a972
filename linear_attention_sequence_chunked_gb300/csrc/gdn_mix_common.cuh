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

// E consecutive elements as they lie in memory, held as the 32-bit words that
// wide loads fill, so that nothing touches them before they are unpacked.
template <typename T, int E>
struct alignas(sizeof(T) * E >= 16 ? 16 : (sizeof(T) * E + 3) / 4 * 4) Raw {
    static constexpr int kWords = (static_cast<int>(sizeof(T)) * E + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

// Read-only loads under a predicate, zero where it is false.  Written as
// volatile assembly so that a prefetch stays where it is issued and nothing
// that uses the value is folded into the branch around it.
__device__ __forceinline__ uint4 load_16(const void* p, bool on) {
    uint4 r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
        "mov.b32 %3, 0;\n\t@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
        : "l"(p), "r"(static_cast<int>(on)));
    return r;
}
__device__ __forceinline__ uint2 load_8(const void* p, bool on) {
    uint2 r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.nc.v2.b32 {%0, %1}, [%2];\n\t}"
        : "=&r"(r.x), "=&r"(r.y)
        : "l"(p), "r"(static_cast<int>(on)));
    return r;
}
__device__ __forceinline__ uint32_t load_4(const void* p, bool on) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}"
                 : "=&r"(r)
                 : "l"(p), "r"(static_cast<int>(on)));
    return r;
}

// One element where it lies, as the 32-bit register that the load fills (no
// conversion before its use); `on` false: zero.
template <typename T, bool PRED = true>
__device__ __forceinline__ uint32_t load_one(const T* p, bool on = true) {
    uint32_t r;
    if constexpr (PRED && sizeof(T) == 2)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
                     : "=&r"(r)
                     : "l"(p), "r"(static_cast<int>(on)));
    else if constexpr (PRED)
        r = load_4(p, on);
    else if constexpr (sizeof(T) == 2)
        asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(r) : "l"(p));
    else
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}
template <typename T>
__device__ __forceinline__ float one_f32(uint32_t r) {
    return __uint_as_float(sizeof(T) == 2 ? r << 16 : r);
}

// Elements [0, n) of the E at p (n < E at the right edge of a row; 0: none).
// VEC: p is aligned to the vector and n is 0 or E, one access of up to 16
// bytes each; else element by element.
template <typename T, int E, bool VEC = true>
__device__ __forceinline__ Raw<T, E> load_raw(const T* p, int n) {
    Raw<T, E> r;
    constexpr int bytes = static_cast<int>(sizeof(T)) * E;
    if constexpr (VEC && bytes % 16 == 0) {
#pragma unroll
        for (int i = 0; i < bytes / 16; ++i) {
            const uint4 x = load_16(reinterpret_cast<const uint4*>(p) + i, n > 0);
            r.w[4 * i] = x.x; r.w[4 * i + 1] = x.y; r.w[4 * i + 2] = x.z; r.w[4 * i + 3] = x.w;
        }
    } else if constexpr (VEC && bytes == 8) {
        const uint2 x = load_8(p, n > 0);
        r.w[0] = x.x; r.w[1] = x.y;
    } else if constexpr (VEC && bytes == 4) {
        r.w[0] = load_4(p, n > 0);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < E; ++i) r.w[i] = load_4(p + i, i < n);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            r.w[i / 2] = load_one(p + i, i < n);
            if (i + 1 < E) r.w[i / 2] |= load_one(p + i + 1, i + 1 < n) << 16;
        }
    }
    return r;
}

template <typename T, int E, bool VEC = true>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, E>& r, int n) {
    constexpr int bytes = static_cast<int>(sizeof(T)) * E;
    if constexpr (VEC && bytes >= 4) {
        if (n <= 0) return;
        if constexpr (bytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < bytes / 16; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
        } else if constexpr (bytes == 8) {
            *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
        } else {
            *reinterpret_cast<uint32_t*>(p) = r.w[0];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (i >= n) continue;
            if constexpr (sizeof(T) == 4)
                p[i] = __uint_as_float(r.w[i]);
            else
                p[i] = static_cast<uint16_t>(i & 1 ? r.w[i / 2] >> 16 : r.w[i / 2]);
        }
    }
}

template <typename T, int E>
__device__ __forceinline__ void unpack(const Raw<T, E>& r, float* x) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = r.get(i);
}
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> pack(const float* x) {
    Raw<T, E> r;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if constexpr (sizeof(T) == 4)
            r.w[i] = __float_as_uint(x[i]);
        else if (i + 1 == E && !(i & 1))
            r.w[i / 2] = f32_to_bf16(x[i]);
        else if (!(i & 1))
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.w[i / 2]) : "f"(x[i + 1]), "f"(x[i]));
    }
    return r;
}

// A thread's own copies from global to shared memory (it alone reads them, so a
// wait is all they need): E elements of one row, zeros where `on` is false.
template <typename T, int E>
__device__ __forceinline__ void copy_async(void* to, const T* from, bool on) {
    constexpr int bytes = static_cast<int>(sizeof(T)) * E;
    static_assert(bytes == 4 || bytes == 8 || bytes == 16, "copy size");
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(on ? bytes : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(from), "n"(bytes), "r"(on ? bytes : 0) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;

// 2^x in one instruction (relative error about 2^-22, results below the
// normal range become zero)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x in one instruction (relative error about 2^-23; 0 for huge x)
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// softplus without overflow and with a small relative error where it is small
// (a few ulp near zero, about |x| 2^-24 from the product before the exponential
// far below it): max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1], by the series of
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, up to s^13 (the next term is
// below 2^-25 of the sum).  A third of log1pf's instructions and no branch.
__device__ __forceinline__ float softplus(float x) {
    const float e = ex2(-kLog2e * fabsf(x));
    const float s = e * rcp(2.f + e), q = s * s;
    float r = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    r = fmaf(q, r, 1.f / 9.f);
    r = fmaf(q, r, 1.f / 7.f);
    r = fmaf(q, r, 1.f / 5.f);
    r = fmaf(q, r, 1.f / 3.f);
    r = fmaf(q, r, 1.f);
    return fmaf(2.f * s, r, fmaxf(x, 0.f));
}

// Two fp32 values in a register pair: one instruction works on both.
struct Two {
    unsigned long long v;
};
__device__ __forceinline__ Two two(float lo, float hi) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(Two a, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two ex2_2(Two a) {
    float lo, hi;
    split(a, lo, hi);
    return two(ex2(lo), ex2(hi));
}

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

__device__ __forceinline__ Two rcp_2(Two a) {
    float lo, hi;
    split(a, lo, hi);
    return two(rcp(lo), rcp(hi));
}
__device__ __forceinline__ Two sigmoid_2(Two x) {
    return rcp_2(add2(two(1.f, 1.f), ex2_2(mul2(two(-kLog2e, -kLog2e), x))));
}

// softplus of both halves
__device__ __forceinline__ Two softplus_2(Two x) {
    float a, b;
    split(x, a, b);
    const Two e = two(ex2(-kLog2e * fabsf(a)), ex2(-kLog2e * fabsf(b)));
    const Two s = mul2(e, rcp_2(add2(two(2.f, 2.f), e))), q = mul2(s, s);
    const auto same = [](float c) { return two(c, c); };
    Two r = fma2(q, same(1.f / 13.f), same(1.f / 11.f));
    r = fma2(q, r, same(1.f / 9.f));
    r = fma2(q, r, same(1.f / 7.f));
    r = fma2(q, r, same(1.f / 5.f));
    r = fma2(q, r, same(1.f / 3.f));
    r = fma2(q, r, same(1.f));
    return fma2(add2(s, s), r, two(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}

// Pairs of elements: E elements are (E + 1) / 2 pairs (an odd one is alone in
// its pair's low half).
template <typename T, int E>
__device__ __forceinline__ void unpack_2(const Raw<T, E>& r, Two* x) {
#pragma unroll
    for (int i = 0; i < (E + 1) / 2; ++i) x[i] = two(r.get(2 * i), 2 * i + 1 < E ? r.get(2 * i + 1) : 0.f);
}
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> pack_2(const Two* x) {
    float v[E + 1];
#pragma unroll
    for (int i = 0; i < (E + 1) / 2; ++i) split(x[i], v[2 * i], v[2 * i + 1]);
    return pack<T, E>(v);
}

}  // namespace mix
}  // namespace gdn
