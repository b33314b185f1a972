// Products of registers (mma.sync), where an operand is too small or too rare for
// tensor memory: 16 rows of A by 8 columns of B, fp32 sums.  With g = lane / 4 and t =
// lane % 4 a lane holds D's rows g and g + 8, columns 2 t and 2 t + 1.
#pragma once

#include <stdint.h>

namespace gdn {
namespace mma {

// bf16: A (g, 2 t), (g + 8, 2 t), (g, 2 t + 8), (g + 8, 2 t + 8), B (2 t, g), (2 t + 8,
// g), each with its neighbour in k.
__device__ __forceinline__ void bf16_16x8x16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// tf32: A (g, t), (g + 8, t), (g, t + 4), (g + 8, t + 4), B (t, g), (t + 4, g).
__device__ __forceinline__ void tf32_16x8x8(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The nearest number of eleven bits.
__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
// One of a pair of bf16 as fp32 bits
__device__ __forceinline__ uint32_t widen(uint32_t pair, bool second) { return second ? pair & 0xffff0000u : pair << 16; }
__device__ __forceinline__ uint32_t word(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

}  // namespace mma
}  // namespace gdn
