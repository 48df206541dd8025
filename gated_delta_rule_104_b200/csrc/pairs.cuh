// Pairs of floats, for the norm, the convolution and the scan (apart from
// common.cuh, to whose code the recorded memory traffic of the log's read is tied).
#pragma once

#include "common.cuh"

namespace dl {

// Pairs of floats in 64-bit registers: one instruction for two products or sums.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) { return pair(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ uint64_t pair_bf(uint32_t w) { return pair(bf_lo(w), bf_hi(w)); }  // of a bfloat16 pair
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ void unpair(uint64_t p, uint32_t &a, uint32_t &b) { asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(p)); }
// A pair rounded to nearest-even bf16, packed.
__device__ __forceinline__ uint32_t pack_bf2(uint64_t p) {
    float a, b;
    unpair(p, a, b);
    return pack_bf2(a, b);
}

}  // namespace dl
