// Pairs of fp32 in one register pair: one instruction for two sums or products.
#pragma once

#include <cstdint>

namespace tsfn {

__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// a + b of products, each rounded on its own: the compiler fuses mul2 into an add2 after it, but
// not into this.  one: 1, of which it must not know.
__device__ __forceinline__ uint64_t add_products2(uint64_t a, uint64_t b, uint64_t one) { return fma2(a, one, b); }

// The two bf16 of a word.
__device__ __forceinline__ uint64_t widen2(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

__device__ __forceinline__ uint64_t twice(float v) { return pair(v, v); }

}  // namespace tsfn
