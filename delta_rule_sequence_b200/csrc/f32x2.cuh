// f32x2.cuh -- packed pairs of floats in a 64-bit register pair: one instruction for two fp32 operations.
#pragma once

#include <stdint.h>

namespace prism {

using F2 = unsigned long long;

__device__ __forceinline__ F2 pack2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float first(F2 r) { return __uint_as_float((uint32_t)r); }
__device__ __forceinline__ float second(F2 r) { return __uint_as_float((uint32_t)(r >> 32)); }
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float total(F2 a) { return first(a) + second(a); }

// The same names on single floats, for code that is built for either.
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float total(float a) { return a; }

}  // namespace prism
