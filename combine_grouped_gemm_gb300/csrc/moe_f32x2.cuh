// Pairs of fp32 numbers in one 64-bit register pair, for the instructions that work on both at
// once: half as many instructions for products, and for those with a sum. (The compiler joins a
// product and a sum of pairs into one operation that rounds once. Where each is to be rounded by
// itself, scalars are used.)
#pragma once

#include <stdint.h>

namespace moe {

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pair(float x, float y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
__device__ __forceinline__ float2 halves(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float sum_of(f32x2 v) {
  const float2 f = halves(v);
  return f.x + f.y;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two bf16 values of a 32-bit word, and back.
__device__ __forceinline__ f32x2 pair_of_bf16(uint32_t v) {
  return pair(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16_of_pair(f32x2 v) {
  uint32_t r;
  const float2 f = halves(v);
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(f.x), "f"(f.y));
  return r;
}

}  // namespace moe
