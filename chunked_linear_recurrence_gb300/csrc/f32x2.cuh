// f32x2.cuh -- two FP32 operations an instruction, and BF16 pairs as pairs of floats.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace sfg {

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
// a - b
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  return fma2(b, make_float2(-1.f, -1.f), a);
}
// The two BF16 values of a word, the one in the low half first.
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 x) {
  __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<uint32_t*>(&v);
}

}  // namespace sfg
