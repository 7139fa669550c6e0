// Arithmetic on two fp32 values at once (sm_100's packed forms, each half rounded
// like the single operation).
#pragma once

namespace infini {

// float2, or float for single channels.
template <int V> struct LaneOf { using type = float2; };
template <> struct LaneOf<1> { using type = float; };
__device__ __forceinline__ unsigned long long bits(float2 x) {
  return (unsigned long long)__float_as_uint(x.y) << 32 | __float_as_uint(x.x);
}
__device__ __forceinline__ float2 pair(unsigned long long x) {
  return {__uint_as_float((unsigned)x), __uint_as_float((unsigned)(x >> 32))};
}
__device__ __forceinline__ float2 mul(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ float2 add(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(d);
}
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sum(float2 x) { return x.x + x.y; }
__device__ __forceinline__ float sum(float x) { return x; }
__device__ __forceinline__ void put(float* to, int e, float2 x) {
  to[2 * e] = x.x;
  to[2 * e + 1] = x.y;
}
__device__ __forceinline__ void put(float* to, int e, float x) { to[e] = x; }
template <typename L> __device__ __forceinline__ L both(float x);
template <> __device__ __forceinline__ float2 both<float2>(float x) { return {x, x}; }
template <> __device__ __forceinline__ float both<float>(float x) { return x; }

}  // namespace infini
