// Loads, stores and conversions of short runs of bf16 or fp32 elements, shared
// by the pooled recurrent rule and the query/key norms.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace gdn {

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// fp32 -> the stored type: to nearest even, the type's own rounding.
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}

// Four consecutive elements, 8-byte (bf16) or 16-byte (fp32) aligned.
__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *p) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  return make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
}
__device__ __forceinline__ void st4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void st4(__nv_bfloat16 *p, float4 x) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(bf_pack(x.x, x.y), bf_pack(x.z, x.w));
}
// The same with the streaming hint, for data that is used once a call.
__device__ __forceinline__ float4 ld4_stream(const float *p) {
  return __ldcs(reinterpret_cast<const float4 *>(p));
}
__device__ __forceinline__ float4 ld4_stream(const __nv_bfloat16 *p) {
  const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(p));
  return make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
}
__device__ __forceinline__ void st4_stream(float *p, float4 x) {
  __stcs(reinterpret_cast<float4 *>(p), x);
}
__device__ __forceinline__ void st4_stream(__nv_bfloat16 *p, float4 x) {
  __stcs(reinterpret_cast<uint2 *>(p), make_uint2(bf_pack(x.x, x.y), bf_pack(x.z, x.w)));
}

// Two fp32 lanes of one instruction (a Blackwell fused multiply-add of pairs).
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ float2 unpair(Pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// a + b with a rounding of its own: two single additions, since a paired
// product and a paired addition come out as one fused operation.
__device__ __forceinline__ Pair add2_apart(Pair a, Pair b) {
  const float2 x = unpair(a), y = unpair(b);
  return pair(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

}  // namespace gdn
