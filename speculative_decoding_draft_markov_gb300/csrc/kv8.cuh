// The 8-bit paged cache: a slot holds one position's K and V of one KV head, D values of e4m3 each, and an exponent byte
// for each of the two in kv_scale[page, head, slot, 2].  Their value is code * 2^(byte - 127); byte 255: the vector is NaN.
//
// The factor is a power of two: a floating code loses nothing by that (its relative error is 2^-4 wherever it is normal),
// and every value of the cache is then exact in bf16, in fp16 up to a factor, and in fp32.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dspark {
namespace kv8 {

constexpr uint32_t kNan = 255;  // exponent byte of a vector that holds a NaN or an infinity

// 2^e, -126 <= e <= 127
__host__ __device__ __forceinline__ float power(int e) {
#ifdef __CUDA_ARCH__
  return __uint_as_float(uint32_t(e + 127) << 23);
#else
  union { uint32_t u; float f; } x;
  x.u = uint32_t(e + 127) << 23;
  return x.f;
#endif
}

// The exponent byte of a vector whose largest magnitude has the bits `top` (of fp32, without the sign): the smallest power of two
// 2^e with top <= 448 * 2^e, at least 2^-126.  448 = 1.75 * 2^8.
__host__ __device__ __forceinline__ uint32_t exponent_byte(uint32_t top) {
  if (top >= 0x7F800000u) return kNan;
  const int e = int(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return uint32_t((e < -126 ? -126 : e) + 127);
}
// The factor that an exponent byte stands for.  Byte 0, which no append writes, counts as 1.
__device__ __forceinline__ float factor(uint32_t byte) {
  return byte == kNan ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(max(byte, 1u) << 23);
}

// Two codes, a in the low byte: rounded to nearest, ties to even; what lies beyond 448 becomes 448.
__device__ __forceinline__ uint32_t code2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}
// The values of two codes, as halves (exact).
__device__ __forceinline__ uint32_t halves(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
__device__ __forceinline__ float2 values(uint32_t codes) {
  const uint32_t h = halves(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two halves as codes of their first parts and of what those leave (exact in fp16: a part has four bits), times 16 if asked.
template <bool kTimes16>
__device__ __forceinline__ void split2(__half2 x, uint32_t& first, uint32_t& rest) {
  uint16_t f, r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(f) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  const uint32_t got = halves(f);
  __half2 left = __hsub2(x, *reinterpret_cast<const __half2*>(&got));
  if (kTimes16) left = __hmul2(left, __float2half2_rn(16.f));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&left)));
  first = f, rest = r;
}

}  // namespace kv8
}  // namespace dspark
