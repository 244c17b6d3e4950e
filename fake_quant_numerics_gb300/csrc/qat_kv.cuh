// qat_kv.cuh -- rows of the paged key-value cache on the device: their place, and
// the conversions of 16 elements to and from codes.
#pragma once

#include <cuda_fp16.h>

#include "qat_device.cuh"

namespace qat {

__host__ __device__ constexpr bool kv_is_int(int f) { return f == QAT_CACHE_INT8 || f == QAT_CACHE_INT4; }
// Bytes of 16 elements.
__host__ __device__ constexpr int kv_unit_bytes(int f) {
  return f == QAT_CACHE_BF16 ? 32 : f == QAT_CACHE_INT4 ? 8 : 16;
}

// Two FP8 codes (low byte first) of two floats: round to nearest even, saturating.
template <int F>
__device__ __forceinline__ uint32_t fp8_pair(float lo, float hi) {
  uint16_t r;
  if (F == QAT_CACHE_E4M3)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int F>
__device__ __forceinline__ float2 fp8_values(uint32_t pair) {
  uint32_t h;
  if (F == QAT_CACHE_E4M3)
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  else
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The values of E codes (E = 8 or 16): (q - zp) * scale, c * scale, or the bf16.
template <int F, int E>
__device__ __forceinline__ void kv_decode(const uint32_t* w, float scale, int zp, float* v) {
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    if (F == QAT_CACHE_BF16) {
      v[i] = __uint_as_float(w[i / 2] << 16);
      v[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
    } else if (F == QAT_CACHE_INT8) {
      const int32_t a = (int32_t)(w[i / 4] << (24 - 8 * (i % 4))) >> 24;
      const int32_t b = (int32_t)(w[i / 4] << (16 - 8 * (i % 4))) >> 24;
      v[i] = __fmul_rn((float)(a - zp), scale);
      v[i + 1] = __fmul_rn((float)(b - zp), scale);
    } else if (F == QAT_CACHE_INT4) {
      const int byte = 8 * ((i / 2) % 4);  // the even element in the high nibble
      const int32_t a = (int32_t)(w[i / 8] << (24 - byte)) >> 28;
      const int32_t b = (int32_t)(w[i / 8] << (28 - byte)) >> 28;
      v[i] = __fmul_rn((float)(a - zp), scale);
      v[i + 1] = __fmul_rn((float)(b - zp), scale);
    } else {
      const float2 c = fp8_values<F>((w[i / 4] >> (8 * (i % 4))) & 0xffffu);
      v[i] = __fmul_rn(c.x, scale);
      v[i + 1] = __fmul_rn(c.y, scale);
    }
  }
}

}  // namespace qat
