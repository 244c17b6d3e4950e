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

// The values of 16 codes: (q - zp) * scale, c * scale, or the bf16.  An integer code
// comes as the low byte of a float of 2^23 (its sign bit turned), from which the same
// number for the zero point is taken: exact.
template <int F>
__device__ __forceinline__ void kv_decode(const uint32_t* w, float scale, int zp, float* v) {
  if constexpr (F == QAT_CACHE_BF16) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      v[i] = __uint_as_float(w[i / 2] << 16);
      v[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
    }
  } else if constexpr (kv_is_int(F)) {
    const float base = 8388608.0f + (float)(zp + (F == QAT_CACHE_INT8 ? 128 : 8));
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      uint32_t a, b;
      if (F == QAT_CACHE_INT8) {
        const uint32_t x = w[i / 4] ^ 0x80808080u;
        a = __byte_perm(x, 0x4b000000u, 0x7550 + i % 4);
        b = __byte_perm(x, 0x4b000000u, 0x7551 + i % 4);
      } else {  // the even element in the high nibble
        const uint32_t x = w[i / 8] ^ 0x88888888u;
        a = __byte_perm((x >> 4) & 0x0f0f0f0fu, 0x4b000000u, 0x7550 + i / 2 % 4);
        b = __byte_perm(x & 0x0f0f0f0fu, 0x4b000000u, 0x7550 + i / 2 % 4);
      }
      sub2(__uint_as_float(a), __uint_as_float(b), base, base, v[i], v[i + 1]);
      mul2(v[i], v[i + 1], scale, scale, v[i], v[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 c = fp8_values<F>((w[i / 4] >> (8 * (i % 4))) & 0xffffu);
      mul2(c.x, c.y, scale, scale, v[i], v[i + 1]);
    }
  }
}

}  // namespace qat
