// qat_layer.cuh -- device helpers shared by the layer operators' kernels.
#pragma once

#include <cuda_bf16.h>

#include "qat_device.cuh"

namespace qat {

template <typename T>
__device__ __forceinline__ float ld_elem(const void* p, int64_t i) {
  return __uint_as_float(load_elem_bits<T>(p, i));
}

template <typename T>
__device__ __forceinline__ void st_elem(void* p, int64_t i, float v);
template <>
__device__ __forceinline__ void st_elem<F32>(void* p, int64_t i, float v) {
  static_cast<float*>(p)[i] = v;
}
template <>
__device__ __forceinline__ void st_elem<BF16>(void* p, int64_t i, float v) {
  static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// The next bf16 part of a float, which keeps the remainder: three calls take all
// 24 bits.  Truncation, so that no part overflows; an infinity leaves nothing
// and a NaN keeps a mantissa bit.
__device__ __forceinline__ float take_bf16(float& x) {
  const uint32_t u = __float_as_uint(x);
  const bool special = (u & 0x7f800000u) == 0x7f800000u;
  uint32_t h = u & 0xffff0000u;
  if (special && (u & 0x007fffffu)) h |= 0x00400000u;
  x = special ? 0.0f : x - __uint_as_float(h);
  return __uint_as_float(h);
}

// act(g) and act'(g): silu (0), gelu in the erf form (1), relu (2).  A NaN
// stays NaN; relu'(0) = 0.  FAST takes the hardware's exponential and reciprocal
// for the sigmoid (2 + 1.173 |g| ulp of the exponential: within 2^-18 for |g| < 20,
// where it matters): enough under a bf16 result, at a third of the instructions.
template <bool FAST>
__device__ __forceinline__ void act_grad(int act, float g, float& a, float& da) {
  if (act == QAT_ACT_SILU) {
    const float s = FAST ? __fdividef(1.0f, 1.0f + __expf(-g)) : __frcp_rn(1.0f + expf(-g));
    a = g * s;
    da = s * fmaf(g, 1.0f - s, 1.0f);
  } else if (act == QAT_ACT_GELU) {
    const float phi = 0.5f * erfcf(g * -0.70710678118654752f);  // keeps the tail's digits
    a = g * phi;
    da = fmaf(g * 0.39894228040143268f, expf(-0.5f * g * g), phi);
  } else {
    a = g > 0.0f ? g : (g != g ? g : 0.0f);
    da = g > 0.0f ? 1.0f : 0.0f;
  }
}
template <bool FAST>
__device__ __forceinline__ float act_value(int act, float g) {
  float a, da;
  act_grad<FAST>(act, g, a, da);
  return a;
}

}  // namespace qat
