// kernels_kvcache.cu -- keys and values quantized as they are written to the paged
// cache, and read back.
//
// A row (one position's key or value of one head) has its own scale: the per-row
// calibration of the integer calls, the amax scale of the FP8 call.  Both
// directions are bound by their bytes.  A group of lanes holds a row in registers,
// 16 elements a lane, so the statistics, the codes and the store take one read.
#include "qat_attention.h"
#include "qat_kv.cuh"
#include "qat_layer.cuh"

namespace qat {
namespace {

constexpr int kKvThreads = 256;

struct KvPlace {
  void *codes[2];
  float *scales[2];
  int8_t *zps[2];
  int64_t slots;  // pages * page_size
  int heads, page_size, d, row_bytes, units;
};

KvPlace place_of(const qat_kv_cache& c) {
  KvPlace p = {{c.k, c.v}, {c.k_scales, c.v_scales}, {c.k_zero_points, c.v_zero_points}};
  p.slots = c.pages * c.page_size;
  p.heads = (int)c.heads, p.page_size = (int)c.page_size, p.d = (int)c.head_dim;
  p.row_bytes = (int)kv_row_bytes(c.format, c.head_dim);
  p.units = (p.row_bytes + kv_unit_bytes(c.format) - 1) / kv_unit_bytes(c.format);
  return p;
}
int kv_lanes(int units) {
  int lanes = 1;
  while (lanes < units) lanes *= 2;
  return lanes;
}

// The row of a slot and head: [page][head][offset].
__device__ __forceinline__ int64_t kv_row(const KvPlace& p, int64_t slot, int head) {
  const int page = (int)slot / p.page_size;  // slots fit 31 bits
  return ((int64_t)page * p.heads + head) * p.page_size + ((int)slot - page * p.page_size);
}

// Half `i` of a lane's unit: 8 elements from a run's start.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const void* x, int64_t at, float* v) {
  if constexpr (!VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ld_elem<T>(x, at + e);
  } else if constexpr (T::BYTES == 2) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at * 2));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      v[e] = __uint_as_float(w[e / 2] << 16);
      v[e + 1] = __uint_as_float(w[e / 2] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 r =
          __ldg(reinterpret_cast<const float4*>(static_cast<const char*>(x) + at * 4) + j);
      v[4 * j] = r.x, v[4 * j + 1] = r.y, v[4 * j + 2] = r.z, v[4 * j + 3] = r.w;
    }
  }
}

template <typename T, int F, bool AFFINE, bool VEC>
__global__ void __launch_bounds__(kKvThreads) k_kv_write(KvRows x, KvPlace p, int64_t rows,
                                                         const int64_t* slots, int lanes) {
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t row = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / lanes;
  int64_t slot = -1, token = 0;
  int which = 0, head = 0;
  if (row < rows) {
    token = row / (2 * p.heads);
    const int r = (int)(row - token * 2 * p.heads);
    which = r >= p.heads;
    head = r - which * p.heads;
    slot = __ldg(slots + token);
  }
  const bool on = slot >= 0 && slot < p.slots;
  float v[16];
  const int e0 = 16 * lane;
  const int64_t from = token * x.token_stride[which] + head * x.head_stride[which] + e0;
  const void* src = which ? x.v : x.k;
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = 0.0f;
  if (on && e0 < p.d) load8<T, VEC>(src, from, v);
  if (on && e0 + 8 < p.d) load8<T, VEC>(src, from + 8, v + 8);
  const int64_t to = on ? kv_row(p, slot, head) : 0;
  uint32_t w[8];
  if constexpr (F == QAT_CACHE_BF16) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) w[e / 2] = pack_bf16x2(v[e], v[e + 1]);
  } else {
    constexpr int BITS = F == QAT_CACHE_INT4 ? 4 : 8;
    constexpr int qmin = QRange<BITS, AFFINE>::qmin, qmax = QRange<BITS, AFFINE>::qmax;
    // Extremes over the finite elements and zero, and whether all are finite.
    float lo = 0.0f, hi = 0.0f;
    int bad = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      bad |= (__float_as_uint(v[e]) & 0x7f800000u) == 0x7f800000u;
      if (AFFINE) lo = fminf(lo, v[e]);
      hi = fmaxf(hi, AFFINE ? v[e] : fabsf(v[e]));
    }
    for (int o = lanes >> 1; o; o >>= 1) {
      if (AFFINE) lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
      bad |= __shfl_xor_sync(kFull, bad, o);
    }
    float scale, zp = 0.0f;
    if constexpr (kv_is_int(F)) {
      scale = __fdiv_rn(AFFINE ? __fsub_rn(hi, lo) : hi, (float)(AFFINE ? qmax - qmin : qmax));
    } else {
      scale = __fdiv_rn(hi, F == QAT_CACHE_E4M3 ? 448.0f : 57344.0f);
    }
    if (bad || isinf(scale)) scale = __uint_as_float(0x7fc00000u);
    const bool usable = scale > 0.0f;
    if (AFFINE && usable)
      zp = fminf(fmaxf(rintf(__fsub_rn((float)qmin, __fdiv_rn(lo, scale))), (float)qmin),
                 (float)qmax);
    const bool fast = quot_scale_ok(scale);
    const float rcp = fast ? __frcp_rn(scale) : 0.0f;
    float q[16];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      if (fast) {
        quotient_rn2(v[e], v[e + 1], rcp, -scale, q[e], q[e + 1]);
      } else {
        q[e] = usable ? __fdiv_rn(v[e], scale) : 0.0f;
        q[e + 1] = usable ? __fdiv_rn(v[e + 1], scale) : 0.0f;
      }
    }
    if constexpr (kv_is_int(F)) {
      uint32_t c[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float k = fminf(fmaxf(__fadd_rn(rintf(q[e]), zp), (float)qmin), (float)qmax);
        // (a row's padding is code 0, whatever its zero point)
        c[e] = e0 + e < p.d && usable ? (uint32_t)(int)k : 0u;
      }
#pragma unroll
      for (int j = 0; j < 16 / (32 / BITS); ++j) {
        uint32_t word = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (BITS == 8)
            word |= (c[4 * j + b] & 255u) << (8 * b);
          else
            word |= ((c[8 * j + 2 * b] & 15u) << 4 | (c[8 * j + 2 * b + 1] & 15u)) << (8 * b);
        }
        w[j] = word;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = usable ? fp8_pair<F>(q[4 * j], q[4 * j + 1]) | fp8_pair<F>(q[4 * j + 2], q[4 * j + 3]) << 16 : 0u;
    }
    if (on && lane == 0) {
      p.scales[which][to] = scale;
      if (AFFINE) p.zps[which][to] = (int8_t)zp;
    }
  }
  constexpr int UB = kv_unit_bytes(F);
  char* dst = static_cast<char*>(p.codes[which]) + to * p.row_bytes + lane * UB;
  const int left = p.row_bytes - lane * UB;
  if (!on || left <= 0) return;
  if constexpr (UB == 8) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    if (UB == 32 && left > 16)
      *reinterpret_cast<uint4*>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <typename T, int F>
__global__ void __launch_bounds__(kKvThreads) k_kv_read(KvPlace p, int64_t rows,
                                                        const int64_t* slots, int lanes, void* k,
                                                        void* v) {
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t row = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / lanes;
  const int e0 = 16 * lane;
  if (row >= rows || e0 >= p.d) return;
  const int64_t token = row / (2 * p.heads);
  const int r = (int)(row - token * 2 * p.heads);
  const int which = r >= p.heads, head = r - which * p.heads;
  const int64_t slot = __ldg(slots + token);
  const bool two = e0 + 8 < p.d;
  float x[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = 0.0f;
  if (slot >= 0 && slot < p.slots) {
    constexpr int UB = kv_unit_bytes(F);
    const int64_t from = kv_row(p, slot, head);
    const char* src = static_cast<const char*>(p.codes[which]) + from * p.row_bytes + lane * UB;
    uint32_t w[8] = {};
    if constexpr (UB == 8) {
      const uint2 a = *reinterpret_cast<const uint2*>(src);
      w[0] = a.x, w[1] = a.y;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(src);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      if (UB == 32 && two) {
        const uint4 b = *reinterpret_cast<const uint4*>(src + 16);
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      }
    }
    const float scale = F == QAT_CACHE_BF16 ? 1.0f : p.scales[which][from];
    const int zp = kv_is_int(F) && p.zps[which] ? p.zps[which][from] : 0;
    kv_decode<F, 16>(w, scale, zp, x);
  }
  char* dst = static_cast<char*>(which ? v : k) +
              ((token * p.heads + head) * p.d + e0) * (int64_t)T::BYTES;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (j && !two) break;
    if constexpr (T::BYTES == 2) {
      uint4 o;
      o.x = pack_bf16x2(x[8 * j], x[8 * j + 1]), o.y = pack_bf16x2(x[8 * j + 2], x[8 * j + 3]);
      o.z = pack_bf16x2(x[8 * j + 4], x[8 * j + 5]), o.w = pack_bf16x2(x[8 * j + 6], x[8 * j + 7]);
      reinterpret_cast<uint4*>(dst)[j] = o;
    } else {
      reinterpret_cast<float4*>(dst)[2 * j] =
          make_float4(x[8 * j], x[8 * j + 1], x[8 * j + 2], x[8 * j + 3]);
      reinterpret_cast<float4*>(dst)[2 * j + 1] =
          make_float4(x[8 * j + 4], x[8 * j + 5], x[8 * j + 6], x[8 * j + 7]);
    }
  }
}

template <typename T, int F, bool AFFINE>
qat_status write_rows(const qat_kv_cache& c, const KvRows& x, int64_t tokens, const int64_t* slots,
                      cudaStream_t s) {
  const KvPlace p = place_of(c);
  const int lanes = kv_lanes(p.units);
  const int64_t rows = tokens * 2 * p.heads;
  const int64_t blocks = (rows * lanes + kKvThreads - 1) / kKvThreads;
  if (blocks > INT32_MAX) return QAT_ERR_INVALID_ARGUMENT;
  bool vec = true;
  for (const void* q : {x.k, x.v}) vec = vec && reinterpret_cast<uintptr_t>(q) % 16 == 0;
  for (int i = 0; i < 2; ++i)
    vec = vec && x.token_stride[i] * T::BYTES % 16 == 0 && x.head_stride[i] * T::BYTES % 16 == 0;
  auto k = vec ? k_kv_write<T, F, AFFINE, true> : k_kv_write<T, F, AFFINE, false>;
  k<<<(unsigned)blocks, kKvThreads, 0, s>>>(x, p, rows, slots, lanes);
  count_launch(1);
  return launch_status();
}

template <typename T>
qat_status write_any(const qat_kv_cache& c, const KvRows& x, int64_t tokens, const int64_t* slots,
                     cudaStream_t s) {
  const bool affine = c.k_zero_points != nullptr;
  switch (c.format) {
    case QAT_CACHE_INT8:
      return affine ? write_rows<T, QAT_CACHE_INT8, true>(c, x, tokens, slots, s)
                    : write_rows<T, QAT_CACHE_INT8, false>(c, x, tokens, slots, s);
    case QAT_CACHE_INT4:
      return affine ? write_rows<T, QAT_CACHE_INT4, true>(c, x, tokens, slots, s)
                    : write_rows<T, QAT_CACHE_INT4, false>(c, x, tokens, slots, s);
    case QAT_CACHE_E4M3: return write_rows<T, QAT_CACHE_E4M3, false>(c, x, tokens, slots, s);
    case QAT_CACHE_E5M2: return write_rows<T, QAT_CACHE_E5M2, false>(c, x, tokens, slots, s);
    default: return write_rows<T, QAT_CACHE_BF16, false>(c, x, tokens, slots, s);
  }
}

template <typename T>
qat_status read_any(const qat_kv_cache& c, const int64_t* slots, int64_t tokens, void* k, void* v,
                    cudaStream_t s) {
  const KvPlace p = place_of(c);
  const int lanes = kv_lanes(p.units);
  const int64_t rows = tokens * 2 * p.heads;
  const int64_t blocks = (rows * lanes + kKvThreads - 1) / kKvThreads;
  if (blocks > INT32_MAX) return QAT_ERR_INVALID_ARGUMENT;
  auto kernel = k_kv_read<T, QAT_CACHE_BF16>;
  if (c.format == QAT_CACHE_INT8) kernel = k_kv_read<T, QAT_CACHE_INT8>;
  if (c.format == QAT_CACHE_INT4) kernel = k_kv_read<T, QAT_CACHE_INT4>;
  if (c.format == QAT_CACHE_E4M3) kernel = k_kv_read<T, QAT_CACHE_E4M3>;
  if (c.format == QAT_CACHE_E5M2) kernel = k_kv_read<T, QAT_CACHE_E5M2>;
  kernel<<<(unsigned)blocks, kKvThreads, 0, s>>>(p, rows, slots, lanes, k, v);
  count_launch(1);
  return launch_status();
}

}  // namespace

qat_status launch_kv_write(const qat_kv_cache& c, const KvRows& x, qat_dtype dt, int64_t tokens,
                           const int64_t* slots, cudaStream_t s) {
  return dt == QAT_F32 ? write_any<F32>(c, x, tokens, slots, s)
                       : write_any<BF16>(c, x, tokens, slots, s);
}
qat_status launch_kv_read(const qat_kv_cache& c, const int64_t* slots, int64_t tokens, void* k,
                          void* v, qat_dtype dt, cudaStream_t s) {
  return dt == QAT_F32 ? read_any<F32>(c, slots, tokens, k, v, s)
                       : read_any<BF16>(c, slots, tokens, k, v, s);
}

}  // namespace qat
