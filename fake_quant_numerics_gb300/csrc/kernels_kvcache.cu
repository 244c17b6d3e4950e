// kernels_kvcache.cu -- keys and values quantized as they are written to the paged
// cache, and read back.
//
// A row (one position's key or value of one head) has its own scale: the per-row
// calibration of the integer calls, the amax scale of the FP8 call.  Both
// directions are bound by their bytes.  A group of lanes holds a row in registers,
// 16 elements a lane, so the statistics, the codes and the store take one read.
// Measured: 65536 int8 positions x 8 heads of 128 to bf16 61 us (6.6 TB/s); 16384 tokens
// of bf16 to affine 4-bit codes 22 us (3.9 TB/s, bound by the instructions of the exact
// quotients) and back 14; blocks of 256 threads in place of 128 2.4 us more.
#include "qat_attention.h"
#include "qat_kv.cuh"
#include "qat_layer.cuh"

namespace qat {
namespace {

constexpr int kKvThreads = 128;

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

// (an index that is not known would put the parameters into local memory)
template <typename A>
__device__ __forceinline__ A one(A const (&two)[2], int which) {
  return which ? two[1] : two[0];
}
// Where a token's rows lie, [page][head][offset]: head 0's, and the slot's validity.
struct KvToken {
  int64_t row;
  bool on;
};
__device__ __forceinline__ KvToken kv_token(const KvPlace& p, int64_t slot) {
  const bool on = slot >= 0 && slot < p.slots;
  const uint32_t at = on ? (uint32_t)slot : 0u, page = at / (uint32_t)p.page_size;  // (31 bits)
  return {(int64_t)page * p.heads * p.page_size + (at - page * p.page_size), on};
}
// x / n for a constant n: as the division rounds it, by its reciprocal and two remainders
// where nothing of them is lost.
template <int N>
__device__ __forceinline__ float over(float x) {
  constexpr float n = (float)N, r = 1.0f / n;
  return x >= 0x1p-80f && x <= 0x1p100f ? quotient_rn(x, r, -n) : __fdiv_rn(x, n);
}

// A lane's 16 elements of a row, as they lie in memory; elements behind the row's end
// are zeros.  How they are loaded: one by one, 16 bytes at a time, or 32 (bf16).
enum { kSingle = 0, kVec16 = 1, kVec32 = 2 };
template <typename T>
struct Unit {
  V32 v[T::BYTES / 2];
  template <int HOW>
  __device__ __forceinline__ void load(const void* x, int64_t at, int left) {
    const char* p = static_cast<const char*>(x) + at * T::BYTES;
#pragma unroll
    for (int i = 0; i < T::BYTES / 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i].w[j] = 0u;
    if constexpr (HOW == kVec32) {
      if (left > 0) v[0] = ld_v32(p);
    } else if constexpr (HOW == kVec16) {
      constexpr int E = 16 / T::BYTES;  // elements a load
#pragma unroll
      for (int i = 0; i < 16 / E; ++i)
        if (i * E < left) {
          const uint4 r = __ldg(reinterpret_cast<const uint4*>(p) + i);
          uint32_t* w = v[i / 2].w + 4 * (i % 2);
          w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
        }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e >= left) break;
        const uint32_t b = load_elem_bits<T>(x, at + e);
        if (T::BYTES == 4)
          v[e / 8].w[e % 8] = b;
        else
          v[0].w[e / 2] |= e & 1 ? b & 0xffff0000u : b >> 16;
      }
    }
  }
  __device__ __forceinline__ float get(int e) const {
    return elem<T>(v[T::BYTES == 4 ? e / 8 : 0], T::BYTES == 4 ? e % 8 : e);
  }
  // max |x|, NaN where one is; and the extremes beside zero
  __device__ __forceinline__ float top() const {
    if constexpr (T::BYTES == 2) {
      uint32_t m = 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = bf16x2_max_nan(m, v[0].w[k] & 0x7fff7fffu);
      return fmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; e += 2) m = fmax3_nan(m, fabsf(get(e)), fabsf(get(e + 1)));
      return m;
    }
  }
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    if constexpr (T::BYTES == 2) {
      uint32_t a = 0u, b = 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(v[0].w[k]));
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(v[0].w[k]));
      }
      lo = fmin3_nan(0.0f, __uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
      hi = fmax3_nan(0.0f, __uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
    } else {
      lo = hi = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        lo = fmin3_nan(lo, get(e), get(e + 1));
        hi = fmax3_nan(hi, get(e), get(e + 1));
      }
    }
  }
};

// Blocks (x: tokens, y: runs of U rows of the token's keys, then values), a group of
// lanes a token; the U rows are loaded together.
template <typename T, int F, bool AFFINE, int HOW, int U>
__global__ void __launch_bounds__(kKvThreads) k_kv_write(KvRows x, KvPlace p, int64_t tokens,
                                                         const int64_t* slots, int lanes) {
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t token = (int64_t)blockIdx.x * (kKvThreads / lanes) + threadIdx.x / lanes;
  const KvToken at = kv_token(p, token < tokens ? __ldg(slots + token) : -1);
  const int left = p.d - 16 * lane;  // elements from this lane's on
  Unit<T> unit[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int row = blockIdx.y * U + i;
    const int which = row >= p.heads, head = row - (which ? p.heads : 0);
    unit[i].template load<HOW>(
        which ? x.v : x.k, token * one(x.token_stride, which) + head * one(x.head_stride, which) + 16 * lane,
        at.on && row < 2 * p.heads ? left : 0);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int row = blockIdx.y * U + i;
    const int which = row >= p.heads, head = row - (which ? p.heads : 0);
    const bool on = at.on && row < 2 * p.heads;
    const int64_t to = at.row + (int64_t)head * p.page_size;
    const Unit<T>& u = unit[i];
    uint32_t w[8];
    if constexpr (F == QAT_CACHE_BF16) {
#pragma unroll
      for (int e = 0; e < 16; e += 2) w[e / 2] = pack_bf16x2(u.get(e), u.get(e + 1));
    } else {
      constexpr int BITS = F == QAT_CACHE_INT4 ? 4 : 8;
      constexpr int qmin = QRange<BITS, AFFINE>::qmin, qmax = QRange<BITS, AFFINE>::qmax;
      float lo = 0.0f, hi;
      if constexpr (AFFINE)
        u.range(lo, hi);
      else
        hi = u.top();
      for (int o = lanes >> 1; o; o >>= 1) {
        if (AFFINE) {
          const float other = __shfl_xor_sync(kFull, lo, o);
          lo = fmin3_nan(lo, lo, other);
        }
        hi = fmax_nan(hi, __shfl_xor_sync(kFull, hi, o));
      }
      // (a NaN or an infinity in the row is one here, and the scale not finite)
      float scale, zp = 0.0f;
      if constexpr (kv_is_int(F))
        scale = over<AFFINE ? qmax - qmin : qmax>(AFFINE ? __fsub_rn(hi, lo) : hi);
      else
        scale = over<F == QAT_CACHE_E4M3 ? 448 : 57344>(hi);
      if (!(scale < __uint_as_float(0x7f800000u))) scale = __uint_as_float(0x7fc00000u);
      const bool usable = scale > 0.0f;
      const bool fast = quot_scale_ok(scale);
      const float rcp = fast ? __frcp_rn(scale) : 0.0f;
      if (AFFINE && usable) {
        const float z = fast ? quotient_rn(lo, rcp, -scale) : __fdiv_rn(lo, scale);
        zp = fminf(fmaxf(rintf(__fsub_rn((float)qmin, z)), (float)qmin), (float)qmax);
      }
      float q[16];
      if (fast) {
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          quotient_rn2(u.get(e), u.get(e + 1), rcp, -scale, q[e], q[e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) q[e] = usable ? __fdiv_rn(u.get(e), scale) : 0.0f;
      }
      if constexpr (kv_is_int(F)) {
        // rint by the magic constant (|q| stays below 2^9), then the zero point.  Packing
        // saturates, which is an affine code's clamp; a symmetric one's quotient can pass
        // qmax only where the scale is subnormal.
        const uint32_t bias = kRintMagicBits - (uint32_t)(int)zp;
        const bool clamp = !AFFINE && scale < 0x1p-126f;
#pragma unroll
        for (int j = 0; j < BITS / 2; ++j) w[j] = 0u;
#pragma unroll
        for (int e = 14; e >= 0; e -= 2) {
          float a, b;
          add2(q[e], q[e + 1], kRintMagic, kRintMagic, a, b);
          int qa = (int)(__float_as_uint(a) - bias), qb = (int)(__float_as_uint(b) - bias);
          if (clamp) qa = min(max(qa, qmin), qmax), qb = min(max(qb, qmin), qmax);
          if (BITS == 8)
            w[e / 4] = pack_s8x2(qb, qa, w[e / 4]);
          else
            w[e / 8] = pack_s4x2(qa, qb, w[e / 8]);
        }
        // a row's padding, and a row without a scale, is code 0 whatever its zero point
        const int codes = usable ? left : 0;
#pragma unroll
        for (int j = 0; j < BITS / 2; ++j) {
          const int n = (codes - j * 32 / BITS) * BITS;  // bits of the word in use
          if (n < 32) w[j] = n <= 0 ? 0u : w[j] & (0xffffffffu >> (32 - n));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = usable ? fp8_pair<F>(q[4 * j], q[4 * j + 1]) | fp8_pair<F>(q[4 * j + 2], q[4 * j + 3]) << 16
                        : 0u;
      }
      if (on && lane == 0) {
        one(p.scales, which)[to] = scale;
        if (AFFINE) one(p.zps, which)[to] = (int8_t)zp;
      }
    }
    constexpr int UB = kv_unit_bytes(F);
    char* dst = static_cast<char*>(one(p.codes, which)) + to * p.row_bytes + lane * UB;
    const int bytes = on ? p.row_bytes - lane * UB : 0;
    if (bytes <= 0) continue;
    if constexpr (UB == 8) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      if (UB == 32 && bytes > 16)
        *reinterpret_cast<uint4*>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// The same walk the other way.  WIDE: rows start on 32 bytes and hold whole units.
template <typename T, int F, bool WIDE, int U>
__global__ void __launch_bounds__(kKvThreads) k_kv_read(KvPlace p, int64_t tokens,
                                                        const int64_t* slots, int lanes, void* k,
                                                        void* v) {
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t token = (int64_t)blockIdx.x * (kKvThreads / lanes) + threadIdx.x / lanes;
  const int left = p.d - 16 * lane;
  if (token >= tokens || left <= 0) return;
  const KvToken at = kv_token(p, __ldg(slots + token));
  constexpr int UB = kv_unit_bytes(F);
  uint32_t w[U][UB / 4];
  float scale[U];
  int zp[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int row = blockIdx.y * U + i;
    const int which = row >= p.heads, head = row - (which ? p.heads : 0);
#pragma unroll
    for (int j = 0; j < UB / 4; ++j) w[i][j] = 0u;
    scale[i] = 0.0f, zp[i] = 0;
    if (!at.on || row >= 2 * p.heads) continue;
    const int64_t from = at.row + (int64_t)head * p.page_size;
    const char* src = static_cast<const char*>(one(p.codes, which)) + from * p.row_bytes + lane * UB;
    if constexpr (UB == 8) {
      const uint2 a = *reinterpret_cast<const uint2*>(src);
      w[i][0] = a.x, w[i][1] = a.y;
    } else {
#pragma unroll
      for (int j = 0; j < UB / 16; ++j)
        if (j == 0 || left > 8) {
          const uint4 a = *reinterpret_cast<const uint4*>(src + 16 * j);
          w[i][4 * j] = a.x, w[i][4 * j + 1] = a.y, w[i][4 * j + 2] = a.z, w[i][4 * j + 3] = a.w;
        }
    }
    if constexpr (F != QAT_CACHE_BF16) scale[i] = one(p.scales, which)[from];
    if constexpr (kv_is_int(F))
      if (one(p.zps, which)) zp[i] = one(p.zps, which)[from];
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int row = blockIdx.y * U + i;
    if (row >= 2 * p.heads) break;
    const int which = row >= p.heads, head = row - (which ? p.heads : 0);
    float x[16];
    kv_decode<F>(w[i], scale[i], zp[i], x);
    uint32_t o[4 * T::BYTES];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      if (T::BYTES == 2)
        o[e / 2] = pack_bf16x2(x[e], x[e + 1]);
      else
        o[e] = __float_as_uint(x[e]), o[e + 1] = __float_as_uint(x[e + 1]);
    }
    char* dst = static_cast<char*>(which ? v : k) +
                ((token * p.heads + head) * p.d + 16 * lane) * (int64_t)T::BYTES;
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < T::BYTES / 2; ++j) {
        V32 y;
#pragma unroll
        for (int e = 0; e < 8; ++e) y.w[e] = o[8 * j + e];
        st_v32(dst + 32 * j, y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < T::BYTES; ++j)
        if (j * 16 / T::BYTES < left)
          reinterpret_cast<uint4*>(dst)[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    }
  }
}

// Rows a group takes at a time: four (two of fp32) once that leaves every SM full, so
// that their loads are in flight together; one for fewer, which then run side by side
// (write and read of 16384 tokens x 8 heads as affine int4: 41 us with one row, 36 with
// four; 16 tokens 3.5 us with one).
bool many_rows(int64_t rows, int lanes) {
  return rows * lanes >= (int64_t)device_info().sms * 2048 * 4;
}
// A grid for runs of U rows of each token; false where it does not fit.
bool kv_grid(const KvPlace& p, int64_t tokens, int lanes, int u, dim3* grid) {
  const int64_t x = (tokens + kKvThreads / lanes - 1) / (kKvThreads / lanes);
  const int64_t y = (2 * (int64_t)p.heads + u - 1) / u;
  *grid = dim3((unsigned)x, (unsigned)y);
  return x <= INT32_MAX && y <= 65535;
}

template <typename T, int F, bool AFFINE>
qat_status write_rows(const qat_kv_cache& c, const KvRows& x, int64_t tokens, const int64_t* slots,
                      cudaStream_t s) {
  const KvPlace p = place_of(c);
  const int lanes = kv_lanes(p.units);
  const auto on = [&](int64_t bytes) {
    bool fits = true;
    for (const void* q : {x.k, x.v}) fits = fits && reinterpret_cast<uintptr_t>(q) % bytes == 0;
    for (int i = 0; i < 2; ++i)
      fits = fits && x.token_stride[i] * T::BYTES % bytes == 0 && x.head_stride[i] * T::BYTES % bytes == 0;
    return fits;
  };
  constexpr int MOST = T::BYTES == 2 ? kVec32 : kVec16, U = T::BYTES == 2 ? 4 : 2;
  const bool vec = on(16), wide = T::BYTES == 4 ? vec : on(32) && p.d % 16 == 0;
  const bool many = wide && many_rows(tokens * 2 * p.heads, lanes);
  dim3 grid;
  if (!kv_grid(p, tokens, lanes, many ? U : 1, &grid)) return QAT_ERR_INVALID_ARGUMENT;
  auto k = many   ? k_kv_write<T, F, AFFINE, MOST, U>
           : wide ? k_kv_write<T, F, AFFINE, MOST, 1>
           : vec  ? k_kv_write<T, F, AFFINE, kVec16, 1>
                  : k_kv_write<T, F, AFFINE, kSingle, 1>;
  k<<<grid, kKvThreads, 0, s>>>(x, p, tokens, slots, lanes);
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

template <typename T, int F>
qat_status read_rows(const qat_kv_cache& c, const int64_t* slots, int64_t tokens, void* k, void* v,
                     cudaStream_t s) {
  const KvPlace p = place_of(c);
  const int lanes = kv_lanes((p.d + 15) / 16);
  const bool wide = p.d % 16 == 0 && reinterpret_cast<uintptr_t>(k) % 32 == 0 &&
                    reinterpret_cast<uintptr_t>(v) % 32 == 0;
  const bool many = wide && many_rows(tokens * 2 * p.heads, lanes);
  dim3 grid;
  if (!kv_grid(p, tokens, lanes, many ? 4 : 1, &grid)) return QAT_ERR_INVALID_ARGUMENT;
  auto kernel = many   ? k_kv_read<T, F, true, 4>
                : wide ? k_kv_read<T, F, true, 1>
                       : k_kv_read<T, F, false, 1>;
  kernel<<<grid, kKvThreads, 0, s>>>(p, tokens, slots, lanes, k, v);
  count_launch(1);
  return launch_status();
}

template <typename T>
qat_status read_any(const qat_kv_cache& c, const int64_t* slots, int64_t tokens, void* k, void* v,
                    cudaStream_t s) {
  switch (c.format) {
    case QAT_CACHE_INT8: return read_rows<T, QAT_CACHE_INT8>(c, slots, tokens, k, v, s);
    case QAT_CACHE_INT4: return read_rows<T, QAT_CACHE_INT4>(c, slots, tokens, k, v, s);
    case QAT_CACHE_E4M3: return read_rows<T, QAT_CACHE_E4M3>(c, slots, tokens, k, v, s);
    case QAT_CACHE_E5M2: return read_rows<T, QAT_CACHE_E5M2>(c, slots, tokens, k, v, s);
    default: return read_rows<T, QAT_CACHE_BF16>(c, slots, tokens, k, v, s);
  }
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
