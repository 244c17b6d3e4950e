// kernels_kvattn.cu -- attention of one new token of each sequence over a paged,
// quantized key-value cache.
//
//   y = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - m),  t < length
//
// One block per sequence and query head; its warps take positions in turn, each
// with a running maximum and sum, and are joined at the end.  A lane holds eight
// elements of the head.
#include <cmath>

#include "qat_attention.h"
#include "qat_kv.cuh"
#include "qat_layer.cuh"

namespace qat {
namespace {

constexpr int kWarps = 4;

struct CacheView {
  const char *k, *v;
  const float *ks, *vs;
  const int8_t *kz, *vz;
  int64_t pages;
  int heads, page_size, d, row_bytes;
};

template <int F>
__device__ __forceinline__ void row8(const char* codes, const float* scales, const int8_t* zps,
                                     int64_t row, int row_bytes, int lane, bool on, float* x) {
  uint32_t w[4] = {};
  constexpr int UB = kv_unit_bytes(F) / 2;
  const char* p = codes + row * row_bytes + lane * UB;
  if (on) {
#pragma unroll
    for (int i = 0; i < UB / 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
  const float scale = F == QAT_CACHE_BF16 ? 1.0f : scales[row];
  kv_decode<F, 8>(w, scale, kv_is_int(F) && zps ? zps[row] : 0, x);
  if (!on) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
  }
}

template <typename T, int F>
__global__ void __launch_bounds__(32 * kWarps) k_kv_attn(CacheView c, KvAttnArgs a) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.y;
  const int h = blockIdx.x, kvh = h / (int)(a.q_heads / c.heads);
  const int64_t length = a.lengths[b];
  const bool on = 8 * lane < c.d;
  float q[8], o[8] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    q[e] = on ? ld_elem<T>(a.q, b * a.q_batch_stride + h * a.q_head_stride + 8 * lane + e) : 0.0f;
  bool bad = length > a.table_cols * c.page_size;
  for (int64_t t = warp; t < length && !bad; t += kWarps) {
    const int page = a.table[b * a.table_stride + t / c.page_size];
    if (page < 0 || page >= c.pages) {
      bad = true;
      break;
    }
    const int64_t row = ((int64_t)page * c.heads + kvh) * c.page_size + t % c.page_size;
    float k[8], v[8], s = 0.0f;
    row8<F>(c.k, c.ks, c.kz, row, c.row_bytes, lane, on, k);
    row8<F>(c.v, c.vs, c.vz, row, c.row_bytes, lane, on, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __fmaf_rn(q[e], k[e], s);
    for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(kFull, s, i);
    s *= a.scale;
    const float top = fmaxf(m, s);
    const float was = m == top ? 1.0f : expf(m - top), p = s == top ? 1.0f : expf(s - top);
    m = top;
    l = __fmaf_rn(l, was, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __fmaf_rn(o[e], was, __fmul_rn(p, v[e]));
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = bad ? NAN : l;
#pragma unroll
  for (int e = 0; e < 8; ++e) s_o[warp][8 * lane + e] = o[e];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  for (int w = 0; w < kWarps; ++w)
    if (s_m[w] > -INFINITY || s_l[w] != 0.0f) sum += s_l[w] * expf(s_m[w] - top);
  for (int e = threadIdx.x; e < c.d; e += 32 * kWarps) {
    float y = 0.0f;
    for (int w = 0; w < kWarps; ++w)
      if (s_m[w] > -INFINITY || s_l[w] != 0.0f) y += s_o[w][e] * expf(s_m[w] - top);
    if (sum != 0.0f) y /= sum;
    st_elem<T>(a.y, (b * a.q_heads + h) * c.d + e, y);
  }
  if (a.lse && threadIdx.x == 0) a.lse[b * a.q_heads + h] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

template <typename T>
qat_status launch_any(const qat_kv_cache& c, const KvAttnArgs& a, cudaStream_t s) {
  const CacheView v = {(const char*)c.k, (const char*)c.v, c.k_scales, c.v_scales, c.k_zero_points,
                       c.v_zero_points, c.pages, (int)c.heads, (int)c.page_size, (int)c.head_dim,
                       (int)kv_row_bytes(c.format, c.head_dim)};
  auto k = k_kv_attn<T, QAT_CACHE_BF16>;
  if (c.format == QAT_CACHE_INT8) k = k_kv_attn<T, QAT_CACHE_INT8>;
  if (c.format == QAT_CACHE_INT4) k = k_kv_attn<T, QAT_CACHE_INT4>;
  if (c.format == QAT_CACHE_E4M3) k = k_kv_attn<T, QAT_CACHE_E4M3>;
  if (c.format == QAT_CACHE_E5M2) k = k_kv_attn<T, QAT_CACHE_E5M2>;
  k<<<dim3((unsigned)a.q_heads, (unsigned)a.batch), 32 * kWarps, 0, s>>>(v, a);
  count_launch(1);
  return launch_status();
}

}  // namespace

size_t kv_attn_ws_bytes(int64_t, int64_t, int64_t) { return 16; }

qat_status launch_kv_attn(const qat_kv_cache& c, const KvAttnArgs& a, qat_dtype dt, void*,
                          cudaStream_t s) {
  return dt == QAT_F32 ? launch_any<F32>(c, a, s) : launch_any<BF16>(c, a, s);
}

}  // namespace qat
