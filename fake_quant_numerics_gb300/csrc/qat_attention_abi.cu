// qat_attention_abi.cu -- the exported C entry points of the attention operators:
// argument validation, then the launchers.  See include/qat.h.
#include <cmath>
#include <cstdint>

#include "qat_attention.h"

using namespace qat;

namespace {

constexpr int64_t kMaxElems = INT64_C(1) << 50;

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool dtype_ok(qat_dtype d) { return d == QAT_F32 || d == QAT_BF16; }
uintptr_t esize(qat_dtype d) { return d == QAT_F32 ? 4 : 2; }
// a * b with a, b >= 0 stays within the library's element limit
bool fits(int64_t a, int64_t b) { return a >= 0 && b >= 0 && (b == 0 || a <= kMaxElems / b); }
// every offset below `tokens` and `heads` strides fits 62 bits
bool stride_ok(int64_t s, int64_t n) {
  const int64_t most = INT64_C(1) << 60;
  return n <= 1 || (s >= -(most / n) && s <= most / n);
}

struct RopeSizes {
  int64_t tokens, q_heads, k_heads, head_dim, rotary_dim;
  int64_t q_ts, q_hs, k_ts, k_hs;
};

qat_status check_rope(const RopeSizes& z, qat_dtype dtype, int layout, float amplitude, int norm,
                      float eps, const void* q_weight, const void* k_weight) {
  if (!dtype_ok(dtype) || (layout != QAT_ROPE_HALF && layout != QAT_ROPE_INTERLEAVED))
    return QAT_ERR_UNSUPPORTED;
  if (z.head_dim < 1 || z.head_dim > 512 || z.rotary_dim < 0 || z.rotary_dim > z.head_dim ||
      z.rotary_dim % 2)
    return QAT_ERR_INVALID_ARGUMENT;
  if (z.q_heads < 0 || z.k_heads < 0 || z.q_heads > 32767 || z.k_heads > 32767 ||
      !fits(z.tokens, (z.q_heads + z.k_heads) * z.head_dim))
    return QAT_ERR_INVALID_ARGUMENT;
  if (!stride_ok(z.q_ts, z.tokens) || !stride_ok(z.k_ts, z.tokens) ||
      !stride_ok(z.q_hs, z.q_heads) || !stride_ok(z.k_hs, z.k_heads))
    return QAT_ERR_INVALID_ARGUMENT;
  if (!(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(amplitude))
    return QAT_ERR_INVALID_ARGUMENT;
  if (!norm && (q_weight || k_weight)) return QAT_ERR_INVALID_ARGUMENT;
  return QAT_OK;
}

RopeArgs rope_args(const RopeSizes& z, const void* q, const void* k, const int64_t* positions,
                   const uint64_t* turns, int layout, float amplitude, int norm, float eps,
                   const void* q_weight, const void* k_weight) {
  RopeArgs a = {};
  a.x[0] = q, a.x[1] = k, a.w[0] = q_weight, a.w[1] = k_weight;
  a.token_stride[0] = z.q_ts, a.token_stride[1] = z.k_ts;
  a.head_stride[0] = z.q_hs, a.head_stride[1] = z.k_hs;
  a.heads[0] = (int)z.q_heads, a.heads[1] = (int)z.k_heads;
  a.positions = positions, a.turns = turns, a.tokens = z.tokens;
  a.d = (int)z.head_dim, a.rotary = (int)z.rotary_dim, a.norm = norm != 0;
  a.interleaved = layout == QAT_ROPE_INTERLEAVED, a.amplitude = amplitude, a.eps = eps;
  a.inv_d = 1.0f / (float)z.head_dim;
  return a;
}

qat_status check_cache(const qat_kv_cache* c) {
  if (!c) return QAT_ERR_INVALID_ARGUMENT;
  const int f = c->format;
  if (f < QAT_CACHE_BF16 || f > QAT_CACHE_E5M2) return QAT_ERR_UNSUPPORTED;
  if (c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8) return QAT_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size % 16 || c->page_size > INT32_MAX)
    return QAT_ERR_INVALID_ARGUMENT;
  if (c->pages < 0 || c->pages > INT32_MAX / c->page_size || c->heads < 1 || c->heads > 32767)
    return QAT_ERR_INVALID_ARGUMENT;
  // (tiles of 16 rows are counted in 31 bits; their bytes would fill more than any memory)
  if (c->pages * (c->page_size / 16) > INT32_MAX / c->heads) return QAT_ERR_INVALID_ARGUMENT;
  const bool ints = f == QAT_CACHE_INT8 || f == QAT_CACHE_INT4;
  if (!c->k_zero_points != !c->v_zero_points || (c->k_zero_points && !ints))
    return QAT_ERR_INVALID_ARGUMENT;
  if (c->pages == 0) return QAT_OK;
  if (!c->k || !c->v || (f != QAT_CACHE_BF16 && (!c->k_scales || !c->v_scales)))
    return QAT_ERR_INVALID_ARGUMENT;
  if (!on(c->k, 16) || !on(c->v, 16) || !on(c->k_scales, 16) || !on(c->v_scales, 16) ||
      !on(c->k_zero_points, 16) || !on(c->v_zero_points, 16))
    return QAT_ERR_MISALIGNED;
  return QAT_OK;
}

}  // namespace

extern "C" {

qat_status qat_head_norm_rope(const void* q, const void* k, qat_dtype dtype, int64_t tokens,
                              int64_t q_heads, int64_t k_heads, int64_t head_dim,
                              int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                              int64_t k_head_stride, const int64_t* positions, const uint64_t* turns,
                              int64_t rotary_dim, qat_rope_layout layout, float amplitude, int norm,
                              const void* q_weight, const void* k_weight, float eps, void* q_out,
                              void* k_out, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_head_norm_rope");
  const RopeSizes z = {tokens, q_heads, k_heads, head_dim, rotary_dim,
                       q_token_stride, q_head_stride, k_token_stride, k_head_stride};
  const qat_status st = check_rope(z, dtype, layout, amplitude, norm, eps, q_weight, k_weight);
  if (st) return st;
  if (tokens == 0 || (q_heads == 0 && k_heads == 0)) return QAT_OK;
  if ((q_heads > 0 && (!q || !q_out)) || (k_heads > 0 && (!k || !k_out)) || !positions ||
      (rotary_dim > 0 && !turns))
    return QAT_ERR_INVALID_ARGUMENT;
  const uintptr_t e = esize(dtype);
  if (!on(q, e) || !on(k, e) || !on(q_out, e) || !on(k_out, e) || !on(q_weight, e) ||
      !on(k_weight, e) || !on(positions, 8) || !on(turns, 8))
    return QAT_ERR_MISALIGNED;
  RopeArgs a =
      rope_args(z, q, k, positions, turns, layout, amplitude, norm, eps, q_weight, k_weight);
  a.y[0] = q_out, a.y[1] = k_out;
  return launch_rope_fwd(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t qat_head_norm_rope_backward_workspace_bytes(int64_t head_dim) {
  if (head_dim < 1 || head_dim > 512) return 0;
  return (size_t)kRopeParts * (size_t)head_dim * 4;
}

qat_status qat_head_norm_rope_backward(
    const void* dq_out, const void* dk_out, const void* q, const void* k, qat_dtype dtype,
    int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim, int64_t q_token_stride,
    int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride, const int64_t* positions,
    const uint64_t* turns, int64_t rotary_dim, qat_rope_layout layout, float amplitude, int norm,
    const void* q_weight, const void* k_weight, float eps, void* dq, void* dk, void* dq_weight,
    void* dk_weight, void* workspace, size_t workspace_bytes, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_head_norm_rope_backward");
  const RopeSizes z = {tokens, q_heads, k_heads, head_dim, rotary_dim,
                       q_token_stride, q_head_stride, k_token_stride, k_head_stride};
  const qat_status st = check_rope(z, dtype, layout, amplitude, norm, eps, q_weight, k_weight);
  if (st) return st;
  if (!norm && (dq_weight || dk_weight)) return QAT_ERR_INVALID_ARGUMENT;
  const bool q_on = tokens > 0 && q_heads > 0 && (dq || dq_weight);
  const bool k_on = tokens > 0 && k_heads > 0 && (dk || dk_weight);
  if (!q_on && !k_on && !dq_weight && !dk_weight) return QAT_OK;
  if ((q_on && (!dq_out || !q)) || (k_on && (!dk_out || !k)) ||
      ((q_on || k_on) && (!positions || (rotary_dim > 0 && !turns))))
    return QAT_ERR_INVALID_ARGUMENT;
  const uintptr_t e = esize(dtype);
  for (const void* p : {dq_out, dk_out, q, k, q_weight, k_weight, (const void*)dq,
                        (const void*)dk, (const void*)dq_weight, (const void*)dk_weight})
    if (!on(p, e)) return QAT_ERR_MISALIGNED;
  if (!on(positions, 8) || !on(turns, 8)) return QAT_ERR_MISALIGNED;
  if ((dq_weight || dk_weight) && (q_on || k_on)) {
    if (!workspace || workspace_bytes < qat_head_norm_rope_backward_workspace_bytes(head_dim))
      return QAT_ERR_WORKSPACE;
    if (!on(workspace, 16)) return QAT_ERR_MISALIGNED;
  }
  RopeArgs a =
      rope_args(z, q, k, positions, turns, layout, amplitude, norm, eps, q_weight, k_weight);
  a.g[0] = dq_out, a.g[1] = dk_out, a.y[0] = dq, a.y[1] = dk, a.dw[0] = dq_weight,
  a.dw[1] = dk_weight;
  if (!q_on) a.heads[0] = 0;
  if (!k_on) a.heads[1] = 0;
  return launch_rope_bwd(a, dtype, static_cast<float*>(workspace),
                         reinterpret_cast<cudaStream_t>(stream));
}

size_t qat_kv_row_bytes(int format, int64_t head_dim) {
  if (format < QAT_CACHE_BF16 || format > QAT_CACHE_E5M2 || head_dim < 8 || head_dim > 256 ||
      head_dim % 8)
    return 0;
  return (size_t)kv_row_bytes(format, head_dim);
}

qat_status qat_kv_write(const qat_kv_cache* cache, const void* k, const void* v, qat_dtype dtype,
                        int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                        int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                        qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_kv_write");
  if (!dtype_ok(dtype)) return QAT_ERR_UNSUPPORTED;
  const qat_status st = check_cache(cache);
  if (st) return st;
  if (!fits(tokens, cache->heads * cache->head_dim)) return QAT_ERR_INVALID_ARGUMENT;
  if (!stride_ok(k_token_stride, tokens) || !stride_ok(v_token_stride, tokens) ||
      !stride_ok(k_head_stride, cache->heads) || !stride_ok(v_head_stride, cache->heads))
    return QAT_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || cache->pages == 0) return QAT_OK;
  if (!k || !v || !slots) return QAT_ERR_INVALID_ARGUMENT;
  const uintptr_t e = esize(dtype);
  if (!on(k, e) || !on(v, e) || !on(slots, 8)) return QAT_ERR_MISALIGNED;
  const KvRows x = {k, v, {k_token_stride, v_token_stride}, {k_head_stride, v_head_stride}};
  return launch_kv_write(*cache, x, dtype, tokens, slots, reinterpret_cast<cudaStream_t>(stream));
}

qat_status qat_kv_read(const qat_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k,
                       void* v, qat_dtype dtype, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_kv_read");
  if (!dtype_ok(dtype)) return QAT_ERR_UNSUPPORTED;
  const qat_status st = check_cache(cache);
  if (st) return st;
  if (!fits(tokens, cache->heads * cache->head_dim)) return QAT_ERR_INVALID_ARGUMENT;
  if (tokens == 0) return QAT_OK;
  if (!k || !v || !slots) return QAT_ERR_INVALID_ARGUMENT;
  if (!on(k, 16) || !on(v, 16) || !on(slots, 8)) return QAT_ERR_MISALIGNED;
  return launch_kv_read(*cache, slots, tokens, k, v, dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t qat_kv_attention_workspace_bytes(const qat_kv_cache* cache, int64_t q_heads) {
  if (check_cache(cache) || q_heads < 1 || q_heads % cache->heads || q_heads > INT32_MAX) return 0;
  return kv_attn_ws_bytes(q_heads, cache->heads, cache->head_dim);
}

qat_status qat_kv_attention(const void* q, qat_dtype dtype, int64_t batch, int64_t q_heads,
                            int64_t q_batch_stride, int64_t q_head_stride, const qat_kv_cache* cache,
                            const int32_t* table, int64_t table_cols, int64_t table_stride,
                            const int32_t* lengths, float scale, void* y, float* lse,
                            void* workspace, size_t workspace_bytes, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_kv_attention");
  if (!dtype_ok(dtype)) return QAT_ERR_UNSUPPORTED;
  const qat_status st = check_cache(cache);
  if (st) return st;
  if (batch < 0 || batch > 65535 || q_heads < 0 || table_cols < 0 || table_cols > INT32_MAX ||
      !std::isfinite(scale) || (batch > 0 && q_heads > INT32_MAX / batch) ||
      !stride_ok(q_batch_stride, batch) || !stride_ok(q_head_stride, q_heads) ||
      !stride_ok(table_stride, batch))
    return QAT_ERR_INVALID_ARGUMENT;
  if (q_heads % cache->heads) return QAT_ERR_DIMENSION_MISMATCH;
  if (batch == 0 || q_heads == 0) return QAT_OK;
  if (!q || !y || !lengths || (table_cols > 0 && !table)) return QAT_ERR_INVALID_ARGUMENT;
  const uintptr_t e = esize(dtype);
  if (!on(q, e) || !on(y, e) || !on(lse, 4) || !on(table, 4) || !on(lengths, 4))
    return QAT_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < qat_kv_attention_workspace_bytes(cache, q_heads))
    return QAT_ERR_WORKSPACE;
  if (!on(workspace, 16)) return QAT_ERR_MISALIGNED;
  const KvAttnArgs a = {q, batch, q_heads, q_batch_stride, q_head_stride, table, table_cols,
                        table_stride, lengths, scale, y, lse};
  return launch_kv_attn(*cache, a, dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
