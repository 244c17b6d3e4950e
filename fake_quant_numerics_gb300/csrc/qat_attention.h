// qat_attention.h -- launchers of the attention operators (internal; not part of
// the C ABI).  Arguments are validated by qat_attention_abi.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qat.h"
#include "qat_launch.h"

namespace qat {

// Queries (0) and keys (1) of a head norm with rotation, forward or backward.
struct RopeArgs {
  const void *x[2], *g[2], *w[2];   // inputs, gradients of the outputs, norm weights
  void *y[2], *dw[2];               // outputs or input gradients, weight gradients
  int64_t token_stride[2], head_stride[2];
  int heads[2];
  const int64_t* positions;
  const uint64_t* turns;
  int64_t tokens;
  int d, rotary, norm, interleaved;
  float amplitude, eps, inv_d;
};
// Blocks of the backward pass at most, one row of partial weight gradients each:
// float[kRopeParts][d] in the workspace.
constexpr int kRopeParts = 320;
qat_status launch_rope_fwd(const RopeArgs& a, qat_dtype dt, cudaStream_t s);
qat_status launch_rope_bwd(const RopeArgs& a, qat_dtype dt, float* ws, cudaStream_t s);

// Bytes of a cache row: whole 16-byte vectors.
constexpr int64_t kv_row_bytes(int format, int64_t d) {
  return format == QAT_CACHE_BF16 ? 2 * d
                                  : ((format == QAT_CACHE_INT4 ? d / 2 : d) + 15) / 16 * 16;
}
struct KvRows {
  const void *k, *v;
  int64_t token_stride[2], head_stride[2];
};
qat_status launch_kv_write(const qat_kv_cache& c, const KvRows& x, qat_dtype dt, int64_t tokens,
                           const int64_t* slots, cudaStream_t s);
qat_status launch_kv_read(const qat_kv_cache& c, const int64_t* slots, int64_t tokens, void* k,
                          void* v, qat_dtype dt, cudaStream_t s);

struct KvAttnArgs {
  const void* q;
  int64_t batch, q_heads, q_batch_stride, q_head_stride;
  const int32_t* table;
  int64_t table_cols, table_stride;
  const int32_t* lengths;
  float scale;
  void* y;
  float* lse;
};
size_t kv_attn_ws_bytes(int64_t q_heads, int64_t kv_heads, int64_t d);
qat_status launch_kv_attn(const qat_kv_cache& c, const KvAttnArgs& a, qat_dtype dt, void* ws,
                          cudaStream_t s);

}  // namespace qat
