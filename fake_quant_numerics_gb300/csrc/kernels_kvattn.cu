// kernels_kvattn.cu -- attention of one new token of each sequence over a paged
// cache: the split kernel of the cache's format, and the join of what it cut.
#include <cmath>

#include "qat_kv.cuh"
#include "qat_kvsplit.h"
#include "qat_layer.cuh"

namespace qat {
namespace {

// For each block of the split kernel (x) whose end cut a sequence off, a query head of
// it (y): the parts - the block's second slot, then the first slots of the blocks
// behind it - are added in that order within each of four warps, every fourth one a
// warp's, and then over the warps.
constexpr int kJoinWarps = 4;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) k_kv_join(SplitWs ws, KvAttnArgs a, int d,
                                                             int group, int tiles, int tile) {
  __shared__ __align__(16) float share[kJoinWarps][256];
  __shared__ float sums[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  pdl_wait();
  const int4 cut = ws.cut[blockIdx.x];
  const int kvh = cut.y / tiles, h0 = kvh * group + (cut.y - kvh * tiles) * tile;
  if (cut.z == 0 || h >= min(tile, (kvh + 1) * group - h0)) return;
  auto slot = [&](int part) {
    return ((int64_t)(blockIdx.x + part) * 2 + (part == 0)) * tile + h;
  };
  float top = -INFINITY, sum = 0.0f, y[8] = {};
  for (int p = lane; p < cut.z; p += 32) top = fmaxf(top, ws.ml[slot(p)].x);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
#pragma unroll 4
  for (int p = warp; p < cut.z; p += kJoinWarps) {
    const float2 ml = ws.ml[slot(p)];
    const float f = ml.x == top ? 1.0f : exp2f(ml.x - top);
    sum = __fmaf_rn(f, ml.y, sum);
    const float* from = ws.o + slot(p) * d;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (4 * (lane + 32 * i) < d) {
        const float4 v = *reinterpret_cast<const float4*>(from + 4 * (lane + 32 * i));
        y[4 * i] = __fmaf_rn(f, v.x, y[4 * i]);
        y[4 * i + 1] = __fmaf_rn(f, v.y, y[4 * i + 1]);
        y[4 * i + 2] = __fmaf_rn(f, v.z, y[4 * i + 2]);
        y[4 * i + 3] = __fmaf_rn(f, v.w, y[4 * i + 3]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<float4*>(&share[warp][4 * (lane + 32 * i)]) =
        make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) sum += sums[w];
  const int64_t row = (int64_t)cut.x * a.q_heads + h0 + h;
  for (int e = threadIdx.x; e < d; e += 32 * kJoinWarps) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) v += share[w][e];
    st_elem<T>(a.y, row * d + e, sum == 0.0f ? 0.0f : __fdiv_rn(v, sum));
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

constexpr size_t kCutBytes = kSplitBlocks * sizeof(int4);
size_t ml_bytes(int tile) { return (size_t)kSplitBlocks * 2 * tile * sizeof(float2); }

}  // namespace

size_t kv_attn_ws_bytes(int64_t q_heads, int64_t kv_heads, int64_t d) {
  const int tile = head_tiles(q_heads, kv_heads, d, false).tile;  // (the larger of both types)
  return kCutBytes + ml_bytes(tile) + (size_t)kSplitBlocks * 2 * tile * (size_t)d * 4;
}

qat_status launch_kv_attn(const qat_kv_cache& c, const KvAttnArgs& a, qat_dtype dt, void* ws,
                          cudaStream_t s) {
  const KvCacheView v = {(const char*)c.k, (const char*)c.v, c.k_scales, c.v_scales, c.k_zero_points,
                         c.v_zero_points, c.pages, (int)c.heads, (int)c.page_size, (int)c.head_dim,
                         (int)kv_row_bytes(c.format, c.head_dim)};
  const HeadTiles t = head_tiles(a.q_heads, c.heads, c.head_dim, dt == QAT_F32);
  char* p = static_cast<char*>(ws);
  const SplitWs w = {reinterpret_cast<int4*>(p), reinterpret_cast<float2*>(p + kCutBytes),
                     reinterpret_cast<float*>(p + kCutBytes + ml_bytes(t.tile))};
  int grid = 0;
  qat_status st;
  switch (c.format) {
    case QAT_CACHE_INT8: st = launch_kv_split<QAT_CACHE_INT8>(v, a, dt, w, &grid, s); break;
    case QAT_CACHE_INT4: st = launch_kv_split<QAT_CACHE_INT4>(v, a, dt, w, &grid, s); break;
    case QAT_CACHE_E4M3: st = launch_kv_split<QAT_CACHE_E4M3>(v, a, dt, w, &grid, s); break;
    case QAT_CACHE_E5M2: st = launch_kv_split<QAT_CACHE_E5M2>(v, a, dt, w, &grid, s); break;
    default: st = launch_kv_split<QAT_CACHE_BF16>(v, a, dt, w, &grid, s);
  }
  if (st) return st;
  const auto k = dt == QAT_F32 ? k_kv_join<F32> : k_kv_join<BF16>;
  if (launch_kernel(k, dim3(grid, t.tile), dim3(32 * kJoinWarps), 0, s, true, w, a, (int)c.head_dim,
                    t.group, t.tiles, t.tile) != cudaSuccess)
    return QAT_ERR_CUDA;
  count_launch(1);
  return QAT_OK;
}

}  // namespace qat
