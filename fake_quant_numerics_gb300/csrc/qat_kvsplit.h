// qat_kvsplit.h -- what the split attention kernel and its join share (internal).
#pragma once

#include "qat_attention.h"

namespace qat {

// Blocks of the split kernel at most, one on each SM; a block leaves up to two parts
// of sequences that it shares with its neighbours.
constexpr int kSplitBlocks = 160;

// The longest sequence.
constexpr int kKvMaxLength = INT32_MAX - 1024;

struct KvCacheView {
  const char *k, *v;
  const float *ks, *vs;
  const int8_t *kz, *vz;
  int64_t pages;
  int heads, page_size, d, row_bytes;
};

// Workspace: one int4 a block - sequence, group of heads, number of parts of the
// sequence that its end cuts off (0: none) -, then for each block and slot [heads]
// maximum and sum, then [heads][d] sums of weighted values.  Slot 0 holds a sequence
// that began in an earlier block, slot 1 the one cut off.
struct SplitWs {
  int4* cut;
  float2* ml;
  float* o;
};
// Query heads that share a cache head, `tile` at a time: tiles of 8, or of 16
// where a group has more heads, the products are bf16 and the head is short.
struct HeadTiles {
  int group, tile, tiles;
};
inline HeadTiles head_tiles(int64_t q_heads, int64_t kv_heads, int64_t d, bool f32) {
  const int group = (int)(q_heads / kv_heads);
  const int tile = group > 8 && !f32 && d <= 128 ? 16 : 8;
  return {group, tile, (group + tile - 1) / tile};
}

template <int F>
qat_status launch_kv_split(const KvCacheView& c, const KvAttnArgs& a, qat_dtype dt, const SplitWs& ws,
                           int* grid, cudaStream_t s);

}  // namespace qat
