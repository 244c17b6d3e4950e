// kernels_kvsplit.cu -- attention of one new token of each sequence over a paged,
// quantized key-value cache (compiled once for each cache format QAT_KV_FORMAT).
//
//   s_t = scale ks_t (q . kq_t - kz_t sum q),  p_t = exp(s_t - m),  w_t = p_t vs_t
//   y = (sum w_t vq_t - sum w_t vz_t) / sum p_t        (kq, vq codes; kz, vz zero points)
//
// The floor is reading the codes once.  The query heads of a cache head share a
// read: they are the eight columns of m16n8k16 products whose rows are positions
// (scores) or head elements (values), both operands' codes exact in bf16.
//
// Work is cut evenly whatever the lengths: the blocks of kBlockKeys positions of
// every (sequence, head group), in one row, are dealt to the resident blocks in
// equal runs.  A run that starts or ends inside a sequence leaves a partial result
// (maximum, sum, weighted values), joined in order by k_kv_join.
//
// A warp takes every fourth tile of its block's run, with a maximum, a sum and
// weighted values of its own, joined over the block's warps where a sequence's
// piece ends.  Each lane copies exactly the codes that it multiplies (cp.async into
// slots of its own), so that only scales are exchanged between lanes: rows of the
// product are positions lane / 4 (+ 8) for keys, and the lane's share of a key is
// every fourth 16-byte run; of a value every eighth.  Which head element a product's
// k index stands for is free, so the codes' own order is taken for both operands.
#include <cmath>

#include "qat_kv.cuh"
#include "qat_kvsplit.h"
#include "qat_layer.cuh"

namespace qat {
namespace {

constexpr int kFormat = QAT_KV_FORMAT;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;  // scores may exceed the running maximum by 2^8 before it moves

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// `bytes` (4, 8 or 16) from global to shared memory, or zeros
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool on) {
  const int n = on ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of 16-bit elements, transposed over the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int BYTES>
__device__ __forceinline__ void load_run(const char* p, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// ---------------------------------------------------------------------------
// codes: the pairs of bf16 that a 32-bit word holds, in the order of its bits
// ---------------------------------------------------------------------------
template <int F>
struct Word {
  static constexpr int CODES = F == QAT_CACHE_INT4 ? 8 : F == QAT_CACHE_BF16 ? 2 : 4;
  static constexpr int PAIRS = CODES / 2;
  // the elements of pair i: `lo` in the low half, HALF elements on the one in the high
  static constexpr int HALF = CODES / 2;
  __host__ __device__ static constexpr int lo(int i) { return F == QAT_CACHE_INT4 ? i ^ 1 : i; }

  __device__ __forceinline__ static void decode(uint32_t w, uint32_t (&out)[PAIRS]) {
    if constexpr (F == QAT_CACHE_BF16) {
      out[0] = w;
    } else if constexpr (F == QAT_CACHE_INT4) {
      // 128 + (q + 8) in bf16, less 136
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[i] = sub2(((w >> (4 * i)) & 0x000f000fu) ^ 0x43084308u, 0x43084308u);
    } else if constexpr (F == QAT_CACHE_INT8) {
      // 128 + the low seven bits, less 128 or, where the sign is set, 256
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = w >> (8 * i);
        out[i] = sub2((x & 0x007f007fu) | 0x43004300u, (x & 0x00800080u) | 0x43004300u);
      }
    } else {
      // the code's exponent and fraction at bf16's place, times 2^(127 - bias); codes
      // are finite, as the cache's rows are written
      constexpr int SH = F == QAT_CACHE_E4M3 ? 4 : 3;
      constexpr uint32_t M = F == QAT_CACHE_E4M3 ? 0x07f007f0u : 0x0fe00fe0u;
      constexpr uint32_t UP = F == QAT_CACHE_E4M3 ? 0x7b807b80u : 0x77807780u;  // 2^120, 2^112
      out[0] = mul2(((w << (8 - SH)) & M) | ((w << 8) & 0x80008000u), UP);
      out[1] = mul2(((w >> SH) & M) | (w & 0x80008000u), UP);
    }
  }
  __device__ __forceinline__ static uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ static uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

// ---------------------------------------------------------------------------
// shapes: DP the head dimension the products take (64, 128, 256; elements behind
// head_dim are zeros), HT tiles of eight query heads
// ---------------------------------------------------------------------------
__device__ __forceinline__ int smaller_of(int a, int b) { return a < b ? a : b; }
constexpr int smaller(int a, int b) { return a < b ? a : b; }
constexpr int larger(int a, int b) { return a > b ? a : b; }

template <typename T, int F, int DP, int HT>
struct Shape {
  using W = Word<F>;
  static constexpr bool kF32 = T::BYTES == 4;
  static constexpr int ROW = DP / W::CODES * 4;  // bytes of a row of DP codes
  // a lane's share of a key: NK runs of CK bytes, every fourth one; of a value NV of
  // CV bytes, every eighth
  static constexpr int CK = smaller(16, ROW / 4), NK = ROW / 4 / CK, EK = CK / 4 * W::CODES;
  static constexpr int CV = smaller(16, ROW / 8), NV = ROW / 8 / CV, EV = CV / 4 * W::CODES;
  static constexpr int TILE = 32 * ROW;  // 16 keys and values
  static constexpr int PARAMS = kFormat == QAT_CACHE_BF16 ? 0 : 160;  // 16 scales each, 16 zero points each
  static constexpr int NT = smaller(2, larger(1, 4096 / TILE));  // tiles a step
  static constexpr int STAGES = TILE > 8192 ? 2 : TILE > 4096 ? 3 : 4;
  static constexpr int STAGE = NT * (TILE + PARAMS);
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int KEYS = kWarps * NT * 16;  // a block's step
  static constexpr int H = 8 * HT, KS = DP / 16, MT = DP / 16;
  static constexpr int QP = kF32 ? 3 : 1, PP = kF32 ? 3 : 2;  // bf16 parts of q and of the weights
  static constexpr int OPAD = DP + 4;
  static constexpr int JOIN = kWarps * H * OPAD * 4;  // (reuses the ring)
  static constexpr int QRAW = H * (DP + 1) * 4;       // (likewise)
  static constexpr int BODY = larger(larger(RING, JOIN), QRAW);
  static constexpr int QFRAG = kF32 ? QP * KS * 32 * 8 : 0;
  static constexpr int ML = kWarps * H * 3 * 4;
  static constexpr int SMEM = (BODY + 15) / 16 * 16 + QFRAG + ML;

  // The head element of half `hi` of pair p of lane t's share of a key.
  __device__ __forceinline__ static int key_elem(int p, int hi, int t) {
    const int word = p / W::PAIRS, i = p % W::PAIRS, run = word / (CK / 4);
    return (4 * run + t) * EK + (word % (CK / 4)) * W::CODES + W::lo(i) + hi * W::HALF;
  }
  // The place of head element e in the order of the value products' rows: eight
  // lanes side by side, pairs in the order in which they are decoded.
  __device__ __forceinline__ static int value_place(int e) {
    const int chunk = e / EV, g = chunk % 8, run = chunk / 8, in = e % EV;
    const int word = run * (CV / 4) + in / W::CODES, c = in % W::CODES;
    const int half = c / W::HALF, i = W::lo(c % W::HALF);  // (lo is its own inverse)
    return ((word * 2 + half) * W::PAIRS + i) * 8 + g;
  }
};

struct Piece {  // blocks [from, to) of `blocks` of sequence b's head group hg
  int b, hg, from, to, blocks;
};

template <typename T, int F, int DP, int HT>
__global__ void __launch_bounds__(kThreads, DP * HT <= 128 && T::BYTES == 2 ? 3 : 2)
    k_kv_split(KvCacheView c, KvAttnArgs a, int group, int tiles, SplitWs ws) {
  using S = Shape<T, F, DP, HT>;
  using W = typename S::W;
  extern __shared__ __align__(16) char smem[];
  __shared__ int64_t s_sum[kWarps + 1];
  __shared__ int s_at[3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  pdl_trigger();

  // --- this block's run of the work ---------------------------------------------
  // (a position's number plus a block's step fits 31 bits)
  const int64_t capacity = min(a.table_cols * c.page_size, (int64_t)kKvMaxLength);
  const int hgs = c.heads * tiles;
  auto length_of = [&](int b) -> int {  // 0 where there is nothing to read
    const int n = __ldg(a.lengths + b);
    return n <= 0 || n > capacity ? 0 : n;
  };
  auto blocks_of = [&](int b) { return (length_of(b) + S::KEYS - 1) / S::KEYS; };
  const int batch = (int)a.batch;
  const int each = (batch + kThreads - 1) / kThreads;
  const int b_lo = smaller_of(threadIdx.x * each, batch), b_hi = smaller_of(b_lo + each, batch);
  int64_t own = 0;
  for (int b = b_lo; b < b_hi; ++b) own += blocks_of(b);
  int64_t before = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(kFull, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) s_sum[warp] = before;
  if (threadIdx.x == 0) s_at[0] = -1;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  before -= own;
  total *= hgs;
  // equal runs for as many blocks as there is work for; the others have none
  const int64_t runs = max((int64_t)1, min((int64_t)gridDim.x, total));
  const bool idle = blockIdx.x >= runs || total == 0;
  const int64_t first = idle ? 0 : total * blockIdx.x / runs;
  const int64_t end = idle ? 0 : total * (blockIdx.x + 1) / runs;
  if (first < end && before * hgs <= first && first < (before + own) * hgs) {
    int b = b_lo;
    int64_t at = before * hgs;
    while (first >= at + (int64_t)blocks_of(b) * hgs) at += (int64_t)blocks_of(b++) * hgs;
    const int n = blocks_of(b);
    s_at[0] = b;
    s_at[1] = (int)((first - at) / n);
    s_at[2] = (int)((first - at) % n);
  }
  // sequences that have nothing to read
  const int64_t y_row = a.q_heads * c.d;
  for (int b = blockIdx.x; b < batch; b += gridDim.x) {
    if (length_of(b)) continue;
    const bool none = __ldg(a.lengths + b) <= 0;
    for (int64_t i = threadIdx.x; i < y_row; i += kThreads)
      st_elem<T>(a.y, b * y_row + i, none ? 0.0f : NAN);
    if (a.lse)
      for (int64_t i = threadIdx.x; i < a.q_heads; i += kThreads)
        a.lse[b * a.q_heads + i] = none ? -INFINITY : NAN;
  }
  __syncthreads();
  int4 cut = make_int4(0, 0, 0, 0);
  int64_t left = end - first;
  Piece pc = {s_at[0], s_at[1], s_at[2], 0, 0};

  const uint32_t ring = smem_at(smem) + warp * (S::STAGES * S::STAGE);
  char* const ring_p = smem + warp * (S::STAGES * S::STAGE);
  uint2* const qfrag = reinterpret_cast<uint2*>(smem + (S::BODY + 15) / 16 * 16);
  float* const ml = reinterpret_cast<float*>(smem + (S::BODY + 15) / 16 * 16 + S::QFRAG);
  const int tiles_page = c.page_size / 16;
  const float to_log2 = a.scale * kLog2e;

  while (left > 0) {
    const int length = length_of(pc.b);
    pc.blocks = (length + S::KEYS - 1) / S::KEYS;
    pc.to = (int)min((int64_t)pc.blocks, pc.from + left);
    left -= pc.to - pc.from;
    const int kvh = pc.hg / tiles, h0 = kvh * group + (pc.hg - kvh * tiles) * S::H;
    const int heads = min(S::H, (kvh + 1) * group - h0);
    const int steps = pc.to - pc.from;

    // --- the queries as products take them ----------------------------------------
    float* const raw = reinterpret_cast<float*>(smem);
    for (int i = threadIdx.x; i < S::H * DP; i += kThreads) {
      const int h = i / DP, e = i % DP;
      raw[h * (DP + 1) + e] =
          h < heads && e < c.d
              ? ld_elem<T>(a.q, pc.b * a.q_batch_stride + (h0 + h) * a.q_head_stride + e)
              : 0.0f;
    }
    __syncthreads();
    uint32_t qr[S::kF32 ? 1 : HT][S::kF32 ? 1 : S::KS][2];
    float qsum[HT][2];  // of heads 2 t4, 2 t4 + 1
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      float sum = 0.0f;
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = raw[(8 * ht + g) * (DP + 1) + S::key_elem(2 * ks + i / 2, i % 2, t4)];
          sum += v[i];
        }
        if constexpr (!S::kF32) {
          qr[ht][ks][0] = pack_bf16x2(v[0], v[1]);
          qr[ht][ks][1] = pack_bf16x2(v[2], v[3]);
        } else if (ks % kWarps == warp) {
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            uint2 f;
            const float x0 = take_bf16(v[0]), x1 = take_bf16(v[1]);
            const float x2 = take_bf16(v[2]), x3 = take_bf16(v[3]);
            f.x = __float_as_uint(x0) >> 16 | (__float_as_uint(x1) & 0xffff0000u);
            f.y = __float_as_uint(x2) >> 16 | (__float_as_uint(x3) & 0xffff0000u);
            qfrag[(p * S::KS + ks) * 32 + lane] = f;
          }
        }
      }
      sum += __shfl_xor_sync(kFull, sum, 1);
      sum += __shfl_xor_sync(kFull, sum, 2);
      qsum[ht][0] = __shfl_sync(kFull, sum, 8 * t4);
      qsum[ht][1] = __shfl_sync(kFull, sum, 8 * t4 + 4);
    }
    __syncthreads();

    // --- copies: the lane's share of tile after tile --------------------------------
    // The warp's tiles of this piece in order; lane l knows the place (in tiles of 16
    // rows) of the l-th of the 32 from `known` on: -1 a page that does not exist, -2
    // behind the sequence.
    const int n_tiles = (length + 15) / 16;
    int64_t place = -2;
    bool bad = false;
    auto look_up = [&](int from) {
      const int e = from + lane;
      const int tile = ((pc.from + e / S::NT) * kWarps + warp) * S::NT + e % S::NT;
      place = -2;
      if (e < steps * S::NT && tile < n_tiles) {
        const int col = tile / tiles_page;
        const int page = __ldg(a.table + pc.b * a.table_stride + col);
        place = page < 0 || page >= c.pages
                    ? -1
                    : ((int64_t)page * c.heads + kvh) * tiles_page + (tile - col * tiles_page);
      }
    };
    auto issue = [&](int step) {
      if (step < steps) {
        if ((step * S::NT) % 32 == 0) look_up(step * S::NT);
#pragma unroll
        for (int t = 0; t < S::NT; ++t) {
          const int64_t at = __shfl_sync(kFull, place, (step * S::NT + t) % 32);
          if (at == -1) bad = true;
          if (at < 0) continue;
          const int key0 = (((pc.from + step) * kWarps + warp) * S::NT + t) * 16;
          const uint32_t slot = ring + (step % S::STAGES) * S::STAGE + t * (S::TILE + S::PARAMS);
          const char* kp = c.k + at * 16 * c.row_bytes;
          const char* vp = c.v + at * 16 * c.row_bytes;
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < S::NK; ++j) {
              const int off = (4 * j + t4) * S::CK;
              copy_async<S::CK>(slot + ((r * S::NK + j) * 32 + lane) * S::CK,
                                kp + (g + 8 * r) * c.row_bytes + off,
                                key0 + g + 8 * r < length && off < c.row_bytes);
            }
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < S::NV; ++j) {
              const int row = 2 * t4 + (r & 1) + 8 * (r >> 1), off = (8 * j + g) * S::CV;
              copy_async<S::CV>(slot + S::TILE / 2 + ((r * S::NV + j) * 32 + lane) * S::CV,
                                vp + row * c.row_bytes + off,
                                key0 + row < length && off < c.row_bytes);
            }
          if constexpr (F != QAT_CACHE_BF16) {
            // 16 scales of keys, of values, then the zero points: runs of 16 bytes
            const char* src = reinterpret_cast<const char*>(lane < 4 ? c.ks : c.vs) + at * 64 +
                              (lane & 3) * 16;
            if (lane >= 8)
              src = reinterpret_cast<const char*>(lane == 8 ? c.kz : c.vz) + at * 16;
            if (lane < (kv_is_int(F) && c.kz ? 10 : 8))
              copy_async<16>(slot + S::TILE + lane * 16, src, true);
          }
        }
      }
      copy_commit();
    };

    float m[HT][2], l[HT][2], zsum[HT][2], o[HT][S::MT][4];
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
      for (int i = 0; i < 2; ++i) m[ht][i] = -INFINITY, l[ht][i] = 0.0f, zsum[ht][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < S::MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[ht][i][j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; ++i) issue(i);

    for (int step = 0; step < steps; ++step) {
      copy_wait<S::STAGES - 2>();
      __syncwarp();  // scales of other lanes' copies; and the slot of the step before is free
      issue(step + S::STAGES - 1);
      const char* const stage = ring_p + (step % S::STAGES) * S::STAGE;
#pragma unroll
      for (int t = 0; t < S::NT; ++t) {
        const int key0 = (((pc.from + step) * kWarps + warp) * S::NT + t) * 16;
        if (key0 >= length) break;
        const char* const slot = stage + t * (S::TILE + S::PARAMS);
        // scores of positions g, g + 8 (rows) and heads 2 t4, 2 t4 + 1 (columns)
        float s[HT][4];
        {
          float acc[S::QP][HT][4];
#pragma unroll
          for (int p = 0; p < S::QP; ++p)
#pragma unroll
            for (int ht = 0; ht < HT; ++ht)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[p][ht][i] = 0.0f;
#pragma unroll
          for (int j = 0; j < S::NK; ++j) {
            uint32_t w[2][S::CK / 4];
#pragma unroll
            for (int r = 0; r < 2; ++r)
              load_run<S::CK>(slot + ((r * S::NK + j) * 32 + lane) * S::CK, w[r]);
            uint32_t pr[2][S::CK / 4 * W::PAIRS];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int i = 0; i < S::CK / 4; ++i) {
                uint32_t d[W::PAIRS];
                W::decode(w[r][i], d);
#pragma unroll
                for (int k = 0; k < W::PAIRS; ++k) pr[r][i * W::PAIRS + k] = d[k];
              }
#pragma unroll
            for (int k = 0; k < S::EK / 4; ++k) {
              const int ks = j * (S::EK / 4) + k;
              const uint32_t fa[4] = {pr[0][2 * k], pr[1][2 * k], pr[0][2 * k + 1], pr[1][2 * k + 1]};
              if constexpr (S::kF32) {
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                  const uint2 f = qfrag[(p * S::KS + ks) * 32 + lane];
                  mma(acc[p][0], fa, f.x, f.y);
                }
              } else {
#pragma unroll
                for (int ht = 0; ht < HT; ++ht) mma(acc[0][ht], fa, qr[ht][ks][0], qr[ht][ks][1]);
              }
            }
          }
#pragma unroll
          for (int ht = 0; ht < HT; ++ht)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s[ht][i] = acc[0][ht][i];
              if constexpr (S::kF32) s[ht][i] += acc[1][ht][i] + acc[2][ht][i];
            }
        }
        float vs[2] = {1.0f, 1.0f}, vz[2] = {0.0f, 0.0f};
        {
          float ks[2] = {1.0f, 1.0f}, kz[2] = {0.0f, 0.0f};
          if constexpr (F != QAT_CACHE_BF16) {
            const float* sc = reinterpret_cast<const float*>(slot + S::TILE);
            ks[0] = sc[g], ks[1] = sc[g + 8], vs[0] = sc[16 + g], vs[1] = sc[24 + g];
            if (kv_is_int(F) && c.kz) {
              const int8_t* z = reinterpret_cast<const int8_t*>(slot + S::TILE + 128);
              kz[0] = z[g], kz[1] = z[g + 8], vz[0] = z[16 + g], vz[1] = z[24 + g];
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float f = ks[r] * to_log2;
#pragma unroll
            for (int ht = 0; ht < HT; ++ht)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float& x = s[ht][2 * r + i];
                x = f * __fmaf_rn(-kz[r], qsum[ht][i], x);
              }
          }
          if (key0 + 16 > length) {  // rows behind the sequence
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (key0 + g + 8 * r >= length) {
                vs[r] = vz[r] = 0.0f;
#pragma unroll
                for (int ht = 0; ht < HT; ++ht) s[ht][2 * r] = s[ht][2 * r + 1] = -INFINITY;
              }
          }
        }
        // the running maximum moves only where a score is far above it
        bool above = false;
#pragma unroll
        for (int ht = 0; ht < HT; ++ht)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            above = above || fmaxf(s[ht][i], s[ht][2 + i]) > m[ht][i] + kSlack;
        if (__any_sync(kFull, above)) {
#pragma unroll
          for (int ht = 0; ht < HT; ++ht)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = fmaxf(s[ht][i], s[ht][2 + i]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
              top = fmaxf(top, m[ht][i]);
              const float was = m[ht][i] == top ? 1.0f : exp2_fast(m[ht][i] - top);
              m[ht][i] = top;
              l[ht][i] *= was;
              zsum[ht][i] *= was;
#pragma unroll
              for (int j = 0; j < S::MT; ++j) o[ht][j][i] *= was, o[ht][j][2 + i] *= was;
            }
        }
        // weights, as the second operand of the value products
        uint32_t wb[HT][S::PP][2];
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float base = m[ht][i & 1] == -INFINITY ? 0.0f : m[ht][i & 1];
            const float p = exp2_fast(s[ht][i] - base);
            l[ht][i & 1] += p;
            w[i] = p * vs[i >> 1];
            zsum[ht][i & 1] = __fmaf_rn(w[i], vz[i >> 1], zsum[ht][i & 1]);
          }
#pragma unroll
          for (int p = 0; p < S::PP; ++p)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t two = pack_bf16x2(w[2 * r], w[2 * r + 1]);
              wb[ht][p][r] = transpose8(two);
              w[2 * r] -= __uint_as_float(two << 16);
              w[2 * r + 1] -= __uint_as_float(two & 0xffff0000u);
            }
        }
        // weighted values: rows are head elements, k the positions
#pragma unroll
        for (int j = 0; j < S::NV; ++j) {
          uint32_t v[4][S::CV / 4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            load_run<S::CV>(slot + S::TILE / 2 + ((r * S::NV + j) * 32 + lane) * S::CV, v[r]);
#pragma unroll
          for (int i = 0; i < S::CV / 4; ++i) {
            uint32_t pr[2][2 * W::PAIRS];  // positions 2 t4, + 1; and those + 8
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t d[W::PAIRS];
              W::decode(__byte_perm(v[2 * k][i], v[2 * k + 1][i], 0x5410), d);
#pragma unroll
              for (int q = 0; q < W::PAIRS; ++q) pr[k][q] = d[q];
              W::decode(__byte_perm(v[2 * k][i], v[2 * k + 1][i], 0x7632), d);
#pragma unroll
              for (int q = 0; q < W::PAIRS; ++q) pr[k][W::PAIRS + q] = d[q];
            }
#pragma unroll
            for (int q = 0; q < W::PAIRS; ++q) {
              const int mt = (j * (S::CV / 4) + i) * W::PAIRS + q;
              const uint32_t fa[4] = {pr[0][2 * q], pr[0][2 * q + 1], pr[1][2 * q], pr[1][2 * q + 1]};
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) {
                if constexpr (S::kF32) {
                  // (sums of many tiles on the tensor cores would drift: 16 positions only)
                  float part[4] = {};
#pragma unroll
                  for (int p = S::PP - 1; p >= 0; --p) mma(part, fa, wb[ht][p][0], wb[ht][p][1]);
#pragma unroll
                  for (int x = 0; x < 4; ++x) o[ht][mt][x] += part[x];
                } else {
#pragma unroll
                  for (int p = 0; p < S::PP; ++p) mma(o[ht][mt], fa, wb[ht][p][0], wb[ht][p][1]);
                }
              }
            }
          }
        }
      }
    }
    copy_wait<0>();

    // --- the block's warps joined ------------------------------------------------------
#pragma unroll
    for (int ht = 0; ht < HT; ++ht)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[ht][i] += __shfl_xor_sync(kFull, l[ht][i], d);
          zsum[ht][i] += __shfl_xor_sync(kFull, zsum[ht][i], d);
        }
    __syncthreads();  // every warp is done with its ring
    float* const part = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int ht = 0; ht < HT; ++ht)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = 8 * ht + 2 * t4 + i;
        float* row = part + (warp * S::H + h) * S::OPAD;
#pragma unroll
        for (int j = 0; j < S::MT; ++j) {
          row[2 * j * 8 + g] = o[ht][j][i];
          row[(2 * j + 1) * 8 + g] = o[ht][j][2 + i];
        }
        if (g == 0) {
          ml[(warp * S::H + h) * 3] = m[ht][i];
          ml[(warp * S::H + h) * 3 + 1] = bad ? NAN : l[ht][i];
          ml[(warp * S::H + h) * 3 + 2] = zsum[ht][i];
        }
      }
    __syncthreads();
    const bool whole = pc.from == 0 && pc.to == pc.blocks;
    const int64_t at = ((int64_t)blockIdx.x * 2 + (pc.from == 0)) * S::H;
    for (int i = threadIdx.x; i < heads * c.d; i += kThreads) {
      const int h = i / c.d, e = i - h * c.d;
      float top = -INFINITY, sum = 0.0f, y = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[(w * S::H + h) * 3]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* r = ml + (w * S::H + h) * 3;
        const float f = r[0] == top ? 1.0f : exp2_fast(r[0] - top);
        sum = __fmaf_rn(f, r[1], sum);
        y = __fmaf_rn(f, part[(w * S::H + h) * S::OPAD + S::value_place(e)] - r[2], y);
      }
      if (whole) {
        st_elem<T>(a.y, ((int64_t)pc.b * a.q_heads + h0 + h) * c.d + e,
                   sum == 0.0f ? 0.0f : __fdiv_rn(y, sum));
        if (e == 0 && a.lse)
          a.lse[(int64_t)pc.b * a.q_heads + h0 + h] =
              sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
      } else {
        ws.o[(at + h) * c.d + e] = y;
        if (e == 0) ws.ml[at + h] = make_float2(top, sum);
      }
    }
    if (!whole && pc.from == 0) {
      // cut off by the run's end: the blocks behind this one hold the rest
      const int64_t rest = pc.blocks - pc.to;
      const int64_t last = end + rest - 1;  // its last block's place in the row
      int n = 1;
      while (total * (blockIdx.x + n + 1) / runs <= last) ++n;
      cut = make_int4(pc.b, pc.hg, n + 1, 0);
    }
    __syncthreads();
    // --- the next piece -----------------------------------------------------------------
    if (left > 0) {
      pc.from = 0;
      if (++pc.hg == hgs) {
        pc.hg = 0;
        do ++pc.b;
        while (blocks_of(pc.b) == 0);
      }
    }
  }
  if (threadIdx.x == 0) ws.cut[blockIdx.x] = cut;
}

template <typename T, int F, int DP, int HT>
qat_status go(const KvCacheView& c, const KvAttnArgs& a, const SplitWs& ws, int* grid,
              cudaStream_t s) {
  using S = Shape<T, F, DP, HT>;
  static_assert(S::SMEM <= 227 * 1024, "shared memory");
  const auto k = k_kv_split<T, F, DP, HT>;
  if (S::SMEM > 48 * 1024 &&
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) != cudaSuccess) {
    (void)cudaGetLastError();
    return QAT_ERR_CUDA;
  }
  const HeadTiles t = head_tiles(a.q_heads, c.heads, c.d, S::kF32);
  int per = 227 * 1024 / (S::SMEM + 2048);
  if (per > 3) per = 3;
  if (DP * HT > 128 || S::kF32) per = per < 2 ? per : 2;
  *grid = device_info().sms * per;
  if (*grid > kSplitBlocks) *grid = kSplitBlocks;
  if (launch_kernel(k, dim3(*grid), dim3(kThreads), S::SMEM, s, false, c, a, t.group, t.tiles, ws) !=
      cudaSuccess)
    return QAT_ERR_CUDA;
  count_launch(1);
  return QAT_OK;
}

}  // namespace

template <int F>
qat_status launch_kv_split(const KvCacheView& c, const KvAttnArgs& a, qat_dtype dt, const SplitWs& ws,
                           int* grid, cudaStream_t s) {
  const bool wide = head_tiles(a.q_heads, c.heads, c.d, dt == QAT_F32).tile == 16;
  if (dt == QAT_F32) {
    if (c.d <= 64) return go<F32, F, 64, 1>(c, a, ws, grid, s);
    if (c.d <= 128) return go<F32, F, 128, 1>(c, a, ws, grid, s);
    return go<F32, F, 256, 1>(c, a, ws, grid, s);
  }
  if (c.d <= 64) return wide ? go<BF16, F, 64, 2>(c, a, ws, grid, s) : go<BF16, F, 64, 1>(c, a, ws, grid, s);
  if (c.d <= 128)
    return wide ? go<BF16, F, 128, 2>(c, a, ws, grid, s) : go<BF16, F, 128, 1>(c, a, ws, grid, s);
  return go<BF16, F, 256, 1>(c, a, ws, grid, s);
}
template qat_status launch_kv_split<kFormat>(const KvCacheView&, const KvAttnArgs&, qat_dtype,
                                             const SplitWs&, int*, cudaStream_t);

}  // namespace qat
