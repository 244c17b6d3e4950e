// kernels_dense.cu -- the dense products of the gated feed-forward block on the
// fifth-generation tensor cores.
//
//   C[m, n] = sum over segments s of sum_k A_s(m, k) B_s(n, k)
//
// with the block's element-wise steps as epilogues.  An operand is read by
// bulk tensor copies either along k (K-major) or along its own rows
// (MN-major), so no transpose is ever written.
//
// A CTA stages up to 128 rows of A and of B, 64 deep, per step (32 KB, six or
// five steps in flight) in 128-byte swizzled rows.  One thread issues the copies, one the
// MMAs; the sums stay in tensor memory, in two buffers, so that eight warps
// finish one tile while the next is multiplied.  CG = 2: two CTAs share a
// 256 x 256 tile, each holding half of A and half of B, which halves the
// shared-memory traffic per product (a single CTA's 128 x 128 tile reads its
// operands faster than shared memory delivers them).  CG = 1: 128 x 128 tiles,
// and where those are few a cluster of up to eight CTAs splits k and adds its
// sums through distributed shared memory in rank order.
//
// With few rows the weights are all that is read, and bytes in flight count: A
// then holds 32 or 64 rows and more stages fit.  The MMA still reads 128 rows,
// the others from whatever follows in the stage; they end in sums of rows that do
// not exist.
//
// Measured at 4096 x 4096 x 14336 (tokens, dim, hidden; calls repeated for a second
// each, power capped): forward 946 us, keeping g and u 980 (1472 TFLOP/s); backward
// 2019 (1429), of which dw_down 326 (1478) and, by differences, dh 377 (1276, the
// epilogue reads and writes 12 bytes an element), dx 678 (1419, its tiles fill 3.4
// waves of 76 pairs) and the other two weight gradients 639 (1506).  cuBLAS, the same
// way, runs plain products of these shapes at 1738 and 1798.  fp32 at 2048 x 4096 x
// 14336: 247 TFLOP/s forward, 236 backward, six bf16 products each.  With one token
// the weights are read at 4.3 TB/s forward and for dx (128 rows of A in every stage:
// 3.8; tiles of 96 columns, for fuller waves, moved nothing there and cost 16% at 16 x
// 1024 x 4096).

#include "qat_dense.h"
#include "qat_layer.cuh"
#include "qat_tc.cuh"

#include <atomic>

namespace qat {

constexpr int kBK = 64;
constexpr int kRows = 128;                      // rows of A and of B per CTA and stage
constexpr uint32_t kOpBytes = kRows * kBK * 2;  // 16 KB
constexpr uint32_t kStageBytes = 2 * kOpBytes;
constexpr uint32_t kBarBytes = 256;
constexpr int kFinishWarps = 8;  // two for each quarter of the tile's rows
// The backward epilogue reads g and u: each finishing warp has 32 x 32 floats of
// both in shared memory, in the place of one stage.
constexpr uint32_t kSideBytes = 2 * 32 * 32 * 4;
// Outputs whose rows are off the vector grid leave by pieces of rows: each
// finishing warp turns 32 rows x 16 columns in shared memory.
constexpr uint32_t kTurnBytes = 32 * 17 * 4;
__host__ __device__ constexpr uint32_t stage_room(int epi) {
  return (epi == kDenseGatedBwd ? 5 : 6) * kStageBytes;
}
constexpr int kMaxStages = 9;
__host__ __device__ constexpr uint32_t dense_smem(int epi) {
  return stage_room(epi) + kBarBytes + 1024 +
         kFinishWarps * (epi == kDenseGatedBwd ? kSideBytes : kTurnBytes);
}
constexpr int kDenseThreads = 64 + 32 * kFinishWarps;
constexpr uint32_t kDrainPolls = 1u << 16;  // of a wait for what is in flight at the block's end

struct DenseArgs {
  CUtensorMap a[2], b[2];
  int64_t m, n;            // output size (gated: n = hidden)
  int mt, nt, problems;    // tiles of the output; outputs that share B
  int kt, segs;            // k steps of a segment; segments
  int split;               // CTAs of a cluster that share k (CG = 1)
  int bn;                  // columns of a pair's tile (store)
  int stages;
  uint32_t a_bytes, stage_bytes;  // of a stage; A may hold fewer rows than the MMA reads
  int act;
  void* c[2];              // outputs (gated: c[0] = h), rows of n
  float* gp;
  float* up;
  void* q[2];              // outputs kept as operands (bf16 parts): gated h
  int64_t q_pitch, q_part;  // (nullable), gated backward dg and du
  int32_t* flags;
  uint32_t limit;
};

// N (8 or 16) consecutive outputs of one row: full vectors where the row allows
template <typename T, int N>
__device__ __forceinline__ void st_row(void* p, int64_t at, int left, uint32_t align,
                                       const float (&v)[N]) {
  if (left >= N && align >= 16) {
    constexpr int W = N * T::BYTES / 4;  // words
    uint32_t w[W];
    if (T::BYTES == 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    char* q = static_cast<char*>(p) + at * T::BYTES;
    if (align >= 32) {
#pragma unroll
      for (int i = 0; i < W; i += 8) {
        V32 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.w[j] = w[i + j];
        st_v32(q + i * 4, o);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4)
        *reinterpret_cast<uint4*>(q + i * 4) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) st_elem<T>(p, at + i, v[i]);
  }
}
// 16 consecutive bf16 outputs as an operand of a later product
__device__ __forceinline__ void st_parts16(const DenseArgs& p, int which, int64_t row, int64_t c,
                                           int left, const float (&v)[16]) {
  st_row<BF16>(p.q[which], row * p.q_pitch + c, left, 16, v);
}
// the largest of 32, 16 or 1 that divides the address and the row pitch
__device__ __forceinline__ uint32_t row_align(const void* p, int64_t pitch_bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p) | (uint64_t)pitch_bytes;
  return a % 32 == 0 ? 32 : a % 16 == 0 ? 16 : 1;
}

// One row's 16 columns of a bf16 layer from column c on
// (gated: v = g, u beside it; backward: v = dh, g and w = u as kept)
template <int EPI>
__device__ __forceinline__ void finish16(const DenseArgs& p, int prob, int64_t row, int64_t c,
                                         const float (&v)[16], const float (&u)[16],
                                         const float (&g)[16], const float (&w)[16]) {
  const int64_t at = row * p.n + c;
  const int left = (int)min((int64_t)16, p.n - c);
  if (EPI == kDenseStore) {
    st_row<BF16>(p.c[prob], at, left, row_align(p.c[prob], p.n * 2), v);
  } else if (EPI == kDenseGated) {
    float h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = act_value<true>(p.act, v[i]) * u[i];
    st_row<BF16>(p.c[0], at, left, row_align(p.c[0], p.n * 2), h);
    if (p.q[0]) st_parts16(p, 0, row, c, left, h);
    if (p.gp) {
      st_row<F32>(p.gp, at, left, row_align(p.gp, p.n * 4), v);
      st_row<F32>(p.up, at, left, row_align(p.up, p.n * 4), u);
    }
  } else {
    float dg[16], du[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a, da;
      act_grad<true>(p.act, g[i], a, da);
      dg[i] = v[i] * w[i] * da;
      du[i] = v[i] * a;
    }
    st_parts16(p, 0, row, c, left, dg);
    st_parts16(p, 1, row, c, left, du);
  }
}
__device__ __forceinline__ void st_parts8(const DenseArgs& p, int which, int64_t row, int64_t c,
                                          int left, const float (&v)[8]) {
  const int64_t at = row * p.q_pitch + c;
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = take_bf16(r[i]);
    // pitch, part and c are multiples of 8; the padding of a row may be written
    __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p.q[which]) + at + k * p.q_part;
    if (left > 0)
      *reinterpret_cast<uint4*>(q) = make_uint4(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]),
                                                pack_bf16x2(h[4], h[5]), pack_bf16x2(h[6], h[7]));
  }
}
// The same for eight columns of a gated fp32 layer, whose sums leave fewer registers.
template <int EPI>
__device__ __forceinline__ void finish8(const DenseArgs& p, int64_t row, int64_t c,
                                        const float (&v)[8], const float (&u)[8],
                                        const float (&g)[8], const float (&w)[8]) {
  const int64_t at = row * p.n + c;
  const int left = (int)min((int64_t)8, p.n - c);
  const auto put = [&](void* q, const float (&o)[8]) {
    st_row<F32>(q, at, left, row_align(q, p.n * 4), o);
  };
  if (EPI == kDenseGated) {
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = act_value<false>(p.act, v[i]) * u[i];
    put(p.c[0], h);
    st_parts8(p, 0, row, c, left, h);
    if (p.gp) {
      put(p.gp, v);
      put(p.up, u);
    }
  } else {
    float dg[8], du[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, da;
      act_grad<false>(p.act, g[i], a, da);
      dg[i] = v[i] * w[i] * da;
      du[i] = v[i] * a;
    }
    st_parts8(p, 0, row, c, left, dg);
    st_parts8(p, 1, row, c, left, du);
  }
}
// The same for four columns.
template <typename T>
__device__ __forceinline__ void st_row4(void* p, int64_t at, int left, bool vec, const float (&v)[4]) {
  if (vec && left >= 4) {
    if constexpr (T::BYTES == 4)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + at) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) st_elem<T>(p, at + i, v[i]);
}
template <typename T>
__device__ __forceinline__ void st_parts4(const DenseArgs& p, int which, int64_t row, int64_t c,
                                          int left, const float (&v)[4]) {
  const int64_t at = row * p.q_pitch + c;
  if constexpr (T::BYTES == 2) {
    st_row4<BF16>(p.q[which], at, left, true, v);
  } else {
    float r[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = take_bf16(r[i]);
      st_row4<BF16>(p.q[which], at + k * p.q_part, left, true, h);
    }
  }
}
template <typename T, int EPI>
__device__ __forceinline__ void finish4(const DenseArgs& p, int prob, int64_t row, int64_t c,
                                        const float (&v)[4], const float (&u)[4]) {
  const int64_t at = row * p.n + c;
  const int left = (int)min((int64_t)4, p.n - c);
  const bool whole = p.n % 4 == 0;
  const auto vec = [&](const void* q, int bytes) {
    return whole && reinterpret_cast<uint64_t>(q) % (4 * bytes) == 0;
  };
  if (EPI == kDenseStore) {
    st_row4<T>(p.c[prob], at, left, vec(p.c[prob], T::BYTES), v);
  } else if (EPI == kDenseGated) {
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = act_value<T::BYTES == 2>(p.act, v[i]) * u[i];
    st_row4<T>(p.c[0], at, left, vec(p.c[0], T::BYTES), h);
    if (p.q[0]) st_parts4<T>(p, 0, row, c, left, h);
    if (p.gp) {
      st_row4<F32>(p.gp, at, left, vec(p.gp, 4), v);
      st_row4<F32>(p.up, at, left, vec(p.up, 4), u);
    }
  } else {
    float g[4], w[4], dg[4], du[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[i] = i < left ? p.gp[at + i] : 0.0f;
      w[i] = i < left ? p.up[at + i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, da;
      act_grad<T::BYTES == 2>(p.act, g[i], a, da);
      dg[i] = v[i] * w[i] * da;
      du[i] = v[i] * a;
    }
    st_parts4<T>(p, 0, row, c, left, dg);
    st_parts4<T>(p, 1, row, c, left, du);
  }
}
// floats from one row of a tile's joined sums to the next: 16-byte accesses by
// neighbouring rows then fall into different banks
constexpr int kJoinPitch = kRows + 4;
__device__ __forceinline__ void put4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
}

struct Tile {
  int prob;
  int64_t m0, n0;  // first output row and column (of the CTA pair)
};
// Tiles in groups of 16 row tiles, columns outermost inside a group: the tiles
// at work together then reread few operand rows, from L2.
template <int CG, int EPI>
__device__ __forceinline__ Tile tile_at(const DenseArgs& p, int64_t t) {
  constexpr int BM = kRows * CG;
  const int BN = EPI == kDenseGated ? kRows * CG / 2 : CG == 2 && EPI == kDenseStore ? p.bn : kRows * CG;
  const int64_t per = (int64_t)p.mt * p.nt;
  Tile r;
  r.prob = (int)(t / per);
  t -= r.prob * per;
  constexpr int G = 16;
  const int64_t g = t / ((int64_t)G * p.nt), in = t - g * G * p.nt;
  const int rows = (int)min((int64_t)G, p.mt - g * G);
  r.m0 = (g * G + in % rows) * BM;
  r.n0 = (in / rows) * BN;
  return r;
}

// fp32 operands are held as three bf16 parts (high, middle, low: all 24 bits);
// the six products that reach 2^-24 of the whole, smallest first.  The tensor
// cores round their binary32 sums toward zero, which would cost a few digits
// over a long k, so fp32 products are summed there over 256 k only and then in
// registers.
__device__ __constant__ const uint8_t kPairA[6] = {2, 0, 1, 1, 0, 0};
__device__ __constant__ const uint8_t kPairB[6] = {0, 2, 1, 0, 1, 0};
constexpr int kChunk = 4;  // k steps of such a sum

// The k work of a segment in units: one step, or for fp32 one chunk of up to
// four steps for each of the six pairs.
template <typename T>
struct Units {
  static constexpr bool kParts = T::BYTES == 4;
  __host__ __device__ static int per_segment(int kt) { return kParts ? (kt + kChunk - 1) / kChunk : kt; }
  __device__ static int steps(int kt, int in_seg) {
    return kParts ? 6 * min(kChunk, kt - in_seg * kChunk) : 1;
  }
};

template <typename T, int CG, int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kDenseThreads, 1) k_dense(const __grid_constant__ DenseArgs p) {
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tc::smem(raw) + 1023) & ~1023u;
  const uint32_t bars = base + stage_room(EPI);
  const int stages = CG == 2 ? stage_room(EPI) / kStageBytes : p.stages;
  const uint32_t a_bytes = CG == 2 ? kOpBytes : p.a_bytes;
  const uint32_t stage_bytes = CG == 2 ? kStageBytes : p.stage_bytes;
  // full[stages], empty[stages], acc_full[2], acc_empty[2], drain
  const auto full = [&](int s) { return bars + 8 * s; };
  const auto empty = [&](int s) { return bars + 8 * (kMaxStages + s); };
  const auto acc_full = [&](int b) { return bars + 8 * (2 * kMaxStages + b); };
  const auto acc_empty = [&](int b) { return bars + 8 * (2 * kMaxStages + 2 + b); };
  const uint32_t drain = bars + 8 * (2 * kMaxStages + 4);
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();  // CG = 2: half of the tile; else k slice
  const bool leader = CG == 1 || rank == 0;
  constexpr int kAccCols = kRows * CG;  // TMEM columns of a buffer
  constexpr int kTmemCols = 2 * kAccCols;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      tc::bar_init(full(s), 1);
      tc::bar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::bar_init(acc_full(b), 1);
      tc::bar_init(acc_empty(b), kFinishWarps * CG);
    }
    tc::bar_init(drain, 1);
    tc::bar_init_fence();
    abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      tc::prefetch_map(&p.a[i]);
      tc::prefetch_map(&p.b[i]);
    }
  }
  if (warp == 1) tc::tmem_alloc<CG>(tc::smem(&tmem_slot), kTmemCols);
  tc::fence_before();
  __syncthreads();
  if (CG == 2 || p.split > 1) tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_trigger();  // the call's next kernel may take each SM as this one leaves it
  pdl_wait();     // and this one's set-up overlapped the previous kernel's end

  // columns of the tile's sums, and the bytes of a stage of B
  const int tile_cols = CG == 2 && EPI == kDenseStore ? p.bn : kAccCols;
  const uint32_t b_bytes = CG == 2 && !B_MN ? (uint32_t)tile_cols / 2 * kBK * 2 : kOpBytes;
  using U = Units<T>;
  const int per_seg = U::per_segment(p.kt), units = p.segs * per_seg;
  // this CTA's share of them
  const int u0 = CG == 1 ? (int)((int64_t)units * rank / p.split) : 0;
  const int u1 = CG == 1 ? (int)((int64_t)units * (rank + 1) / p.split) : units;
  const int64_t tiles = (int64_t)p.mt * p.nt * p.problems;
  const int per_cluster = CG == 2 ? 2 : p.split;
  const int64_t first = blockIdx.x / per_cluster, stride = gridDim.x / per_cluster;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 1;  // a fresh barrier passes the wait for "already empty"
      int64_t issued = 0;
      for (int64_t t = first; ok && t < tiles; t += stride) {
        const Tile w = tile_at<CG, EPI>(p, t);
        const int am = (int)(w.m0 + (CG == 2 ? (int64_t)rank * kRows : 0));
        const int bn = (int)(w.n0 + (CG == 2 && EPI != kDenseGated ? (int64_t)rank * (tile_cols / 2) : 0));
        for (int un = u0; ok && un < u1; ++un) {
          const int seg = un / per_seg, in_seg = un - seg * per_seg;
          const int steps = U::steps(p.kt, in_seg);
          for (int st = 0; st < steps; ++st) {
            ok = tc::bar_wait(empty(stage), phase, &abort_flag, p.limit);
            if (!ok) break;
            const int nk = steps / 6;
            const int pr = U::kParts ? st / nk : 0;
            const int k0 = (U::kParts ? in_seg * kChunk + st - pr * nk : in_seg) * kBK;
            const int pa = U::kParts ? kPairA[pr] : 0, pb = U::kParts ? kPairB[pr] : 0;
            const uint32_t sa = base + stage * stage_bytes, sb = sa + a_bytes;
            uint32_t bar = full(stage);
            if (leader) tc::bar_expect(bar, (a_bytes + b_bytes) * CG);
            if (CG == 2) bar = tc::map_rank(bar, 0);
            const CUtensorMap* ma = &p.a[p.problems > 1 ? w.prob : seg];
            if (A_MN) {
              tc::load_box<CG == 2>(ma, sa, bar, am, k0, pa);
              tc::load_box<CG == 2>(ma, sa + kOpBytes / 2, bar, am + 64, k0, pa);
            } else {
              tc::load_box<CG == 2>(ma, sa, bar, k0, am, pa);
            }
            if (EPI == kDenseGated) {
              // gate rows then up rows; a pair's CTAs hold one each
              if (CG == 2) {
                tc::load_box<true>(&p.b[rank], sb, bar, k0, bn, pb);
              } else {
                tc::load_box<false>(&p.b[0], sb, bar, k0, bn, pb);
                tc::load_box<false>(&p.b[1], sb + kOpBytes / 2, bar, k0, bn, pb);
              }
            } else if (B_MN) {
              tc::load_box<CG == 2>(&p.b[seg], sb, bar, bn, k0, pb);
              tc::load_box<CG == 2>(&p.b[seg], sb + kOpBytes / 2, bar, bn + 64, k0, pb);
            } else {
              tc::load_box<CG == 2>(&p.b[seg], sb, bar, k0, bn, pb);
            }
            ++issued;
            if (++stage == stages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
      // The last copies land before the block ends, also where other warps gave up
      // on them (a pair's are counted in its leader, see the block's end).
      volatile int none = 0;
      if (leader)
        for (int64_t i = issued > stages ? issued - stages : 0; i < issued; ++i)
          if (!tc::bar_wait(full((int)(i % stages)), (uint32_t)(i / stages) & 1, &none, kDrainPolls))
            abort_flag = 1;
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      const uint32_t idesc = tc::idesc_bf16(kRows * CG, tile_cols, A_MN, B_MN);
      int stage = 0;
      uint32_t phase = 0;
      int64_t run = 0;  // sums begun: the accumulators alternate
      for (int64_t t = first; ok && t < tiles; t += stride) {
        for (int un = u0; ok && un < u1; ++un) {
          const uint32_t acc = tmem + (uint32_t)(run & 1) * kAccCols;
          const bool begin = U::kParts || un == u0, end = U::kParts || un + 1 == u1;
          if (begin) {
            ok = tc::bar_wait(acc_empty((int)(run & 1)), (uint32_t)(run >> 1 & 1) ^ 1, &abort_flag,
                              p.limit);
            tc::fence_after();
          }
          const int steps = U::steps(p.kt, U::kParts ? un % per_seg : 0);
          for (int st = 0; ok && st < steps; ++st) {
            ok = tc::bar_wait(full(stage), phase, &abort_flag, p.limit);
            if (!ok) break;
            tc::fence_after();
            const uint32_t sa = base + stage * stage_bytes, sb = sa + a_bytes;
            const uint64_t da = tc::desc_sw128(sa, A_MN ? kOpBytes / 2 : 16);
            const uint64_t db = tc::desc_sw128(sb, B_MN ? kOpBytes / 2 : 16);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              tc::mma_bf16<CG>(acc, da + (A_MN ? 2048 : 32) / 16 * k,
                               db + (B_MN ? 2048 : 32) / 16 * k, idesc, !begin || st > 0 || k > 0);
            tc::mma_commit<CG>(empty(stage));
            if (++stage == stages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (ok && end) {
            tc::mma_commit<CG>(acc_full((int)(run & 1)));
            ++run;
          }
        }
      }
      // The last MMAs end before tensor memory is freed, also where the finishing
      // warps gave up on them.
      volatile int none = 0;
      tc::mma_commit<CG>(drain);
      if (!tc::bar_wait(drain, 0, &none, kDrainPolls)) abort_flag = 1;
    }
  } else {
    const int quad = warp & 3;
    constexpr int kOut = EPI == kDenseGated ? kAccCols / 2 : kAccCols;
    constexpr int kHalf = kOut / 2;
    const int c_first = (warp - 2) / 4 * kHalf;  // this warp's columns
    const int c_count = EPI == kDenseGated ? kHalf : min(kHalf, tile_cols - c_first);
    constexpr float kBad = __builtin_nanf("");
    int64_t run = 0;
    // waits for the next sum; the address of this warp's lanes of it
    const auto next_sum = [&]() {
      const int buf = (int)(run & 1);
      if (ok) ok = tc::bar_wait(acc_full(buf), (uint32_t)(run >> 1 & 1), &abort_flag, p.limit);
      ok = __all_sync(~0u, ok);
      tc::fence_after();
      return tmem + buf * kAccCols + ((uint32_t)(quad * 32) << 16) + c_first;
    };
    // the sum is read: MMAs may use its buffer again
    const auto sum_read = [&]() {
      tc::fence_before();
      if (lane == 0) tc::bar_arrive_cluster(tc::map_rank(acc_empty((int)(run & 1)), CG == 2 ? 0 : rank));
      ++run;
    };
    // Backward: g and u of 32 rows x 32 columns come in by rows of 128 bytes,
    // asynchronously, and are taken back a row a thread; the 16-byte pieces of a
    // row are permuted by it so that both ways are free of bank conflicts.
    // Rows off the vector grid come in an element a lane.
    const bool pieces = p.n % 4 == 0 &&
                        ((reinterpret_cast<uint64_t>(p.gp) | reinterpret_cast<uint64_t>(p.up)) & 15) == 0;
    const uint32_t side_at = bars + kBarBytes + (warp - 2) * kSideBytes;
    const auto side_load = [&](int64_t row0, int64_t c) {
      if (!pieces) {
        const int64_t from = row0 * p.n + c + lane;
        const int rows = c + lane < p.n ? (int)max((int64_t)0, min((int64_t)32, p.m - row0)) : 0;
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
          const uint32_t to = side_at + r * 128 + (((lane / 4) ^ (r & 7)) * 16) + lane % 4 * 4;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p.gp + from + r * p.n) : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4096), "l"(p.up + from + r * p.n)
                       : "memory");
        }
      }
#pragma unroll
      for (int i = 0; pieces && i < 8; ++i) {
        const int r = i * 4 + lane / 8, k = lane % 8;
        if (row0 + r < p.m && c + k * 4 < p.n) {
          const int64_t at = (row0 + r) * p.n + c + k * 4;
          const uint32_t to = side_at + r * 128 + ((k ^ (r & 7)) * 16);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p.gp + at) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 4096), "l"(p.up + at)
                       : "memory");
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto side_wait = [&]() {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
    };
    // g and u of four columns of this thread's row
    const auto side_get = [&](int k, float4& g, float4& u) {
      const uint8_t* at = raw + (side_at - tc::smem(raw)) + lane * 128 + ((k ^ (lane & 7)) * 16);
      g = *reinterpret_cast<const float4*>(at);
      u = *reinterpret_cast<const float4*>(at + 4096);
    };
    // taken: the next 32 columns may come in
    const auto side_next = [&](int64_t row, int64_t c, bool more) {
      __syncwarp();
      if (more) side_load(row - lane, c);
    };
    // g and u of this thread's row, 16 columns from c on (c = c32 within 32)
    const auto kept = [&](float (&g)[16], float (&u)[16], int64_t row, int64_t c, int c32, bool more) {
      if constexpr (EPI == kDenseGatedBwd) {
        if (c32 == 0) side_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float4 a, b;
          side_get(c32 / 4 + k, a, b);
          g[4 * k] = a.x, g[4 * k + 1] = a.y, g[4 * k + 2] = a.z, g[4 * k + 3] = a.w;
          u[4 * k] = b.x, u[4 * k + 1] = b.y, u[4 * k + 2] = b.z, u[4 * k + 3] = b.w;
        }
        if (c32) side_next(row, c + 16, more);
      }
    };
    // N columns of a row a thread, stored by N columns of 32 / N rows: a store of
    // one element of 32 rows would take 32 sectors (dw_gate and dw_up of 300 tokens,
    // 510 x 1363, fp32: 49 us in place of 57; the gated product of bf16 layers of
    // 4000 x 1001 x 4003 makes their forward 135 us in place of 243)
    float* turn = reinterpret_cast<float*>(raw + (bars + kBarBytes - tc::smem(raw)) + (warp - 2) * kTurnBytes);
    const auto st_turned = [&](auto type, void* to, int64_t row0, int64_t c, const auto& v) {
      constexpr int N = sizeof(v) / 4, kPitch = N + 1;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) turn[lane * kPitch + i] = v[i];
      __syncwarp();
      const int64_t at = c + lane % N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = i * (32 / N) + lane / N;
        if (row0 + r < p.m && at < p.n)
          st_elem<decltype(type)>(to, (row0 + r) * p.n + at, turn[r * kPitch + lane % N]);
      }
    };
    const auto off_grid = [&](const void* q, int bytes) { return q && row_align(q, p.n * bytes) < 16; };
    // the same of a gated layer's h, g and u
    const auto gated_turned = [&](int64_t row, int64_t c, const auto& g, const auto& u) {
      constexpr int N = sizeof(g) / 4;
      float h[N];
#pragma unroll
      for (int i = 0; i < N; ++i) h[i] = act_value<T::BYTES == 2>(p.act, g[i]) * u[i];
      st_turned(T{}, p.c[0], row - lane, c, h);
      if (p.q[0] && row < p.m) {
        const int left = (int)min((int64_t)N, p.n - c);
        if constexpr (N == 8)
          st_parts8(p, 0, row, c, left, h);
        else
          st_parts16(p, 0, row, c, left, h);
      }
      if (p.gp) {
        st_turned(F32{}, p.gp, row - lane, c, g);
        st_turned(F32{}, p.up, row - lane, c, u);
      }
    };
    for (int64_t t = first; t < tiles; t += stride) {
      const Tile w = tile_at<CG, EPI>(p, t);
      const bool turned = EPI == kDenseStore ? off_grid(p.c[w.prob], T::BYTES)
                          : EPI == kDenseGated ? off_grid(p.c[0], T::BYTES) || off_grid(p.gp, 4) || off_grid(p.up, 4)
                                               : false;
      const int64_t row = w.m0 + (CG == 2 ? (int64_t)rank * kRows : 0) + quad * 32 + lane;
      const int64_t col = w.n0 + c_first;
      if (EPI == kDenseGatedBwd && (CG == 2 || p.split == 1)) side_load(row - lane, col);
      // where k is split: this row of the CTA's sums, in the stage buffers (every
      // stage has been multiplied by then, unless a wait ran out)
      float* sums = reinterpret_cast<float*>(raw + (base - tc::smem(raw))) +
                    (quad * 32 + lane) * kJoinPitch + c_first;
      if constexpr (U::kParts) {
        constexpr int kU = EPI == kDenseGated ? kHalf : 1;
        float sv[kHalf], su[kU];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) sv[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < kU; ++i) su[i] = 0.0f;
        uint32_t acc = 0;
        for (int un = u0; un < u1; ++un) {
          acc = next_sum();
#pragma unroll
          for (int c = 0; c < kHalf; c += 32) {
            uint32_t r[32];
            tc::tmem_ld32(acc + c, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) sv[c + i] += ok ? __uint_as_float(r[i]) : kBad;
            if constexpr (EPI == kDenseGated) {
              tc::tmem_ld32(acc + kOut + c, r);
              tc::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) su[c + i] += ok ? __uint_as_float(r[i]) : kBad;
            }
          }
          if (un + 1 < u1) sum_read();
        }
        if (CG == 1 && p.split > 1) {
#pragma unroll
          for (int c = 0; c < kHalf; c += 4) {
            put4(sums + c, sv[c], sv[c + 1], sv[c + 2], sv[c + 3]);
            if constexpr (EPI == kDenseGated)
              put4(sums + kOut + c, su[c], su[c + 1], su[c + 2], su[c + 3]);
          }
          break;  // joined below
        }
        // the whole sums go back to their place in tensor memory, from where a
        // short loop takes them: the code for all columns at once, unrolled for
        // the registers, would not fit the instruction cache
#pragma unroll
        for (int c = 0; c < kHalf; c += 32) {
          tc::tmem_st32(acc + c, sv + c);
          if constexpr (EPI == kDenseGated) tc::tmem_st32(acc + kOut + c, su + c);
        }
        tc::tmem_st_wait();
        if constexpr (EPI == kDenseStore) {
#pragma unroll 1
          for (int c = 0; c < c_count; c += 16) {
            uint32_t r[16];
            tc::tmem_ld16(acc + c, r);
            tc::tmem_ld_wait();
            if (c + 16 >= c_count) sum_read();
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
            const int64_t at = col + c;
            if (turned)
              st_turned(F32{}, p.c[w.prob], row - lane, at, v);
            else if (row < p.m && at < p.n)
              st_row<F32>(p.c[w.prob], row * p.n + at, (int)min((int64_t)16, p.n - at),
                          row_align(p.c[w.prob], p.n * 4), v);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < c_count; c += 8) {
            uint32_t r[8], q[8];
            tc::tmem_ld8(acc + c, r);
            if (EPI == kDenseGated) tc::tmem_ld8(acc + kOut + c, q);
            tc::tmem_ld_wait();
            if (c + 8 >= c_count) sum_read();
            float v[8], u[8], g[8], k[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v[i] = __uint_as_float(r[i]);
              u[i] = EPI == kDenseGated ? __uint_as_float(q[i]) : 0.0f;
            }
            const int64_t at = col + c;
            if constexpr (EPI == kDenseGatedBwd) {
              if (c % 32 == 0) side_wait();
#pragma unroll
              for (int i = 0; i < 8; i += 4) {
                float4 a, b;
                side_get((c % 32 + i) / 4, a, b);
                g[i] = a.x, g[i + 1] = a.y, g[i + 2] = a.z, g[i + 3] = a.w;
                k[i] = b.x, k[i + 1] = b.y, k[i + 2] = b.z, k[i + 3] = b.w;
              }
              if (c % 32 == 24) side_next(row, at + 8, c + 8 < c_count);
            }
            if (EPI == kDenseGated && turned)
              gated_turned(row, at, v, u);
            else if (row < p.m && at < p.n)
              finish8<EPI>(p, row, at, v, u, g, k);
          }
        }
      } else {
        const uint32_t acc = next_sum();
#pragma unroll 1
        for (int c = 0; c < c_count; c += 16) {
          uint32_t r[16], q[16];
          tc::tmem_ld16(acc + c, r);
          if (EPI == kDenseGated) tc::tmem_ld16(acc + kOut + c, q);
          tc::tmem_ld_wait();
          if (c + 16 >= c_count) sum_read();
          float v[16], u[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = ok ? __uint_as_float(r[i]) : kBad;
            u[i] = EPI != kDenseGated ? 0.0f : ok ? __uint_as_float(q[i]) : kBad;
          }
          if (CG == 1 && p.split > 1) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              put4(sums + c + i, v[i], v[i + 1], v[i + 2], v[i + 3]);
              if (EPI == kDenseGated) put4(sums + kOut + c + i, u[i], u[i + 1], u[i + 2], u[i + 3]);
            }
          } else {
            float g[16], k[16];
            kept(g, k, row, col + c, c % 32, c + 16 < c_count);
            if (EPI == kDenseStore && turned)
              st_turned(T{}, p.c[w.prob], row - lane, col + c, v);
            else if (EPI == kDenseGated && turned)
              gated_turned(row, col + c, v, u);
            else if (row < p.m && col + c < p.n)
              finish16<EPI>(p, w.prob, row, col + c, v, u, g, k);
          }
        }
        if (CG == 1 && p.split > 1) break;  // joined below
      }
    }
  }
  __syncthreads();
  if (CG == 1 && p.split > 1) {
    // A finishing warp that gave up left its NaN in the stage buffers while copies
    // could still land there: once more, now that none is in flight.
    if (!ok && warp >= 2) {
      float* row = reinterpret_cast<float*>(raw + (base - tc::smem(raw))) +
                   ((warp & 3) * 32 + lane) * kJoinPitch;
      constexpr float kBad = __builtin_nanf("");
      for (int c = 0; c < kAccCols; c += 4) put4(row + c, kBad, kBad, kBad, kBad);
    }
    tc::cluster_sync();
    // the cluster's CTAs finish the tile together, four columns of a row a
    // thread, adding the k slices in rank order with every slice's load in flight
    constexpr int kOut = EPI == kDenseGated ? kAccCols / 2 : kAccCols;
    const Tile w = tile_at<CG, EPI>(p, first);
    const int rows = (int)min((int64_t)kRows, p.m - w.m0);
    for (int i = (int)rank * kDenseThreads + threadIdx.x; i < rows * (kOut / 4);
         i += kDenseThreads * p.split) {
      const int r = i / (kOut / 4), c = i % (kOut / 4) * 4;
      if (w.n0 + c >= p.n) continue;
      float4 v = make_float4(0, 0, 0, 0), u = v;
      const uint32_t at = base + (r * kJoinPitch + c) * 4;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (q >= p.split) break;
        const uint32_t peer = tc::map_rank(at, q);
        add4(v, tc::ld_cluster4(peer));
        if (EPI == kDenseGated) add4(u, tc::ld_cluster4(peer + kOut * 4));
      }
      const float vs[4] = {v.x, v.y, v.z, v.w}, us[4] = {u.x, u.y, u.z, u.w};
      finish4<T, EPI>(p, w.prob, w.m0 + r, w.n0 + c, vs, us);
    }
  }
  if (CG == 2) {
    volatile int none = 0;
    if (leader && threadIdx.x == 0 && abort_flag)
      tc::st_cluster(tc::map_rank(tc::smem(const_cast<int*>(&abort_flag)), 1), 1);
    // the MMAs' end has been signalled here too
    if (!leader && threadIdx.x == 0) tc::bar_wait(drain, 0, &none, kDrainPolls);
    __syncwarp();
  }
  if (CG == 2 || p.split > 1) tc::cluster_sync();  // peers have read this CTA's memory
  // The leader has seen the pair's copies land unless one of the two gave up; then
  // those it did not wait for have a millisecond, which is ample, before the CTA they
  // write to and the one that counts them may end.
  if (CG == 2 && threadIdx.x == 0 && abort_flag)
    for (int i = 0; i < 1024; ++i) __nanosleep(1000);
  if (threadIdx.x == 0 && abort_flag && p.flags) atomicOr(p.flags, QAT_FLAG_DEVICE_TIMEOUT);
  if (warp == 1) tc::tmem_free<CG>(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);
static EncodeTiled encoder() {
  static std::atomic<EncodeTiled> fn{nullptr};
  EncodeTiled f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* q = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault,
                                         &st) != cudaSuccess ||
        st != cudaDriverEntryPointSuccess)
      return nullptr;
    f = reinterpret_cast<EncodeTiled>(q);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// Operand of `rows` m or n and `depth` k: boxes of `box` rows x 64 k (K-major)
// or 64 rows x 64 k (MN-major).
static bool encode(CUtensorMap* map, const DenseOp& o, int64_t rows, int64_t depth, int parts,
                   int box) {
  EncodeTiled f = encoder();
  if (!f) return false;
  const cuuint64_t inner = o.mn_major ? rows : depth, outer = o.mn_major ? depth : rows;
  const cuuint64_t dims[3] = {inner, outer, (cuuint64_t)parts};
  const cuuint64_t pitch = (cuuint64_t)o.pitch * 2;
  const cuuint64_t strides[2] = {pitch, parts > 1 ? (cuuint64_t)o.part * 2 : pitch * outer};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)(o.mn_major ? 64 : box), 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides, boxes,
           unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int CG, int EPI, bool A_MN, bool B_MN>
static qat_status launch(DenseArgs& p, bool pdl, cudaStream_t s) {
  const auto kernel = k_dense<T, CG, EPI, A_MN, B_MN>;
  constexpr uint32_t smem = dense_smem(EPI);
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return QAT_ERR_CUDA;
  }
  const int sms = device_info().sms;
  const int64_t tiles = (int64_t)p.mt * p.nt * p.problems;
  const int cluster = CG == 2 ? 2 : p.split;
  int64_t most = sms / cluster;
  const int64_t clusters = CG == 1 && p.split > 1 ? tiles : tiles < most ? tiles : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * cluster));
  cfg.blockDim = dim3(kDenseThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return QAT_ERR_CUDA;
  }
  count_launch(1);
  return QAT_OK;
}

template <typename T, int CG>
static qat_status launch_majors(DenseArgs& p, const Dense& d, cudaStream_t s) {
  const bool a_mn = d.a[0].mn_major, b_mn = d.b[0].mn_major;
  if (d.epi == kDenseGated) return launch<T, CG, kDenseGated, false, false>(p, d.pdl, s);
  if (d.epi == kDenseGatedBwd) return launch<T, CG, kDenseGatedBwd, false, true>(p, d.pdl, s);
  if (a_mn) return launch<T, CG, kDenseStore, true, true>(p, d.pdl, s);
  if (b_mn) return launch<T, CG, kDenseStore, false, true>(p, d.pdl, s);
  return launch<T, CG, kDenseStore, false, false>(p, d.pdl, s);
}

// Clusters of c CTAs that run at the same time (one CTA a SM; a cluster stays
// inside a group of SMs, so eight times fifteen is all of 152).
static int resident_clusters(int c) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> cache[kMaxDev][9];  // 0 = unknown
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
  int n = cache[dev][c].load(std::memory_order_relaxed);
  if (n > 0) return n;
  const auto kernel = k_dense<BF16, 1, kDenseStore, false, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c);
  cfg.blockDim = dim3(kDenseThreads);
  constexpr uint32_t smem = dense_smem(kDenseStore);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  cache[dev][c].store(n, std::memory_order_relaxed);
  return n;
}

qat_status launch_dense(const Dense& d, cudaStream_t s) {
  if (d.m == 0 || d.n == 0) return QAT_OK;
  DenseArgs p = {};
  const bool gated = d.epi == kDenseGated, f32 = d.dtype == QAT_F32;
  const int sms = device_info().sms, parts = f32 ? 3 : 1;
  const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  p.m = d.m;
  p.n = d.n;
  p.problems = d.problems;
  p.segs = d.segs;
  p.kt = (int)up(d.k, kBK);
  // Pairs of CTAs, single CTAs, or clusters that split k, whichever should end
  // first: waves of tiles times k steps, and the end of a tile.  Measured cycles
  // of a step: 620 of a pair's (256 x 256 x 64), 680 of a single CTA's (128 x 128
  // x 64); a pair's tile ends in about 6000, a split one is joined in as many, a
  // single one ends in 2500.  With 128 rows or fewer half a pair would idle.  At
  // 1001 x 4096, k = 14336, pairs take 84 us and single CTAs 158; at 128 x 4096 it
  // is 150 and 31 (split).
  const auto tiles_of = [&](int side) {
    return up(d.m, side) * up(d.n, gated ? side / 2 : side) * d.problems;
  };
  const int64_t units = (int64_t)p.segs * (f32 ? Units<F32>::per_segment(p.kt) : p.kt);
  const int64_t steps = f32 ? (int64_t)p.segs * p.kt * 6 : units;
  // A pair's tile has 256 columns, or 224 where that fills its last wave (560
  // cycles a step): 4096 x 4096 is 256 tiles of 256 on 76 pairs, four waves, and
  // 304 of 224, four waves too.
  p.bn = 256;
  int64_t pair_cost = up(tiles_of(256), sms / 2) * steps * 620 + 6000;
  if (d.epi == kDenseStore) {
    const int64_t narrow = up(d.m, 256) * up(d.n, 224) * d.problems;
    const int64_t cost = up(narrow, sms / 2) * steps * 560 + 6000;
    if (cost < pair_cost) {
      p.bn = 224;
      pair_cost = cost;
    }
  }
  int64_t best = up(tiles_of(128), sms) * steps * 680 + 2500;
  p.split = 1;
  const int least = f32 ? 1 : 4;
  for (int c = 2; c <= 8; ++c) {
    if (units < c * least || tiles_of(128) > resident_clusters(c)) break;
    const int64_t cost = up(steps, c) * 680 + 6000;
    if (cost < best) {
      best = cost;
      p.split = c;
    }
  }
  const bool pair = d.m > 128 && pair_cost <= best;
  if (pair) p.split = 1;
  const int bm = pair ? 256 : 128, bn = gated ? bm / 2 : pair ? p.bn : bm;
  p.mt = (int)up(d.m, bm);
  p.nt = (int)up(d.n, bn);
  // 32 rows of A leave room for nine stages (1 token x 4096 x 14336 forward 82 us,
  // with six of 128 rows 93), 64 for eight
  const int a_rows = d.a[0].mn_major || d.m > 64 ? 128 : d.m > 32 ? 64 : 32;
  p.a_bytes = (uint32_t)a_rows * kBK * 2;
  p.stage_bytes = p.a_bytes + kOpBytes;
  p.stages = (int)(stage_room(d.epi) / p.stage_bytes);
  const int nb = gated ? 2 : d.segs, na = d.problems > 1 ? d.problems : d.segs;
  for (int i = 0; i < 2; ++i) {
    if (!encode(&p.a[i], d.a[i < na ? i : 0], d.m, d.k, parts, a_rows)) return QAT_ERR_CUDA;
    if (!encode(&p.b[i], d.b[i < nb ? i : 0], d.n, d.k, parts, gated ? bn : pair ? bn / 2 : 128))
      return QAT_ERR_CUDA;
  }
  p.act = d.act;
  for (int i = 0; i < 2; ++i) {
    p.c[i] = d.c[i];
    p.q[i] = d.q[i];
  }
  p.q_pitch = d.q_pitch;
  p.q_part = d.q_part;
  p.gp = d.gp;
  p.up = d.up;
  p.flags = d.flags;
  p.limit = device_wait_limit();
  if (f32) return pair ? launch_majors<F32, 2>(p, d, s) : launch_majors<F32, 1>(p, d, s);
  return pair ? launch_majors<BF16, 2>(p, d, s) : launch_majors<BF16, 1>(p, d, s);
}

// ---------------------------------------------------------------------------
// Operands the copies cannot read in place (rows that are not whole 16-byte
// vectors, fp32) as bf16 parts with padded rows.  One launch for up to six
// tensors; a thread takes eight elements of a row.
// ---------------------------------------------------------------------------
struct PackArgs {
  DensePack t[6];
};
template <typename T>
__global__ void __launch_bounds__(256) k_dense_pack(const __grid_constant__ PackArgs p) {
  const DensePack& t = p.t[blockIdx.y];
  pdl_trigger();
  const int64_t wide = t.pitch / 8, total = t.rows * wide;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / wide, c = (i - r * wide) * 8;
    float v[8];
    const int64_t at = r * t.cols + c;
    if (T::BYTES == 4 && t.cols % 4 == 0 && c + 8 <= t.cols) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(t.src) + at);
      const float4 a = q[0], b = q[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e < t.cols ? ld_elem<T>(t.src, at + e) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < (T::BYTES == 4 ? 3 : 1); ++k) {
      float h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = T::BYTES == 4 ? take_bf16(v[e]) : v[e];
      *reinterpret_cast<uint4*>(static_cast<char*>(t.dst) + (k * t.part + r * t.pitch + c) * 2) =
          make_uint4(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]), pack_bf16x2(h[4], h[5]),
                     pack_bf16x2(h[6], h[7]));
    }
  }
}

qat_status launch_dense_pack(qat_dtype dt, const DensePack* list, int n, cudaStream_t s) {
  if (n == 0) return QAT_OK;
  PackArgs p = {};
  int64_t most = 0;
  for (int i = 0; i < n; ++i) {
    p.t[i] = list[i];
    const int64_t b = (list[i].rows * (list[i].pitch / 8) + 255) / 256;
    most = b > most ? b : most;
  }
  const int64_t room = (int64_t)device_info().sms * 16;
  const dim3 grid((unsigned)(most < room ? most : room), (unsigned)n);
  if (dt == QAT_F32)
    k_dense_pack<F32><<<grid, 256, 0, s>>>(p);
  else
    k_dense_pack<BF16><<<grid, 256, 0, s>>>(p);
  count_launch(1);
  return launch_status();
}

}  // namespace qat
