// kernels_kvsplit.cu -- attention of one new token of each sequence over a paged,
// quantized key-value cache (compiled once for each cache format QAT_KV_FORMAT).
//
//   s_t = scale ks_t (q . kq_t - kz_t sum q),  p_t = exp(s_t - m),  w_t = p_t vs_t
//   y = (sum w_t vq_t - sum w_t vz_t) / sum p_t        (kq, vq codes; kz, vz zero points)
//
// The floor is reading the codes once.  The query heads of a cache head share a
// read: they are the eight columns of m16n8k16 products whose rows are positions
// (scores) or head elements (values).  Codes are exact in fp16, which takes fewer
// operations to reach than bf16 (a code is the low bits of a number of exponent 10;
// FP8 converts), so quantized rows are multiplied in fp16: queries and weights (with
// their value's scale) are first scaled by powers of two, so that a head's largest lie near
// the top of its range; what falls below it is 2^-38 of the largest element of q and 2^-33
// of the largest weight.  bf16 rows are multiplied in bf16.
//
// Work is cut evenly whatever the lengths: the tiles of 16 positions of every
// (sequence, head group), in one row, are dealt to the resident warps in equal runs.
// A run that starts or ends inside a sequence leaves a part (maximum, sum, weighted
// values): a block joins what its warps, whose runs follow each other, hold of the same
// sequence, and k_kv_join the rest.  Until then warps share nothing, so that the start
// and the end of a piece, a few latencies each, pass behind the others' work; what they
// cost a warp counts as kPieceTiles tiles when the runs are cut.
//
// Tiles come by cp.async, each warp's own ring, 512 consecutive bytes an operation
// (copies of 64 bytes of eight rows took nearly twice the bytes from L2), to places
// that are swizzled so that both products' operands are read without conflicts.  Rows
// of a product are positions lane / 4 (+ 8) for keys, and the lane's share of a key is
// every fourth 16-byte run; of a value every eighth.  Which head element a product's k
// index stands for is free, so the codes' own order is taken for both operands.
//
// Twelve warps an SM (168 registers, 17 KB of ring each, two tiles and more in flight)
// walk through tiles at 0.8 to 1.1 us each.  Measured (both launches, in a graph): 64
// sequences of up to 8192 positions, 32 heads over 8 of 128 in affine 4-bit codes, 68 us
// (2.9 TB/s; 486 instructions a tile with the pieces' starts and ends, 53% of the issue
// slots); two of 131072 in E4M3 103 us (5.4 TB/s, 79% of the copy bandwidth); 32 of up to
// 2048, 16 heads of 64 in bf16, 23 us; one of 700 in int8 10.9 us, of which 8 are the
// latencies of lengths, table, codes and the two joins.
#include <atomic>
#include <cmath>

#include "qat_kv.cuh"
#include "qat_kvsplit.h"
#include "qat_layer.cuh"

namespace qat {
namespace {

constexpr int kFormat = QAT_KV_FORMAT;
constexpr float kLog2e = 1.4426950408889634f;
// What a piece costs beside its tiles, in tiles (64 sequences of up to 8192 positions
// in 4-bit codes: 68.5 us with 4, 68.1 with 6, 67.7 with 8, 67.3 with 11, 68.5 with 14; two
// of 131072 in E4M3 100.5 to 102.5, the fewest with 11).
constexpr int kPieceTiles = 8;
// Tiles of a run at least (one sequence of 700 positions: 10.9 us with 1 or 2, 11.7 with
// 4; a run's first tiles may be a piece's cost).
constexpr int kLeastRun = 2;
constexpr float kSlack = 4.0f;  // scores may exceed the running maximum by 2^4 before it moves

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes from global to shared memory, or zeros
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// (FIRST: with no sum before it)
template <bool HALF, bool FIRST = false>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
#define QAT_MMA(TYPE)                                                                              \
  if constexpr (FIRST)                                                                             \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                    \
        ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"                 \
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                                           \
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));                \
  else                                                                                             \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                    \
        ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"                     \
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                           \
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1))
  if constexpr (HALF) {
    QAT_MMA("f16");
  } else {
    QAT_MMA("bf16");
  }
#undef QAT_MMA
}
// The number one binary32 step nearer to 0, cut off to its upper half (0 stays): never the
// number itself, so that a remainder is left, of its sign.
template <bool SIGNED>
__device__ __forceinline__ uint32_t upper_below(float x) {
  const uint32_t u = __float_as_uint(x);
  if constexpr (!SIGNED) return (max(u, 1u) - 1u) & 0xffff0000u;
  return ((max(u & 0x7fffffffu, 1u) - 1u) & 0x7fff0000u) | (u & 0x80000000u);
}
// The next 16-bit parts of two numbers, packed; they keep the remainders.  bf16 parts before
// the LAST are cut off, so that none overflows, and none is 0 unless the number is (or lies
// below 2^-110): 0 times an infinity of the cache's would make NaN of what is infinite.
// SIGNED: numbers that may be negative.
template <bool HALF, bool LAST, bool SIGNED>
__device__ __forceinline__ uint32_t take_pair(float& x, float& y) {
  if constexpr (HALF) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    if constexpr (!LAST) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r));
      x -= v.x, y -= v.y;
    }
    return r;
  } else if constexpr (LAST) {
    return pack_bf16x2(x, y);
  } else {
    const uint32_t u = upper_below<SIGNED>(x), v = upper_below<SIGNED>(y);
    x -= __uint_as_float(u), y -= __uint_as_float(v);
    return u >> 16 | v;
  }
}
// an 8 x 8 matrix of 16-bit elements, transposed over the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x *= f in x's own register: the branch that rescales the sums must not leave them
// in others, from which every pass of the loop would move them back
__device__ __forceinline__ void scale_in_place(float& x, float f) {
  asm volatile("mul.rn.f32 %0, %0, %1;" : "+f"(x) : "f"(f));
}
// Loads from shared memory (as one instruction each: vectors that the compiler takes
// apart it does not always put together again).
template <int BYTES>
__device__ __forceinline__ void load_run(uint32_t at, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at)
                 : "memory");
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
}
__device__ __forceinline__ float load_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float load_s8(uint32_t at) {
  int v;
  asm volatile("ld.shared.s8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return (float)v;
}

// ---------------------------------------------------------------------------
// codes: the pairs of fp16 (or bf16) that a 32-bit word holds, in the order in which
// they are cheapest to reach
// ---------------------------------------------------------------------------
template <int F>
struct Word {
  static constexpr bool kHalf = F != QAT_CACHE_BF16;
  static constexpr bool kFp8 = F == QAT_CACHE_E4M3 || F == QAT_CACHE_E5M2;
  static constexpr int CODES = F == QAT_CACHE_INT4 ? 8 : F == QAT_CACHE_BF16 ? 2 : 4;
  static constexpr int PAIRS = CODES / 2;
  // Keys: the places of pair i's halves in the word.  Integer codes lie 16 bits apart.
  __host__ __device__ static constexpr int lo(int i) {
    return kFp8 ? 2 * i : F == QAT_CACHE_INT4 ? i ^ 1 : i;
  }
  __host__ __device__ static constexpr int hi(int i) { return kFp8 ? 2 * i + 1 : lo(i) + PAIRS; }
  // Values: words of two positions are first brought together, one half (0, 1) of each
  // at a time, so that a pair is the same element of both.
  static constexpr uint32_t kLower = kFp8 ? 0x5140 : 0x5410, kUpper = kFp8 ? 0x7362 : 0x7632;
  // element c of the word among the pairs of both halves
  __host__ __device__ static constexpr int rank(int c) {
    return F == QAT_CACHE_INT4 ? c ^ 1 : c;
  }

  __device__ __forceinline__ static void decode(uint32_t w, uint32_t (&out)[PAIRS]) {
    if constexpr (F == QAT_CACHE_BF16) {
      out[0] = w;
    } else if constexpr (F == QAT_CACHE_INT4) {
      // a low nibble is 1024 + (q + 8), less 1032; a high one 1024 + 16 (q + 8), by 1/16, less 72
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const uint32_t x = w >> (4 * i);
        out[i] = sub2(pick(x, 0x000f000fu, 0x64086408u), 0x64086408u);
        out[i + 1] = fma2(pick(x, 0x00f000f0u, 0x64806480u), 0x2c002c00u, 0xd480d480u);
      }
    } else if constexpr (F == QAT_CACHE_INT8) {
      // 1024 + (q + 128), less 1152
#pragma unroll
      for (int i = 0; i < 2; ++i)
        out[i] = sub2(pick(w >> (8 * i), 0x00ff00ffu, 0x64806480u), 0x64806480u);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint16_t x = (uint16_t)(w >> (16 * i));
        if (F == QAT_CACHE_E4M3)
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(out[i]) : "h"(x));
        else
          asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(out[i]) : "h"(x));
      }
    }
  }
  // (w & mask) ^ bits in one operation
  __device__ __forceinline__ static uint32_t pick(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
  }
  __device__ __forceinline__ static uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ static uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
  }
};

// ---------------------------------------------------------------------------
// shapes: DP the head dimension the products take (64, 128, 256; elements behind
// head_dim are zeros), HT tiles of eight query heads
// ---------------------------------------------------------------------------
constexpr int smaller(int a, int b) { return a < b ? a : b; }
constexpr int larger(int a, int b) { return a > b ? a : b; }

template <typename T, int F, int DP, int HT>
struct Shape {
  using W = Word<F>;
  static constexpr bool kF32 = T::BYTES == 4;
  static constexpr int ROW = DP / W::CODES * 4;  // bytes of a row of DP codes
  // a lane's share of a key: NK runs of CK bytes (EK codes), every fourth one; of a
  // value NV of CV bytes (EV codes), every eighth
  static constexpr int CK = smaller(16, ROW / 4), NK = ROW / 4 / CK, EK = CK / 4 * W::CODES;
  static constexpr int CV = smaller(16, ROW / 8), NV = ROW / 8 / CV, EV = CV / 4 * W::CODES;
  static constexpr int TILE = 32 * ROW;  // 16 keys and values
  static constexpr int UNITS = ROW / 16, LOADS = ROW / 32;  // 16-byte units a row; of a tile's half, a lane
  // 16 scales and 16 zero points of both
  static constexpr int PARAMS = F == QAT_CACHE_BF16 ? 0 : 160;
  // Keys of a tile and, a step later, its values, each with their scales and zero points.
  static constexpr int HALF_STAGE = (TILE + PARAMS) / 2;
  static constexpr int STAGES = smaller(6, larger(2, 13 * 1024 / (TILE + PARAMS)));
  static constexpr int H = 8 * HT, KS = DP / 16, MT = DP / 16;
  // 16-bit parts of q and of the weights: two of fp16 hold 22 bits of a weight (one took five
  // us less for the 4-bit batch, but left a sequence's elements off by up to 2^-12 all alike),
  // three of bf16 all 24 (two: no less time, 16 bits).
  static constexpr int QP = kF32 ? 3 : 1, PP = kF32 || F == QAT_CACHE_BF16 ? 3 : 2;
  static constexpr int QFRAG = kF32 ? QP * KS * 32 * 8 : 0;
  // A warp's ring and queries, then the part it starts with (its run began inside a
  // sequence); the part it ends with takes the ring's place.
  static constexpr int PART = H * DP * 4;
  static constexpr int RING = larger(2 * STAGES * HALF_STAGE + QFRAG, PART), WARP = RING + PART;
  // Registers hold twelve warps of up to 168, eight of up to 255 (64 sequences in 4-bit codes:
  // 70.6 us with eleven, 67.7 with twelve, 82.7 with thirteen, which spill; 32 sequences of
  // short heads in bf16: 21.5, 22.8, 24.5).
  static constexpr int WARPS =
      smaller(224 * 1024 / WARP, DP * HT <= 128 && !kF32 ? 12 : 8);
  static constexpr int THREADS = 32 * WARPS, SMEM = WARPS * WARP;

  // Where a unit of a row lies in a tile's half.  Reads of keys (rows lane / 4, four
  // units side by side) and of values (rows 2 (lane % 4), eight runs side by side) then
  // meet every bank once.  mix() is linear: mix(r + s) = mix(r) ^ mix(s) without carries.
  __host__ __device__ static constexpr int mix(int r) {
    return UNITS >= 8 ? (r & 6) ^ 4 * (r & 1) : UNITS == 4 ? (r >> 1) & 2 : 0;
  }
  __host__ __device__ static constexpr int row_place(int r) {
    return UNITS >= 8 ? r : UNITS == 4 ? r ^ ((r >> 1) & 1) : r ^ ((r >> 2) & 1);
  }
  __host__ __device__ static constexpr int place(int r, int byte) {
    return (row_place(r) * UNITS + ((byte / 16) ^ mix(r))) * 16 + byte % 16;
  }

  // Pair p of a run of a key: the place of its halves in the run.
  __host__ __device__ static constexpr int key_place(int p, int hi) {
    return p / W::PAIRS * W::CODES + (hi ? W::hi(p % W::PAIRS) : W::lo(p % W::PAIRS));
  }
  // Element e of run j of a value: its place among the rows of the products (even
  // and odd ones are rows g and g + 8 of a tile).
  __host__ __device__ static constexpr int value_place(int j, int e) {
    return (j * (CV / 4) + e / W::CODES) * W::CODES + W::rank(e % W::CODES);
  }
};

// Eight consecutive elements of q or y.
template <typename T>
__device__ __forceinline__ void load8(const void* x, int64_t at, bool vec, float* v) {
  if (!vec) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ld_elem<T>(x, at + e);
  } else if constexpr (T::BYTES == 2) {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const char*>(x) + 2 * at);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const char*>(x) + 4 * at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(void* x, int64_t at, bool vec, const float* v) {
  if (!vec) {
#pragma unroll
    for (int e = 0; e < 8; ++e) st_elem<T>(x, at + e, v[e]);
  } else if constexpr (T::BYTES == 2) {
    *reinterpret_cast<uint4*>(static_cast<char*>(x) + 2 * at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<char*>(x) + 4 * at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// The exponent of the power of two at or below x (0 for 0 and what is not finite).
__device__ __forceinline__ int exponent_of(float x) {
  const int e = (int)(__float_as_uint(x) >> 23 & 255u);
  return e == 0 || e == 255 ? 0 : e - 127;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// EXACT: rows of exactly DP codes.
template <typename T, int F, int DP, int HT, bool EXACT>
__global__ void __launch_bounds__(Shape<T, F, DP, HT>::THREADS, 1)
    k_kv_split(KvCacheView c, KvAttnArgs a, int group, int tiles, bool q_vec, bool y_vec,
               SplitWs ws) {
  using S = Shape<T, F, DP, HT>;
  using W = typename S::W;
  constexpr int WARPS = S::WARPS, H = S::H;
  constexpr bool HALF = W::kHalf;
  extern __shared__ __align__(16) char smem[];
  __shared__ int64_t s_sum[WARPS], s_first[WARPS], s_off[WARPS];
  __shared__ int s_b[WARPS];
  // Parts: sequence, head group, tiles from .. to (none: to = 0); maximum and sum, then
  // the factor in its chain; of the chain that starts with it, maximum and sum.
  static_assert(2 * WARPS <= 32, "a lane for each part");
  __shared__ int4 s_part[2 * WARPS];
  __shared__ float2 s_ml[2 * WARPS][H], s_chain[2 * WARPS][H];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int d = EXACT ? DP : c.d, row_bytes = EXACT ? S::ROW : c.row_bytes;
  pdl_trigger();

  // --- this warp's run of the work --------------------------------------------------
  // (a position's number plus a step fits 31 bits)
  const int64_t capacity =
      c.pages > 0 ? min(a.table_cols * c.page_size, (int64_t)kKvMaxLength) : 0;
  const int hgs = c.heads * tiles;
  auto length_of = [&](int b) -> int {  // 0 where there is nothing to read
    const int n = __ldg(a.lengths + b);
    return n <= 0 || n > capacity ? 0 : n;
  };
  // what a head group of sequence b counts for: its tiles and the cost of a piece
  auto cost_of = [&](int b) -> int64_t {
    const int n = length_of(b);
    return n ? (n + 15) / 16 + kPieceTiles : 0;
  };
  const int batch = (int)a.batch;
  const int each = (batch + S::THREADS - 1) / S::THREADS;
  const int b_lo = min((int)threadIdx.x * each, batch), b_hi = min(b_lo + each, batch);
  int64_t own = 0;
  for (int b = b_lo; b < b_hi; ++b) own += cost_of(b);
  int64_t before = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(kFull, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) s_sum[warp] = before;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  before = (before - own) * hgs, own *= hgs, total *= hgs;
  // Equal runs for as many warps as there is work for, on as many blocks as possible.
  const int64_t runs = max((int64_t)1, min((int64_t)gridDim.x * WARPS, total / kLeastRun));
  const int per = (int)((runs + gridDim.x - 1) / gridDim.x);  // of a block
  const int64_t run_least = total / runs, run_more = total - run_least * runs;  // (one more tile)
  auto run_start = [&](int64_t r) { return r < runs ? run_least * r + min(r, run_more) : total; };
  const int64_t run = (int64_t)blockIdx.x * per + warp;
  const int64_t first = run_start(run);
  if (lane == 0) s_first[warp] = first;
  __syncthreads();
  if (own > 0)
    for (int w = 0; w < per; ++w) {
      const int64_t f = s_first[w];
      if (f < before || f >= before + own) continue;
      int b = b_lo;
      int64_t at = before;
      while (f >= at + cost_of(b) * hgs) at += cost_of(b++) * hgs;
      s_b[w] = b;
      s_off[w] = f - at;
    }
  if (threadIdx.x < 2 * WARPS) s_part[threadIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();
  // sequences that have nothing to read
  const int64_t y_row = a.q_heads * c.d;
  for (int64_t b = (int64_t)blockIdx.x * WARPS + warp; b < batch; b += (int64_t)gridDim.x * WARPS) {
    if (length_of((int)b)) continue;
    const bool none = __ldg(a.lengths + b) <= 0;
    for (int64_t i = lane; i < y_row; i += 32) st_elem<T>(a.y, b * y_row + i, none ? 0.0f : NAN);
    if (a.lse)
      for (int64_t i = lane; i < a.q_heads; i += 32)
        a.lse[b * a.q_heads + i] = none ? -INFINITY : NAN;
  }
  int64_t left = 0, skip = 0;  // tiles of the run; of its first piece before it
  int b = 0, hg = 0;
  if (warp < per && run < runs && total > 0) {
    left = run_start(run + 1) - first;
    b = s_b[warp];
    hg = (int)(s_off[warp] / cost_of(b));
    skip = s_off[warp] - hg * cost_of(b);
  }

  char* const ring_p = smem + warp * S::WARP;  // keys' slots, then values'
  const uint32_t ring = smem_at(ring_p);
  constexpr uint32_t kRingEnd = S::STAGES * S::HALF_STAGE;
  uint2* const qfrag = reinterpret_cast<uint2*>(ring_p + 2 * kRingEnd);
  const int tiles_page = c.page_size / 16;
  const float to_log2 = a.scale * kLog2e;
  const bool zeros = kv_is_int(F) && c.kz;
  // Places of the lane's units as they are copied, and of its shares as they are read:
  // of keys in row g, of values in rows 2 t4 and 2 t4 + 1.
  const int units = row_bytes / 16;
  const int c_row = EXACT ? lane / S::UNITS : lane / units;
  const int c_unit = EXACT ? lane % S::UNITS : lane - c_row * units;
  const int c_place = S::place(c_row, c_unit * 16), k_place = S::place(g, t4 * S::CK);
  const int v_places[2] = {S::place(2 * t4, g * S::CV), S::place(2 * t4 + 1, g * S::CV)};
  // 16 scales a tile, then the zero points: lanes 0 to 3 and 4 take 16 bytes each
  const char* const k_params =
      lane == 4 ? reinterpret_cast<const char*>(c.kz) : reinterpret_cast<const char*>(c.ks) + lane * 16;
  const char* const v_params =
      lane == 4 ? reinterpret_cast<const char*>(c.vz) : reinterpret_cast<const char*>(c.vs) + lane * 16;
  const int p_step = lane == 4 ? 16 : 64, p_lanes = zeros ? 5 : 4;
  const int r_step = 32 / units, u_step = 32 - r_step * units;  // from one of a lane's units to its next
  if (!EXACT) {  // elements behind head_dim stay zeros (never NaN, whose product with 0 is NaN)
    for (int i = lane * 16; i < 2 * (int)kRingEnd; i += 512)
      *reinterpret_cast<uint4*>(ring_p + i) = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }

  while (left > 0) {
    const int length = length_of(b), n_tiles = (length + 15) / 16;
    const int64_t cost = n_tiles + kPieceTiles, take = min(cost - skip, left);
    const int from = (int)max((int64_t)0, skip - kPieceTiles);
    const int to = (int)max((int64_t)0, skip + take - kPieceTiles);
    left -= take;
    if (to > from) {
      const int kvh = hg / tiles, h0 = kvh * group + (hg - kvh * tiles) * S::H;
      const int heads = min(S::H, (kvh + 1) * group - h0);
      const int steps = to - from;

      // --- copies, tile after tile ----------------------------------------------------
      // The page of the next tile of keys, its offset there (in tiles), and the place in
      // the cache (in tiles of 16 rows: 31 bits) of the tile whose values come next.
      int rem = from % tiles_page;
      const int32_t* entry = a.table + (int64_t)b * a.table_stride + from / tiles_page;
      int page = __ldg(entry);
      uint32_t v_at = 0;
      bool bad = false;
      // 16 rows, their scales and zero points; zeros in place of the rows from `rows` on.
      auto copy = [&](uint32_t slot, const char* codes, const char* params, uint32_t at, int rows,
                      bool on) {
        const char* src = codes + (uint64_t)at * (uint32_t)(16 * row_bytes);
        const int left = on ? rows - c_row : 0;
        if constexpr (EXACT) {
#pragma unroll
          for (int i = 0; i < S::LOADS; ++i)
            copy_async(slot + 512 * i + (c_place ^ S::mix(i * 32 / S::UNITS) * 16), src + 512 * i,
                       left > i * 32 / S::UNITS);
        } else {
          int r = 0, u = c_unit;
#pragma unroll 1
          for (int i = 0; lane + i < 16 * units; i += 32) {
            copy_async(slot + S::place(c_row + r, u * 16), src + i * 16, left > r);
            r += r_step, u += u_step;
            if (u >= units) u -= units, ++r;
          }
        }
        if constexpr (F != QAT_CACHE_BF16)
          if (lane < p_lanes)
            copy_async(slot + S::TILE / 2 + lane * 16, params + (uint64_t)at * (uint32_t)p_step, on);
      };
      const char* const k_codes = c.k + lane * 16;
      const char* const v_codes = c.v + lane * 16;
      int rows_ahead = length - from * 16 + 16;  // of the tile whose values come next
      // keys of tile `step` + 1 and values of tile `step`
      auto issue = [&](int step, uint32_t k_slot, uint32_t v_slot) {
        copy(ring + kRingEnd + v_slot, v_codes, v_params, v_at, rows_ahead, step >= 0 && step < steps);
        rows_ahead -= 16;
        const bool on = step + 1 < steps;
        const bool there = (uint32_t)page < (uint32_t)c.pages;
        bad = bad || (on && !there);
        v_at = ((uint32_t)(there ? page : 0) * (uint32_t)c.heads + kvh) * tiles_page + rem;
        copy(ring + k_slot, k_codes, k_params, v_at, rows_ahead, on && there);
        if (++rem == tiles_page) {
          rem = 0, ++entry;
          if (step + 2 < steps) page = __ldg(entry);
        }
        copy_commit();
      };
      auto after = [&](uint32_t slot) {
        return slot == kRingEnd - S::HALF_STAGE ? 0 : slot + S::HALF_STAGE;
      };
      // (no slot has two copies under way: before the first tile the last slot gets zeros)
#pragma unroll 1
      for (int i = -1; i < S::STAGES - 1; ++i)
        issue(i, (i + 1) * S::HALF_STAGE, (i < 0 ? S::STAGES - 1 : i) * S::HALF_STAGE);

      // --- the queries as products take them ------------------------------------------
      uint32_t qr[S::kF32 ? 1 : HT][S::kF32 ? 1 : S::KS][2];
      // of heads 2 t4, 2 t4 + 1: the sum of the scaled query, and the factor of its scores
      float qsum[HT][2], qscale[HT][2];
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        float v[S::NK][S::EK], sum = 0.0f, top = 0.0f;
#pragma unroll
        for (int j = 0; j < S::NK; ++j)
#pragma unroll
          for (int e = 0; e < S::EK; e += 8) {
            const int at = (4 * j + t4) * S::EK + e;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][e + i] = 0.0f;
            if (8 * ht + g < heads && at < d)
              load8<T>(a.q, (int64_t)b * a.q_batch_stride + (h0 + 8 * ht + g) * a.q_head_stride + at,
                       q_vec, v[j] + e);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[j][e + i]));
          }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // fp16: the largest element between 2^13 and 2^14 (or, below 2^-100, as near as that)
        const int up = HALF ? 13 - max(exponent_of(top), -87) : 0;
#pragma unroll
        for (int j = 0; j < S::NK; ++j) {
#pragma unroll
          for (int e = 0; e < S::EK; ++e) {
            if constexpr (HALF) v[j][e] *= power_of_two(up);
            sum += v[j][e];
          }
#pragma unroll
          for (int k = 0; k < S::EK / 4; ++k) {
            const int ks = j * (S::EK / 4) + k;
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = v[j][S::key_place(2 * k + i / 2, i % 2)];
            if constexpr (!S::kF32) {
              qr[ht][ks][0] = take_pair<HALF, true, true>(x[0], x[1]);
              qr[ht][ks][1] = take_pair<HALF, true, true>(x[2], x[3]);
            } else {
#pragma unroll
              for (int p = 0; p < 3; ++p) {
                uint2 y;
                y.x = p < 2 ? take_pair<HALF, false, true>(x[0], x[1])
                            : take_pair<HALF, true, true>(x[0], x[1]);
                y.y = p < 2 ? take_pair<HALF, false, true>(x[2], x[3])
                            : take_pair<HALF, true, true>(x[2], x[3]);
                qfrag[(p * S::KS + ks) * 32 + lane] = y;
              }
            }
          }
        }
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        const float factor = to_log2 * power_of_two(-up);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qsum[ht][i] = __shfl_sync(kFull, sum, 8 * t4 + 4 * i);
          qscale[ht][i] = __shfl_sync(kFull, factor, 8 * t4 + 4 * i);
        }
      }

      // m: the maximum that weights refer to; limit: where it moves; base: m, but 0 before
      // the first score.  Weighted values of codes are summed times `unit`, a head's power of
      // two that keeps p vs unit within 2^15 and `most`, which the largest p vs has reached,
      // between 2^8 and 2^9: what p vs loses below fp16's last bit is 2^-33 of the largest, and
      // rows of small weights count for what they add, whatever their scale.
      float m[HT][2], limit[HT][2], base[HT][2], l[HT][2], zsum[HT][2], o[HT][S::MT][4];
      float unit[HT][2], most[HT][2];
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          m[ht][i] = limit[ht][i] = -INFINITY, base[ht][i] = l[ht][i] = zsum[ht][i] = 0.0f,
          unit[ht][i] = HALF ? 0x1p123f : 1.0f, most[ht][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < S::MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[ht][i][j] = 0.0f;
      }

      // Scores of a tile: positions g, g + 8 (rows) and heads 2 t4, 2 t4 + 1 (columns).
      float s[HT][4];
      auto scores = [&](uint32_t slot) {
        // (two sums: a product waits for the one before the last)
        float acc[S::kF32 ? 3 : 2][HT][4];
#pragma unroll
        for (int j = 0; j < S::NK; ++j) {
          uint32_t w[2][S::CK / 4];
#pragma unroll
          for (int r = 0; r < 2; ++r)
            load_run<S::CK>(slot + 8 * r * S::ROW + (k_place ^ (j & 1) * 64) + j / 2 * 128, w[r]);
          uint32_t pr[2][S::CK / 4 * W::PAIRS];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < S::CK / 4; ++i) {
              uint32_t x[W::PAIRS];
              W::decode(w[r][i], x);
#pragma unroll
              for (int k = 0; k < W::PAIRS; ++k) pr[r][i * W::PAIRS + k] = x[k];
            }
#pragma unroll
          for (int k = 0; k < S::EK / 4; ++k) {
            const int ks = j * (S::EK / 4) + k;
            const uint32_t fa[4] = {pr[0][2 * k], pr[1][2 * k], pr[0][2 * k + 1], pr[1][2 * k + 1]};
            if constexpr (S::kF32) {
#pragma unroll
              for (int p = 0; p < 3; ++p) {
                const uint2 f = qfrag[(p * S::KS + ks) * 32 + lane];
                if (ks == 0)
                  mma<HALF, true>(acc[p][0], fa, f.x, f.y);
                else
                  mma<HALF>(acc[p][0], fa, f.x, f.y);
              }
            } else {
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) {
                if (ks < 2)
                  mma<HALF, true>(acc[ks % 2][ht], fa, qr[ht][ks][0], qr[ht][ks][1]);
                else
                  mma<HALF>(acc[ks % 2][ht], fa, qr[ht][ks][0], qr[ht][ks][1]);
              }
            }
          }
        }
#pragma unroll
        for (int ht = 0; ht < HT; ++ht)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[ht][i] = acc[0][ht][i] + acc[1][ht][i];
            if constexpr (S::kF32) s[ht][i] += acc[2][ht][i];
          }
      };
      // The tile's weights, as the second operand of the value products.
      uint32_t wb[HT][S::PP][2];
      float ks[2] = {1.0f, 1.0f}, kz[2] = {0.0f, 0.0f};
      auto key_params = [&](uint32_t slot) {
        if constexpr (F != QAT_CACHE_BF16) {
          const uint32_t at = slot + S::TILE / 2;
          ks[0] = load_f32(at + 4 * g), ks[1] = load_f32(at + 4 * g + 32);
          if (zeros) kz[0] = load_s8(at + 64 + g), kz[1] = load_s8(at + 72 + g);
        }
      };
      auto weigh = [&](int tile, uint32_t v_slot) {
        float vs[2] = {1.0f, 1.0f}, vz[2] = {0.0f, 0.0f};
        if constexpr (F != QAT_CACHE_BF16) {
          const uint32_t at = v_slot + S::TILE / 2;
          vs[0] = load_f32(at + 4 * g), vs[1] = load_f32(at + 4 * g + 32);
          if (zeros) vz[0] = load_s8(at + 64 + g), vz[1] = load_s8(at + 72 + g);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int ht = 0; ht < HT; ++ht)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& x = s[ht][2 * r + i];
              if constexpr (kv_is_int(F)) x = __fmaf_rn(-kz[r], qsum[ht][i], x);
              x *= F == QAT_CACHE_BF16 ? qscale[ht][i] : qscale[ht][i] * ks[r];
            }
        if (tile * 16 + 16 > length) {  // rows behind the sequence
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (tile * 16 + g + 8 * r >= length) {
              vs[r] = vz[r] = 0.0f;
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) s[ht][2 * r] = s[ht][2 * r + 1] = -INFINITY;
            }
        }
        float p[HT][4], w[HT][4];
        auto weights = [&] {
#pragma unroll
          for (int ht = 0; ht < HT; ++ht)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[ht][i] = p[ht][i] = exp2_fast(s[ht][i] - base[ht][i & 1]);
              if constexpr (HALF) w[ht][i] = p[ht][i] * unit[ht][i & 1] * vs[i >> 1];
            }
        };
        weights();
        // the maximum and the unit move only where a score or a weighted scale is far above them
        bool above = false;
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
          for (int i = 0; i < 2; ++i) above = above || fmaxf(s[ht][i], s[ht][2 + i]) > limit[ht][i];
          if constexpr (HALF)
            above = above || fmaxf(fmaxf(fabsf(w[ht][0]), fabsf(w[ht][1])),
                                   fmaxf(fabsf(w[ht][2]), fabsf(w[ht][3]))) > 0x1p15f;
        }
        if (__any_sync(kFull, above)) {
#pragma unroll
          for (int ht = 0; ht < HT; ++ht)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = fmaxf(s[ht][i], s[ht][2 + i]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
              top = fmaxf(top, m[ht][i]);
              const float was = m[ht][i] == top ? 1.0f : exp2_fast(m[ht][i] - top);
              m[ht][i] = top;
              limit[ht][i] = top + kSlack;
              base[ht][i] = top == -INFINITY ? 0.0f : top;
              l[ht][i] *= was;
              float both = was;
              if constexpr (HALF) {
                // (Below 2^-115 as near to 2^8 as that: the unit times p stays finite, and what is
                // lost lies below the smallest number.  The unit grows by more than 1 / was only
                // beside sums of 0, and falls by more than 2^126 from sums that no longer count.)
                float here = fmaxf(fabsf(exp2_fast(s[ht][i] - base[ht][i]) * vs[0]),
                                   fabsf(exp2_fast(s[ht][2 + i] - base[ht][i]) * vs[1]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) here = fmaxf(here, __shfl_xor_sync(kFull, here, x));
                most[ht][i] = fmaxf(fmaxf(here, most[ht][i] * was), 0x1p-115f);
                const int old = exponent_of(unit[ht][i]), now = 8 - exponent_of(most[ht][i]);
                unit[ht][i] = power_of_two(now);
                both *= power_of_two(min(max(now - old, -126), 127));
              }
              zsum[ht][i] *= both;
#pragma unroll
              for (int j = 0; j < S::MT; ++j)
                scale_in_place(o[ht][j][i], both), scale_in_place(o[ht][j][2 + i], both);
            }
          weights();
        }
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            l[ht][i & 1] += p[ht][i];
            if constexpr (kv_is_int(F))
              zsum[ht][i & 1] = __fmaf_rn(w[ht][i], vz[i >> 1], zsum[ht][i & 1]);
          }
#pragma unroll
          for (int k = 0; k < S::PP; ++k)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              wb[ht][k][r] =
                  transpose8(k + 1 < S::PP ? take_pair<HALF, false, false>(w[ht][2 * r], w[ht][2 * r + 1])
                                           : take_pair<HALF, true, false>(w[ht][2 * r], w[ht][2 * r + 1]));
        }
      };
      // Weighted values: rows are head elements, k the positions.
      auto values = [&](uint32_t slot) {
#pragma unroll
        for (int j = 0; j < S::NV; ++j) {
          uint32_t v[4][S::CV / 4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            load_run<S::CV>(slot + (r >> 1) * 8 * S::ROW + v_places[r & 1] + 128 * j, v[r]);
#pragma unroll
          for (int i = 0; i < S::CV / 4; ++i) {
            uint32_t pr[2][2 * W::PAIRS];  // positions 2 t4, + 1; and those + 8
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t x[W::PAIRS];
              W::decode(__byte_perm(v[2 * k][i], v[2 * k + 1][i], W::kLower), x);
#pragma unroll
              for (int q = 0; q < W::PAIRS; ++q) pr[k][q] = x[q];
              W::decode(__byte_perm(v[2 * k][i], v[2 * k + 1][i], W::kUpper), x);
#pragma unroll
              for (int q = 0; q < W::PAIRS; ++q) pr[k][W::PAIRS + q] = x[q];
            }
#pragma unroll
            for (int q = 0; q < W::PAIRS; ++q) {
              const int mt = (j * (S::CV / 4) + i) * W::PAIRS + q;
              const uint32_t fa[4] = {pr[0][2 * q], pr[0][2 * q + 1], pr[1][2 * q], pr[1][2 * q + 1]};
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) {
                // 16 positions only: the tensor cores cut their sums off toward zero, a loss that
                // grows with the run (2^-7 of the result after 2^20 positions; the additions take
                // 3 us of the 4-bit batch's 68)
                float part[4];
                mma<HALF, true>(part, fa, wb[ht][S::PP - 1][0], wb[ht][S::PP - 1][1]);
#pragma unroll
                for (int p = S::PP - 2; p >= 0; --p) mma<HALF>(part, fa, wb[ht][p][0], wb[ht][p][1]);
                add2(o[ht][mt][0], o[ht][mt][1], part[0], part[1], o[ht][mt][0], o[ht][mt][1]);
                add2(o[ht][mt][2], o[ht][mt][3], part[2], part[3], o[ht][mt][2], o[ht][mt][3]);
              }
            }
          }
        }
      };

      // A tile's scores are computed beside the weighted values of the tile before: one
      // chain of products alone would leave the warp waiting.
      uint32_t prev = kRingEnd - S::HALF_STAGE, slot = 0, next = after(0);  // of this step
      copy_wait<S::STAGES - 1>();
      __syncwarp();  // (scales are other lanes' copies)
      scores(ring);
      key_params(ring);
      for (int step = 0; step < steps; ++step) {
        copy_wait<S::STAGES - 2>();
        __syncwarp();  // also: this step's keys and the values of the step before are done with
        weigh(from + step, ring + kRingEnd + slot);
        issue(step + S::STAGES - 1, slot, prev);
        if (step + 1 < steps) {
          scores(ring + next);
          key_params(ring + next);
        }
        values(ring + kRingEnd + slot);
        prev = slot, slot = next, next = after(next);
      }
      copy_wait<0>();
      __syncwarp();  // (the next piece's copies write where other lanes read scales)

      // --- the piece's result -----------------------------------------------------------
      const bool whole = from == 0 && to == n_tiles;
      const int which = 2 * warp + (from == 0);
      float* const part = reinterpret_cast<float*>(ring_p + (from == 0 ? 0 : S::RING));
      if (!whole && lane == 0) s_part[which] = make_int4(b, hg, from, to);
#pragma unroll
      for (int ht = 0; ht < HT; ++ht)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float sum = bad ? NAN : l[ht][i], z = zsum[ht][i];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            sum += __shfl_xor_sync(kFull, sum, x);
            if constexpr (kv_is_int(F)) z += __shfl_xor_sync(kFull, z, x);
          }
          const int h = 8 * ht + 2 * t4 + i;
          if (h >= heads) continue;
          const float by = !whole ? 1.0f : sum == 0.0f ? 0.0f : __frcp_rn(sum), down = __frcp_rn(unit[ht][i]);
          const int64_t y_at = ((int64_t)b * a.q_heads + h0 + h) * d;
#pragma unroll
          for (int j = 0; j < S::NV; ++j)
#pragma unroll
            for (int e = 0; e < S::EV; e += 8) {
              const int at = (8 * j + g) * S::EV + e;
              if (!EXACT && at >= d) continue;
              float y[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                constexpr auto pl = &S::value_place;
                const int p = pl(j, e + x);
                y[x] = (o[ht][p / 2][i + 2 * (p % 2)] - z) * by * down;
              }
              if (whole)
                store8<T>(a.y, y_at + at, y_vec, y);
              else
                store8<F32>(part, h * d + at, true, y);
            }
          if (g == 0) {
            if (!whole)
              s_ml[which][h] = make_float2(m[ht][i], sum);
            else if (a.lse)
              a.lse[(int64_t)b * a.q_heads + h0 + h] =
                  sum == 0.0f ? -INFINITY : (m[ht][i] + log2f(sum)) * 0.69314718055994531f;
          }
        }
    }
    // --- the next piece -------------------------------------------------------------------
    skip = 0;
    if (left > 0 && ++hg == hgs) {
      hg = 0;
      do ++b;
      while (cost_of(b) == 0);
    }
  }
  __syncthreads();

  // --- parts of one sequence that the block's warps hold, one after the other, joined ------
  // Lane k looks at part k.  A chain is a row of neighbours: the same sequence and group,
  // each beginning where the one before it ends.
  const int4 mine = lane < 2 * per ? s_part[lane] : make_int4(0, 0, 0, 0);
  const uint32_t valid = __ballot_sync(kFull, mine.w > 0);
  const uint32_t before_me = valid & ((1u << lane) - 1u);
  const int prev = before_me ? 31 - __clz(before_me) : 0;
  // (every lane takes part in each exchange: none may hang on the outcome of another)
  const int prev_b = __shfl_sync(kFull, mine.x, prev), prev_g = __shfl_sync(kFull, mine.y, prev);
  const int prev_to = __shfl_sync(kFull, mine.w, prev);
  const bool follows = before_me && prev_b == mine.x && prev_g == mine.y && prev_to == mine.z;
  const uint32_t starts = __ballot_sync(kFull, mine.w > 0 && !follows);
  auto chain_of = [&](uint32_t rest) {  // its parts; `rest`: the starts from it on
    const uint32_t after = rest & (rest - 1);
    return valid & ~((rest & -rest) - 1u) & (after ? (after & -after) - 1u : kFull);
  };
  for (int h = warp; h < H; h += WARPS)
    for (uint32_t rest = starts; rest; rest &= rest - 1) {
      const bool in = chain_of(rest) >> lane & 1u;
      const float2 x = in ? s_ml[lane][h] : make_float2(-INFINITY, 0.0f);
      float top = x.x;
      for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
      const float f = x.x == top ? 1.0f : exp2_fast(x.x - top);
      float sum = in ? f * x.y : 0.0f;
      for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(kFull, sum, i);
      if (in) s_ml[lane][h].x = f;
      if (lane == 0) s_chain[__ffs(rest) - 1][h] = make_float2(top, sum);
    }
  __syncthreads();
  int4 cut = make_int4(0, 0, 0, 0);
  for (uint32_t rest = starts; rest; rest &= rest - 1) {
    const uint32_t chain = chain_of(rest);
    const int head = __ffs(rest) - 1, tail = 31 - __clz(chain);
    const int pb = __shfl_sync(kFull, mine.x, head), pg = __shfl_sync(kFull, mine.y, head);
    const int from = __shfl_sync(kFull, mine.z, head), to = __shfl_sync(kFull, mine.w, tail);
    const int n_tiles = (length_of(pb) + 15) / 16;
    const int kvh = pg / tiles, h0 = kvh * group + (pg - kvh * tiles) * H;
    const int heads = min(H, (kvh + 1) * group - h0);
    const bool whole = from == 0 && to == n_tiles;
    const int64_t slot = ((int64_t)blockIdx.x * 2 + (from == 0)) * H;
    for (int i = threadIdx.x; i < heads * (d / 4); i += S::THREADS) {
      const int h = i / (d / 4), e = (i - h * (d / 4)) * 4;
      float y[4] = {};
      for (uint32_t m = chain; m; m &= m - 1) {
        const int k = __ffs(m) - 1;
        const float f = s_ml[k][h].x;
        const float4 v = *reinterpret_cast<const float4*>(
            smem + (k / 2) * S::WARP + (k % 2 ? 0 : S::RING) + (h * d + e) * 4);
        y[0] = __fmaf_rn(f, v.x, y[0]), y[1] = __fmaf_rn(f, v.y, y[1]);
        y[2] = __fmaf_rn(f, v.z, y[2]), y[3] = __fmaf_rn(f, v.w, y[3]);
      }
      const float2 t = s_chain[head][h];
      if (whole) {
        const int64_t row = (int64_t)pb * a.q_heads + h0 + h;
        const float by = t.y == 0.0f ? 0.0f : __frcp_rn(t.y);
#pragma unroll
        for (int x = 0; x < 4; ++x) st_elem<T>(a.y, row * d + e + x, y[x] * by);
        if (e == 0 && a.lse)
          a.lse[row] = t.y == 0.0f ? -INFINITY : (t.x + log2f(t.y)) * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float4*>(ws.o + (slot + h) * d + e) = make_float4(y[0], y[1], y[2], y[3]);
        if (e == 0) ws.ml[slot + h] = t;
      }
    }
    if (from == 0 && to < n_tiles && threadIdx.x == 0) {
      // cut off by the end of the block's last run: the blocks behind it hold the rest, up
      // to the run of its last tile's place x
      const int64_t x = run_start((int64_t)(blockIdx.x + 1) * per) + (n_tiles - to) - 1;
      const int64_t longer = run_more * (run_least + 1);
      const int64_t r = x < longer ? x / (run_least + 1) : run_more + (x - longer) / run_least;
      cut = make_int4(pb, pg, (int)(r / per) - (int)blockIdx.x + 1, 0);
    }
  }
  if (threadIdx.x == 0) ws.cut[blockIdx.x] = cut;
}

template <typename T, int F, int DP, int HT, bool EXACT>
qat_status go(const KvCacheView& c, const KvAttnArgs& a, const SplitWs& ws, int* grid,
              cudaStream_t s) {
  using S = Shape<T, F, DP, HT>;
  static_assert(S::WARPS >= 2, "shared memory");
  const auto k = k_kv_split<T, F, DP, HT, EXACT>;
  // (once for each device: the attribute stays)
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 63;
  const uint64_t bit = uint64_t{1} << dev;
  if (!(done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) != cudaSuccess) {
      (void)cudaGetLastError();
      return QAT_ERR_CUDA;
    }
    if (dev < 63) done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const HeadTiles t = head_tiles(a.q_heads, c.heads, c.d, S::kF32);
  const int sms = device_info().sms;
  *grid = sms < kSplitBlocks ? sms : kSplitBlocks;
  const auto vec = [](const void* p, int64_t s0, int64_t s1) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 * T::BYTES % 16 == 0 &&
           s1 * T::BYTES % 16 == 0;
  };
  if (launch_kernel(k, dim3(*grid), dim3(S::THREADS), S::SMEM, s, false, c, a, t.group, t.tiles,
                    vec(a.q, a.q_batch_stride, a.q_head_stride), vec(a.y, 8, 8), ws) != cudaSuccess)
    return QAT_ERR_CUDA;
  count_launch(1);
  return QAT_OK;
}
template <typename T, int F, int DP, int HT>
qat_status go_any(const KvCacheView& c, const KvAttnArgs& a, const SplitWs& ws, int* grid,
                  cudaStream_t s) {
  return c.d == DP ? go<T, F, DP, HT, true>(c, a, ws, grid, s)
                   : go<T, F, DP, HT, false>(c, a, ws, grid, s);
}

}  // namespace

template <int F>
qat_status launch_kv_split(const KvCacheView& c, const KvAttnArgs& a, qat_dtype dt, const SplitWs& ws,
                           int* grid, cudaStream_t s) {
  const bool wide = head_tiles(a.q_heads, c.heads, c.d, dt == QAT_F32).tile == 16;
  if (dt == QAT_F32) {
    if (c.d <= 64) return go_any<F32, F, 64, 1>(c, a, ws, grid, s);
    if (c.d <= 128) return go_any<F32, F, 128, 1>(c, a, ws, grid, s);
    return go_any<F32, F, 256, 1>(c, a, ws, grid, s);
  }
  if (c.d <= 64)
    return wide ? go_any<BF16, F, 64, 2>(c, a, ws, grid, s) : go_any<BF16, F, 64, 1>(c, a, ws, grid, s);
  if (c.d <= 128)
    return wide ? go_any<BF16, F, 128, 2>(c, a, ws, grid, s)
                : go_any<BF16, F, 128, 1>(c, a, ws, grid, s);
  return go_any<BF16, F, 256, 1>(c, a, ws, grid, s);
}
template qat_status launch_kv_split<kFormat>(const KvCacheView&, const KvAttnArgs&, qat_dtype,
                                             const SplitWs&, int*, cudaStream_t);

}  // namespace qat
