// kernels_w4.cu -- products of a few tokens with 4-bit weights.
//
//   y[t, n] = sum_u s[n, u] * sum_{k in u} (q[n, k] - z[n, u]) * x[t, k]
//
// and the gated pair h = act(x gate^T) * (x up^T), whose h goes to the second
// product as bf16 planes.  The floor is reading the codes (rows * cols / 2 bytes)
// and their parameters while the tokens are few.
#include "qat_layer.cuh"
#include "qat_layer.h"
#include "qat_tc.cuh"

namespace qat {

struct W4 {
  const uint8_t* codes;
  const void* scales;
  const int32_t* zp;
  const float* super;
  int64_t unit;  // elements of a unit, flat (units never straddle rows but for
                 // the two-level blocks and the whole tensor)
};

// scale and zero point of a unit
template <bool DOUBLE>
__device__ __forceinline__ void w4_params(const W4& w, int64_t u, float& s, float& z) {
  if (DOUBLE) {
    s = __fmul_rn(__fdiv_rn((float)static_cast<const uint8_t*>(w.scales)[u], 255.0f),
                  w.super[u >> 8]);
    z = 0.0f;
  } else {
    s = static_cast<const float*>(w.scales)[u];
    z = w.zp ? (float)w.zp[u] : 0.0f;
  }
}

constexpr int kGenTokens = 8;  // tokens a generic block keeps

// Any shape (rows that start inside a byte or a word, blocks that straddle rows,
// units that are not whole runs of 32): a warp per output row, lanes along k, one
// element at a time.  Bound by its instructions.
template <typename T, bool DOUBLE>
__device__ __forceinline__ void w4_row_generic(const void* x, int64_t t0, int nt, const W4& w,
                                               int64_t n, int64_t cols, int lane,
                                               float (&acc)[kGenTokens]) {
#pragma unroll
  for (int t = 0; t < kGenTokens; ++t) acc[t] = 0.0f;
  const int64_t base = n * cols;
  int64_t k = 0;
  while (k < cols) {  // one run of the row inside one unit at a time
    const int64_t u = (base + k) / w.unit;
    const int64_t left = (u + 1) * w.unit - base - k;
    const int64_t end = left < cols - k ? k + left : cols;
    float s, z, part[kGenTokens];
    w4_params<DOUBLE>(w, u, s, z);
#pragma unroll
    for (int t = 0; t < kGenTokens; ++t) part[t] = 0.0f;
    for (int64_t j = k + lane; j < end; j += 32) {
      const int64_t i = base + j;
      const int nib = (w.codes[i >> 1] >> ((i & 1) ? 0 : 4)) & 15;
      const float q = (float)((nib ^ 8) - 8) - z;
#pragma unroll
      for (int t = 0; t < kGenTokens; ++t)
        if (t < nt) part[t] = fmaf(q, ld_elem<T>(x, (t0 + t) * cols + j), part[t]);
    }
#pragma unroll
    for (int t = 0; t < kGenTokens; ++t) acc[t] = fmaf(part[t], s, acc[t]);
    k = end;
  }
#pragma unroll
  for (int t = 0; t < kGenTokens; ++t)
    for (int o = 16; o; o >>= 1) acc[t] += __shfl_xor_sync(~0u, acc[t], o);
}

template <typename T, bool DOUBLE, int NW>
__global__ void __launch_bounds__(128) k_w4_generic(const void* x, int64_t tokens, W4 wa, W4 wb,
                                                    int64_t rows, int64_t cols, int act, void* y,
                                                    int y_bf16) {
  pdl_trigger();
  pdl_wait();  // x may be the previous kernel's output
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (n >= rows) return;
  const int64_t t0 = (int64_t)blockIdx.y * kGenTokens;
  const int nt = (int)min((int64_t)kGenTokens, tokens - t0);
  float a[kGenTokens], b[kGenTokens];
  w4_row_generic<T, DOUBLE>(x, t0, nt, wa, n, cols, lane, a);
  if (NW == 2) w4_row_generic<T, DOUBLE>(x, t0, nt, wb, n, cols, lane, b);
  if (lane) return;
#pragma unroll
  for (int t = 0; t < kGenTokens; ++t) {
    if (t >= nt) break;
    const float v = NW == 2 ? act_value<false>(act, a[t]) * b[t] : a[t];
    if (y_bf16)
      st_elem<BF16>(y, (t0 + t) * rows + n, v);
    else
      st_elem<F32>(y, (t0 + t) * rows + n, v);
  }
}

// ---------------------------------------------------------------------------
// Rows of whole 8-code words whose units are whole runs of 32 codes.
//
// A warp multiplies two tiles of 16 rows (two of one weight, or one of each of
// the gated pair) by 8 NT tokens with m16n8k16 tensor-core products: a code is
// exact in bf16 (128 + q with the low mantissa bits, one logic operation for two
// codes, then an exact subtraction of 136 + zero point), so is a bf16 x, and the
// sums are binary32.  Decoding is then about 1.5 instructions a code where scalar
// multiply-adds would need three or four in all.  A float x comes as TERMS bf16
// planes (high, middle, low: three hold all its 24 bits, two hold 16, enough
// under a bf16 output), one product each.
//
// k runs in blocks of 128 codes, in parts of 32 CH: lane t of a row's four takes
// 8 CH consecutive codes of each part (one load), so that a part's codes share a
// unit; lane t brings the scale of part t.  The order of k inside a word is the
// codes' bit order, the same for both operands.  The warps of a block split k
// (and, with more tokens, also the rows, so that they read the same x from L1)
// and walk over the block's row tiles with the codes of the next blocks of k in
// flight across the tiles.  Where rows are few a cluster splits k once more.
// Partial sums are added in shared memory, then over the cluster, in a fixed
// order.
//
// Measured (GPU time of a call, codes and parameters read per second):
// [14336, 4096] in groups of 128, one token 12.0 us (2.6 TB/s), 8 tokens 13.6,
// 32 tokens 42.5; [57344, 4096] one token 35.6 us (3.5 TB/s).  Reading bounds
// the floor (4.6 us for the first); what holds it now is latency: four warps a
// scheduler (125 registers) keep 57% of the issue slots busy, the ALU and the
// tensor pipe are below half.  Codes decoded into tensor memory for tcgen05,
// 64 a step behind a block barrier, took 20.7 us at one token and 30.7 at 32.
// ---------------------------------------------------------------------------
constexpr int kW4Warps = 16;
constexpr int kW4Block = 128;  // codes of a row in a block of k
enum { kOutF32 = 0, kOutBf16 = 1, kOutPlanes = 2 };

struct W4Fast {
  const uint8_t* codes;
  const void* scales;
  const int32_t* zp;
  const float* super;
};
struct W4Args {
  W4Fast w[2];
  const void* x;           // bf16 rows, or planes
  int64_t x_pitch, x_plane;
  void* y;
  int64_t y_pitch, y_plane;  // planes
  int64_t rows, tokens;
  int64_t row_units;       // units from one row to the next
  int64_t unit;            // codes of a unit
  int cols, tiles;
  uint32_t unit_magic;
  int dbl, act, out, y_terms, split;
};

// two codes of a word (bits 0-3 and 16-19 after the shift) as bf16 q - zp: the bits of
// an integer under a fixed exponent are a float (the conversion of arXiv 2211.10017)
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t bias) {
  uint32_t v;
  // (w & 0x000f000f) ^ 0x43084308: bf16 128 + (q + 8)
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43084308, 0x6a;" : "=r"(v) : "r"(w));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(v), "r"(bias));
  return v;
}
// 136 + zp as a bf16 pair (exact)
__device__ __forceinline__ uint32_t w4_bias(int zp) { return (uint32_t)(0x4308 + zp) * 0x10001u; }
// 8 bf16 of x.  PLANES: what a kernel of this call may have written, by a coherent
// load that is free to move among the products (a C++ load is not: 32 fp32 tokens by
// [14336, 4096] take 132 us in place of 95); else the caller's rows, which nobody
// writes meanwhile (32 bf16 tokens: 50 us in place of 52).
template <bool PLANES>
__device__ __forceinline__ uint4 ld_x(const uint4* p) {
  if (!PLANES) return __ldg(p);
  uint4 v;
  asm("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(__cvta_generic_to_global(p)));
  return v;
}
// what a lane past the end of a row takes for x
__device__ const uint4 kZeros[4] = {};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with no sum before it
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The place of element e of 8 in the codes' order, pairs (1,5) (0,4) (3,7) (2,6).
__device__ __forceinline__ int w4_place(int e) { return (0x57134602 >> (4 * e)) & 7; }
// x of 8 consecutive k in that order: as stored in planes, or a bf16 row's
template <bool PLANES>
__device__ __forceinline__ uint4 x_pairs(const uint4& v) {
  if (PLANES) return v;
  return make_uint4(__byte_perm(v.x, v.z, 0x7632), __byte_perm(v.x, v.z, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632), __byte_perm(v.y, v.w, 0x5410));
}

// a lane's 4 words of a block of 128 codes of a row: 16 bytes at once, or 8 of
// each half, or 4 of each quarter
struct CodeWords {
  uint32_t v[4];
};
template <int CH>
__device__ __forceinline__ void load_codes(uint32_t* v, const uint8_t* p) {
  if constexpr (CH == 4) {
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else if constexpr (CH == 2) {
    const uint2 q = __ldcs(reinterpret_cast<const uint2*>(p));
    v[0] = q.x, v[1] = q.y;
  } else {
    v[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
  }
}

template <int NT, int NW>
struct W4Shape {
  static constexpr int R = 2 / NW;              // row tiles of each weight
  static constexpr int WR = NT;                 // warps along the rows
  static constexpr int WK = kW4Warps / WR;      // warps along k
  static constexpr int kRows = 16 * R * WR;     // output rows of a block's tile
  static constexpr int kTok = 8 * NT;
  static constexpr int kDepth = NT == 4 ? 1 : 2;  // blocks of k in flight
  static constexpr int kSlots = NT == 1 ? 2 : 1;  // tiles between joins
  static constexpr int kOne = NW * kRows * kTok;  // one k slice's sums of a tile
  static constexpr int kSmem = kSlots * WK * kOne * 4;
};

// TERMS 0: x is bf16 rows; else that many planes.  CH 2 with DBL: the two-level
// scales.
template <int TERMS, int CH, bool DBL, int NT, int NW>
__global__ void __launch_bounds__(kW4Warps * 32, 1) k_w4(const __grid_constant__ W4Args p) {
  using S = W4Shape<NT, NW>;
  constexpr int KB = kW4Block, SUB = 4 / CH, D = S::kDepth, kTerms = TERMS ? TERMS : 1, R = S::R;
  extern __shared__ __align__(16) float red[];  // [slot][k slice][weight][row][token]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wr = warp % S::WR, wk = warp / S::WR, split = p.split;
  const int rank = split > 1 ? (int)(blockIdx.x % split) : 0;
  const int first = blockIdx.x / split, stride = gridDim.x / split;
  const int mine = (p.tiles - first + stride - 1) / stride;  // tiles of this block
  const int64_t tok0 = (int64_t)blockIdx.y * S::kTok;
  const int tokens = (int)min((int64_t)S::kTok, p.tokens - tok0);
  const int cols = p.cols, blocks = (cols + KB - 1) / KB, step = S::WK * split;
  const int start = rank * S::WK + wk;
  const int per_tile = start < blocks ? (blocks - start + step - 1) / step : 0;

  // tokens past the end read the first one's x: their columns are not used
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q)
    xp[q] = static_cast<const __nv_bfloat16*>(p.x) +
            (q * 8 + g < tokens ? tok0 + q * 8 + g : 0) * p.x_pitch + t * 8 * CH;

  // The loads in flight, as loaded: codes, scales and zero points of D blocks of
  // k, for the rows g and g + 8 of the two row tiles.  Offsets are 32-bit and the
  // same for both weights.
  CodeWords code[D][2][2];
  uint32_t sc[D][2][2];
  float sup[D][2][2];
  int zp[D][2][2];
  uint32_t co[R][2], so[R][2];  // codes, units
  int f_tile = 0, f_kb = start;
  const int part_t = t & (SUB - 1);                // the part whose scale this lane brings
  const int parts = (cols + 32 * CH - 1) / (32 * CH);  // parts of a row
  // rows past the end read row 0 and are dropped at the end
  const auto rows_of = [&](int tile) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t n = (uint32_t)(first + tile * stride) * S::kRows + (wr * R + r) * 16 + h * 8 + g;
        const uint32_t m = n < p.rows ? n : 0;
        co[r][h] = (uint32_t)(((uint64_t)m * cols) >> 1) + t * 4 * CH;
        so[r][h] = m * (uint32_t)p.row_units;
      }
  };
  const uint32_t co_step = (uint32_t)(((uint64_t)stride * S::kRows * cols) >> 1);
  const uint32_t so_step = (uint32_t)(stride * S::kRows) * (uint32_t)p.row_units;
  const bool affine = p.w[0].zp != nullptr;
  const auto fetch = [&](int d) {
    const uint32_t run = (uint32_t)min(f_kb * SUB + part_t, parts - 1);
    const uint32_t u = __umulhi(2 * run + 1, p.unit_magic);
    uint32_t off[SUB];
    // past the row's end (in its last block) the lane reads the row's first
    // codes; x is zero there
#pragma unroll
    for (int s = 0; s < SUB; ++s)
      off[s] = f_kb * KB + s * 32 * CH + t * 8 * CH < cols
                   ? (uint32_t)f_kb * (KB / 2) + s * 16 * CH : 0u - t * 4 * CH;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const W4Fast& w = p.w[i / R];
#pragma unroll
        for (int s = 0; s < SUB; ++s)
          load_codes<CH>(code[d][i][h].v + s * CH, w.codes + (co[i % R][h] + off[s]));
        const uint32_t at = so[i % R][h] + u;
        if (DBL) {
          sc[d][i][h] = __ldg(static_cast<const uint8_t*>(w.scales) + at);
          sup[d][i][h] = __ldg(w.super + (at >> 8));
        } else {
          sc[d][i][h] = __ldg(static_cast<const uint32_t*>(w.scales) + at);
          if (affine) zp[d][i][h] = __ldg(w.zp + at);
        }
      }
    f_kb += step;
    if (f_kb >= blocks) {
      f_kb = start;
      ++f_tile;
      if ((int64_t)(first + f_tile * stride + 1) * S::kRows > p.rows) {
        if (f_tile < mine) rows_of(f_tile);
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            co[r][h] += co_step;
            so[r][h] += so_step;
          }
      }
    }
  };

  // Adds the partial sums of the tiles in the first `used` slots, of which the
  // last holds tile `last`: an output a thread.
  constexpr int kOne = S::kOne;
  const auto put = [&](int r, int c, int64_t n0, float v, float u) {
    const int64_t n = n0 + r, tok = tok0 + c;
    if (n >= p.rows) return;
    if (NW == 2) v = act_value<false>(p.act, v) * u;
    if (p.out == kOutBf16) {
      st_elem<BF16>(p.y, tok * p.rows + n, v);
    } else if (p.out == kOutF32) {
      st_elem<F32>(p.y, tok * p.rows + n, v);
    } else {
      const int64_t o = tok * p.y_pitch + (n & ~INT64_C(7)) + w4_place((int)(n & 7));
      for (int q = 0; q < p.y_terms; ++q) st_elem<BF16>(p.y, o + q * p.y_plane, take_bf16(v));
    }
  };
  const auto join = [&](int last, int used) {
    __syncthreads();
    if (split > 1) {  // one tile: the CTAs of the cluster add theirs, then share the outputs
      float* base = red;
      for (int i = threadIdx.x; i < kOne; i += kW4Warps * 32) {
        float v = base[i];
#pragma unroll
        for (int w = 1; w < S::WK; ++w) v += base[w * kOne + i];
        base[i] = v;
      }
      tc::cluster_sync();
      for (int i = threadIdx.x + rank * kW4Warps * 32; i < S::kRows * tokens;
           i += kW4Warps * 32 * split) {
        const int r = i % S::kRows, c = i / S::kRows, at = r * S::kTok + c;
        float v = 0.0f, u = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (q >= split) break;
          v += tc::ld_cluster(tc::map_rank(tc::smem(base + at), q));
          if (NW == 2) u += tc::ld_cluster(tc::map_rank(tc::smem(base + kOne / 2 + at), q));
        }
        put(r, c, (int64_t)first * S::kRows, v, u);
      }
      tc::cluster_sync();  // the other CTAs have read these sums
      return;
    }
    const int each = S::kRows * tokens;
    for (int i = threadIdx.x; i < used * each; i += kW4Warps * 32) {
      const int s = i / each, j = i - s * each, r = j % S::kRows, c = j / S::kRows;
      const float* at = red + s * S::WK * kOne + r * S::kTok + c;
      float v = 0.0f, u = 0.0f;
#pragma unroll
      for (int w = 0; w < S::WK; ++w) {
        v += at[w * kOne];
        if (NW == 2) u += at[w * kOne + kOne / 2];
      }
      put(r, c, (int64_t)(first + (last - used + 1 + s) * stride) * S::kRows, v, u);
    }
    __syncthreads();
  };

  float total[2][NT][4] = {};
  int tile = 0, left = per_tile, slot = 0;
  const auto flush = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = (i / R) * S::kRows + (wr * R + i % R) * 16 + h * 8 + g;
          *reinterpret_cast<float2*>(red + (slot * S::WK + wk) * kOne + row * S::kTok + q * 8 + 2 * t) =
              make_float2(total[i][q][2 * h], total[i][q][2 * h + 1]);
          total[i][q][2 * h] = total[i][q][2 * h + 1] = 0.0f;
        }
    if (++slot == S::kSlots || tile + 1 == mine) {
      join(tile, slot);
      slot = 0;
    }
    ++tile;
    left = per_tile;
  };

  const int work = per_tile * mine;
  if (work) rows_of(0);
  pdl_trigger();
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < work) fetch(d);
  // Planes may be the previous kernel's output; the weights, which come through the
  // read-only path, are not.  No load of a plane moves above this: its address is
  // known here.
  pdl_wait();
  if (TERMS) {
#pragma unroll
    for (int q = 0; q < NT; ++q) asm volatile("" : "+l"(xp[q])::"memory");
  }
  int kb = start;
  for (int it = 0; it < work; it += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (it + d >= work) break;
      uint32_t bias[2][2];
      float scale[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bias[i][h] = !DBL && affine ? w4_bias(zp[d][i][h]) : 0x43084308u;
          // two-level: within an ulp of (q / 255) * super
          scale[i][h] = DBL ? (float)sc[d][i][h] * (1.0f / 255.0f) * sup[d][i][h]
                            : __uint_as_float(sc[d][i][h]);
        }
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        const int k = kb * KB + s * 32 * CH;
        const bool in = k + t * 8 * CH < cols;
        const uint4* xs[NT][kTerms];
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int m = 0; m < kTerms; ++m)
            xs[q][m] = in ? reinterpret_cast<const uint4*>(xp[q] + m * p.x_plane + k) : kZeros;
        // this part's parameters, from the lane that has them
        uint32_t bs[2][2];
        float ss[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            bs[i][h] = bias[i][h];
            ss[i][h] = scale[i][h];
            if (SUB > 1) {
              ss[i][h] = __shfl_sync(~0u, ss[i][h], s, 4);
              if (!DBL && affine) bs[i][h] = __shfl_sync(~0u, bs[i][h], s, 4);
            }
          }
        float part[2][NT][4];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          uint4 b[NT][kTerms];
#pragma unroll
          for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int m = 0; m < kTerms; ++m) b[q][m] = x_pairs<TERMS != 0>(ld_x<TERMS != 0>(xs[q][m] + j));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                a[h][e] = w4_pair(code[d][i][h].v[s * CH + j] >> (4 * e), bs[i][h]);
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
              for (int m = kTerms - 1; m >= 0; --m) {
                if (j == 0 && m == kTerms - 1)
                  mma_16816_first(part[i][q], a[0][0], a[1][0], a[0][1], a[1][1], b[q][m].x, b[q][m].y);
                else
                  mma_16816(part[i][q], a[0][0], a[1][0], a[0][1], a[1][1], b[q][m].x, b[q][m].y);
                mma_16816(part[i][q], a[0][2], a[1][2], a[0][3], a[1][3], b[q][m].z, b[q][m].w);
              }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              total[i][q][e] = fmaf(part[i][q][e], ss[i][e >> 1], total[i][q][e]);
      }
      if (it + d + D < work) fetch(d);
      kb += step;
      if (--left == 0) {
        kb = start;
        flush();
      }
    }
  }
  if (!work)  // more warps than blocks of k: nothing to add, but the joins to make
    while (tile < mine) flush();
}

// x [tokens, cols] as planes (cols a multiple of 8): a thread takes 8 elements.
template <typename T>
__global__ void __launch_bounds__(256) k_w4_planes(const void* x, int64_t total, int terms,
                                                   int64_t plane, __nv_bfloat16* out) {
  pdl_trigger();
  pdl_wait();
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= total) return;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = ld_elem<T>(x, i + e);
  for (int q = 0; q < terms; ++q) {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = take_bf16(v[e]);
    *reinterpret_cast<uint4*>(out + q * plane + i) =
        make_uint4(pack_bf16x2(h[1], h[5]), pack_bf16x2(h[0], h[4]), pack_bf16x2(h[3], h[7]),
                   pack_bf16x2(h[2], h[6]));
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static cudaError_t launch_w4_kernel(void (*k)(W4Args), dim3 grid, int smem, int cluster, bool pdl,
                                    const W4Args& p, cudaStream_t s) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return e;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kW4Warps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, p);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

template <int TERMS, int CH, bool DBL, int NT, int NW>
static qat_status launch_fast(W4Args p, bool pdl, cudaStream_t s) {
  using S = W4Shape<NT, NW>;
  p.tiles = (int)((p.rows + S::kRows - 1) / S::kRows);
  const int kblocks = (p.cols + kW4Block - 1) / kW4Block;
  // the unit of part j of a row is j / d, as (2 j + 1) ceil(2^31 / d) >> 32 (exact
  // while 2 j d < 2^31); rows that are one unit: 0
  const int64_t d = p.unit / (32 * CH);
  p.unit_magic = p.unit >= p.cols ? 0u : (uint32_t)(((INT64_C(1) << 31) + d - 1) / d);
  const int room = device_info().sms;
  // a cluster splits k while the GPU has room and every warp keeps a block
  p.split = 1;
  while (p.split < 8 && p.tiles * p.split * 2 <= room && kblocks >= p.split * 2 * S::WK)
    p.split *= 2;
  const unsigned blocks = (unsigned)(p.split > 1 ? p.tiles * p.split : p.tiles < room ? p.tiles : room);
  const dim3 grid(blocks, (unsigned)((p.tokens + S::kTok - 1) / S::kTok));
  if (launch_w4_kernel(k_w4<TERMS, CH, DBL, NT, NW>, grid, S::kSmem, p.split, pdl, p, s) != cudaSuccess)
    return QAT_ERR_CUDA;
  count_launch(1);
  return QAT_OK;
}
template <int TERMS, int CH, bool DBL, int NW>
static qat_status fast_tokens(const W4Args& p, bool pdl, cudaStream_t s) {
  if (p.tokens <= 8) return launch_fast<TERMS, CH, DBL, 1, NW>(p, pdl, s);
  if (p.tokens <= 16) return launch_fast<TERMS, CH, DBL, 2, NW>(p, pdl, s);
  return launch_fast<TERMS, CH, DBL, 4, NW>(p, pdl, s);
}
template <int TERMS, int NW>
static qat_status fast_chunk(const W4Args& p, int ch, bool pdl, cudaStream_t s) {
  if (p.dbl) return fast_tokens<TERMS, 2, true, NW>(p, pdl, s);
  if (ch == 4) return fast_tokens<TERMS, 4, false, NW>(p, pdl, s);
  if (ch == 2) return fast_tokens<TERMS, 2, false, NW>(p, pdl, s);
  return fast_tokens<TERMS, 1, false, NW>(p, pdl, s);
}

// Words of 8 codes a lane takes at once: the widest load that rows, units and
// blocks of k allow; 0 when the shape needs the generic kernel (rows longer and
// weights larger than the 32-bit offsets reach too).
static int w4_chunk(const qat_weight4& w) {
  if (w.cols <= 0 || w.cols % 8 || w.cols > (1 << 19) || w.rows > (1 << 28) ||
      w.rows * w.cols >= (INT64_C(1) << 32))
    return 0;
  if (w.layout == QAT_PER_TENSOR || w.layout == QAT_PER_ROW)
    return w.cols % 32 == 0 ? 4 : w.cols % 16 == 0 ? 2 : 1;
  const int64_t unit = w.layout == QAT_W4_DOUBLE ? 64 : w.group;
  if (w.layout == QAT_W4_DOUBLE && w.cols % 64) return 0;
  return unit % 128 == 0 ? 4 : unit % 64 == 0 ? 2 : unit % 32 == 0 ? 1 : 0;
}

// A product's x: its type's rows, or planes of `terms` parts.
struct X4 {
  const void* p;
  qat_dtype dt;
  int terms;  // 0: rows
  int64_t pitch, plane;
};
// Its y, likewise (planes only from the gated pair).
struct Y4 {
  void* p;
  qat_dtype dt;
  int terms;
  int64_t pitch, plane;
};

static qat_status run_fast(const X4& x, int64_t tokens, const qat_weight4* w, int nw, int act,
                           const Y4& y, int ch, bool pdl, cudaStream_t s) {
  W4Args p = {};
  for (int i = 0; i < nw; ++i)
    p.w[i] = W4Fast{static_cast<const uint8_t*>(w[i].codes), w[i].scales, w[i].zero_points,
                    w[i].super_scales};
  p.x = x.p;
  p.x_pitch = x.terms ? x.pitch : w->cols;
  p.x_plane = x.plane;
  p.y = y.p;
  p.y_pitch = y.pitch;
  p.y_plane = y.plane;
  p.y_terms = y.terms;
  p.out = y.terms ? kOutPlanes : y.dt == QAT_BF16 ? kOutBf16 : kOutF32;
  p.rows = w->rows;
  p.cols = (int)w->cols;
  p.tokens = tokens;
  p.dbl = w->layout == QAT_W4_DOUBLE;
  p.unit = w->layout == QAT_PER_GROUP ? w->group : p.dbl ? 64 : w->cols;
  p.row_units = w->layout == QAT_PER_TENSOR ? 0 : w->cols / p.unit;
  p.act = act;
  if (nw == 2)
    return x.terms == 0 ? fast_chunk<0, 2>(p, ch, pdl, s) : fast_chunk<3, 2>(p, ch, pdl, s);
  return x.terms == 0   ? fast_chunk<0, 1>(p, ch, pdl, s)
         : x.terms == 2 ? fast_chunk<2, 1>(p, ch, pdl, s)
                        : fast_chunk<3, 1>(p, ch, pdl, s);
}

static W4 w4_of(const qat_weight4& w) {
  W4 r;
  r.codes = static_cast<const uint8_t*>(w.codes);
  r.scales = w.scales;
  r.zp = w.zero_points;
  r.super = w.super_scales;
  r.unit = w.layout == QAT_W4_DOUBLE      ? 64
           : w.layout == QAT_PER_GROUP    ? w.group
           : w.layout == QAT_PER_ROW      ? w.cols
                                          : w.rows * w.cols;
  if (r.unit <= 0) r.unit = 1;
  return r;
}

static qat_status run_generic(const void* x, qat_dtype xdt, int64_t tokens, const qat_weight4* w,
                              int nw, int act, void* y, qat_dtype ydt, bool pdl, cudaStream_t s) {
  const W4 a = w4_of(w[0]), b = w4_of(w[nw - 1]);
  const bool dbl = w->layout == QAT_W4_DOUBLE;
  // gridDim.y holds 65535 token tiles: longer inputs in several launches
  constexpr int64_t kMost = (int64_t)65535 * kGenTokens;
  for (int64_t t0 = 0; t0 < tokens; t0 += kMost) {
    const int64_t nt = tokens - t0 < kMost ? tokens - t0 : kMost;
    const dim3 grid((unsigned)((w->rows + 3) / 4), (unsigned)((nt + kGenTokens - 1) / kGenTokens));
    const void* xp = static_cast<const char*>(x) + t0 * w->cols * (xdt == QAT_F32 ? 4 : 2);
    void* yp = static_cast<char*>(y) + t0 * w->rows * (ydt == QAT_F32 ? 4 : 2);
    const int yb = ydt == QAT_BF16;
    const auto go = [&](auto kernel) {
      return launch_kernel(kernel, grid, dim3(128), 0, s, pdl || t0 > 0, xp, nt, a, b, w->rows,
                           w->cols, act, yp, yb);
    };
    cudaError_t e;
    if (xdt == QAT_F32)
      e = nw == 2 ? (dbl ? go(k_w4_generic<F32, true, 2>) : go(k_w4_generic<F32, false, 2>))
                  : (dbl ? go(k_w4_generic<F32, true, 1>) : go(k_w4_generic<F32, false, 1>));
    else
      e = nw == 2 ? (dbl ? go(k_w4_generic<BF16, true, 2>) : go(k_w4_generic<BF16, false, 2>))
                  : (dbl ? go(k_w4_generic<BF16, true, 1>) : go(k_w4_generic<BF16, false, 1>));
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return QAT_ERR_CUDA;
    }
    count_launch(1);
  }
  return QAT_OK;
}

// Tokens of a launch of the fast kernel at most (gridDim.y).
constexpr int64_t kFastTokens = (int64_t)65535 * 8;
static bool fast_ok(const qat_weight4& w, int64_t tokens) {
  return w4_chunk(w) != 0 && tokens <= kFastTokens;
}

// Planes x is taken as: none where bf16 rows can be read as they are (others
// come as three of which two are zero: one kernel less for a rare case)
static int x_terms(const void* x, qat_dtype dt, qat_dtype ydt) {
  if (dt == QAT_BF16) return reinterpret_cast<uintptr_t>(x) % 16 == 0 ? 0 : 3;
  return ydt == QAT_BF16 ? 2 : 3;
}
static int64_t plane_of(int64_t tokens, int64_t pitch) { return (tokens * pitch + 7) / 8 * 8; }

static qat_status make_planes(const void* x, qat_dtype dt, int64_t tokens, int64_t cols, int terms,
                              void* out, bool pdl, X4* r, cudaStream_t s) {
  *r = X4{out, QAT_BF16, terms, cols, plane_of(tokens, cols)};
  const int64_t total = tokens * cols;
  const dim3 grid((unsigned)((total / 8 + 255) / 256));
  auto* o = static_cast<__nv_bfloat16*>(out);
  const cudaError_t e =
      dt == QAT_F32
          ? launch_kernel(k_w4_planes<F32>, grid, dim3(256), 0, s, pdl, x, total, terms, r->plane, o)
          : launch_kernel(k_w4_planes<BF16>, grid, dim3(256), 0, s, pdl, x, total, terms, r->plane, o);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return QAT_ERR_CUDA;
  }
  count_launch(1);
  return QAT_OK;
}

// y = act(x W0^T) * (x W1^T) (nw = 2) or x W^T; `planes` is room for x's planes.
// *launched: a kernel of this call ran before.
static qat_status product(const void* x, qat_dtype dt, int64_t tokens, const qat_weight4* w, int nw,
                          int act, const Y4& y, void* planes, bool* launched, cudaStream_t s) {
  const int ch = w4_chunk(*w);
  if (!fast_ok(*w, tokens)) {
    const bool pdl = *launched;
    *launched = true;
    return run_generic(x, dt, tokens, w, nw, act, y.p, y.dt, pdl, s);
  }
  // the gated pair's sums go through act, and its planes hold what y needs
  const int terms = x_terms(x, dt, nw == 2 ? QAT_F32 : y.dt);
  X4 xv = {x, dt, 0, 0, 0};
  if (terms) {
    const qat_status st = make_planes(x, dt, tokens, w->cols, terms, planes, *launched, &xv, s);
    if (st) return st;
    *launched = true;
  }
  const bool pdl = *launched;
  *launched = true;
  return run_fast(xv, tokens, w, nw, act, y, ch, pdl, s);
}

static size_t r256(size_t b) { return (b + 255) / 256 * 256; }
static size_t planes_bytes(int64_t tokens, int64_t cols, int terms) {
  return r256((size_t)plane_of(tokens, (cols + 7) / 8 * 8) * terms * 2);
}

size_t linear4_ws_bytes(const void* x, qat_dtype dt, int64_t tokens, int64_t cols) {
  if (x && x_terms(x, dt, dt) == 0) return 0;
  return planes_bytes(tokens, cols, 3);
}
qat_status launch_linear4(const void* x, qat_dtype dt, int64_t tokens, const qat_weight4& w, void* y,
                          void* ws, cudaStream_t s) {
  bool launched = false;
  return product(x, dt, tokens, &w, 1, 0, Y4{y, dt, 0, 0, 0}, ws, &launched, s);
}

// workspace: x's planes, then h (float, or its planes), then planes of a float h
size_t gated4_ws_bytes(int64_t tokens, int64_t dim, int64_t hidden) {
  return planes_bytes(tokens, dim, 3) +
         r256((size_t)tokens * hidden * 4) + planes_bytes(tokens, hidden, 3);
}
qat_status launch_gated4(const void* x, qat_dtype dt, int64_t tokens, const qat_weight4* gate_up,
                         const qat_weight4& down, int act, void* y, void* ws, cudaStream_t s) {
  const int64_t dim = gate_up->cols, hidden = gate_up->rows;
  char* base = static_cast<char*>(ws);
  char* h = base + planes_bytes(tokens, dim, 3);
  char* h_planes = h + r256((size_t)tokens * hidden * 4);
  bool launched = false;
  // no hidden values: the second product is an empty sum, the first has no rows to launch
  if (hidden == 0)
    return product(h, QAT_F32, tokens, &down, 1, 0, Y4{y, dt, 0, 0, 0}, h_planes, &launched, s);
  if (fast_ok(*gate_up, tokens) && fast_ok(down, tokens)) {
    // h straight as the second product's planes
    const int terms = dt == QAT_BF16 ? 2 : 3;
    const Y4 hy = {h_planes, QAT_F32, terms, hidden, plane_of(tokens, hidden)};
    const qat_status st = product(x, dt, tokens, gate_up, 2, act, hy, base, &launched, s);
    if (st) return st;
    return run_fast(X4{h_planes, QAT_BF16, terms, hy.pitch, hy.plane}, tokens, &down, 1, 0,
                    Y4{y, dt, 0, 0, 0}, w4_chunk(down), true, s);
  }
  const qat_status st =
      product(x, dt, tokens, gate_up, 2, act, Y4{h, QAT_F32, 0, 0, 0}, base, &launched, s);
  if (st) return st;
  return product(h, QAT_F32, tokens, &down, 1, 0, Y4{y, dt, 0, 0, 0}, h_planes, &launched, s);
}

}  // namespace qat
