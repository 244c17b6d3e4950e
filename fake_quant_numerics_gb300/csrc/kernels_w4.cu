// kernels_w4.cu -- products of a few tokens with 4-bit weights.
//
//   y[t, n] = sum_u s[n, u] * sum_{k in u} (q[n, k] - z[n, u]) * x[t, k]
//
// and the gated pair h = act(x gate^T) * (x up^T).  Bound by reading the codes
// (rows * cols / 2 bytes and the parameters) while the tokens are few.
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
    z = w.zp ? (float)min(max(w.zp[u], -8), 7) : 0.0f;
  }
}

constexpr int kGenTokens = 8;  // tokens a generic block keeps

// Any shape: a warp per output row, lanes along k, one element at a time.
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
__global__ void __launch_bounds__(128) k_w4_generic(const void* __restrict__ x, int64_t tokens,
                                                    W4 wa, W4 wb, int64_t rows, int64_t cols,
                                                    int act, void* __restrict__ y, int y_bf16) {
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
    const float v = NW == 2 ? act_value(act, a[t]) * b[t] : a[t];
    if (y_bf16)
      st_elem<BF16>(y, (t0 + t) * rows + n, v);
    else
      st_elem<F32>(y, (t0 + t) * rows + n, v);
  }
}

// ---------------------------------------------------------------------------
// Rows of whole 8-code words whose units are whole runs of 32 codes.
//
// A warp multiplies 16 rows (of each of R row tiles and NW weights) by 8 NT
// tokens with m16n8k16 tensor-core products: a code is exact in bf16 (128 + q
// with the low mantissa bits, one logic operation for two codes, then an exact
// subtraction of 136 + zero point), so is a bf16 x, and the sums are binary32.
// Arithmetic per code is then about 1.4 instructions, which keeps reading the
// codes the bound; scalar multiply-adds would need four.  A float x is split
// into TERMS bf16 values (high, middle, low: 3 hold all its 24 bits, 2 hold 16,
// enough under a bf16 output), one product each.
//
// k runs in blocks of 32 CH codes: lane t of a row's four takes 8 CH
// consecutive codes (one load), so a load instruction covers 16 CH bytes of
// each of 8 rows.  The order of k inside a block is the codes' bit order, the
// same for both operands.  The block's 8 warps take blocks in turn, the CTAs of
// a cluster split them once more where rows are few; partial sums are added in
// shared memory, then over the cluster in rank order.
// ---------------------------------------------------------------------------
constexpr int kW4Warps = 8;

struct W4Fast {
  const uint8_t* codes;
  const void* scales;
  const int32_t* zp;
  const float* super;
};
struct W4Args {
  W4Fast w[2];
  const void* x;
  void* y;
  int64_t rows, tokens;
  int64_t row_units;  // units from one row to the next
  int64_t unit;       // codes of a unit
  int cols;
  uint32_t unit_magic;
  int dbl, act, y_bf16, vec_x, split;
};

// two codes of a word (bits 0-3 and 16-19 after the shift) as bf16 q - zp
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t bias) {
  uint32_t v;
  // (w & 0x000f000f) ^ 0x43084308: bf16 128 + (q + 8)
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43084308, 0x6a;" : "=r"(v) : "r"(w));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(v), "r"(bias));
  return v;
}

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

// x of 8 consecutive k as bf16 pairs in the codes' order (1,5) (0,4) (3,7) (2,6)
__device__ __forceinline__ void pairs_bf16(const uint4& v, uint32_t (&b)[4]) {
  b[0] = __byte_perm(v.x, v.z, 0x7632);
  b[1] = __byte_perm(v.x, v.z, 0x5410);
  b[2] = __byte_perm(v.y, v.w, 0x7632);
  b[3] = __byte_perm(v.y, v.w, 0x5410);
}
// the bf16 terms of one float, in the high halves
template <int TERMS>
__device__ __forceinline__ void split_f32(float x, uint32_t (&h)[TERMS]) {
#pragma unroll
  for (int i = 0; i < TERMS; ++i) h[i] = __float_as_uint(take_bf16(x));
}

template <typename T, int CH>
struct XWords {
  uint32_t v[CH * (T::BYTES == 2 ? 4 : 8)];
};
// a lane's x of 8 CH consecutive k of one token (zeros where there is none)
template <typename T, int CH>
__device__ __forceinline__ void load_x(XWords<T, CH>& o, const char* p, bool in, bool vec) {
  constexpr int W = CH * (T::BYTES == 2 ? 4 : 8);
#pragma unroll
  for (int i = 0; i < W; ++i) o.v[i] = 0u;
  if (!in) return;
  if (vec) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
      o.v[i] = q.x, o.v[i + 1] = q.y, o.v[i + 2] = q.z, o.v[i + 3] = q.w;
    }
  } else if (T::BYTES == 4) {
#pragma unroll
    for (int i = 0; i < W; ++i) o.v[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
  } else {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < W; ++i)
      o.v[i] = (uint32_t)__ldg(q + 2 * i) | (uint32_t)__ldg(q + 2 * i + 1) << 16;
  }
}
// the B registers of word j, TERMS sets of four pairs
template <typename T, int TERMS, int CH>
__device__ __forceinline__ void x_pairs(const XWords<T, CH>& x, int j, uint32_t (&b)[TERMS][4]) {
  if constexpr (T::BYTES == 2) {
    pairs_bf16(make_uint4(x.v[j * 4], x.v[j * 4 + 1], x.v[j * 4 + 2], x.v[j * 4 + 3]), b[0]);
  } else {
    uint32_t h[8][TERMS];
#pragma unroll
    for (int i = 0; i < 8; ++i) split_f32<TERMS>(__uint_as_float(x.v[j * 8 + i]), h[i]);
    constexpr int lo[4] = {1, 0, 3, 2};
#pragma unroll
    for (int q = 0; q < TERMS; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) b[q][i] = __byte_perm(h[lo[i]][q], h[lo[i] + 4][q], 0x7632);
  }
}

template <int CH>
struct CodeWords {
  uint32_t v[CH];
};
template <int CH>
__device__ __forceinline__ void load_codes(CodeWords<CH>& o, const uint8_t* p, bool in) {
  if constexpr (CH == 4) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (in) q = __ldcs(reinterpret_cast<const uint4*>(p));
    o.v[0] = q.x, o.v[1] = q.y, o.v[2] = q.z, o.v[3] = q.w;
  } else if constexpr (CH == 2) {
    uint2 q = make_uint2(0, 0);
    if (in) q = __ldcs(reinterpret_cast<const uint2*>(p));
    o.v[0] = q.x, o.v[1] = q.y;
  } else {
    o.v[0] = in ? __ldcs(reinterpret_cast<const uint32_t*>(p)) : 0u;
  }
}

// 136 + zp as a bf16 pair (exact)
__device__ __forceinline__ uint32_t w4_bias(int zp) {
  const uint32_t h = 0x4308u + (uint32_t)min(max(zp, -8), 7);
  return h | h << 16;
}

// Row tiles of a warp and the warps that share a block of k: with more tokens
// the warps of a CTA sit side by side along the rows, so that they read the
// same x from L1.
template <int NT, int NW>
struct W4Shape {
  static constexpr int R = NW == 2 && NT == 4 ? 1 : 2;  // row tiles of each weight
  static constexpr int RT = R * NW;
  static constexpr int WR = NT;              // warps along the rows
  static constexpr int WK = kW4Warps / WR;   // warps along k
  static constexpr int kRows = 16 * R * WR;  // output rows of a CTA
};

template <typename T, int TERMS, int CH, int NT, int NW>
__global__ void __launch_bounds__(kW4Warps * 32, NT == 1 && NW == 1 ? 2 : 1)
    k_w4(const __grid_constant__ W4Args p) {
  using S = W4Shape<NT, NW>;
  constexpr int R = S::R, RT = S::RT, kTok = 8 * NT, KB = 32 * CH;
  __shared__ float red[S::WK][NW][S::kRows][kTok];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wr = warp % S::WR, wk = warp / S::WR;
  const int split = p.split;
  const int rank = split > 1 ? (int)(blockIdx.x % split) : 0;
  const int64_t n0 = (int64_t)(blockIdx.x / split) * S::kRows;
  const int64_t tok0 = (int64_t)blockIdx.y * kTok;
  const int cols = p.cols, blocks = (cols + KB - 1) / KB, step = S::WK * split;
  const bool vec_x = p.vec_x;

  // this lane's rows: g and g + 8 of each tile (rows past the end read row 0
  // and are dropped at the end)
  const uint8_t* cp[RT][2];
  uint32_t ru[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = n0 + (wr * R + r) * 16 + h * 8 + g, m = n < p.rows ? n : 0;
      ru[r][h] = (uint32_t)(m * p.row_units);
#pragma unroll
      for (int w = 0; w < NW; ++w) cp[w * R + r][h] = p.w[w].codes + ((m * cols) >> 1) + t * 4 * CH;
    }
  const char* xp[NT];
  bool xin[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int64_t tok = tok0 + q * 8 + g;
    xin[q] = tok < p.tokens;
    xp[q] = static_cast<const char*>(p.x) + ((xin[q] ? tok : 0) * cols + t * 8 * CH) * T::BYTES;
  }

  float total[RT][NT][4] = {};
  CodeWords<CH> next[RT][2];
  const auto fetch = [&](int kb) {
    const bool in = kb * KB + t * 8 * CH < cols;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) load_codes<CH>(next[i][h], cp[i][h] + kb * (KB / 2), in);
  };
  int kb = rank * S::WK + wk;
  fetch(kb);
#pragma unroll 1
  for (; kb < blocks; kb += step) {
    CodeWords<CH> now[RT][2];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) now[i][h] = next[i][h];
    const bool in = kb * KB + t * 8 * CH < cols;
    XWords<T, CH> xw[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q)
      load_x<T, CH>(xw[q], xp[q] + (int64_t)kb * (KB * T::BYTES), in && xin[q], vec_x);
    fetch(kb + step);
    const uint32_t u = p.unit_magic ? __umulhi((uint32_t)kb, p.unit_magic) : 0u;
    float sc[RT][2];
    uint32_t bias[RT][2];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const W4Fast& w = p.w[i / R];
        const uint32_t at = ru[i % R][h] + (p.unit_magic == 1 ? (uint32_t)kb : u);
        if (p.dbl)  // within an ulp of (q / 255) * super
          sc[i][h] = (float)__ldg(static_cast<const uint8_t*>(w.scales) + at) * (1.0f / 255.0f) *
                     __ldg(w.super + (at >> 8));
        else
          sc[i][h] = __ldg(static_cast<const float*>(w.scales) + at);
        bias[i][h] = w.zp ? w4_bias(__ldg(w.zp + at)) : 0x43084308u;
      }
    float part[RT][NT][4];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      uint32_t b[NT][TERMS][4];
#pragma unroll
      for (int q = 0; q < NT; ++q) x_pairs<T, TERMS, CH>(xw[q], j, b[q]);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        uint32_t a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) a[h][e] = w4_pair(now[i][h].v[j] >> (4 * e), bias[i][h]);
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int m = TERMS - 1; m >= 0; --m) {
            if (j == 0 && m == TERMS - 1)
              mma_16816_first(part[i][q], a[0][0], a[1][0], a[0][1], a[1][1], b[q][m][0], b[q][m][1]);
            else
              mma_16816(part[i][q], a[0][0], a[1][0], a[0][1], a[1][1], b[q][m][0], b[q][m][1]);
            mma_16816(part[i][q], a[0][2], a[1][2], a[0][3], a[1][3], b[q][m][2], b[q][m][3]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          total[i][q][e] = fmaf(part[i][q][e], sc[i][e >> 1], total[i][q][e]);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(
            &red[wk][i / R][(wr * R + i % R) * 16 + h * 8 + g][q * 8 + 2 * t]) =
            make_float2(total[i][q][2 * h], total[i][q][2 * h + 1]);
  __syncthreads();
  const int tokens = (int)min((int64_t)kTok, p.tokens - tok0);
  // this CTA's sums over its warps, in red[0]
  for (int i = threadIdx.x; i < NW * S::kRows * tokens; i += kW4Warps * 32) {
    const int r = i % (NW * S::kRows), c = i / (NW * S::kRows);
    float* at = &red[0][0][r][c];
    float v = *at;
#pragma unroll
    for (int w = 1; w < S::WK; ++w) v += at[w * NW * S::kRows * kTok];
    *at = v;
  }
  if (split > 1)
    tc::cluster_sync();
  else
    __syncthreads();
  for (int i = threadIdx.x + rank * kW4Warps * 32; i < S::kRows * tokens;
       i += kW4Warps * 32 * split) {
    const int r = i % S::kRows, c = i / S::kRows;
    if (n0 + r >= p.rows) continue;
    float v = 0.0f, u = 0.0f;
    if (split > 1) {
      for (int q = 0; q < split; ++q) {
        v += tc::ld_cluster(tc::map_rank(tc::smem(&red[0][0][r][c]), q));
        if (NW == 2) u += tc::ld_cluster(tc::map_rank(tc::smem(&red[0][NW - 1][r][c]), q));
      }
    } else {
      v = red[0][0][r][c];
      if (NW == 2) u = red[0][NW - 1][r][c];
    }
    if (NW == 2) v = act_value(p.act, v) * u;
    const int64_t at = (tok0 + c) * p.rows + n0 + r;
    if (p.y_bf16)
      st_elem<BF16>(p.y, at, v);
    else
      st_elem<F32>(p.y, at, v);
  }
  if (split > 1) tc::cluster_sync();  // the other CTAs have read red
}

template <typename T, int TERMS, int CH, int NT, int NW>
static qat_status launch_fast(W4Args p, cudaStream_t s) {
  using S = W4Shape<NT, NW>;
  const int64_t row_blocks = (p.rows + S::kRows - 1) / S::kRows;
  const int kblocks = (p.cols + 32 * CH - 1) / (32 * CH);
  // units of a row: none (whole rows), one a block, or kb / per_unit by
  // multiplication (exact while blocks^2 < 2^32)
  const int64_t per_unit = p.unit / (32 * CH);
  p.unit_magic = p.unit >= p.cols ? 0u
                 : per_unit == 1  ? 1u
                                  : (uint32_t)((UINT64_C(1) << 32) / per_unit + 1);
  // a cluster splits k while two CTAs a SM are not reached and every warp keeps
  // a block
  p.split = 1;
  const int64_t room = (int64_t)device_info().sms * 2;
  while (p.split < 8 && row_blocks * p.split * 2 <= room && kblocks >= p.split * 2 * S::WK)
    p.split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(row_blocks * p.split), (unsigned)((p.tokens + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3(kW4Warps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_w4<T, TERMS, CH, NT, NW>, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return QAT_ERR_CUDA;
  }
  count_launch(1);
  return QAT_OK;
}
template <typename T, int TERMS, int CH, int NW>
static qat_status fast_tokens(const W4Args& p, cudaStream_t s) {
  if (p.tokens <= 8) return launch_fast<T, TERMS, CH, 1, NW>(p, s);
  if (p.tokens <= 16) return launch_fast<T, TERMS, CH, 2, NW>(p, s);
  return launch_fast<T, TERMS, CH, 4, NW>(p, s);
}
template <typename T, int TERMS, int NW>
static qat_status fast_chunk(const W4Args& p, int ch, cudaStream_t s) {
  if (ch == 4) return fast_tokens<T, TERMS, 4, NW>(p, s);
  if (ch == 2) return fast_tokens<T, TERMS, 2, NW>(p, s);
  return fast_tokens<T, TERMS, 1, NW>(p, s);
}

// Words of 8 codes a lane takes at once: the widest load that rows, units and
// blocks of k allow; 0 when the shape needs the generic kernel (longer rows and
// more units than the 32-bit indexes hold too).
static int w4_chunk(const qat_weight4& w) {
  if (w.cols % 8 || w.cols > (1 << 20) || w.rows > (1 << 30)) return 0;
  if (w.layout != QAT_PER_TENSOR && w.layout != QAT_PER_ROW && w.rows * w.cols >= (INT64_C(1) << 36))
    return 0;
  if (w.layout == QAT_PER_TENSOR || w.layout == QAT_PER_ROW)
    return w.cols % 32 == 0 ? 4 : w.cols % 16 == 0 ? 2 : 1;
  const int64_t unit = w.layout == QAT_W4_DOUBLE ? 64 : w.group;
  if (w.layout == QAT_W4_DOUBLE && w.cols % 64) return 0;
  return unit % 128 == 0 ? 4 : unit % 64 == 0 ? 2 : unit % 32 == 0 ? 1 : 0;
}

static qat_status launch_w4_fast(const void* x, qat_dtype xdt, int64_t tokens,
                                 const qat_weight4* w, int nw, int act, void* y, qat_dtype ydt,
                                 int ch, cudaStream_t s) {
  W4Args p = {};
  for (int i = 0; i < nw; ++i)
    p.w[i] = W4Fast{static_cast<const uint8_t*>(w[i].codes), w[i].scales, w[i].zero_points,
                    w[i].super_scales};
  p.x = x;
  p.y = y;
  p.rows = w->rows;
  p.cols = (int)w->cols;
  p.tokens = tokens;
  p.vec_x = w->cols % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  p.dbl = w->layout == QAT_W4_DOUBLE;
  p.unit = w->layout == QAT_PER_GROUP ? w->group : p.dbl ? 64 : w->cols;
  p.row_units = w->layout == QAT_PER_TENSOR ? 0 : w->cols / p.unit;
  p.act = act;
  p.y_bf16 = ydt == QAT_BF16;
  if (xdt == QAT_BF16)
    return nw == 2 ? fast_chunk<BF16, 1, 2>(p, ch, s) : fast_chunk<BF16, 1, 1>(p, ch, s);
  if (nw == 2) return fast_chunk<F32, 3, 2>(p, ch, s);
  return p.y_bf16 ? fast_chunk<F32, 2, 1>(p, ch, s) : fast_chunk<F32, 3, 1>(p, ch, s);
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

qat_status launch_w4(const void* x, qat_dtype xdt, int64_t tokens, const qat_weight4* w, int nw,
                     int act, void* y, qat_dtype ydt, cudaStream_t s) {
  const W4 a = w4_of(w[0]), b = w4_of(w[nw - 1]);
  const bool dbl = w->layout == QAT_W4_DOUBLE;
  const int ch = w->cols > 0 && tokens <= 65535 * 8 ? w4_chunk(*w) : 0;
  if (ch) return launch_w4_fast(x, xdt, tokens, w, nw, act, y, ydt, ch, s);
  // gridDim.y holds 65535 token tiles: longer inputs in several launches
  constexpr int64_t kMost = (int64_t)65535 * kGenTokens;
  for (int64_t t0 = 0; t0 < tokens; t0 += kMost) {
    const int64_t nt = tokens - t0 < kMost ? tokens - t0 : kMost;
    const dim3 grid((unsigned)((w->rows + 3) / 4), (unsigned)((nt + kGenTokens - 1) / kGenTokens));
    const char* xp = static_cast<const char*>(x) + t0 * w->cols * (xdt == QAT_F32 ? 4 : 2);
    char* yp = static_cast<char*>(y) + t0 * w->rows * (ydt == QAT_F32 ? 4 : 2);
    const int yb = ydt == QAT_BF16;
#define QAT_W4_GO(T, D, N) \
  k_w4_generic<T, D, N><<<grid, 128, 0, s>>>(xp, nt, a, b, w->rows, w->cols, act, yp, yb)
#define QAT_W4_D(T, D) (nw == 2 ? QAT_W4_GO(T, D, 2) : QAT_W4_GO(T, D, 1))
    if (xdt == QAT_F32) {
      if (dbl) QAT_W4_D(F32, true); else QAT_W4_D(F32, false);
    } else {
      if (dbl) QAT_W4_D(BF16, true); else QAT_W4_D(BF16, false);
    }
#undef QAT_W4_D
#undef QAT_W4_GO
    count_launch(1);
  }
  return launch_status();
}

}  // namespace qat
