// kernels_w4.cu -- products of a few tokens with 4-bit weights.
//
//   y[t, n] = sum_u s[n, u] * sum_{k in u} (q[n, k] - z[n, u]) * x[t, k]
//
// and the gated pair h = act(x gate^T) * (x up^T).  Bound by reading the codes
// (rows * cols / 2 bytes and the parameters) while the tokens are few.
#include "qat_layer.cuh"
#include "qat_layer.h"

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
