// kernels_norm.cu -- layer norm, forward and backward.
//
//   z = (x - mean) * rstd,  y = z * w + b
//   p = dy * w;  dx = rstd * (p - mean(p) - z * mean(p * z))
//   dw = sum_rows dy * z,  db = sum_rows dy
//
// Every kernel is bound by reading its rows.  Sums are binary32 trees around
// the mean; dw and db are added over the rows in a fixed order.
#include "qat_layer.cuh"
#include "qat_layer.h"

namespace qat {

constexpr int kRowThreads = 512;

// sums over a block of kRowThreads threads (red: 2 * 16 floats), to every thread
__device__ __forceinline__ float2 block_sum2(float a, float b, float* red) {
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(~0u, a, o);
    b += __shfl_xor_sync(~0u, b, o);
  }
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  __syncthreads();  // red may still be read from the previous sum
  if (lane == 0) {
    red[wid] = a;
    red[16 + wid] = b;
  }
  __syncthreads();
  a = lane < nw ? red[lane] : 0.0f;
  b = lane < nw ? red[16 + lane] : 0.0f;
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(~0u, a, o);
    b += __shfl_xor_sync(~0u, b, o);
  }
  return make_float2(a, b);
}

// Rows of any length and alignment: a block per row, three passes over it.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    k_norm_fwd_row(const void* __restrict__ x, int64_t rows, int64_t cols,
                   const void* __restrict__ w, const void* __restrict__ b, float eps,
                   void* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[32];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t base = r * cols;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) s += ld_elem<T>(x, base + c);
    const float m = block_sum2(s, 0.0f, red).x / (float)cols;
    float v = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float d = ld_elem<T>(x, base + c) - m;
      v = fmaf(d, d, v);
    }
    const float rs = 1.0f / sqrtf(block_sum2(v, 0.0f, red).x / (float)cols + eps);
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float z = (ld_elem<T>(x, base + c) - m) * rs;
      st_elem<T>(y, base + c, fmaf(z, w ? ld_elem<T>(w, c) : 1.0f, b ? ld_elem<T>(b, c) : 0.0f));
    }
    if (threadIdx.x == 0) {
      if (mean) mean[r] = m;
      if (rstd) rstd[r] = rs;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    k_norm_bwd_row(const void* __restrict__ dy, const void* __restrict__ x, int64_t rows,
                   int64_t cols, const void* __restrict__ w, const float* __restrict__ mean,
                   const float* __restrict__ rstd, void* __restrict__ dx) {
  __shared__ float red[32];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t base = r * cols;
    const float m = mean[r], rs = rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float z = (ld_elem<T>(x, base + c) - m) * rs;
      const float p = ld_elem<T>(dy, base + c) * (w ? ld_elem<T>(w, c) : 1.0f);
      s1 += p;
      s2 = fmaf(p, z, s2);
    }
    const float2 t = block_sum2(s1, s2, red);
    const float c1 = t.x / (float)cols, c2 = t.y / (float)cols;
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float z = (ld_elem<T>(x, base + c) - m) * rs;
      const float p = ld_elem<T>(dy, base + c) * (w ? ld_elem<T>(w, c) : 1.0f);
      st_elem<T>(dx, base + c, rs * (fmaf(-z, c2, p - c1)));
    }
  }
}

// Partial column sums: block (column tile, part) adds rows part, part + parts,
// ...; ws holds [2][parts][cols].
template <typename T>
__global__ void __launch_bounds__(256)
    k_norm_cols(const void* __restrict__ dy, const void* __restrict__ x, int64_t rows,
                int64_t cols, const float* __restrict__ mean, const float* __restrict__ rstd,
                int parts, float* __restrict__ ws) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  float sw = 0.0f, sb = 0.0f;
  for (int64_t r = blockIdx.y; r < rows; r += parts) {
    const float g = ld_elem<T>(dy, r * cols + c);
    sw = fmaf(g, (ld_elem<T>(x, r * cols + c) - mean[r]) * rstd[r], sw);
    sb += g;
  }
  ws[(int64_t)blockIdx.y * cols + c] = sw;
  ws[((int64_t)parts + blockIdx.y) * cols + c] = sb;
}

// The partials' sum, in order of the parts.
template <typename T>
__global__ void __launch_bounds__(256)
    k_norm_cols_join(const float* __restrict__ ws, int parts, int64_t cols, void* __restrict__ dw,
                     void* __restrict__ db) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  float sw = 0.0f, sb = 0.0f;
  for (int p = 0; p < parts; ++p) {
    sw += ws[(int64_t)p * cols + c];
    sb += ws[((int64_t)parts + p) * cols + c];
  }
  if (dw) st_elem<T>(dw, c, sw);
  if (db) st_elem<T>(db, c, sb);
}

template <typename T>
static qat_status norm_fwd(const void* x, int64_t rows, int64_t cols, const void* w, const void* b,
                           float eps, void* y, float* mean, float* rstd, cudaStream_t s) {
  const unsigned grid = (unsigned)(rows < 65535 ? rows : 65535);
  k_norm_fwd_row<T><<<grid, kRowThreads, 0, s>>>(x, rows, cols, w, b, eps, y, mean, rstd);
  count_launch(1);
  return launch_status();
}

template <typename T>
static qat_status norm_bwd(const void* dy, const void* x, int64_t rows, int64_t cols,
                           const void* w, const float* mean, const float* rstd, void* dx, void* dw,
                           void* db, float* ws, cudaStream_t s) {
  if (dx && rows > 0) {
    const unsigned grid = (unsigned)(rows < 65535 ? rows : 65535);
    k_norm_bwd_row<T><<<grid, kRowThreads, 0, s>>>(dy, x, rows, cols, w, mean, rstd, dx);
    count_launch(1);
  }
  if (dw || db) {
    const int parts = (int)(rows < kNormMaxParts ? rows : kNormMaxParts);
    const unsigned tiles = (unsigned)((cols + 255) / 256);
    if (parts) {
      k_norm_cols<T><<<dim3(tiles, parts), 256, 0, s>>>(dy, x, rows, cols, mean, rstd, parts, ws);
      count_launch(1);
    }
    k_norm_cols_join<T><<<tiles, 256, 0, s>>>(ws, parts, cols, dw, db);
    count_launch(1);
  }
  return launch_status();
}

qat_status launch_norm_fwd(const void* x, qat_dtype dt, int64_t rows, int64_t cols, const void* w,
                           const void* b, float eps, void* y, float* mean, float* rstd,
                           cudaStream_t s) {
  return dt == QAT_F32 ? norm_fwd<F32>(x, rows, cols, w, b, eps, y, mean, rstd, s)
                       : norm_fwd<BF16>(x, rows, cols, w, b, eps, y, mean, rstd, s);
}

qat_status launch_norm_bwd(const void* dy, const void* x, qat_dtype dt, int64_t rows, int64_t cols,
                           const void* w, const float* mean, const float* rstd, void* dx, void* dw,
                           void* db, float* ws, cudaStream_t s) {
  return dt == QAT_F32 ? norm_bwd<F32>(dy, x, rows, cols, w, mean, rstd, dx, dw, db, ws, s)
                       : norm_bwd<BF16>(dy, x, rows, cols, w, mean, rstd, dx, dw, db, ws, s);
}

}  // namespace qat
