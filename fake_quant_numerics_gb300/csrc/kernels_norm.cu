// kernels_norm.cu -- layer norm, forward and backward.
//
//   z = (x - mean) * rstd,  y = z * w + b
//   p = dy * w;  dx = rstd * (p - mean(p) - z * mean(p * z))
//   dw = sum_rows dy * z,  db = sum_rows dy
//
// The floor is reading the rows once and writing as many.  Sums are binary32
// trees around the mean; dw and db are added over the rows in a fixed order.
//
// Measured, bytes that have to move over the copy rate: bf16 16384 x 4096 forward
// 48 us (82%), backward 72 us (83%, its second kernel, which joins the column
// sums, 7 us of it); fp32 8192 x 4096 forward 43 us (93%), backward 65 us (92%);
// bf16 is held back by instruction issue (56% and 46% of the slots) as much as
// by memory.  fp32 2053 x 5003, whose rows are not whole vectors: 20 and 38 us
// (60% and 47%), one element a load.  4 x 4096: 3.2 and 4.4 us.
#include "qat_layer.cuh"
#include "qat_layer.h"

#include <initializer_list>

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

// ---------------------------------------------------------------------------
// Rows that fit in the registers of W warps, 8 R elements a thread: one read of
// the row, the mean, then the deviations around it.  VEC: 16-byte vectors (rows
// of whole ones); else neighbouring threads take neighbouring elements.
// ---------------------------------------------------------------------------
// Eight elements as loaded: bf16 vectors stay packed until they are used.
template <typename T, bool VEC>
struct Raw8 {
  static constexpr bool kPacked = VEC && T::BYTES == 2;
  uint32_t w[kPacked ? 4 : 8];
  __device__ __forceinline__ float get(int e) const {
    if (kPacked) return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    return __uint_as_float(w[kPacked ? 0 : e]);
  }
};
// Two binary32 operations at a time (add, multiply, fused multiply-add): with
// bf16 rows the kernels would otherwise be bound by instruction issue.
struct Pair {
  float x, y;
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair r;
  add2(a.x, a.y, b.x, b.y, r.x, r.y);
  return r;
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) {
  Pair r;
  sub2(a.x, a.y, b.x, b.y, r.x, r.y);
  return r;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair r;
  mul2(a.x, a.y, b.x, b.y, r.x, r.y);
  return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair r;
  fma2(a.x, a.y, b.x, b.y, c.x, c.y, r.x, r.y);
  return r;
}
__device__ __forceinline__ Pair both(float v) { return Pair{v, v}; }
template <typename T, bool VEC>
__device__ __forceinline__ Pair pair(const Raw8<T, VEC>& v, int e) {
  return Pair{v.get(2 * e), v.get(2 * e + 1)};
}
// The columns of chunk q of thread i, eight of them: with vectors runs of 16
// bytes, side by side for neighbouring threads (a 32-byte run would be fetched
// as two half sectors); else one element at a time.
template <typename T, int W, bool VEC>
struct Cols {
  static constexpr int kRun = VEC ? 16 / T::BYTES : 1;  // elements of a run
  static constexpr int kRuns = 8 / kRun;
  int first;
  __device__ __forceinline__ Cols(int q, int i) : first(q * 256 * W + i * kRun) {}
  __device__ __forceinline__ int at(int e) const { return first + e / kRun * (32 * W * kRun) + e % kRun; }
  __device__ __forceinline__ bool has(int e, int cols) const { return at(e / kRun * kRun) < cols; }
};
template <typename T, int W, bool VEC>
__device__ __forceinline__ void ld_cols(Raw8<T, VEC>& v, const void* p, int64_t base,
                                        const Cols<T, W, VEC>& c, int cols) {
  using C = Cols<T, W, VEC>;
#pragma unroll
  for (int k = 0; k < C::kRuns; ++k) {
    const int64_t at = base + c.at(k * C::kRun);
    const bool in = c.has(k * C::kRun, cols);
    if constexpr (VEC) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (in) u = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * T::BYTES);
      v.w[4 * k] = u.x, v.w[4 * k + 1] = u.y, v.w[4 * k + 2] = u.z, v.w[4 * k + 3] = u.w;
    } else {
      v.w[k] = in ? load_elem_bits<T>(p, at) : 0u;
    }
  }
}
template <typename T, int W, bool VEC>
__device__ __forceinline__ void st_cols(void* p, int64_t base, const Cols<T, W, VEC>& c, int cols,
                                        const Pair (&v)[4]) {
  using C = Cols<T, W, VEC>;
#pragma unroll
  for (int k = 0; k < C::kRuns; ++k) {
    const int64_t at = base + c.at(k * C::kRun);
    if (!c.has(k * C::kRun, cols)) continue;
    if constexpr (VEC) {
      uint4 u;
      if constexpr (T::BYTES == 2)
        u = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                       pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
      else
        u = make_uint4(__float_as_uint(v[2 * k].x), __float_as_uint(v[2 * k].y),
                       __float_as_uint(v[2 * k + 1].x), __float_as_uint(v[2 * k + 1].y));
      *reinterpret_cast<uint4*>(static_cast<char*>(p) + at * T::BYTES) = u;
    } else {
      st_elem<T>(p, at, k & 1 ? v[k / 2].y : v[k / 2].x);
    }
  }
}
// sums over the W warps of a row, to every thread; red holds 2 W floats that the
// previous sum of the same buffer no longer needs
template <int W>
__device__ __forceinline__ float2 row_sum2(float a, float b, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(~0u, a, o);
    b += __shfl_xor_sync(~0u, b, o);
  }
  if (W > 1) {
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
      red[wid] = a;
      red[W + wid] = b;
    }
    __syncthreads();
    a = lane < W ? red[lane] : 0.0f;
    b = lane < W ? red[W + lane] : 0.0f;
#pragma unroll
    for (int o = W / 2; o; o >>= 1) {
      a += __shfl_xor_sync(~0u, a, o);
      b += __shfl_xor_sync(~0u, b, o);
    }
    if (W < 32) {
      a = __shfl_sync(~0u, a, 0);
      b = __shfl_sync(~0u, b, 0);
    }
  }
  return make_float2(a, b);
}

template <typename T, int W, int R, bool VEC>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W, W == 1 ? 4 : 32 / W)
    k_norm_fwd(const void* __restrict__ x, int64_t rows, int cols, const void* __restrict__ w,
               const void* __restrict__ b, float eps, void* __restrict__ y,
               float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[2][2 * W];
  const int i = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t r = W == 1 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (r >= rows) return;
  const int64_t base = r * cols;
  Raw8<T, VEC> v[R];
#pragma unroll
  for (int q = 0; q < R; ++q) ld_cols<T>(v[q], x, base, Cols<T, W, VEC>(q, i), cols);
  Pair s = {0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < R; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = s + pair(v[q], e);
  const float m = row_sum2<W>(s.x + s.y, 0.0f, red[0]).x / (float)cols;
  Pair d2 = {0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const Cols<T, W, VEC> c(q, i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      Pair d = pair(v[q], e) - both(m);
      if (!c.has(2 * e, cols)) d.x = 0.0f;
      if (!c.has(2 * e + 1, cols)) d.y = 0.0f;
      d2 = fma(d, d, d2);
    }
  }
  const float rs = 1.0f / sqrtf(row_sum2<W>(d2.x + d2.y, 0.0f, red[1]).x / (float)cols + eps);
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const Cols<T, W, VEC> c(q, i);
    Raw8<T, VEC> g, h;
    if (w) ld_cols<T>(g, w, 0, c, cols);
    if (b) ld_cols<T>(h, b, 0, c, cols);
    Pair o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] = (pair(v[q], e) - both(m)) * both(rs);
      if (w) o[e] = o[e] * pair(g, e);
      if (b) o[e] = o[e] + pair(h, e);
    }
    st_cols<T>(y, base, c, cols, o);
  }
  if (i == 0) {
    if (mean) mean[r] = m;
    if (rstd) rstd[r] = rs;
  }
}

// dx of a row and this block's column sums over its rows (block, block + grid,
// ...; eight rows at a time where a warp takes one): x and dy are read once, dw
// and db stay in registers until the block's partial sums go to ws
// ([2][blocks][cols]).  With vectors every thread copies its own 8 elements of
// the next rows asynchronously into its own slots of shared memory, so no
// barrier guards them and enough bytes are in flight.
template <typename T, int R, bool VEC>
struct NormBwd {
  static constexpr int kStages = VEC ? (T::BYTES == 2 ? 4 : 3) : 0;
  static constexpr int kSlot = 16 * T::BYTES * R;  // x and dy of a row, per thread
};
template <typename T, int W, int R, bool VEC>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W, W == 1 ? 2 : 16 / W)
    k_norm_bwd(const void* __restrict__ dy, const void* __restrict__ x, int64_t rows, int cols,
               const void* __restrict__ w, const float* __restrict__ mean,
               const float* __restrict__ rstd, void* __restrict__ dx, float* __restrict__ ws) {
  constexpr int G = W == 1 ? 8 : 1;  // rows at a time
  constexpr int NT = W == 1 ? 256 : 32 * W;
  constexpr int ST = NormBwd<T, R, VEC>::kStages;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][2 * W];
  __shared__ __align__(16) float join[G == 1 ? 1 : G][G == 1 ? 1 : 256 * R];
  const int i = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t first = (int64_t)blockIdx.x * G + (G == 1 ? 0 : threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * G;
  Pair aw[R][4] = {}, ab[R][4] = {};
  Raw8<T, VEC> wv[R];
  if (w)
#pragma unroll
    for (int q = 0; q < R; ++q) ld_cols<T>(wv[q], w, 0, Cols<T, W, VEC>(q, i), cols);
  const float inv = 1.0f / (float)cols;

  // 16-byte pieces of a thread's slots lie NT * 16 bytes apart (no conflicts)
  constexpr int P = T::BYTES / 2;  // pieces of 8 elements
  const auto piece = [&](int st, int which, int q, int k) {
    return ((((st * 2 + which) * R + q) * P + k) * NT + (int)threadIdx.x) * 16;
  };
  const auto copy = [&](int64_t r, int st) {
    if (r < rows) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const Cols<T, W, VEC> c(q, i);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          if (!c.has(k * c.kRun, cols)) continue;
          const int64_t at = (r * cols + c.at(k * c.kRun)) * T::BYTES;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           (uint32_t)__cvta_generic_to_shared(ring + piece(st, 0, q, k))),
                       "l"(static_cast<const char*>(x) + at)
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           (uint32_t)__cvta_generic_to_shared(ring + piece(st, 1, q, k))),
                       "l"(static_cast<const char*>(dy) + at)
                       : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const auto take = [&](Raw8<T, VEC>& v, int st, int which, int q) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (Cols<T, W, VEC>(q, i).has(k * (16 / T::BYTES), cols))
        u = *reinterpret_cast<const uint4*>(ring + piece(st, which, q, k));
      v.w[4 * k] = u.x, v.w[4 * k + 1] = u.y, v.w[4 * k + 2] = u.z, v.w[4 * k + 3] = u.w;
    }
  };

  if constexpr (VEC) {
#pragma unroll
    for (int k = 0; k < ST - 1; ++k) copy(first + k * step, k);
  }
  int stage = 0, buf = 0;
  float m_next = 0.0f, rs_next = 0.0f;
  if (first < rows) {
    m_next = mean[first];
    rs_next = rstd[first];
  }
  for (int64_t r = first; r < rows; r += step) {
    const int64_t base = r * cols;
    const float m = m_next, rs = rs_next;
    if (r + step < rows) {
      m_next = mean[r + step];
      rs_next = rstd[r + step];
    }
    Raw8<T, VEC> xv[R], gv[R];
    if constexpr (VEC) {
      int into = stage + ST - 1;
      if (into >= ST) into -= ST;
      copy(r + (ST - 1) * step, into);
      asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
#pragma unroll
      for (int q = 0; q < R; ++q) {
        take(xv[q], stage, 0, q);
        take(gv[q], stage, 1, q);
      }
      if (++stage == ST) stage = 0;
    } else {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        ld_cols<T>(xv[q], x, base, Cols<T, W, VEC>(q, i), cols);
        ld_cols<T>(gv[q], dy, base, Cols<T, W, VEC>(q, i), cols);
      }
    }
    Pair z[R][4], p[R][4], s1 = {0.0f, 0.0f}, s2 = {0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < R; ++q) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[q][e] = (pair(xv[q], e) - both(m)) * both(rs);
        p[q][e] = pair(gv[q], e);
        aw[q][e] = fma(p[q][e], z[q][e], aw[q][e]);
        ab[q][e] = ab[q][e] + p[q][e];
        if (w) p[q][e] = p[q][e] * pair(wv[q], e);
        s1 = s1 + p[q][e];
        s2 = fma(p[q][e], z[q][e], s2);
      }
    }
    if (!dx) continue;
    const float2 t = row_sum2<W>(s1.x + s1.y, s2.x + s2.y, red[buf]);
    buf ^= 1;
    const Pair c1 = both(t.x * inv), c2 = both(-t.y * inv);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      Pair o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = both(rs) * fma(z[q][e], c2, p[q][e] - c1);
      st_cols<T>(dx, base, Cols<T, W, VEC>(q, i), cols, o);
    }
  }
  pdl_trigger();
  if (!ws) return;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float* out = ws + ((int64_t)half * gridDim.x + blockIdx.x) * cols;
    if (G > 1) __syncthreads();
    float* to = G == 1 ? out : join[threadIdx.x >> 5];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const Cols<T, W, VEC> c(q, i);
#pragma unroll
      for (int e = 0; e < 4; e += VEC ? 2 : 1) {  // pairs
        const Pair v = half ? ab[q][e] : aw[q][e];
        if (VEC) {
          const Pair u = half ? ab[q][e + 1] : aw[q][e + 1];
          if (G > 1 || c.has(2 * e, cols))
            *reinterpret_cast<float4*>(to + c.at(2 * e)) = make_float4(v.x, v.y, u.x, u.y);
        } else {
          if (G > 1 || c.has(2 * e, cols)) to[c.at(2 * e)] = v.x;
          if (G > 1 || c.has(2 * e + 1, cols)) to[c.at(2 * e + 1)] = v.y;
        }
      }
    }
    if (G > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += 256) {
        float v = join[0][c];
#pragma unroll
        for (int k = 1; k < G; ++k) v += join[k][c];
        out[c] = v;
      }
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

// The partials' sum in a fixed order: 32 columns a block, 32 warps that take
// every 32nd part, their sums added in order.
template <typename T>
__global__ void __launch_bounds__(1024)
    k_norm_cols_join(const float* ws, int parts, int64_t cols, void* dw, void* db) {
  __shared__ float sums[2][32][33];
  pdl_wait();  // the partials are the previous kernel's
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float sw = 0.0f, sb = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int p = wid; p < parts; p += 32) {
      sw += ws[(int64_t)p * cols + c];
      sb += ws[((int64_t)parts + p) * cols + c];
    }
  }
  sums[0][wid][lane] = sw;
  sums[1][wid][lane] = sb;
  __syncthreads();
  if (wid > 1 || c >= cols) return;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) v += sums[wid][k][lane];
  void* out = wid ? db : dw;
  if (out) st_elem<T>(out, c, v);
}

static bool vectors(int64_t cols, std::initializer_list<const void*> ps) {
  if (cols % 8) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}

template <typename T, int W, int R>
static void go_fwd(bool vec, const void* x, int64_t rows, int64_t cols, const void* w,
                   const void* b, float eps, void* y, float* mean, float* rstd, cudaStream_t s) {
  const unsigned grid = (unsigned)(W == 1 ? (rows + 7) / 8 : rows);
  const auto k = vec ? k_norm_fwd<T, W, R, true> : k_norm_fwd<T, W, R, false>;
  k<<<grid, W == 1 ? 256 : 32 * W, 0, s>>>(x, rows, (int)cols, w, b, eps, y, mean, rstd);
}

template <typename T>
static qat_status norm_fwd(const void* x, int64_t rows, int64_t cols, const void* w, const void* b,
                           float eps, void* y, float* mean, float* rstd, cudaStream_t s) {
  const bool vec = vectors(cols, {x, w, b, y});
#define QAT_FWD(W, R) go_fwd<T, W, R>(vec, x, rows, cols, w, b, eps, y, mean, rstd, s)
  if (cols > 16384 || rows > INT32_MAX) {
    const unsigned grid = (unsigned)(rows < 65535 ? rows : 65535);
    k_norm_fwd_row<T><<<grid, kRowThreads, 0, s>>>(x, rows, cols, w, b, eps, y, mean, rstd);
  } else if (cols <= 256) {
    QAT_FWD(1, 1);
  } else if (cols <= 512) {
    QAT_FWD(1, 2);
  } else if (cols <= 1024) {  // 32 elements a thread: enough bytes in flight
    QAT_FWD(1, 4);
  } else if (cols <= 2048) {
    QAT_FWD(2, 4);
  } else if (cols <= 4096) {
    QAT_FWD(4, 4);
  } else if (cols <= 8192) {
    QAT_FWD(8, 4);
  } else {
    QAT_FWD(16, 4);
  }
#undef QAT_FWD
  count_launch(1);
  return launch_status();
}

template <typename T, int W, int R>
static int go_bwd(bool vec, const void* dy, const void* x, int64_t rows, int64_t cols,
                  const void* w, const float* mean, const float* rstd, void* dx, float* ws,
                  cudaStream_t s) {
  const int64_t groups = W == 1 ? (rows + 7) / 8 : rows;
  constexpr int threads = W == 1 ? 256 : 32 * W;
  int64_t grid = (int64_t)device_info().sms * (W == 1 ? 2 : 16 / W);  // all resident
  const int most = norm_parts(INT64_MAX, cols);
  if (grid > most) grid = most;
  if (grid > groups) grid = groups;
  using N = NormBwd<T, R, true>;
  const int smem = vec ? N::kStages * N::kSlot * threads : 0;
  const auto k = vec ? k_norm_bwd<T, W, R, true> : k_norm_bwd<T, W, R, false>;
  if (smem > 40000 &&
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return -1;
  }
  k<<<(unsigned)grid, threads, smem, s>>>(dy, x, rows, (int)cols, w, mean, rstd, dx, ws);
  count_launch(1);
  return (int)grid;
}

template <typename T>
static qat_status norm_bwd(const void* dy, const void* x, int64_t rows, int64_t cols,
                           const void* w, const float* mean, const float* rstd, void* dx, void* dw,
                           void* db, float* ws, cudaStream_t s) {
  const bool sums = dw || db;
  int parts = 0;
  if (rows > 0 && cols <= 8192) {
    const bool vec = vectors(cols, {dy, x, w, dx});
    float* part = sums ? ws : nullptr;
#define QAT_BWD(W, R) parts = go_bwd<T, W, R>(vec, dy, x, rows, cols, w, mean, rstd, dx, part, s)
    if (cols <= 256)
      QAT_BWD(1, 1);
    else if (cols <= 512)
      QAT_BWD(1, 2);
    else if (cols <= 1024)
      QAT_BWD(2, 2);
    else if (cols <= 2048)
      QAT_BWD(4, 2);
    else if (cols <= 4096)
      QAT_BWD(8, 2);
    else
      QAT_BWD(16, 2);
    if (parts < 0) return QAT_ERR_CUDA;
#undef QAT_BWD
  } else if (rows > 0) {
    if (dx) {
      const unsigned grid = (unsigned)(rows < 65535 ? rows : 65535);
      k_norm_bwd_row<T><<<grid, kRowThreads, 0, s>>>(dy, x, rows, cols, w, mean, rstd, dx);
      count_launch(1);
    }
    if (sums) {
      parts = norm_parts(rows, cols);
      k_norm_cols<T><<<dim3((unsigned)((cols + 255) / 256), parts), 256, 0, s>>>(
          dy, x, rows, cols, mean, rstd, parts, ws);
      count_launch(1);
    }
  }
  if (sums) {
    if (launch_kernel(k_norm_cols_join<T>, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, s,
                      parts > 0, ws, parts, cols, dw, db) != cudaSuccess) {
      (void)cudaGetLastError();
      return QAT_ERR_CUDA;
    }
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
