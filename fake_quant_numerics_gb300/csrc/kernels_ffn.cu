// kernels_ffn.cu -- the gated feed-forward block, forward and backward.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) * u, y = h Wd^T
//   dh = dy Wd; dg = dh * u * act'(g), du = dh * act(g)
//   dx = dg Wg + du Wu; dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// One tiled product kernel with the element-wise steps as its epilogues.
#include "qat_layer.cuh"
#include "qat_layer.h"

namespace qat {

// A matrix read as M(i, j) = p[i * si + j * sj].
struct Mat {
  const void* p;
  int64_t si, sj;
};

enum { kEpiStore = 0, kEpiGated = 1, kEpiGatedBwd = 2 };

struct FfnEpi {
  int act;
  void* c;        // store / gated: the output [m, n]
  float* gp;      // gated: g and u kept (nullable); backward: read
  float* up;
  void* dg;       // backward: outputs
  void* du;
};

constexpr int kTM = 64, kTN = 64, kTK = 16;

// C[m, n] = sum_k A0(m, k) B0(k, n) (+ A1 B1 for a store; a second
// accumulator with B1 for the gated epilogue).
template <typename T, int EPI>
__global__ void __launch_bounds__(256) k_ffn_tile(Mat a0, Mat b0, Mat a1, Mat b1, int terms,
                                                  int64_t m, int64_t n, int64_t k, FfnEpi e) {
  __shared__ float sa[kTK][kTM + 4], sb[2][kTK][kTN + 4];
  constexpr int NB = EPI == kEpiGated ? 2 : 1;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * kTM, n0 = (int64_t)blockIdx.x * kTN;
  float acc[NB][4][4] = {};
  for (int t = 0; t < terms; ++t) {
    const Mat a = t ? a1 : a0;
    for (int64_t k0 = 0; k0 < k; k0 += kTK) {
      for (int i = threadIdx.x; i < kTK * kTM; i += 256) {
        // neighbouring threads along the contiguous direction
        const int mm = a.sj == 1 ? i / kTK : i % kTM, kk = a.sj == 1 ? i % kTK : i / kTM;
        sa[kk][mm] = m0 + mm < m && k0 + kk < k
                         ? ld_elem<T>(a.p, (m0 + mm) * a.si + (k0 + kk) * a.sj) : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < NB; ++q) {
        const Mat b = (NB == 2 ? q : t) ? b1 : b0;
        for (int i = threadIdx.x; i < kTK * kTN; i += 256) {
          const int nn = b.sj == 1 ? i % kTN : i / kTK, kk = b.sj == 1 ? i / kTN : i % kTK;
          sb[q][kk][nn] = n0 + nn < n && k0 + kk < k
                              ? ld_elem<T>(b.p, (k0 + kk) * b.si + (n0 + nn) * b.sj) : 0.0f;
        }
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kTK; ++kk) {
        float av[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = sa[kk][ty * 4 + i];
#pragma unroll
        for (int q = 0; q < NB; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float bv = sb[q][kk][tx * 4 + j];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][i][j] = fmaf(av[i], bv, acc[q][i][j]);
          }
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = m0 + ty * 4 + i, c = n0 + tx * 4 + j;
      if (r >= m || c >= n) continue;
      const int64_t o = r * n + c;
      const float v = acc[0][i][j];
      if (EPI == kEpiStore) {
        st_elem<T>(e.c, o, v);
      } else if (EPI == kEpiGated) {
        const float u = acc[NB - 1][i][j];
        st_elem<T>(e.c, o, act_value(e.act, v) * u);
        if (e.gp) {
          e.gp[o] = v;
          e.up[o] = u;
        }
      } else {
        float ga, da;
        act_grad(e.act, e.gp[o], ga, da);
        st_elem<T>(e.dg, o, v * e.up[o] * da);
        st_elem<T>(e.du, o, v * ga);
      }
    }
}

template <typename T, int EPI>
static void tile(Mat a0, Mat b0, Mat a1, Mat b1, int terms, int64_t m, int64_t n, int64_t k,
                 const FfnEpi& e, cudaStream_t s) {
  if (m == 0 || n == 0) return;
  // gridDim.y holds 65535 tiles of rows: taller outputs in several launches
  const dim3 grid((unsigned)((n + kTN - 1) / kTN), (unsigned)((m + kTM - 1) / kTM));
  k_ffn_tile<T, EPI><<<grid, 256, 0, s>>>(a0, b0, a1, b1, terms, m, n, k, e);
  count_launch(1);
}

static size_t r256(size_t b) { return (b + 255) / 256 * 256; }

size_t ffn_ws_bytes(qat_dtype dt, int64_t tokens, int64_t dim, int64_t hidden, bool backward) {
  (void)dim;
  return backward ? 2 * r256((size_t)tokens * hidden * (dt == QAT_F32 ? 4 : 2)) : 0;
}

template <typename T>
static qat_status fwd(const void* x, int64_t t, int64_t d, int64_t f, const void* wg,
                      const void* wu, const void* wd, int act, void* h, float* gp, float* up,
                      void* y, cudaStream_t s) {
  FfnEpi e = {act, h, gp, up, nullptr, nullptr};
  const Mat mx = {x, d, 1};
  tile<T, kEpiGated>(mx, Mat{wg, 1, d}, mx, Mat{wu, 1, d}, 1, t, f, d, e, s);
  e.c = y;
  tile<T, kEpiStore>(Mat{h, f, 1}, Mat{wd, 1, f}, Mat{}, Mat{}, 1, t, d, f, e, s);
  return launch_status();
}

template <typename T>
static qat_status bwd(const void* dy, const void* x, int64_t t, int64_t d, int64_t f,
                      const void* wg, const void* wu, const void* wd, int act, const void* h,
                      const float* gp, const float* up, void* dx, void* dwg, void* dwu, void* dwd,
                      void* ws, cudaStream_t s) {
  char* dg = static_cast<char*>(ws);
  char* du = dg + r256((size_t)t * f * T::BYTES);
  FfnEpi e = {act, nullptr, const_cast<float*>(gp), const_cast<float*>(up), dg, du};
  if (dx || dwg || dwu)
    tile<T, kEpiGatedBwd>(Mat{dy, d, 1}, Mat{wd, f, 1}, Mat{}, Mat{}, 1, t, f, d, e, s);
  e.c = dx;
  if (dx)
    tile<T, kEpiStore>(Mat{dg, f, 1}, Mat{wg, d, 1}, Mat{du, f, 1}, Mat{wu, d, 1}, 2, t, d, f, e, s);
  e.c = dwg;
  if (dwg) tile<T, kEpiStore>(Mat{dg, 1, f}, Mat{x, d, 1}, Mat{}, Mat{}, 1, f, d, t, e, s);
  e.c = dwu;
  if (dwu) tile<T, kEpiStore>(Mat{du, 1, f}, Mat{x, d, 1}, Mat{}, Mat{}, 1, f, d, t, e, s);
  e.c = dwd;
  if (dwd) tile<T, kEpiStore>(Mat{dy, 1, d}, Mat{h, f, 1}, Mat{}, Mat{}, 1, d, f, t, e, s);
  return launch_status();
}

qat_status launch_ffn_fwd(const void* x, qat_dtype dt, int64_t t, int64_t d, int64_t f,
                          const void* wg, const void* wu, const void* wd, int act, void* h,
                          float* gp, float* up, void* y, void* ws, cudaStream_t s) {
  (void)ws;
  return dt == QAT_F32 ? fwd<F32>(x, t, d, f, wg, wu, wd, act, h, gp, up, y, s)
                       : fwd<BF16>(x, t, d, f, wg, wu, wd, act, h, gp, up, y, s);
}

qat_status launch_ffn_bwd(const void* dy, const void* x, qat_dtype dt, int64_t t, int64_t d,
                          int64_t f, const void* wg, const void* wu, const void* wd, int act,
                          const void* h, const float* gp, const float* up, void* dx, void* dwg,
                          void* dwu, void* dwd, void* ws, cudaStream_t s) {
  return dt == QAT_F32
             ? bwd<F32>(dy, x, t, d, f, wg, wu, wd, act, h, gp, up, dx, dwg, dwu, dwd, ws, s)
             : bwd<BF16>(dy, x, t, d, f, wg, wu, wd, act, h, gp, up, dx, dwg, dwu, dwd, ws, s);
}

}  // namespace qat
