// kernels_ffn.cu -- the gated feed-forward block, forward and backward.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) * u, y = h Wd^T
//   dh = dy Wd; dg = dh * u * act'(g), du = dh * act(g)
//   dx = dg Wg + du Wu; dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// One tiled product kernel with the element-wise steps as its epilogues.
#include "qat_dense.h"
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

static bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The tensor cores take bf16 rows of whole 16-byte vectors.
static bool dense_ok(qat_dtype dt, int64_t d, int64_t f, const void* const* ps, int n) {
  if (dt != QAT_BF16 || d % 8 || f % 8) return false;
  for (int i = 0; i < n; ++i)
    if (!on16(ps[i])) return false;
  return true;
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

static qat_status fwd_dense(const void* x, int64_t t, int64_t d, int64_t f, const void* wg,
                            const void* wu, const void* wd, int act, void* h, float* gp, float* up,
                            void* y, int32_t* flags, cudaStream_t s) {
  Dense g = {};
  g.epi = kDenseGated;
  g.m = t;
  g.n = f;
  g.k = d;
  g.a[0] = DenseOp{x, d, false, 0};
  g.b[0] = DenseOp{wg, d, false, 0};
  g.b[1] = DenseOp{wu, d, false, 0};
  g.act = act;
  g.c[0] = h;
  g.gp = gp;
  g.up = up;
  g.flags = flags;
  const qat_status st = launch_dense(g, s);
  if (st) return st;
  Dense o = {};
  o.epi = kDenseStore;
  o.m = t;
  o.n = d;
  o.k = f;
  o.a[0] = DenseOp{h, f, false, 0};
  o.b[0] = DenseOp{wd, f, false, 0};
  o.c[0] = y;
  o.flags = flags;
  return launch_dense(o, s);
}

static qat_status bwd_dense(const void* dy, const void* x, int64_t t, int64_t d, int64_t f,
                            const void* wg, const void* wu, const void* wd, int act, const void* h,
                            const float* gp, const float* up, void* dx, void* dwg, void* dwu,
                            void* dwd, int32_t* flags, void* ws, cudaStream_t s) {
  char* dg = static_cast<char*>(ws);
  char* du = dg + r256((size_t)t * f * 2);
  qat_status st = QAT_OK;
  if (dx || dwg || dwu) {
    Dense q = {};
    q.epi = kDenseGatedBwd;
    q.m = t;
    q.n = f;
    q.k = d;
    q.a[0] = DenseOp{dy, d, false, 0};
    q.b[0] = DenseOp{wd, f, true, 0};
    q.act = act;
    q.gp = const_cast<float*>(gp);
    q.up = const_cast<float*>(up);
    q.dg = dg;
    q.du = du;
    q.flags = flags;
    st = launch_dense(q, s);
  }
  if (!st && dx) {
    Dense q = {};
    q.epi = kDenseStore;
    q.m = t;
    q.n = d;
    q.k = f;
    q.segs = 2;
    q.a[0] = DenseOp{dg, f, false, 0};
    q.a[1] = DenseOp{du, f, false, 0};
    q.b[0] = DenseOp{wg, d, true, 0};
    q.b[1] = DenseOp{wu, d, true, 0};
    q.c[0] = dx;
    q.flags = flags;
    st = launch_dense(q, s);
  }
  if (!st && (dwg || dwu)) {
    Dense q = {};
    q.epi = kDenseStore;
    q.m = f;
    q.n = d;
    q.k = t;
    q.problems = dwg && dwu ? 2 : 1;
    q.a[0] = DenseOp{dwg ? dg : du, f, true, 0};
    q.a[1] = DenseOp{du, f, true, 0};
    q.b[0] = DenseOp{x, d, true, 0};
    q.c[0] = dwg ? dwg : dwu;
    q.c[1] = dwu;
    q.flags = flags;
    st = launch_dense(q, s);
  }
  if (!st && dwd) {
    Dense q = {};
    q.epi = kDenseStore;
    q.m = d;
    q.n = f;
    q.k = t;
    q.a[0] = DenseOp{dy, d, true, 0};
    q.b[0] = DenseOp{h, f, true, 0};
    q.c[0] = dwd;
    q.flags = flags;
    st = launch_dense(q, s);
  }
  return st;
}

qat_status launch_ffn_fwd(const void* x, qat_dtype dt, int64_t t, int64_t d, int64_t f,
                          const void* wg, const void* wu, const void* wd, int act, void* h,
                          float* gp, float* up, void* y, int32_t* flags, void* ws, cudaStream_t s) {
  (void)ws;
  const void* ps[] = {x, wg, wu, wd, h};
  if (t > 0 && d > 0 && f > 0 && dense_ok(dt, d, f, ps, 5))
    return fwd_dense(x, t, d, f, wg, wu, wd, act, h, gp, up, y, flags, s);
  return dt == QAT_F32 ? fwd<F32>(x, t, d, f, wg, wu, wd, act, h, gp, up, y, s)
                       : fwd<BF16>(x, t, d, f, wg, wu, wd, act, h, gp, up, y, s);
}

qat_status launch_ffn_bwd(const void* dy, const void* x, qat_dtype dt, int64_t t, int64_t d,
                          int64_t f, const void* wg, const void* wu, const void* wd, int act,
                          const void* h, const float* gp, const float* up, void* dx, void* dwg,
                          void* dwu, void* dwd, int32_t* flags, void* ws, cudaStream_t s) {
  const void* ps[] = {dy, x, wg, wu, wd, h};
  if (t > 0 && d > 0 && f > 0 && dense_ok(dt, d, f, ps, 6))
    return bwd_dense(dy, x, t, d, f, wg, wu, wd, act, h, gp, up, dx, dwg, dwu, dwd, flags, ws, s);
  return dt == QAT_F32
             ? bwd<F32>(dy, x, t, d, f, wg, wu, wd, act, h, gp, up, dx, dwg, dwu, dwd, ws, s)
             : bwd<BF16>(dy, x, t, d, f, wg, wu, wd, act, h, gp, up, dx, dwg, dwu, dwd, ws, s);
}

}  // namespace qat
