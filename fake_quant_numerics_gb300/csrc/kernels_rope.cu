// kernels_rope.cu -- RMS norm of each head of queries and keys with the position
// rotation in the same pass, and its backward pass.
//
//   z = x / sqrt(mean x^2 + eps), p = z w, (a', b') = m (a c - b s, b c + a s)
//   g' = the gradient turned back; dw = sum g' z; dx = (g'w - z mean(g'w z)) / sqrt(..)
//
// The angle of pair j at position t is t * turns[j] modulo 2^64 of a turn, by
// integer multiplication: exact for any position, where a binary32 product t * f
// is off by t * 2^-24 of a radian.
//
// Bound by reading and writing the heads.  A group of lanes holds a head in
// registers: each lane the two runs of V elements whose pairs it turns, so that
// norm, weight and rotation need one pass and one reduction over the group.  A
// group walks over several heads of a token, which share its angles.
#include "qat_attention.h"
#include "qat_layer.cuh"

namespace qat {
namespace {

// V consecutive elements as they lie in memory (aligned to their whole size, at
// most to 16 bytes).
template <typename T, int V>
struct Run {
  static constexpr int BYTES = V * T::BYTES, W = (BYTES + 3) / 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const char* p = static_cast<const char*>(base) + i * T::BYTES;
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int j = 0; j < BYTES / 16; ++j) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + j);
        w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
      }
    } else if constexpr (BYTES == 8) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (BYTES == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = 0u;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (T::BYTES == 4) return __uint_as_float(w[e]);
    return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  }
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (T::BYTES == 4) {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 2) w[e >> 1] = pack_bf16x2(v[e], e + 1 < V ? v[e + 1] : 0.0f);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    char* p = static_cast<char*>(base) + i * T::BYTES;
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int j = 0; j < BYTES / 16; ++j)
        reinterpret_cast<uint4*>(p)[j] =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
  }
};

// Cosine and sine of a 2^-64 fraction of a turn: the quarter by its two top bits,
// the rest (|r| <= an eighth of a turn) by the library's function of half turns.
__device__ __forceinline__ void turn_cos_sin(uint64_t t, float m, float& c, float& s) {
  const uint64_t quarter = (t + (UINT64_C(1) << 61)) >> 62;
  const int32_t r = (int32_t)((int64_t)(t - (quarter << 62)) >> 32);
  float sr, cr;
  sincospif((float)r * 0x1p-31f, &sr, &cr);
  const int n = (int)quarter & 3;
  c = (n & 1) ? sr : cr;
  s = (n & 1) ? cr : sr;
  if (n == 1 || n == 2) c = -c;
  if (n >= 2) s = -s;
  c = __fmul_rn(c, m);
  s = __fmul_rn(s, m);
}

// Where the runs A and B of unit u start.  Units of turned pairs come first; a
// later unit is 2 V elements that pass as they are.
template <int V, bool INTER>
__device__ __forceinline__ void unit_runs(int u, int rotary, int& a, int& b) {
  const int turned = rotary / (2 * V);
  if (u < turned) {
    a = INTER ? 2 * V * u : V * u;
    b = a + (INTER ? V : rotary / 2);
  } else {
    a = rotary + (u - turned) * 2 * V;
    b = a + V;
  }
}

// The lane's V pairs turned in place: v holds run A, then run B.
template <int V, bool INTER>
__device__ __forceinline__ void turn_pairs(float (&v)[2 * V], const float (&c)[V],
                                           const float (&s)[V], bool back) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int p = INTER ? 2 * e : e, q = INTER ? 2 * e + 1 : V + e;
    const float se = back ? -s[e] : s[e];
    const float a = v[p], b = v[q];
    v[p] = __fmaf_rn(a, c[e], -__fmul_rn(b, se));
    v[q] = __fmaf_rn(b, c[e], __fmul_rn(a, se));
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// A lane's units of one head, u = lane + lanes * p.
template <int V, int NP, bool INTER>
struct Units {
  int a[NP], b[NP];
  bool has_a[NP], has_b[NP];
  __device__ __forceinline__ Units(int lane, int lanes, int d, int rotary) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      unit_runs<V, INTER>(lane + lanes * p, rotary, a[p], b[p]);
      has_a[p] = a[p] < d;
      has_b[p] = has_a[p] && b[p] < d;
    }
  }
};

template <typename T, int V, int NP>
__device__ __forceinline__ void load_weight(const void* w, const int (&a)[NP], const int (&b)[NP],
                                            const bool (&ha)[NP], const bool (&hb)[NP],
                                            float (&wt)[NP][2 * V]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    Run<T, V> ra, rb;
    ra.zero(), rb.zero();
    if (w && ha[p]) ra.load(w, a[p]);
    if (w && hb[p]) rb.load(w, b[p]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      wt[p][e] = w ? ra.get(e) : 1.0f;
      wt[p][V + e] = w ? rb.get(e) : 1.0f;
    }
  }
}

template <int V, int NP, bool INTER>
__device__ __forceinline__ void load_angles(const RopeArgs& r, int64_t token, int lane, int lanes,
                                            float (&c)[NP][V], float (&s)[NP][V]) {
  const uint64_t pos = (uint64_t)__ldg(r.positions + token);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int u = lane + lanes * p;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int j = u * V + e;
      c[p][e] = 1.0f, s[p][e] = 0.0f;
      if (j < r.rotary / 2) turn_cos_sin(pos * __ldg(r.turns + j), r.amplitude, c[p][e], s[p][e]);
    }
  }
}

constexpr int kRopeThreads = 256;

// `per` heads of one token a group; items are the query heads' runs, then the
// keys'.  All lanes of a warp take the same number of steps (shuffles).
template <typename T, int V, int NP, int U, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) k_rope_fwd(RopeArgs r, int lanes, int per) {
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t item = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / lanes;
  const int runs0 = (r.heads[0] + per - 1) / per, runs1 = (r.heads[1] + per - 1) / per;
  const int64_t items0 = r.tokens * runs0;
  const bool there = item < items0 + r.tokens * runs1;
  const int which = item >= items0;
  const int runs = which ? runs1 : runs0;
  const int64_t at = item - (which ? items0 : 0);
  const int64_t token = there ? at / runs : 0;
  const int h0 = there ? (int)(at - token * runs) * per : 0;
  const int heads = there ? r.heads[which] : 0;
  const void* x = r.x[which];
  const int64_t hs = r.head_stride[which];
  const int64_t xt = token * r.token_stride[which];
  const int64_t yt = (token * r.heads[which]) * r.d;

  const Units<V, NP, INTER> un(lane, lanes, r.d, r.rotary);
  float w[NP][2 * V], c[NP][V], s[NP][V];
  load_weight<T, V, NP>(r.w[which], un.a, un.b, un.has_a, un.has_b, w);
  load_angles<V, NP, INTER>(r, token, lane, lanes, c, s);
  for (int h = 0; h < per; h += U) {
    Run<T, V> ra[U][NP], rb[U][NP];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool on = h + i < per && h0 + h + i < heads;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        ra[i][p].zero(), rb[i][p].zero();
        const int64_t o = xt + (h0 + h + i) * hs;
        if (on && un.has_a[p]) ra[i][p].load(x, o + un.a[p]);
        if (on && un.has_b[p]) rb[i][p].load(x, o + un.b[p]);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool on = h + i < per && h0 + h + i < heads;
      float rstd = 1.0f;
      if (r.norm) {
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            sum = __fmaf_rn(ra[i][p].get(e), ra[i][p].get(e), sum);
            sum = __fmaf_rn(rb[i][p].get(e), rb[i][p].get(e), sum);
          }
        sum = group_sum(sum, lanes);
        rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)r.d), r.eps)));
      }
      const int64_t o = yt + (int64_t)(h0 + h + i) * r.d;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        float v[2 * V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          v[e] = __fmul_rn(__fmul_rn(ra[i][p].get(e), rstd), w[p][e]);
          v[V + e] = __fmul_rn(__fmul_rn(rb[i][p].get(e), rstd), w[p][V + e]);
        }
        turn_pairs<V, INTER>(v, c[p], s[p], false);
        Run<T, V> out;
        if (on && un.has_a[p]) out.set(v), out.store(r.y[which], o + un.a[p]);
        if (on && un.has_b[p]) out.set(v + V), out.store(r.y[which], o + un.b[p]);
      }
    }
  }
}

// The same walk with the gradients; each lane keeps its elements' share of dweight,
// and a block's shares are added over its groups in shared memory, in order.
template <typename T, int V, int NP, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) k_rope_bwd(RopeArgs r, int lanes, int per,
                                                           float* parts) {
  __shared__ float share[kRopeThreads * 2 * V * NP];
  pdl_trigger();
  const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
  const int groups = kRopeThreads / lanes;
  const Units<V, NP, INTER> un(lane, lanes, r.d, r.rotary);
  for (int which = 0; which < 2; ++which) {
    const int heads = r.heads[which];
    const bool sums = r.dw[which] != nullptr;
    const int runs = (heads + per - 1) / per;
    const int64_t items = r.y[which] || sums ? r.tokens * runs : 0;
    const void *x = r.x[which], *g = r.g[which];
    float w[NP][2 * V], acc[NP][2 * V] = {};
    load_weight<T, V, NP>(r.w[which], un.a, un.b, un.has_a, un.has_b, w);
    // (whole blocks step together: the shuffles need every lane)
    for (int64_t base = (int64_t)blockIdx.x * groups; base < items;
         base += (int64_t)gridDim.x * groups) {
      const int64_t item = base + group;
      const bool there = item < items;
      const int64_t token = there ? item / runs : 0;
      const int h0 = there ? (int)(item - token * runs) * per : 0;
      float c[NP][V], s[NP][V];
      load_angles<V, NP, INTER>(r, token, lane, lanes, c, s);
      for (int h = 0; h < per; ++h) {
        const bool on = there && h0 + h < heads;
        Run<T, V> xa[NP], xb[NP], ga[NP], gb[NP];
        const int64_t xo = token * r.token_stride[which] + (h0 + h) * r.head_stride[which];
        const int64_t go = (token * heads + h0 + h) * r.d;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          xa[p].zero(), xb[p].zero(), ga[p].zero(), gb[p].zero();
          if (on && un.has_a[p]) xa[p].load(x, xo + un.a[p]), ga[p].load(g, go + un.a[p]);
          if (on && un.has_b[p]) xb[p].load(x, xo + un.b[p]), gb[p].load(g, go + un.b[p]);
        }
        float v[NP][2 * V], sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
#pragma unroll
          for (int e = 0; e < V; ++e) v[p][e] = ga[p].get(e), v[p][V + e] = gb[p].get(e);
          turn_pairs<V, INTER>(v[p], c[p], s[p], true);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float a = xa[p].get(e), b = xb[p].get(e);
            sum = __fmaf_rn(b, b, __fmaf_rn(a, a, sum));
            dot = __fmaf_rn(__fmul_rn(v[p][e], w[p][e]), a, dot);
            dot = __fmaf_rn(__fmul_rn(v[p][V + e], w[p][V + e]), b, dot);
          }
        }
        float rstd = 1.0f, mean = 0.0f;
        if (r.norm) {
          sum = group_sum(sum, lanes);
          dot = group_sum(dot, lanes);
          rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)r.d), r.eps)));
          mean = __fdiv_rn(__fmul_rn(dot, rstd), (float)r.d);  // of g'w z
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          float dx[2 * V];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float za = __fmul_rn(xa[p].get(e), rstd), zb = __fmul_rn(xb[p].get(e), rstd);
            acc[p][e] = __fmaf_rn(v[p][e], za, acc[p][e]);
            acc[p][V + e] = __fmaf_rn(v[p][V + e], zb, acc[p][V + e]);
            dx[e] = __fmul_rn(rstd, __fmaf_rn(-mean, za, __fmul_rn(v[p][e], w[p][e])));
            dx[V + e] = __fmul_rn(rstd, __fmaf_rn(-mean, zb, __fmul_rn(v[p][V + e], w[p][V + e])));
          }
          Run<T, V> out;
          if (on && r.y[which] && un.has_a[p]) out.set(dx), out.store(r.y[which], go + un.a[p]);
          if (on && r.y[which] && un.has_b[p]) out.set(dx + V), out.store(r.y[which], go + un.b[p]);
        }
      }
    }
    if (!sums) continue;  // (the same for the whole grid)
    float* mine = share + (size_t)threadIdx.x * 2 * V * NP;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) mine[p * 2 * V + e] = acc[p][e];
    __syncthreads();
    for (int i = threadIdx.x; i < lanes * NP * 2 * V; i += kRopeThreads) {
      const int ln = i / (NP * 2 * V), p = i / (2 * V) % NP, e = i % (2 * V);
      int a, b;
      unit_runs<V, INTER>(ln + lanes * p, r.rotary, a, b);
      const int at = e < V ? a + e : b + e - V;
      if (at >= r.d || a >= r.d) continue;
      float total = 0.0f;
      for (int k = 0; k < groups; ++k) total += share[((size_t)k * lanes + ln) * NP * 2 * V + i % (NP * 2 * V)];
      parts[((int64_t)blockIdx.x * 2 + which) * r.d + at] = total;
    }
    __syncthreads();
  }
}

// dweight from the blocks' shares: 32 columns a block, 32 rows at a time, in order.
template <typename T>
__global__ void __launch_bounds__(1024) k_rope_join(const float* parts, int n, int d, void* dwq,
                                                    void* dwk) {
  __shared__ float part[32][33];
  pdl_wait();
  const int col = blockIdx.x * 32 + threadIdx.x;
  float sum = 0.0f;
  if (col < 2 * d)
    for (int i = threadIdx.y; i < n; i += 32) sum += parts[(int64_t)i * 2 * d + col];
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y || col >= 2 * d) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += part[i][threadIdx.x];
  void* dw = col < d ? dwq : dwk;
  if (dw) st_elem<T>(dw, col < d ? col : col - d, sum);
}

// The widest run that fits every run's start: elements of a vector of at most 16
// bytes for bf16, two of them for fp32.
template <typename T>
int run_width(const RopeArgs& r) {
  for (int v = 8; v > 1; v >>= 1) {
    const uintptr_t bytes = v * T::BYTES < 16 ? v * T::BYTES : 16;
    bool fits = r.rotary % (2 * v) == 0 && r.d % v == 0;
    for (int i = 0; i < 2; ++i) {
      if (r.heads[i] == 0) continue;
      for (const void* p : {r.x[i], r.g[i], r.w[i], (const void*)r.y[i]})
        fits = fits && reinterpret_cast<uintptr_t>(p) % bytes == 0;
      fits = fits && r.token_stride[i] * T::BYTES % (int64_t)bytes == 0 &&
             r.head_stride[i] * T::BYTES % (int64_t)bytes == 0 &&
             (int64_t)r.d * T::BYTES % (int64_t)bytes == 0;
    }
    if (fits) return v;
  }
  return 1;
}

int group_lanes(int d, int v) {
  const int units = (d + 2 * v - 1) / (2 * v);
  int lanes = 1;
  while (lanes < units && lanes < 32) lanes *= 2;
  return lanes;
}

template <typename T, int V, int NP, int U>
qat_status fwd(const RopeArgs& r, cudaStream_t s) {
  const int lanes = group_lanes(r.d, V);
  // Heads a group takes (they share a token's angles and weights): as many as
  // leave two waves of full SMs.
  const int64_t rows = r.tokens * (r.heads[0] + r.heads[1]);
  const int64_t want = (int64_t)device_info().sms * 4096 / lanes;
  int per = 1;
  while (per < 8 && rows / (2 * per) >= want) per *= 2;
  const int64_t items = r.tokens * ((r.heads[0] + per - 1) / per + (r.heads[1] + per - 1) / per);
  const int64_t blocks = (items * lanes + kRopeThreads - 1) / kRopeThreads;
  if (blocks > INT32_MAX) return QAT_ERR_INVALID_ARGUMENT;
  auto k = r.interleaved ? k_rope_fwd<T, V, NP, U, true> : k_rope_fwd<T, V, NP, U, false>;
  RopeArgs a = r;
  if (launch_kernel(k, dim3((unsigned)blocks), dim3(kRopeThreads), 0, s, false, a, lanes, per) !=
      cudaSuccess)
    return QAT_ERR_CUDA;
  count_launch(1);
  return QAT_OK;
}

template <typename T, int V, int NP>
qat_status bwd(const RopeArgs& r, float* ws, cudaStream_t s) {
  const int lanes = group_lanes(r.d, V), groups = kRopeThreads / lanes;
  int64_t most = 0;
  for (int i = 0; i < 2; ++i) most = r.heads[i] > most ? r.heads[i] : most;
  int per = 1;
  while (per < 8 && r.tokens * most / (2 * per) >= (int64_t)kRopeParts * groups) per *= 2;
  const int64_t blocks = (r.tokens * ((most + per - 1) / per) + groups - 1) / groups;
  const int grid = (int)(blocks < kRopeParts ? blocks : kRopeParts);
  const bool sums = r.dw[0] || r.dw[1];
  RopeArgs a = r;
  if (grid > 0) {
    auto k = r.interleaved ? k_rope_bwd<T, V, NP, true> : k_rope_bwd<T, V, NP, false>;
    if (launch_kernel(k, dim3(grid), dim3(kRopeThreads), 0, s, false, a, lanes, per, ws) !=
        cudaSuccess)
      return QAT_ERR_CUDA;
    count_launch(1);
  }
  if (sums) {
    if (launch_kernel(k_rope_join<T>, dim3((2 * r.d + 31) / 32), dim3(32, 32), 0, s, grid > 0,
                      (const float*)ws, grid, r.d, r.dw[0], r.dw[1]) != cudaSuccess)
      return QAT_ERR_CUDA;
    count_launch(1);
  }
  return QAT_OK;
}

template <typename T>
qat_status fwd_any(const RopeArgs& r, cudaStream_t s) {
  switch (run_width<T>(r)) {
    case 8: return fwd<T, 8, 1, 2>(r, s);
    case 4: return fwd<T, 4, 2, 1>(r, s);
    case 2: return fwd<T, 2, 4, 1>(r, s);
    default: return fwd<T, 1, 8, 1>(r, s);
  }
}
template <typename T>
qat_status bwd_any(const RopeArgs& r, float* ws, cudaStream_t s) {
  switch (run_width<T>(r)) {
    case 8: return bwd<T, 8, 1>(r, ws, s);
    case 4: return bwd<T, 4, 2>(r, ws, s);
    case 2: return bwd<T, 2, 4>(r, ws, s);
    default: return bwd<T, 1, 8>(r, ws, s);
  }
}

}  // namespace

qat_status launch_rope_fwd(const RopeArgs& a, qat_dtype dt, cudaStream_t s) {
  return dt == QAT_F32 ? fwd_any<F32>(a, s) : fwd_any<BF16>(a, s);
}
qat_status launch_rope_bwd(const RopeArgs& a, qat_dtype dt, float* ws, cudaStream_t s) {
  return dt == QAT_F32 ? bwd_any<F32>(a, ws, s) : bwd_any<BF16>(a, ws, s);
}

}  // namespace qat
