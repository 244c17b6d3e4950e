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
// group walks over several heads of a token, which share its angles and weights, with
// the next head's loads in flight; arithmetic is on pairs of binary32 numbers.
// Measured for 8192 tokens of 32 + 8 heads of 128 in bf16: forward 30 us (5.6 TB/s),
// backward 53 us (4.7 TB/s: 128 registers leave two blocks an SM) and its join 4.5; runs
// of two elements (heads of 80, 20 turned) 1.4 TB/s, single ones 0.7.
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
  __device__ __forceinline__ void load(const char* p) {
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
  __device__ __forceinline__ void store(char* p) const {
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

// Cosine and sine of a 2^-64 fraction of a turn: the quarter by its two top bits, the
// rest (|x| <= pi / 4) by the Taylor series, whose next terms are below 2^-25: within 6 U of m,
// U = 2^-24, with the roundings of the angle and of the steps.
__device__ __forceinline__ void turn_cos_sin(uint64_t t, float m, float& c, float& s) {
  const uint32_t top = (uint32_t)(t >> 32) + 0x20000000u;  // (an eighth of a turn on)
  const int n = (int)(top >> 30);
  const int32_t r = (int32_t)(top & 0x3fffffffu) - 0x20000000;
  const float x = __fmul_rn((float)r, 1.4629180792671596e-9f);  // 2 pi / 2^32
  const float q = __fmul_rn(x, x);
  float sr = __fmaf_rn(q, 1.0f / 362880, -1.0f / 5040), cr = __fmaf_rn(q, 1.0f / 40320, -1.0f / 720);
  sr = __fmaf_rn(q, sr, 1.0f / 120), cr = __fmaf_rn(q, cr, 1.0f / 24);
  sr = __fmaf_rn(q, sr, -1.0f / 6), cr = __fmaf_rn(q, cr, -0.5f);
  sr = __fmaf_rn(__fmul_rn(q, x), sr, x), cr = __fmaf_rn(q, cr, 1.0f);
  c = (n & 1) ? sr : cr;
  s = (n & 1) ? cr : sr;
  c = __fmul_rn(c, n == 1 || n == 2 ? -m : m);
  s = __fmul_rn(s, n >= 2 ? -m : m);
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

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// r = a b + c and r = a b over N elements, two at a time.
template <int N>
__device__ __forceinline__ void vfma(const float (&a)[N], const float (&b)[N], const float (&c)[N],
                                     float (&r)[N]) {
#pragma unroll
  for (int e = 0; e + 1 < N; e += 2) fma2(a[e], a[e + 1], b[e], b[e + 1], c[e], c[e + 1], r[e], r[e + 1]);
  if (N & 1) r[N - 1] = __fmaf_rn(a[N - 1], b[N - 1], c[N - 1]);
}
template <int N>
__device__ __forceinline__ void vmul(const float (&a)[N], const float (&b)[N], float (&r)[N]) {
#pragma unroll
  for (int e = 0; e + 1 < N; e += 2) mul2(a[e], a[e + 1], b[e], b[e + 1], r[e], r[e + 1]);
  if (N & 1) r[N - 1] = __fmul_rn(a[N - 1], b[N - 1]);
}
template <int N>
__device__ __forceinline__ void vmul(const float (&a)[N], float b, float (&r)[N]) {
#pragma unroll
  for (int e = 0; e + 1 < N; e += 2) mul2(a[e], a[e + 1], b, b, r[e], r[e + 1]);
  if (N & 1) r[N - 1] = __fmul_rn(a[N - 1], b);
}
template <int N>
__device__ __forceinline__ void vfma(const float (&a)[N], float b, const float (&c)[N], float (&r)[N]) {
#pragma unroll
  for (int e = 0; e + 1 < N; e += 2) fma2(a[e], a[e + 1], b, b, c[e], c[e + 1], r[e], r[e + 1]);
  if (N & 1) r[N - 1] = __fmaf_rn(a[N - 1], b, c[N - 1]);
}
template <int N>
__device__ __forceinline__ float vsum(const float (&a)[N]) {
  if constexpr (N == 1) {
    return a[0];
  } else if constexpr (N == 2) {
    return a[0] + a[1];
  } else {
    float x = a[0], y = a[1];
#pragma unroll
    for (int e = 2; e < N; e += 2) add2(x, y, a[e], a[e + 1], x, y);
    return x + y;
  }
}

// A lane's units of one head, u = lane + lanes * p: the bytes where their runs lie,
// and whether their pairs are turned.
template <typename T, int V, int NP, bool INTER>
struct Units {
  int a[NP], b[NP];
  bool has_a[NP], has_b[NP], turned[NP];
  __device__ __forceinline__ Units(int lane, int lanes, int d, int rotary) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int u = lane + lanes * p;
      unit_runs<V, INTER>(u, rotary, a[p], b[p]);
      turned[p] = u < rotary / (2 * V);
      has_a[p] = a[p] < d;
      has_b[p] = has_a[p] && b[p] < d;
      a[p] *= T::BYTES, b[p] *= T::BYTES;
    }
  }
};

// The first and second elements of a unit's V pairs, from its runs and back.
template <typename T, int V, bool INTER>
struct Pairs {
  Run<T, V> ra, rb;
  // from a head at p: the runs at bytes a and b of it, where there are any
  __device__ __forceinline__ void load(const char* p, int a, int b, bool ha, bool hb) {
    ra.zero(), rb.zero();
    if (ha) ra.load(p + a);
    if (hb) rb.load(p + b);
  }
  __device__ __forceinline__ void get(float (&x)[V], float (&y)[V]) const {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (INTER) {
        x[e] = 2 * e < V ? ra.get(2 * e) : rb.get(2 * e - V);
        y[e] = 2 * e + 1 < V ? ra.get(2 * e + 1) : rb.get(2 * e + 1 - V);
      } else {
        x[e] = ra.get(e), y[e] = rb.get(e);
      }
    }
  }
  __device__ __forceinline__ void put(const float (&x)[V], const float (&y)[V]) {
    float v[2 * V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[INTER ? 2 * e : e] = x[e];
      v[INTER ? 2 * e + 1 : V + e] = y[e];
    }
    ra.set(v), rb.set(v + V);
  }
  __device__ __forceinline__ void store(char* p, int a, int b, bool ha, bool hb) const {
    if (ha) ra.store(p + a);
    if (hb) rb.store(p + b);
  }
};

template <typename T, int V, int NP, bool INTER>
__device__ __forceinline__ void load_weight(const void* w, const Units<T, V, NP, INTER>& un,
                                            float (&wa)[NP][V], float (&wb)[NP][V]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if (w) {
      Pairs<T, V, INTER> x;
      x.load(static_cast<const char*>(w), un.a[p], un.b[p], un.has_a[p], un.has_b[p]);
      x.get(wa[p], wb[p]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) wa[p][e] = wb[p][e] = 1.0f;
    }
  }
}

template <int V, int NP>
__device__ __forceinline__ void load_angles(const RopeArgs& r, int64_t token, int lane, int lanes,
                                            float (&c)[NP][V], float (&s)[NP][V]) {
  const uint64_t pos = (uint64_t)__ldg(r.positions + token);
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int j = (lane + lanes * p) * V + e;
      c[p][e] = 1.0f, s[p][e] = 0.0f;
      if (j < r.rotary / 2) turn_cos_sin(pos * __ldg(r.turns + j), r.amplitude, c[p][e], s[p][e]);
    }
}

__device__ __forceinline__ float rstd_of(const RopeArgs& r, float sum) {
  return rsqrtf(__fmaf_rn(sum, r.inv_d, r.eps));
}

constexpr int kRopeThreads = 256;

// Blocks (x: tokens, y: runs of `per` heads, the queries' first), a group a token.
// All lanes of a warp take the same number of steps (shuffles).
template <typename T, int V, int NP, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, V == 8 && T::BYTES == 2 ? 3 : 2)
    k_rope_fwd(RopeArgs r, int lanes, int per, int runs0) {
  using P = Pairs<T, V, INTER>;
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t token = (int64_t)blockIdx.x * (kRopeThreads / lanes) + threadIdx.x / lanes;
  const int which = (int)blockIdx.y >= runs0;
  const int h0 = ((int)blockIdx.y - (which ? runs0 : 0)) * per;
  const int steps = min(per, r.heads[which] - h0);
  const bool on = token < r.tokens;
  const Units<T, V, NP, INTER> un(lane, lanes, r.d, r.rotary);
  const int64_t x_step = r.head_stride[which] * T::BYTES, y_step = (int64_t)r.d * T::BYTES;
  const char* x = static_cast<const char*>(r.x[which]) +
                  (on ? token * r.token_stride[which] * T::BYTES + h0 * x_step : 0);
  char* y = static_cast<char*>(r.y[which]) + (on ? (token * r.heads[which] + h0) * y_step : 0);

  P next[NP];
  auto fetch = [&]() {
#pragma unroll
    for (int p = 0; p < NP; ++p)
      next[p].load(x, un.a[p], un.b[p], on && un.has_a[p], on && un.has_b[p]);
    x += x_step;
  };
  fetch();
  // a' = (a wa c - b wb s) rstd, b' = (b wb c + a wa s) rstd
  float ac[NP][V], bs[NP][V], bc[NP][V], as[NP][V];
  {
    float wa[NP][V], wb[NP][V], c[NP][V], s[NP][V];
    load_weight<T, V, NP, INTER>(r.w[which], un, wa, wb);
    load_angles<V, NP>(r, on ? token : 0, lane, lanes, c, s);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      vmul(wa[p], c[p], ac[p]);
      vmul(wb[p], s[p], bs[p]);
      vmul(bs[p], -1.0f, bs[p]);
      vmul(wb[p], c[p], bc[p]);
      vmul(wa[p], s[p], as[p]);
    }
  }
  for (int h = 0; h < steps; ++h) {
    P now[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) now[p] = next[p];
    if (h + 1 < steps) fetch();
    float a[NP][V], b[NP][V], sq[V] = {};
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      now[p].get(a[p], b[p]);
      if (r.norm) vfma(a[p], a[p], sq, sq), vfma(b[p], b[p], sq, sq);
    }
    const float rstd = r.norm ? rstd_of(r, group_sum(vsum(sq), lanes)) : 1.0f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      float u[V], v[V];
      vmul(a[p], ac[p], u);
      vmul(b[p], bc[p], v);
      if (un.turned[p]) {  // (0 times what is not finite would not pass the others as they are)
        vfma(b[p], bs[p], u, u);
        vfma(a[p], as[p], v, v);
      }
      vmul(u, rstd, u);
      vmul(v, rstd, v);
      now[p].put(u, v);
      now[p].store(y, un.a[p], un.b[p], on && un.has_a[p], on && un.has_b[p]);
    }
    y += y_step;
  }
}

// The same walk with the gradients, the first `blocks0` blocks over the queries, the
// others over the keys; each lane keeps its elements' share of dweight, and a block's
// shares are added over its groups in shared memory, in order.
template <typename T, int V, int NP, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, V == 8 && T::BYTES == 2 ? 2 : 1)
    k_rope_bwd(RopeArgs r, int lanes, int per, int blocks0, float* parts) {
  using P = Pairs<T, V, INTER>;
  __shared__ float share[kRopeThreads * 2 * V * NP];
  pdl_trigger();
  const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
  const int groups = kRopeThreads / lanes;
  const Units<T, V, NP, INTER> un(lane, lanes, r.d, r.rotary);
  const int which = (int)blockIdx.x >= blocks0;
  const int64_t block = blockIdx.x - (which ? blocks0 : 0);
  const int64_t blocks = which ? gridDim.x - blocks0 : blocks0;
  {
    const int heads = r.heads[which];
    const bool sums = r.dw[which] != nullptr;
    const int runs = (heads + per - 1) / per;
    const int64_t items = r.tokens * runs;
    float wa[NP][V], wb[NP][V], da[NP][V] = {}, db[NP][V] = {};
    load_weight<T, V, NP, INTER>(r.w[which], un, wa, wb);
    // (whole blocks step together: the shuffles need every lane)
    for (int64_t base = block * groups; base < items; base += blocks * groups) {
      const int64_t item = base + group, token = item < items ? item / runs : 0;
      const int h0 = item < items ? (int)(item - token * runs) * per : 0;
      const int n = item < items ? min(per, heads - h0) : 0;
      const int64_t x_step = r.head_stride[which] * T::BYTES, g_step = (int64_t)r.d * T::BYTES;
      const char* x = static_cast<const char*>(r.x[which]) +
                      token * r.token_stride[which] * T::BYTES + h0 * x_step;
      const char* g = static_cast<const char*>(r.g[which]) + (token * heads + h0) * g_step;
      char* y = r.y[which] ? static_cast<char*>(r.y[which]) + (token * heads + h0) * g_step : nullptr;
      P next_x[NP], next_g[NP];
      auto fetch = [&](bool on) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          next_x[p].load(x, un.a[p], un.b[p], on && un.has_a[p], on && un.has_b[p]);
          next_g[p].load(g, un.a[p], un.b[p], on && un.has_a[p], on && un.has_b[p]);
        }
        x += x_step, g += g_step;
      };
      fetch(n > 0);
      float c[NP][V], s[NP][V];
      load_angles<V, NP>(r, token, lane, lanes, c, s);
      for (int h = 0; h < per; ++h) {
        P now[NP];
        float a[NP][V], b[NP][V], ga[NP][V], gb[NP][V], sq[V] = {}, gx[V] = {};
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          next_x[p].get(a[p], b[p]);
          now[p] = next_g[p];
        }
        if (h + 1 < per) fetch(h + 1 < n);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          float u[V], v[V], t[V];
          now[p].get(u, v);
          vmul(u, c[p], ga[p]);
          vmul(v, c[p], gb[p]);
          if (un.turned[p]) {
            vfma(v, s[p], ga[p], ga[p]);
            vmul(u, -1.0f, t);
            vfma(t, s[p], gb[p], gb[p]);
          }
          if (r.norm) {
            vfma(a[p], a[p], sq, sq), vfma(b[p], b[p], sq, sq);
            vmul(ga[p], wa[p], t), vfma(t, a[p], gx, gx);
            vmul(gb[p], wb[p], t), vfma(t, b[p], gx, gx);
          }
        }
        float rstd = 1.0f, mean = 0.0f;
        if (r.norm) {
          // (a step without a head: zeros, whose norm without an epsilon is not a number)
          rstd = rstd_of(r, group_sum(vsum(sq), lanes));
          if (h >= n) rstd = 0.0f;
          mean = -(group_sum(vsum(gx), lanes) * rstd) * r.inv_d;  // of g'w z
        }
        // dw += g' z; dx = (g'w - z mean) rstd
        auto finish = [&](const float (&gr)[V], const float (&w)[V], float (&z)[V], float (&dw)[V]) {
          float t[V];
          vmul(z, rstd, z);
          vfma(gr, z, dw, dw);
          vmul(gr, w, t);
          vfma(z, mean, t, t);
          vmul(t, rstd, z);
        };
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          if (r.norm) {
            finish(ga[p], wa[p], a[p], da[p]);
            finish(gb[p], wb[p], b[p], db[p]);
            now[p].put(a[p], b[p]);
          } else {
            now[p].put(ga[p], gb[p]);
          }
          const bool on = h < n && y;
          now[p].store(y, un.a[p], un.b[p], on && un.has_a[p], on && un.has_b[p]);
        }
        y += y ? g_step : 0;
      }
    }
    if (!sums) return;
    float* mine = share + (size_t)threadIdx.x * 2 * V * NP;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        mine[p * 2 * V + (INTER ? 2 * e : e)] = da[p][e];
        mine[p * 2 * V + (INTER ? 2 * e + 1 : V + e)] = db[p][e];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < lanes * NP * 2 * V; i += kRopeThreads) {
      const int ln = i / (NP * 2 * V), p = i / (2 * V) % NP, e = i % (2 * V);
      int a, b;
      unit_runs<V, INTER>(ln + lanes * p, r.rotary, a, b);
      const int at = e < V ? a + e : b + e - V;
      if (at >= r.d || a >= r.d) continue;
      float total = 0.0f;
      for (int k = 0; k < groups; ++k)
        total += share[((size_t)k * lanes + ln) * NP * 2 * V + i % (NP * 2 * V)];
      parts[(int64_t)blockIdx.x * r.d + at] = total;
    }
  }
}

// dweight from the blocks' shares: 32 columns of the queries' (y = 0) or the keys' a
// block, 32 rows at a time, in order.
template <typename T>
__global__ void __launch_bounds__(1024) k_rope_join(const float* parts, int blocks0, int blocks, int d,
                                                    void* dwq, void* dwk) {
  __shared__ float part[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  void* const dw = blockIdx.y ? dwk : dwq;
  if (!dw) return;
  const int end = blockIdx.y ? blocks : blocks0;
  float sum = 0.0f;
  pdl_wait();
  if (col < d) {
#pragma unroll 4
    for (int i = (blockIdx.y ? blocks0 : 0) + threadIdx.y; i < end; i += 32)
      sum += parts[(int64_t)i * d + col];
  }
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y || col >= d) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += part[i][threadIdx.x];
  st_elem<T>(dw, col, sum);
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

template <typename T, int V, int NP>
qat_status fwd(const RopeArgs& r, cudaStream_t s) {
  const int lanes = group_lanes(r.d, V), groups = kRopeThreads / lanes;
  // Heads a group takes (they share a token's angles and weights): as many as
  // leave two waves of full SMs.
  const int64_t rows = r.tokens * (r.heads[0] + r.heads[1]);
  const int64_t want = (int64_t)device_info().sms * 2048 / lanes;
  int per = 1;
  while (per < 8 && rows / (2 * per) >= want) per *= 2;
  const int runs0 = (r.heads[0] + per - 1) / per, runs1 = (r.heads[1] + per - 1) / per;
  const int64_t blocks = (r.tokens + groups - 1) / groups;
  if (blocks > INT32_MAX || runs0 + runs1 > 65535) return QAT_ERR_INVALID_ARGUMENT;
  auto k = r.interleaved ? k_rope_fwd<T, V, NP, true> : k_rope_fwd<T, V, NP, false>;
  if (launch_kernel(k, dim3((unsigned)blocks, runs0 + runs1), dim3(kRopeThreads), 0, s, false, r, lanes,
                    per, runs0) != cudaSuccess)
    return QAT_ERR_CUDA;
  count_launch(1);
  return QAT_OK;
}

template <typename T, int V, int NP>
qat_status bwd(const RopeArgs& r, float* ws, cudaStream_t s) {
  const int lanes = group_lanes(r.d, V), groups = kRopeThreads / lanes;
  const int64_t most = 2 * device_info().sms < kRopeParts ? 2 * device_info().sms : kRopeParts;
  const int64_t all = r.heads[0] + r.heads[1];
  int per = 1;
  while (per < 8 && r.tokens * all / (2 * per) >= most * groups) per *= 2;
  // Blocks of both in proportion to their heads.
  int64_t need[2];
  for (int i = 0; i < 2; ++i)
    need[i] = (r.tokens * ((r.heads[i] + per - 1) / per) + groups - 1) / groups;
  if (need[0] + need[1] > most) {
    const int64_t q = (most * r.heads[0] + all / 2) / all;
    const int64_t floor0 = r.heads[0] ? 1 : 0, ceil0 = r.heads[1] ? most - 1 : most;
    need[0] = q < floor0 ? floor0 : q > ceil0 ? ceil0 : q;
    need[1] = most - need[0];
  }
  const int grid = (int)(need[0] + need[1]), blocks0 = (int)need[0];
  if (grid > 0) {
    auto k = r.interleaved ? k_rope_bwd<T, V, NP, true> : k_rope_bwd<T, V, NP, false>;
    if (launch_kernel(k, dim3(grid), dim3(kRopeThreads), 0, s, false, r, lanes, per, blocks0, ws) !=
        cudaSuccess)
      return QAT_ERR_CUDA;
    count_launch(1);
  }
  if (r.dw[0] || r.dw[1]) {
    if (launch_kernel(k_rope_join<T>, dim3((r.d + 31) / 32, 2), dim3(32, 32), 0, s, grid > 0,
                      (const float*)ws, blocks0, grid, r.d, r.dw[0], r.dw[1]) != cudaSuccess)
      return QAT_ERR_CUDA;
    count_launch(1);
  }
  return QAT_OK;
}

// Units a lane of a head holds where 32 lanes are too few: kernels for as few as there
// are (the others' steps would be empty).
template <typename T, typename F>
qat_status by_width(const RopeArgs& r, F f) {
  const int v = run_width<T>(r), units = (r.d + 2 * v - 1) / (2 * v);
  switch (v) {
    case 8: return f.template operator()<8, 1>();
    case 4: return units <= 32 ? f.template operator()<4, 1>() : f.template operator()<4, 2>();
    case 2: return units <= 32 ? f.template operator()<2, 1>() : f.template operator()<2, 4>();
    default:
      return units <= 32   ? f.template operator()<1, 1>()
             : units <= 64 ? f.template operator()<1, 2>()
                           : f.template operator()<1, 8>();
  }
}
template <typename T>
struct Fwd {
  const RopeArgs& r;
  cudaStream_t s;
  template <int V, int NP>
  qat_status operator()() const {
    return fwd<T, V, NP>(r, s);
  }
};
template <typename T>
struct Bwd {
  const RopeArgs& r;
  float* ws;
  cudaStream_t s;
  template <int V, int NP>
  qat_status operator()() const {
    return bwd<T, V, NP>(r, ws, s);
  }
};

}  // namespace

qat_status launch_rope_fwd(const RopeArgs& a, qat_dtype dt, cudaStream_t s) {
  return dt == QAT_F32 ? by_width<F32>(a, Fwd<F32>{a, s}) : by_width<BF16>(a, Fwd<BF16>{a, s});
}
qat_status launch_rope_bwd(const RopeArgs& a, qat_dtype dt, float* ws, cudaStream_t s) {
  return dt == QAT_F32 ? by_width<F32>(a, Bwd<F32>{a, ws, s}) : by_width<BF16>(a, Bwd<BF16>{a, ws, s});
}

}  // namespace qat
