// kernels_few.cu -- binary32 products of a few tokens with a weight that is read
// as it is, for the gated feed-forward block.
//
//   rows:    out[t, n] = sum_k a[t, k] W[n, k]        (and the gated pair)
//   columns: out[t, c] = sum_r a[t, r] W[r, c]        (one or two such sums)
//
// The tensor cores take fp32 weights as three bf16 parts that have to be written
// first, 10 bytes moved an element before the product starts; for up to 32
// tokens reading the weight itself, once per 16 tokens, moves less.  Scalar
// multiply-adds suffice: 16 tokens cost three quarters of their rate at the copy
// bandwidth.  a is staged in shared memory; sums are binary32.
//
// Measured (GPU time of a call in us with a cold L2, here / on the tensor cores):
//
//   dim x hidden     tokens  forward      backward
//   4096 x 14336     16      232 / 657    674 / 955
//                    17      433 / 658    958 / 955
//                    32      448 / 658    1011 / 956
//   1024 x 4096      16      54 / 79      110 / 130
//                    32      75 / 79      124 / 130
//   510 x 1363       16      44 / 42      81 / 71
//                    32      53 / 42      77 / 73
//
// One token by 4096 x 14336 takes 123 us forward (reading the weights takes 104).  From
// 16 tokens on the multiply-adds bound it.  One limit for both passes and all layers:
// past 16 tokens the backward pass of a large layer loses up to 6% by it, and a layer
// whose weights are a few MB, where launches are all that counts, up to 27% of one
// pass; the forward pass of a large layer gains a third to two thirds.

#include "qat_few.h"
#include "qat_layer.cuh"
#include "qat_tc.cuh"

namespace qat {

constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;

struct FewArgs {
  const float* a[2];
  const float* w[2];
  int64_t t, n, k;  // tokens, outputs, length of a sum
  int act, split;
  float* out[2];
  float* gp;
  float* up;
};

// ---------------------------------------------------------------------------
// Rows: a warp takes four weight rows (two of each of the gated pair), lanes
// along k; the next chunk of a is copied while this one is multiplied.
// ---------------------------------------------------------------------------
constexpr int kRowChunk = 512;  // k of a chunk

template <int TT, int NW, bool VEC>
__global__ void __launch_bounds__(kFewThreads, 1) k_few_rows(const __grid_constant__ FewArgs p) {
  constexpr int RW = 4 / NW, STEPS = kRowChunk / 128;
  extern __shared__ __align__(16) float xs[];  // [2][TT][kRowChunk]
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.y * TT;
  const int tokens = (int)min((int64_t)TT, p.t - t0);
  const int64_t n0 = ((int64_t)blockIdx.x * kFewWarps + warp) * RW;
  // element e of step s of this lane
  const auto at = [&](int s, int e) { return VEC ? s * 128 + lane * 4 + e : s * 128 + e * 32 + lane; };
  const float* row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = n0 + i % RW;
    row[i] = p.w[i / RW] + (n < p.n ? n : 0) * p.k;
  }
  const auto stage = [&](int64_t k0, int b) {
    float* to = xs + b * TT * kRowChunk;
    if (k0 < p.k) {
      if (VEC) {
        for (int i = threadIdx.x * 4; i < TT * kRowChunk; i += kFewThreads * 4) {
          const int t = i / kRowChunk, k = i % kRowChunk;
          if (t < tokens && k0 + k < p.k)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem(to + i)),
                         "l"(p.a[0] + (t0 + t) * p.k + k0 + k)
                         : "memory");
          else
            *reinterpret_cast<float4*>(to + i) = make_float4(0, 0, 0, 0);
        }
      } else {
        for (int i = threadIdx.x; i < TT * kRowChunk; i += kFewThreads) {
          const int t = i / kRowChunk, k = i % kRowChunk;
          to[i] = t < tokens && k0 + k < p.k ? p.a[0][(t0 + t) * p.k + k0 + k] : 0.0f;
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float acc[4][TT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = 0.0f;
  stage(0, 0);
  int b = 0;
  for (int64_t k0 = 0; k0 < p.k; k0 += kRowChunk, b ^= 1) {
    float w[STEPS][4][4];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (VEC) {
          float4 v = make_float4(0, 0, 0, 0);
          if (k0 + at(s, 0) < p.k) v = __ldcs(reinterpret_cast<const float4*>(row[i] + k0 + at(s, 0)));
          w[s][i][0] = v.x, w[s][i][1] = v.y, w[s][i][2] = v.z, w[s][i][3] = v.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[s][i][e] = k0 + at(s, e) < p.k ? __ldcs(row[i] + k0 + at(s, e)) : 0.0f;
        }
      }
    stage(k0 + kRowChunk, b ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const float* x = xs + b * TT * kRowChunk;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        float v[4];
        if constexpr (VEC) {
          const float4 q = *reinterpret_cast<const float4*>(x + t * kRowChunk + at(s, 0));
          v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = x[t * kRowChunk + at(s, e)];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][t] = fmaf(w[s][i][e], v[e], acc[i][t]);
      }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[i][t] += __shfl_xor_sync(~0u, acc[i][t], o);
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int64_t n = n0 + i;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (lane != t || t >= tokens || n >= p.n) continue;  // a lane a token
      const int64_t o = (t0 + t) * p.n + n;
      const float v = acc[i][t];
      if (NW == 2) {
        const float u = acc[(i + RW) & 3][t];
        p.out[0][o] = act_value<false>(p.act, v) * u;
        if (p.gp) {
          p.gp[o] = v;
          p.up[o] = u;
        }
      } else {
        p.out[0][o] = v;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Columns: a block takes 128 columns (a thread four), its warps and the blocks of
// a cluster share the rows, whose sums are added in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kColChunk = 64;  // rows of a chunk

template <int TT, bool BWD, bool VEC>
__global__ void __launch_bounds__(kFewThreads, 2) k_few_cols(const __grid_constant__ FewArgs p, int terms) {
  extern __shared__ __align__(16) float sm[];  // a chunk [kColChunk][TT + 4]; then [warps][TT][128]
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, split = p.split;
  const int rank = split > 1 ? (int)(blockIdx.x % split) : 0;
  const int64_t c0 = (int64_t)(blockIdx.x / split) * 128;
  const int64_t t0 = (int64_t)blockIdx.y * TT;
  const int tokens = (int)min((int64_t)TT, p.t - t0);
  const auto col = [&](int j) { return VEC ? lane * 4 + j : j * 32 + lane; };
  const int64_t all = p.k * terms;  // rows of both terms, one after the other
  const int64_t r0 = all * rank / split, r1 = all * (rank + 1) / split;
  float acc[4][TT];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[j][t] = 0.0f;
  constexpr int PER = kColChunk / kFewWarps;  // rows of a chunk a warp
  constexpr int EACH = (kColChunk * TT + kFewThreads - 1) / kFewThreads;  // of a chunk of a, a thread
  constexpr int PITCH = TT + 4;  // neighbouring rows in different banks
  for (int64_t q0 = r0; q0 < r1; q0 += kColChunk) {
    float av[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int at = threadIdx.x + i * kFewThreads, t = at / kColChunk;
      const int64_t q = q0 + at % kColChunk;
      av[i] = 0.0f;
      if (t < tokens && q < r1)
        av[i] = q < p.k ? p.a[0][(t0 + t) * p.k + q] : p.a[1][(t0 + t) * p.k + q - p.k];
    }
    float w[PER][4];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t q = q0 + i * kFewWarps + warp;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i][j] = 0.0f;
      if (q >= r1) continue;
      const float* base = (q < p.k ? p.w[0] + q * p.n : p.w[1] + (q - p.k) * p.n) + c0;
      if constexpr (VEC) {
        if (c0 + col(0) < p.n) {
          const float4 v = __ldcs(reinterpret_cast<const float4*>(base + col(0)));
          w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c0 + col(j) < p.n) w[i][j] = __ldcs(base + col(j));
      }
    }
    __syncthreads();  // the previous chunk has been used
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int at = threadIdx.x + i * kFewThreads;
      if (at < kColChunk * TT) sm[at % kColChunk * PITCH + at / kColChunk] = av[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float* a = sm + (i * kFewWarps + warp) * PITCH;
#pragma unroll
      for (int t = 0; t < TT; t += 4) {
        const float4 v = *reinterpret_cast<const float4*>(a + t);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[j][t] = fmaf(w[i][j], v.x, acc[j][t]);
          acc[j][t + 1] = fmaf(w[i][j], v.y, acc[j][t + 1]);
          acc[j][t + 2] = fmaf(w[i][j], v.z, acc[j][t + 2]);
          acc[j][t + 3] = fmaf(w[i][j], v.w, acc[j][t + 3]);
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) sm[(warp * TT + t) * 128 + col(j)] = acc[j][t];
  __syncthreads();
  if (split > 1) {
    for (int i = threadIdx.x; i < tokens * 128; i += kFewThreads) {
      float v = sm[i];
#pragma unroll
      for (int w = 1; w < kFewWarps; ++w) v += sm[w * TT * 128 + i];
      sm[i] = v;
    }
    tc::cluster_sync();
  }
  for (int i = threadIdx.x + rank * kFewThreads; i < tokens * 128; i += kFewThreads * split) {
    const int64_t c = c0 + i % 128;
    if (c >= p.n) continue;
    float v = 0.0f;
    if (split > 1) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (q >= split) break;
        v += tc::ld_cluster(tc::map_rank(tc::smem(sm + i), q));
      }
    } else {
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) v += sm[w * TT * 128 + i];
    }
    const int64_t o = (t0 + i / 128) * p.n + c;
    if (BWD) {
      float a, da;
      act_grad<false>(p.act, p.gp[o], a, da);
      p.out[0][o] = v * p.up[o] * da;
      p.out[1][o] = v * a;
    } else {
      p.out[0][o] = v;
    }
  }
  if (split > 1) tc::cluster_sync();  // the other blocks have read sm
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
template <typename... A>
static qat_status go(void (*kernel)(A...), dim3 grid, int smem, int cluster, bool pdl, cudaStream_t s,
                     A... args) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return QAT_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
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
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return QAT_ERR_CUDA;
  }
  count_launch(1);
  return QAT_OK;
}

template <int TT, int NW>
static qat_status rows(const FewArgs& p, bool pdl, cudaStream_t s) {
  const bool vec = p.k % 4 == 0;
  const int64_t per = kFewWarps * (4 / NW);
  const dim3 grid((unsigned)((p.n + per - 1) / per), (unsigned)((p.t + TT - 1) / TT));
  const int smem = 2 * TT * kRowChunk * 4;
  return vec ? go(k_few_rows<TT, NW, true>, grid, smem, 1, pdl, s, p)
             : go(k_few_rows<TT, NW, false>, grid, smem, 1, pdl, s, p);
}
template <int TT, bool BWD>
static qat_status cols(FewArgs p, int terms, bool pdl, cudaStream_t s) {
  const bool vec = p.n % 4 == 0;
  const int64_t tiles = (p.n + 127) / 128, tt = (p.t + TT - 1) / TT;
  // a cluster shares the rows while there is room for it and four chunks each
  p.split = 1;
  while (p.split < 8 && tiles * tt * p.split < 2 * device_info().sms &&
         p.k * terms >= p.split * 2 * 4 * kColChunk)
    p.split *= 2;
  const dim3 grid((unsigned)(tiles * p.split), (unsigned)tt);
  const int smem = kFewWarps * TT * 128 * 4;
  return vec ? go(k_few_cols<TT, BWD, true>, grid, smem, p.split, pdl, s, p, terms)
             : go(k_few_cols<TT, BWD, false>, grid, smem, p.split, pdl, s, p, terms);
}

qat_status launch_few_gated(const float* x, int64_t t, int64_t d, int64_t f, const float* wg,
                            const float* wu, int act, float* h, float* gp, float* up, bool pdl,
                            cudaStream_t s) {
  const FewArgs p = {{x, nullptr}, {wg, wu}, t, f, d, act, 1, {h, nullptr}, gp, up};
  return t <= 4 ? rows<4, 2>(p, pdl, s) : rows<16, 2>(p, pdl, s);
}
qat_status launch_few_rows(const float* a, int64_t t, int64_t k, int64_t n, const float* w,
                           float* out, bool pdl, cudaStream_t s) {
  const FewArgs p = {{a, nullptr}, {w, nullptr}, t, n, k, 0, 1, {out, nullptr}, nullptr, nullptr};
  return t <= 4 ? rows<4, 1>(p, pdl, s) : rows<16, 1>(p, pdl, s);
}
qat_status launch_few_gated_bwd(const float* dy, int64_t t, int64_t d, int64_t f, const float* wd,
                                int act, const float* gp, const float* up, float* dg, float* du,
                                bool pdl, cudaStream_t s) {
  const FewArgs p = {{dy, dy}, {wd, wd}, t, f, d, act, 1, {dg, du}, const_cast<float*>(gp),
                     const_cast<float*>(up)};
  return t <= 4 ? cols<4, true>(p, 1, pdl, s) : cols<16, true>(p, 1, pdl, s);
}
qat_status launch_few_cols2(const float* a, const float* b, int64_t t, int64_t k, int64_t n,
                            const float* wa, const float* wb, float* out, bool pdl, cudaStream_t s) {
  const FewArgs p = {{a, b}, {wa, wb}, t, n, k, 0, 1, {out, nullptr}, nullptr, nullptr};
  return t <= 4 ? cols<4, false>(p, 2, pdl, s) : cols<16, false>(p, 2, pdl, s);
}

}  // namespace qat
