// qat_dense.h -- the tensor-core product behind the gated feed-forward block
// (internal; not part of the C ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qat.h"
#include "qat_launch.h"

namespace qat {

enum { kDenseStore = 0, kDenseGated = 1, kDenseGatedBwd = 2 };

// A bf16 operand whose rows (m or n) or whose depth (k) is contiguous.
// 16-byte aligned, pitch a multiple of 8 elements.
struct DenseOp {
  const void* p;
  int64_t pitch;   // elements between rows (K-major) or between k (MN-major)
  bool mn_major;
  int64_t part;    // elements between the parts of an fp32 operand
};

// C[m, n] = sum_s A_s B_s^T (store: segs 1 or 2; with problems = 2 two outputs
// c[i] = A_i B_0^T), or gated: g = A B_0^T, u = A B_1^T, c[0] = act(g) * u (and
// g, u kept in gp, up), or gated_bwd: dh = A B^T, dg = dh * up * act'(gp),
// du = dh * act(gp).  Outputs are [m, n] without padding.
struct Dense {
  int epi;
  int64_t m, n, k;
  int segs = 1, problems = 1, parts = 1;
  DenseOp a[2], b[2];
  int act = 0;
  void* c[2] = {nullptr, nullptr};
  float* gp = nullptr;
  float* up = nullptr;
  void* dg = nullptr;
  void* du = nullptr;
  int32_t* flags = nullptr;
};
qat_status launch_dense(const Dense& d, cudaStream_t s);

}  // namespace qat
