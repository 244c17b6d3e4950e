// qat_dense.h -- the tensor-core product behind the gated feed-forward block
// (internal; not part of the C ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qat.h"
#include "qat_launch.h"

namespace qat {

enum { kDenseStore = 0, kDenseGated = 1, kDenseGatedBwd = 2 };

// An operand whose rows (m or n) or whose depth (k) is contiguous, in bf16:
// 16-byte aligned, pitch a multiple of 8 elements.  An fp32 operand is three
// such parts (high, middle, low), `part` elements apart.
struct DenseOp {
  const void* p;
  int64_t pitch;   // elements between rows (K-major) or between k (MN-major)
  bool mn_major;
  int64_t part;
};

// C[m, n] = sum_s A_s B_s^T (store: segs 1 or 2; with problems = 2 two outputs
// c[i] = A_i B_0^T), or gated: g = A B_0^T, u = A B_1^T, c[0] = act(g) * u, kept
// as an operand in q[0] too where that is set, and g, u in gp, up; or
// gated_bwd: dh = A B^T, q[0] = dg = dh * up * act'(gp), q[1] = du = dh *
// act(gp).  c, gp and up are [m, n] without padding, in dtype and float; q in
// bf16 parts of pitch q_pitch.
struct Dense {
  int epi;
  qat_dtype dtype;
  int64_t m, n, k;
  int segs = 1, problems = 1;
  DenseOp a[2], b[2];
  int act = 0;
  void* c[2] = {nullptr, nullptr};
  void* q[2] = {nullptr, nullptr};
  int64_t q_pitch = 0, q_part = 0;
  float* gp = nullptr;
  float* up = nullptr;
  int32_t* flags = nullptr;
  bool pdl = false;  // the call's previous kernel may still be running
};
qat_status launch_dense(const Dense& d, cudaStream_t s);

// src [rows, cols] as an operand in dst (DenseOp: pitch, part)
struct DensePack {
  const void* src;
  int64_t rows, cols;
  void* dst;
  int64_t pitch, part;
};
qat_status launch_dense_pack(qat_dtype dt, const DensePack* list, int n, cudaStream_t s);

}  // namespace qat
