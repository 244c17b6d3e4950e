// qat_layer.h -- launchers of the layer operators (internal; not part of the
// C ABI).  Arguments are validated by qat_layer_abi.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qat.h"
#include "qat_launch.h"

namespace qat {

// Products with 4-bit weights (y in x's dtype) and the gated block from codes.
// (none for a 16-byte aligned bf16 x)
size_t linear4_ws_bytes(const void* x, qat_dtype dt, int64_t tokens, int64_t cols);
qat_status launch_linear4(const void* x, qat_dtype dt, int64_t tokens, const qat_weight4& w, void* y,
                          void* ws, cudaStream_t s);
size_t gated4_ws_bytes(int64_t tokens, int64_t dim, int64_t hidden);
qat_status launch_gated4(const void* x, qat_dtype dt, int64_t tokens, const qat_weight4* gate_up,
                         const qat_weight4& down, int act, void* y, void* ws, cudaStream_t s);

// Row partials of dweight / dbias that the layer norm's backward pass keeps in
// its workspace: [2][parts][cols] floats.  Enough parts for every resident
// block: eight 128-thread blocks a SM for short rows, four from there on.
constexpr int norm_parts(int64_t rows, int64_t cols) {
  const int most = cols <= 1024 ? 1216 : 608;
  return rows < most ? (int)rows : most;
}
qat_status launch_norm_fwd(const void* x, qat_dtype dt, int64_t rows, int64_t cols, const void* w,
                           const void* b, float eps, void* y, float* mean, float* rstd,
                           cudaStream_t s);
qat_status launch_norm_bwd(const void* dy, const void* x, qat_dtype dt, int64_t rows, int64_t cols,
                           const void* w, const float* mean, const float* rstd, void* dx, void* dw,
                           void* db, float* ws, cudaStream_t s);

size_t ffn_ws_bytes(qat_dtype dt, int64_t tokens, int64_t dim, int64_t hidden, bool backward);
qat_status launch_ffn_fwd(const void* x, qat_dtype dt, int64_t t, int64_t d, int64_t f,
                          const void* wg, const void* wu, const void* wd, int act, void* h,
                          float* gp, float* up, void* y, int32_t* flags, void* ws, cudaStream_t s);
qat_status launch_ffn_bwd(const void* dy, const void* x, qat_dtype dt, int64_t t, int64_t d,
                          int64_t f, const void* wg, const void* wu, const void* wd, int act,
                          const void* h, const float* gp, const float* up, void* dx, void* dwg,
                          void* dwu, void* dwd, int32_t* flags, void* ws, cudaStream_t s);

}  // namespace qat
