// qat_layer_abi.cu -- the exported C entry points of the layer operators:
// argument validation, then the launchers.  See include/qat.h.
#include <cmath>
#include <cstdint>

#include "qat_layer.h"

using namespace qat;

namespace {

constexpr int64_t kMaxElems = INT64_C(1) << 50;
// four rows a block of the 4-bit kernel for any shape: what gridDim.x holds
constexpr int64_t kMaxRows4 = INT64_C(4) * INT32_MAX;

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool dtype_ok(qat_dtype d) { return d == QAT_F32 || d == QAT_BF16; }
uintptr_t esize(qat_dtype d) { return d == QAT_F32 ? 4 : 2; }
// a * b with a, b >= 0 stays within the library's element limit
bool fits(int64_t a, int64_t b) { return a >= 0 && b >= 0 && (b == 0 || a <= kMaxElems / b); }
bool act_ok(qat_activation a) {
  return a == QAT_ACT_SILU || a == QAT_ACT_GELU || a == QAT_ACT_RELU;
}

qat_status check_w4(const qat_weight4* w) {
  if (!w) return QAT_ERR_INVALID_ARGUMENT;
  if (w->layout != QAT_PER_TENSOR && w->layout != QAT_PER_ROW && w->layout != QAT_PER_GROUP &&
      w->layout != QAT_W4_DOUBLE)
    return QAT_ERR_UNSUPPORTED;
  if (!fits(w->rows, w->cols) || w->rows > kMaxRows4) return QAT_ERR_INVALID_ARGUMENT;
  if (w->layout == QAT_PER_GROUP && (w->group <= 0 || w->cols % w->group))
    return QAT_ERR_INVALID_ARGUMENT;
  if (w->layout == QAT_W4_DOUBLE && w->zero_points) return QAT_ERR_INVALID_ARGUMENT;
  if (w->rows == 0 || w->cols == 0) return QAT_OK;
  if (!w->codes || !w->scales) return QAT_ERR_INVALID_ARGUMENT;
  if (w->layout == QAT_W4_DOUBLE && !w->super_scales) return QAT_ERR_INVALID_ARGUMENT;
  if (!on(w->codes, 16) || (w->layout != QAT_W4_DOUBLE && !on(w->scales, 4)) ||
      !on(w->zero_points, 4) || !on(w->super_scales, 4))
    return QAT_ERR_MISALIGNED;
  return QAT_OK;
}

bool ffn_sizes_ok(int64_t t, int64_t d, int64_t f) {
  // coordinates of the tensor copies are 32-bit
  constexpr int64_t most = INT32_MAX - 4096;
  return t <= most && d <= most && f <= most && fits(t, d) && fits(t, f) && fits(d, f);
}

}  // namespace

extern "C" {

size_t qat_linear4_workspace_bytes(qat_dtype dtype, int64_t tokens, int64_t cols) {
  if (!dtype_ok(dtype) || !fits(tokens, cols)) return 0;
  return linear4_ws_bytes(nullptr, dtype, tokens, cols);
}

qat_status qat_linear4(const void* x, qat_dtype dtype, int64_t tokens, const qat_weight4* w, void* y,
                       void* workspace, size_t workspace_bytes, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_linear4");
  if (!dtype_ok(dtype)) return QAT_ERR_UNSUPPORTED;
  const qat_status st = check_w4(w);
  if (st) return st;
  if (!fits(tokens, w->cols) || !fits(tokens, w->rows)) return QAT_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || w->rows == 0) return QAT_OK;
  if ((!x && w->cols > 0) || !y) return QAT_ERR_INVALID_ARGUMENT;
  if (!on(x, esize(dtype)) || !on(y, esize(dtype))) return QAT_ERR_MISALIGNED;
  const size_t need = linear4_ws_bytes(x, dtype, tokens, w->cols);
  if (need && (!workspace || workspace_bytes < need)) return QAT_ERR_WORKSPACE;
  if (need && !on(workspace, 16)) return QAT_ERR_MISALIGNED;
  return launch_linear4(x, dtype, tokens, *w, y, workspace, reinterpret_cast<cudaStream_t>(stream));
}

size_t qat_gated_ffn4_workspace_bytes(qat_dtype dtype, int64_t tokens, int64_t dim,
                                      int64_t hidden) {
  if (!dtype_ok(dtype) || !fits(tokens, dim) || !fits(tokens, hidden)) return 0;
  return gated4_ws_bytes(tokens, dim, hidden);
}

qat_status qat_gated_ffn4(const void* x, qat_dtype dtype, int64_t tokens, const qat_weight4* gate,
                          const qat_weight4* up, const qat_weight4* down, qat_activation act,
                          void* y, void* workspace, size_t workspace_bytes, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_gated_ffn4");
  if (!dtype_ok(dtype) || !act_ok(act)) return QAT_ERR_UNSUPPORTED;
  for (const qat_weight4* w : {gate, up, down}) {
    const qat_status st = check_w4(w);
    if (st) return st;
  }
  if (gate->rows != up->rows || gate->cols != up->cols || gate->layout != up->layout ||
      (gate->layout == QAT_PER_GROUP && gate->group != up->group) ||
      !gate->zero_points != !up->zero_points || down->cols != gate->rows)
    return QAT_ERR_DIMENSION_MISMATCH;
  if (!fits(tokens, gate->cols) || !fits(tokens, gate->rows) || !fits(tokens, down->rows))
    return QAT_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || down->rows == 0) return QAT_OK;
  if ((!x && gate->cols > 0) || !y) return QAT_ERR_INVALID_ARGUMENT;
  if (!on(x, esize(dtype)) || !on(y, esize(dtype))) return QAT_ERR_MISALIGNED;
  const size_t need = gated4_ws_bytes(tokens, gate->cols, gate->rows);
  if (need && (!workspace || workspace_bytes < need)) return QAT_ERR_WORKSPACE;
  if (need && !on(workspace, 16)) return QAT_ERR_MISALIGNED;
  const qat_weight4 both[2] = {*gate, *up};
  return launch_gated4(x, dtype, tokens, both, *down, act, y, workspace,
                       reinterpret_cast<cudaStream_t>(stream));
}

size_t qat_gated_ffn_workspace_bytes(qat_dtype dtype, int64_t tokens, int64_t dim, int64_t hidden,
                                     int backward) {
  if (!dtype_ok(dtype) || !ffn_sizes_ok(tokens, dim, hidden)) return 0;
  return ffn_ws_bytes(dtype, tokens, dim, hidden, backward != 0);
}

qat_status qat_gated_ffn(const void* x, qat_dtype dtype, int64_t tokens, int64_t dim,
                         int64_t hidden, const void* w_gate, const void* w_up, const void* w_down,
                         qat_activation act, void* h, float* gate_pre, float* up_pre, void* y,
                         int32_t* dev_flags, void* workspace, size_t workspace_bytes, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_gated_ffn");
  if (!dtype_ok(dtype) || !act_ok(act)) return QAT_ERR_UNSUPPORTED;
  if (!ffn_sizes_ok(tokens, dim, hidden)) return QAT_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || (dim == 0 && hidden == 0)) return QAT_OK;
  const bool weights = dim > 0 && hidden > 0;
  if (!gate_pre != !up_pre) return QAT_ERR_INVALID_ARGUMENT;
  if ((dim > 0 && (!x || !y)) || (hidden > 0 && !h) ||
      (weights && (!w_gate || !w_up || !w_down)))
    return QAT_ERR_INVALID_ARGUMENT;
  const uintptr_t e = esize(dtype);
  if (!on(x, 16) || !on(w_gate, 16) || !on(w_up, 16) || !on(w_down, 16) || !on(h, 16) ||
      !on(y, e) || !on(gate_pre, 4) || !on(up_pre, 4) || !on(dev_flags, 4))
    return QAT_ERR_MISALIGNED;
  const size_t need = ffn_ws_bytes(dtype, tokens, dim, hidden, false);
  if (need && (!workspace || workspace_bytes < need)) return QAT_ERR_WORKSPACE;
  if (need && !on(workspace, 16)) return QAT_ERR_MISALIGNED;
  return launch_ffn_fwd(x, dtype, tokens, dim, hidden, w_gate, w_up, w_down, act, h, gate_pre,
                        up_pre, y, dev_flags, workspace, reinterpret_cast<cudaStream_t>(stream));
}

qat_status qat_gated_ffn_backward(const void* dy, const void* x, qat_dtype dtype, int64_t tokens,
                                  int64_t dim, int64_t hidden, const void* w_gate,
                                  const void* w_up, const void* w_down, qat_activation act,
                                  const void* h, const float* gate_pre, const float* up_pre,
                                  void* dx, void* dw_gate, void* dw_up, void* dw_down,
                                  int32_t* dev_flags, void* workspace, size_t workspace_bytes, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_gated_ffn_backward");
  if (!dtype_ok(dtype) || !act_ok(act)) return QAT_ERR_UNSUPPORTED;
  if (!ffn_sizes_ok(tokens, dim, hidden)) return QAT_ERR_INVALID_ARGUMENT;
  if (dim == 0 || (tokens == 0 && hidden == 0)) return QAT_OK;
  if ((tokens > 0 && (!dy || !x)) || (hidden > 0 && (!w_gate || !w_up || !w_down)) ||
      (tokens > 0 && hidden > 0 && (!h || !gate_pre || !up_pre)))
    return QAT_ERR_INVALID_ARGUMENT;
  const uintptr_t e = esize(dtype);
  if (!on(dy, 16) || !on(x, 16) || !on(w_gate, 16) || !on(w_up, 16) || !on(w_down, 16) ||
      !on(h, 16) || !on(gate_pre, 4) || !on(up_pre, 4) || !on(dx, e) || !on(dw_gate, e) || !on(dw_up, e) ||
      !on(dw_down, e) || !on(dev_flags, 4))
    return QAT_ERR_MISALIGNED;
  const size_t need = ffn_ws_bytes(dtype, tokens, dim, hidden, true);
  if (need && (!workspace || workspace_bytes < need)) return QAT_ERR_WORKSPACE;
  if (need && !on(workspace, 16)) return QAT_ERR_MISALIGNED;
  return launch_ffn_bwd(dy, x, dtype, tokens, dim, hidden, w_gate, w_up, w_down, act, h, gate_pre,
                        up_pre, dx, dw_gate, dw_up, dw_down, dev_flags, workspace,
                        reinterpret_cast<cudaStream_t>(stream));
}

qat_status qat_layer_norm(const void* x, qat_dtype dtype, int64_t rows, int64_t cols,
                          const void* weight, const void* bias, float eps, void* y, float* mean,
                          float* rstd, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_layer_norm");
  if (!dtype_ok(dtype)) return QAT_ERR_UNSUPPORTED;
  if (!fits(rows, cols) || !(eps >= 0.0f) || std::isinf(eps)) return QAT_ERR_INVALID_ARGUMENT;
  if (rows == 0 || cols == 0) return QAT_OK;
  if (!x || !y) return QAT_ERR_INVALID_ARGUMENT;
  const uintptr_t e = esize(dtype);
  if (!on(x, e) || !on(weight, e) || !on(bias, e) || !on(y, e) || !on(mean, 4) || !on(rstd, 4))
    return QAT_ERR_MISALIGNED;
  return launch_norm_fwd(x, dtype, rows, cols, weight, bias, eps, y, mean, rstd,
                         reinterpret_cast<cudaStream_t>(stream));
}

size_t qat_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (!fits(rows, cols)) return 0;
  return (size_t)norm_parts(rows, cols) * (size_t)cols * 8;
}

qat_status qat_layer_norm_backward(const void* dy, const void* x, qat_dtype dtype, int64_t rows,
                                   int64_t cols, const void* weight, const float* mean,
                                   const float* rstd, void* dx, void* dweight, void* dbias,
                                   void* workspace, size_t workspace_bytes, qat_stream_t stream) {
  qat::NvtxScope nvtx("qat_layer_norm_backward");
  if (!dtype_ok(dtype)) return QAT_ERR_UNSUPPORTED;
  if (!fits(rows, cols)) return QAT_ERR_INVALID_ARGUMENT;
  if (cols == 0 || (rows == 0 && !dweight && !dbias)) return QAT_OK;
  if (rows > 0 && (!dy || !x || !mean || !rstd)) return QAT_ERR_INVALID_ARGUMENT;
  const uintptr_t e = esize(dtype);
  if (!on(dy, e) || !on(x, e) || !on(weight, e) || !on(mean, 4) || !on(rstd, 4) || !on(dx, e) ||
      !on(dweight, e) || !on(dbias, e))
    return QAT_ERR_MISALIGNED;
  if ((dweight || dbias) && rows > 0) {
    if (!workspace || workspace_bytes < qat_layer_norm_backward_workspace_bytes(rows, cols))
      return QAT_ERR_WORKSPACE;
    if (!on(workspace, 16)) return QAT_ERR_MISALIGNED;
  }
  return launch_norm_bwd(dy, x, dtype, rows, cols, weight, mean, rstd, dx, dweight, dbias,
                         static_cast<float*>(workspace), reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
