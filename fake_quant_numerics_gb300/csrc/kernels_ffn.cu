// kernels_ffn.cu -- the gated feed-forward block, forward and backward.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) * u, y = h Wd^T
//   dh = dy Wd; dg = dh * u * act'(g), du = dh * act(g)
//   dx = dg Wg + du Wu; dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// Two products forward (both projections, the activation and the product in
// the first) and four backward (dg and du in the first; dx in one sum over both;
// dWg and dWu in one launch), all on k_dense (kernels_dense.cu).  Operands it
// cannot read in place are packed into the workspace first.
//
// Roundings: h is rounded to the layer's type, as the tensor cores take it, and
// dg and du likewise; g and u are kept in binary32 for the backward pass (a bf16
// copy would double the error of dg).  A bf16 layer's outputs are then 0.0023 to
// 0.0025 of their norm off, where results that are rounded only once are 0.0017 off;
// two bf16 parts each of h, dg and du would close that, for a third more products
// forward and five sixths more backward.
#include "qat_dense.h"
#include "qat_few.h"
#include "qat_layer.h"

namespace qat {

static size_t r256(size_t b) { return (b + 255) / 256 * 256; }

// Lays operands out in the workspace, then packs them in one launch.  With base
// 0 it only counts the bytes.
struct Packer {
  qat_dtype dt;
  uintptr_t base;
  size_t used = 0;
  DensePack list[6];
  int n = 0;

  int64_t parts() const { return dt == QAT_F32 ? 3 : 1; }
  // room for a [rows, cols] operand; its pitch and part
  void* room(int64_t rows, int64_t cols, int64_t* pitch, int64_t* part) {
    *pitch = (cols + 7) / 8 * 8;
    *part = (rows * *pitch + 7) / 8 * 8;
    const uintptr_t p = base + used;
    used += r256((size_t)(*part * parts()) * 2);
    return reinterpret_cast<void*>(p);
  }
  // the operand itself where it can be read in place, else its packed copy
  DenseOp operand(const void* p, int64_t rows, int64_t cols) {
    if (dt == QAT_BF16 && cols % 8 == 0) return DenseOp{p, cols, false, 0};
    DensePack k = {p, rows, cols, nullptr, 0, 0};
    k.dst = room(rows, cols, &k.pitch, &k.part);
    list[n++] = k;
    return DenseOp{k.dst, k.pitch, false, k.part};
  }
  qat_status go(cudaStream_t s) { return launch_dense_pack(dt, list, n, s); }
  // whether a kernel of this call has been launched before
  bool launched = false;
  bool next() {
    const bool was = launched || n > 0;
    launched = true;
    return was;
  }
};
// the same matrix read along its rows
static DenseOp turned(DenseOp o) {
  o.mn_major = true;
  return o;
}

struct FwdOps {
  DenseOp x, wg, wu, wd, h;
  bool keep_h;  // h as an operand beside the caller's
};
static FwdOps fwd_ops(Packer& w, int64_t t, int64_t d, int64_t f, const void* x, const void* wg,
                      const void* wu, const void* wd, void* h) {
  FwdOps o;
  o.x = w.operand(x, t, d);
  o.wg = w.operand(wg, f, d);
  o.wu = w.operand(wu, f, d);
  o.wd = w.operand(wd, d, f);
  o.keep_h = w.dt == QAT_F32 || f % 8;
  o.h = DenseOp{h, f, false, 0};
  if (o.keep_h) o.h.p = w.room(t, f, &o.h.pitch, &o.h.part);
  return o;
}

// fp32 layers of a few tokens read their weights as they are.
static bool few(qat_dtype dt, int64_t t) { return dt == QAT_F32 && t <= kFewTokens; }

// The backward pass of a few fp32 tokens: dg and du in binary32, then they and
// the tokens as operands of the weight gradients (t is short there, the weights
// are outputs).
struct FewOps {
  float *dg32, *du32;
  DenseOp dy, x, h, dg, du;
};
static FewOps few_ops(Packer& w, int64_t t, int64_t d, int64_t f, const void* dy, const void* x,
                      const void* h) {
  FewOps o;
  const size_t bytes = r256((size_t)t * f * 4);
  o.dg32 = reinterpret_cast<float*>(w.base + w.used);
  o.du32 = reinterpret_cast<float*>(w.base + w.used + bytes);
  w.used += 2 * bytes;
  o.dy = w.operand(dy, t, d);
  o.x = w.operand(x, t, d);
  o.h = w.operand(h, t, f);
  o.dg = w.operand(o.dg32, t, f);
  o.du = w.operand(o.du32, t, f);
  return o;
}

struct BwdOps {
  DenseOp dy, x, wg, wu, wd, h, dg, du;
};
static BwdOps bwd_ops(Packer& w, int64_t t, int64_t d, int64_t f, const void* dy, const void* x,
                      const void* wg, const void* wu, const void* wd, const void* h) {
  BwdOps o;
  o.dy = w.operand(dy, t, d);
  o.x = w.operand(x, t, d);
  o.wg = w.operand(wg, f, d);
  o.wu = w.operand(wu, f, d);
  o.wd = w.operand(wd, d, f);
  o.h = w.operand(h, t, f);
  o.dg = o.du = DenseOp{};
  o.dg.p = w.room(t, f, &o.dg.pitch, &o.dg.part);
  o.du.p = w.room(t, f, &o.du.pitch, &o.du.part);
  return o;
}

size_t ffn_ws_bytes(qat_dtype dt, int64_t t, int64_t d, int64_t f, bool backward) {
  Packer w = {dt, 0};
  if (few(dt, t)) {
    if (backward) few_ops(w, t, d, f, nullptr, nullptr, nullptr);
    return w.used;
  }
  if (backward)
    bwd_ops(w, t, d, f, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  else
    fwd_ops(w, t, d, f, nullptr, nullptr, nullptr, nullptr, nullptr);
  return w.used;
}

static qat_status zero(void* p, int64_t n, qat_dtype dt, cudaStream_t s) {
  if (!p || n == 0) return QAT_OK;
  if (cudaMemsetAsync(p, 0, (size_t)n * (dt == QAT_F32 ? 4 : 2), s) == cudaSuccess) return QAT_OK;
  (void)cudaGetLastError();
  return QAT_ERR_CUDA;
}

qat_status launch_ffn_fwd(const void* x, qat_dtype dt, int64_t t, int64_t d, int64_t f,
                          const void* wg, const void* wu, const void* wd, int act, void* h,
                          float* gp, float* up, void* y, int32_t* flags, void* ws, cudaStream_t s) {
  if (d == 0 || f == 0) {  // empty sums: act(0) * 0 = 0
    qat_status st = zero(y, t * d, dt, s);
    if (!st) st = zero(h, t * f, dt, s);
    if (!st) st = zero(gp, t * f, QAT_F32, s);
    return st ? st : zero(up, t * f, QAT_F32, s);
  }
  if (few(dt, t)) {
    const auto f32 = [](const void* p) { return static_cast<const float*>(p); };
    const qat_status st = launch_few_gated(f32(x), t, d, f, f32(wg), f32(wu), act,
                                           static_cast<float*>(h), gp, up, false, s);
    return st ? st : launch_few_rows(f32(h), t, f, d, f32(wd), static_cast<float*>(y), true, s);
  }
  Packer w = {dt, reinterpret_cast<uintptr_t>(ws)};
  const FwdOps o = fwd_ops(w, t, d, f, x, wg, wu, wd, h);
  qat_status st = w.go(s);
  if (st) return st;
  Dense q = {};
  q.epi = kDenseGated;
  q.dtype = dt;
  q.m = t;
  q.n = f;
  q.k = d;
  q.a[0] = o.x;
  q.b[0] = o.wg;
  q.b[1] = o.wu;
  q.act = act;
  q.c[0] = h;
  if (o.keep_h) {
    q.q[0] = const_cast<void*>(o.h.p);
    q.q_pitch = o.h.pitch;
    q.q_part = o.h.part;
  }
  q.gp = gp;
  q.up = up;
  q.flags = flags;
  q.pdl = w.next();
  st = launch_dense(q, s);
  if (st) return st;
  q = {};
  q.epi = kDenseStore;
  q.dtype = dt;
  q.m = t;
  q.n = d;
  q.k = f;
  q.a[0] = o.h;
  q.b[0] = o.wd;
  q.c[0] = y;
  q.flags = flags;
  q.pdl = w.next();
  return launch_dense(q, s);
}

qat_status launch_ffn_bwd(const void* dy, const void* x, qat_dtype dt, int64_t t, int64_t d,
                          int64_t f, const void* wg, const void* wu, const void* wd, int act,
                          const void* h, const float* gp, const float* up, void* dx, void* dwg,
                          void* dwu, void* dwd, int32_t* flags, void* ws, cudaStream_t s) {
  if (t == 0 || f == 0) {
    qat_status st = zero(dx, t * d, dt, s);
    if (!st) st = zero(dwg, f * d, dt, s);
    if (!st) st = zero(dwu, f * d, dt, s);
    return st ? st : zero(dwd, d * f, dt, s);
  }
  Packer w = {dt, reinterpret_cast<uintptr_t>(ws)};
  DenseOp dy_op, x_op, h_op, dg_op, du_op;
  qat_status st = QAT_OK;
  if (few(dt, t)) {
    const auto f32 = [](const void* p) { return static_cast<const float*>(p); };
    const FewOps o = few_ops(w, t, d, f, dy, x, h);
    if (dx || dwg || dwu) {
      st = launch_few_gated_bwd(f32(dy), t, d, f, f32(wd), act, gp, up, o.dg32, o.du32, false, s);
      w.launched = true;
    }
    if (!st && dx)
      st = launch_few_cols2(o.dg32, o.du32, t, f, d, f32(wg), f32(wu), static_cast<float*>(dx), true, s);
    if (!st && (dwg || dwu || dwd)) {
      // without dg and du only dy, x and h are packed
      if (!(dwg || dwu)) w.n = 3;
      st = w.go(s);
    }
    dy_op = o.dy, x_op = o.x, h_op = o.h, dg_op = o.dg, du_op = o.du;
  } else {
    const BwdOps o = bwd_ops(w, t, d, f, dy, x, wg, wu, wd, h);
    dy_op = o.dy, x_op = o.x, h_op = o.h, dg_op = o.dg, du_op = o.du;
    st = w.go(s);
    if (!st && (dx || dwg || dwu)) {
      Dense q = {};
      q.epi = kDenseGatedBwd;
      q.dtype = dt;
      q.m = t;
      q.n = f;
      q.k = d;
      q.a[0] = o.dy;
      q.b[0] = turned(o.wd);
      q.act = act;
      q.gp = const_cast<float*>(gp);
      q.up = const_cast<float*>(up);
      q.q[0] = const_cast<void*>(o.dg.p);
      q.q[1] = const_cast<void*>(o.du.p);
      q.q_pitch = o.dg.pitch;
      q.q_part = o.dg.part;
      q.flags = flags;
      q.pdl = w.next();
      st = launch_dense(q, s);
    }
    if (!st && dx) {
      Dense q = {};
      q.epi = kDenseStore;
      q.dtype = dt;
      q.m = t;
      q.n = d;
      q.k = f;
      q.segs = 2;
      q.a[0] = o.dg;
      q.a[1] = o.du;
      q.b[0] = turned(o.wg);
      q.b[1] = turned(o.wu);
      q.c[0] = dx;
      q.flags = flags;
      q.pdl = w.next();
      st = launch_dense(q, s);
    }
  }
  if (!st && (dwg || dwu)) {
    Dense q = {};
    q.epi = kDenseStore;
    q.dtype = dt;
    q.m = f;
    q.n = d;
    q.k = t;
    q.problems = dwg && dwu ? 2 : 1;
    q.a[0] = turned(dwg ? dg_op : du_op);
    q.a[1] = turned(du_op);
    q.b[0] = turned(x_op);
    q.c[0] = dwg ? dwg : dwu;
    q.c[1] = dwu;
    q.flags = flags;
    q.pdl = w.next();
    st = launch_dense(q, s);
  }
  if (!st && dwd) {
    Dense q = {};
    q.epi = kDenseStore;
    q.dtype = dt;
    q.m = d;
    q.n = f;
    q.k = t;
    q.a[0] = turned(dy_op);
    q.b[0] = turned(h_op);
    q.c[0] = dwd;
    q.flags = flags;
    q.pdl = w.next();
    st = launch_dense(q, s);
  }
  return st;
}

}  // namespace qat
