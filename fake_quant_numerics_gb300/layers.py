"""Layer operators on quantized weights (include/qat.h, "Layer operators").

Products of a few tokens with the 4-bit codes the library writes
(:func:`linear4`), the gated feed-forward block with its backward pass
(:func:`gated_ffn`, :func:`gated_ffn_backward`) and from 4-bit codes
(:func:`gated_ffn4`), and layer norm with its backward pass
(:func:`layer_norm`, :func:`layer_norm_backward`).  The ``qat_*`` functions
mirror the C ABI; the named ones check shapes, allocate the outputs with torch
and run on the current stream of the tensors' device.  Every step of the computation runs in the
library's kernels.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import (BF16, GELU, PER_COLUMN, PER_GROUP, PER_ROW, PER_TENSOR, RELU, SILU, W4_DOUBLE, QatError)
from .api import _GRAN, _dt, _nbytes, _p, _ready, _s, DoubleQuantized4Bit

_ACT = {"silu": SILU, "gelu": GELU, "relu": RELU, SILU: SILU, GELU: GELU, RELU: RELU}


def _mismatch(what: str) -> QatError:
    return QatError(what, _lib.QAT_ERR_DIMENSION_MISMATCH)


def _ptr(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("libqat takes CUDA tensors only")
    return t.data_ptr()


# The current stream of a device as a raw handle (the calls here are short, and a
# Stream object costs as much as a launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name: str, device: torch.device, function, *args):
    """The library's call on the device's current stream.  A launch goes to the
    current device, so the device is made that for the call where it is not."""
    index = device.index
    if index == _current_device():
        st = function(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = function(*args, _raw_stream(index))
    if st:
        _lib.check(name, st)


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """Contiguous and 16-byte aligned (a fresh copy when it is not)."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _leading(t: torch.Tensor, shape) -> int:
    """Rows of t seen as [rows, last dimension]."""
    if len(shape) == 2:
        return shape[0]
    return t.numel() // shape[-1] if shape[-1] else shape[:-1].numel()


def _of_type(like: torch.Tensor, *tensors: Optional[torch.Tensor]):
    """Every tensor has like's dtype and device."""
    for t in tensors:
        if t is None:
            continue
        if t.dtype != like.dtype:
            raise TypeError(f"{t.dtype} beside {like.dtype}: the call's tensors share one dtype")
        _on_device(like.device, t)


def _on_device(device, *tensors):
    """Every tensor (or 4-bit weight) is on this device: the kernels take addresses."""
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {t.device} and {device}")


# ---------------------------------------------------------------------------
# products with 4-bit weights
# ---------------------------------------------------------------------------
class Weight4:
    """A [rows, cols] weight as packed 4-bit codes (see :func:`weight4`).  It holds
    its tensors and the qat_weight4 of their addresses: do not change them."""

    __slots__ = ("codes", "scale", "zero_point", "super_scales", "rows", "cols", "layout", "group",
                 "device", "struct", "address")

    def __init__(self, codes, scale, zero_point, super_scales, rows, cols, layout, group):
        self.device = codes.device
        _on_device(codes.device, scale, zero_point, super_scales)
        self.codes, self.scale, self.zero_point, self.super_scales = codes, scale, zero_point, super_scales
        self.rows, self.cols, self.layout, self.group = rows, cols, layout, group
        self.struct = _lib.Weight4Struct(
            codes.data_ptr(), scale.data_ptr(), None if zero_point is None else zero_point.data_ptr(),
            None if super_scales is None else super_scales.data_ptr(), rows, cols, group, layout)
        self.address = ctypes.addressof(self.struct)


def weight4(codes: torch.Tensor, scale: torch.Tensor, rows: int, cols: int, granularity="group",
            group: int = 128, zero_point: Optional[torch.Tensor] = None) -> Weight4:
    """The [rows, cols] weight of fake_quant_int(bits=4)'s codes, scale and
    zero_point (per tensor, row or group of the last dimension)."""
    layout = _GRAN[granularity]
    if layout == PER_COLUMN:
        raise ValueError("4-bit products take scales per tensor, row or group")
    if layout == PER_GROUP and (group <= 0 or cols % group):
        raise ValueError(f"group {group} must divide the last dimension {cols}")
    units = {PER_TENSOR: 1, PER_ROW: rows}.get(layout) if layout != PER_GROUP else rows * (cols // group)
    if codes.dtype != torch.uint8 or scale.dtype != torch.float32:
        raise TypeError("codes are uint8 (two per byte), scales float32")
    if zero_point is not None and zero_point.dtype != torch.int32:
        raise TypeError("zero points are int32")
    if (codes.numel() != (rows * cols + 1) // 2 or scale.numel() != units
            or (zero_point is not None and zero_point.numel() != units)):
        raise _mismatch("weight4")
    return Weight4(_ready(codes), scale.contiguous(),
                   None if zero_point is None else zero_point.contiguous(), None, rows, cols,
                   layout, group if layout == PER_GROUP else 0)


def weight4_double(dq: DoubleQuantized4Bit, rows: int, cols: int) -> Weight4:
    """The [rows, cols] weight of quantize_4bit_double's result."""
    if (dq.data.dtype != torch.uint8 or dq.quantized_scales.dtype != torch.uint8
            or dq.super_scales.dtype != torch.float32):
        raise TypeError("codes and their scales are uint8, super scales float32")
    blocks = (dq.len + 63) // 64
    if (dq.len != rows * cols or dq.data.numel() < (dq.len + 1) // 2
            or dq.quantized_scales.numel() < blocks or dq.super_scales.numel() < (blocks + 255) // 256):
        raise _mismatch("weight4_double")
    return Weight4(_ready(dq.data), _ready(dq.quantized_scales), None, dq.super_scales.contiguous(),
                   rows, cols, W4_DOUBLE, 0)


def _w4(w: Weight4, x: torch.Tensor):
    """The weight's address, for a call on x (itself refused off the GPU)."""
    if w.device != x.device:
        _on_device(x.device, w)
    return w.address


def qat_linear4_workspace_bytes(dtype, tokens: int, cols: int) -> int:
    return int(_lib.lib().qat_linear4_workspace_bytes(dtype, tokens, cols))


def qat_linear4(x, tokens, w: Weight4, y, workspace, stream=None):
    st = _lib.lib().qat_linear4(_p(x), _dt(x), tokens, _w4(w, x), _p(y), _p(workspace),
                                _nbytes(workspace), _s(stream))
    _lib.check("qat_linear4", st)


def qat_gated_ffn4_workspace_bytes(dtype, tokens: int, dim: int, hidden: int) -> int:
    return int(_lib.lib().qat_gated_ffn4_workspace_bytes(dtype, tokens, dim, hidden))


def qat_gated_ffn4(x, tokens, gate: Weight4, up: Weight4, down: Weight4, act, y, workspace,
                   stream=None):
    st = _lib.lib().qat_gated_ffn4(_p(x), _dt(x), tokens, _w4(gate, x), _w4(up, x), _w4(down, x),
                                   _ACT[act], _p(y), _p(workspace), _nbytes(workspace), _s(stream))
    _lib.check("qat_gated_ffn4", st)


def linear4(x: torch.Tensor, weight: Weight4) -> torch.Tensor:
    """x [..., cols] times the weight's transpose: [..., rows] in x's dtype
    (float32 or bfloat16).  For a few tokens (the weight is read once per 32)."""
    shape, cols = x.shape, weight.cols
    if not shape or shape[-1] != cols:
        raise _mismatch("linear4")
    w = _w4(weight, x)
    x = x.contiguous()
    tokens, dt, dev, lib = _leading(x, shape), _dt(x), x.device, _lib.lib()
    y = torch.empty(shape[:-1] + (weight.rows,), dtype=x.dtype, device=dev)
    xp, ws, n = _ptr(x), None, 0
    if dt != BF16 or xp % 16:
        n = lib.qat_linear4_workspace_bytes(dt, tokens, cols)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _call("qat_linear4", dev, lib.qat_linear4, xp, dt, tokens, w, y.data_ptr(),
          ws.data_ptr() if n else None, n)
    return y


def gated_ffn4(x: torch.Tensor, gate: Weight4, up: Weight4, down: Weight4,
               activation="silu") -> torch.Tensor:
    """The gated feed-forward block from 4-bit codes: (act(x gate^T) * (x up^T)) down^T.
    The hidden values are computed in float32; the second product takes all their 24
    bits for a float32 x and, unless a weight's shape is off the fast kernel's, 16 of
    them for a bfloat16 x."""
    shape = x.shape
    if not shape or shape[-1] != gate.cols or down.cols != gate.rows:
        raise _mismatch("gated_ffn4")
    w_gate, w_up, w_down = _w4(gate, x), _w4(up, x), _w4(down, x)
    x = x.contiguous()
    tokens, dt, dev, lib = _leading(x, shape), _dt(x), x.device, _lib.lib()
    y = torch.empty(shape[:-1] + (down.rows,), dtype=x.dtype, device=dev)
    n = lib.qat_gated_ffn4_workspace_bytes(dt, tokens, gate.cols, gate.rows)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _call("qat_gated_ffn4", dev, lib.qat_gated_ffn4, _ptr(x), dt, tokens, w_gate, w_up, w_down,
          _ACT[activation], y.data_ptr(), ws.data_ptr(), n)
    return y


# ---------------------------------------------------------------------------
# gated feed-forward block
# ---------------------------------------------------------------------------
class GatedFfn(NamedTuple):
    y: torch.Tensor
    h: torch.Tensor                    # act(g) * u, x's dtype
    gate_pre: Optional[torch.Tensor]   # g, float32 (save=True)
    up_pre: Optional[torch.Tensor]     # u, float32 (save=True)


def qat_gated_ffn_workspace_bytes(dtype, tokens, dim, hidden, backward=False) -> int:
    return int(_lib.lib().qat_gated_ffn_workspace_bytes(dtype, tokens, dim, hidden, int(backward)))


def qat_gated_ffn(x, tokens, dim, hidden, w_gate, w_up, w_down, act, h, gate_pre, up_pre, y,
                  dev_flags, workspace, stream=None):
    st = _lib.lib().qat_gated_ffn(_p(x), _dt(x), tokens, dim, hidden, _p(w_gate), _p(w_up),
                                  _p(w_down), _ACT[act], _p(h), _p(gate_pre), _p(up_pre), _p(y),
                                  _p(dev_flags), _p(workspace), _nbytes(workspace), _s(stream))
    _lib.check("qat_gated_ffn", st)


def qat_gated_ffn_backward(dy, x, tokens, dim, hidden, w_gate, w_up, w_down, act, h, gate_pre,
                           up_pre, dx, dw_gate, dw_up, dw_down, dev_flags, workspace, stream=None):
    st = _lib.lib().qat_gated_ffn_backward(
        _p(dy), _p(x), _dt(x), tokens, dim, hidden, _p(w_gate), _p(w_up), _p(w_down), _ACT[act],
        _p(h), _p(gate_pre), _p(up_pre), _p(dx), _p(dw_gate), _p(dw_up), _p(dw_down),
        _p(dev_flags), _p(workspace), _nbytes(workspace), _s(stream))
    _lib.check("qat_gated_ffn_backward", st)


def _ffn_sizes(what, x, w_gate, w_up, w_down):
    if w_gate.dim() != 2 or x.dim() == 0:
        raise _mismatch(what)
    hidden, dim = w_gate.shape
    if x.shape[-1] != dim or tuple(w_up.shape) != (hidden, dim) or tuple(w_down.shape) != (dim, hidden):
        raise _mismatch(what)
    _of_type(x, w_gate, w_up, w_down)
    return x.shape[:-1].numel(), dim, hidden


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
              activation="silu", save: bool = False) -> GatedFfn:
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T for x [..., dim], w_gate and w_up
    [hidden, dim], w_down [dim, hidden], one dtype (float32 or bfloat16).
    save=True keeps the pre-activations for gated_ffn_backward."""
    tokens, dim, hidden = _ffn_sizes("gated_ffn", x, w_gate, w_up, w_down)
    x, w_gate, w_up, w_down = _aligned(x), _aligned(w_gate), _aligned(w_up), _aligned(w_down)
    h = torch.empty((tokens, hidden), dtype=x.dtype, device=x.device)
    g = u = None
    if save:
        g = torch.empty((tokens, hidden), dtype=torch.float32, device=x.device)
        u = torch.empty_like(g)
    y = torch.empty_like(x)
    lib, dt = _lib.lib(), _dt(x)
    n = lib.qat_gated_ffn_workspace_bytes(dt, tokens, dim, hidden, 0)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _call("qat_gated_ffn", x.device, lib.qat_gated_ffn, _ptr(x), dt, tokens, dim, hidden,
          w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), _ACT[activation], h.data_ptr(),
          g.data_ptr() if save else None, u.data_ptr() if save else None, y.data_ptr(), None,
          ws.data_ptr() if n else None, n)
    return GatedFfn(y, h, g, u)


def gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       w_down: torch.Tensor, saved: GatedFfn, activation="silu", want_dx: bool = True,
                       want_dw: bool = True):
    """(dx, dw_gate, dw_up, dw_down) of gated_ffn(..., save=True), in x's dtype; None
    for what is not wanted."""
    tokens, dim, hidden = _ffn_sizes("gated_ffn_backward", x, w_gate, w_up, w_down)
    h, g, u = saved.h, saved.gate_pre, saved.up_pre
    if g is None or u is None:
        raise ValueError("gated_ffn_backward needs the pre-activations of gated_ffn(save=True)")
    if dy.shape != x.shape or any(t.shape != (tokens, hidden) for t in (h, g, u)):
        raise _mismatch("gated_ffn_backward")
    _of_type(x, dy, h)
    if g.dtype != torch.float32 or u.dtype != torch.float32:
        raise TypeError("the saved pre-activations are float32")
    _on_device(x.device, g, u)
    dy, x, h, g, u = _aligned(dy), _aligned(x), _aligned(h), g.contiguous(), u.contiguous()
    w_gate, w_up, w_down = _aligned(w_gate), _aligned(w_up), _aligned(w_down)
    dx = torch.empty_like(x) if want_dx else None
    dwg = dwu = dwd = None
    if want_dw:
        dwg, dwu, dwd = torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(w_down)
    lib, dt = _lib.lib(), _dt(x)
    n = lib.qat_gated_ffn_workspace_bytes(dt, tokens, dim, hidden, 1)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _call("qat_gated_ffn_backward", x.device, lib.qat_gated_ffn_backward, _ptr(dy), _ptr(x), dt, tokens,
          dim, hidden, w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), _ACT[activation],
          h.data_ptr(), g.data_ptr(), u.data_ptr(), dx.data_ptr() if want_dx else None,
          dwg.data_ptr() if want_dw else None, dwu.data_ptr() if want_dw else None,
          dwd.data_ptr() if want_dw else None, None, ws.data_ptr() if n else None, n)
    return dx, dwg, dwu, dwd


class GatedFfnFunction(torch.autograd.Function):
    """gated_ffn with its backward pass (first derivatives; a second one is an error)."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation="silu"):
        r = gated_ffn(x, w_gate, w_up, w_down, activation, save=True)
        ctx.save_for_backward(x, w_gate, w_up, w_down, r.h, r.gate_pre, r.up_pre)
        ctx.activation = activation
        return r.y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, wg, wu, wd, h, g, u = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dg, du, dd = gated_ffn_backward(dy, x, wg, wu, wd, GatedFfn(None, h, g, u),
                                            ctx.activation, want_dx=need[0], want_dw=any(need[1:4]))
        return dx, dg, du, dd, None


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
class LayerNorm(NamedTuple):
    y: torch.Tensor
    mean: torch.Tensor   # float32, one per row
    rstd: torch.Tensor


def qat_layer_norm(x, rows, cols, weight, bias, eps, y, mean, rstd, stream=None):
    st = _lib.lib().qat_layer_norm(_p(x), _dt(x), rows, cols, _p(weight), _p(bias), eps, _p(y),
                                   _p(mean), _p(rstd), _s(stream))
    _lib.check("qat_layer_norm", st)


def qat_layer_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return int(_lib.lib().qat_layer_norm_backward_workspace_bytes(rows, cols))


def qat_layer_norm_backward(dy, x, rows, cols, weight, mean, rstd, dx, dweight, dbias, workspace,
                            stream=None):
    st = _lib.lib().qat_layer_norm_backward(_p(dy), _p(x), _dt(x), rows, cols, _p(weight), _p(mean),
                                            _p(rstd), _p(dx), _p(dweight), _p(dbias), _p(workspace),
                                            _nbytes(workspace), _s(stream))
    _lib.check("qat_layer_norm_backward", st)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5) -> LayerNorm:
    """Layer norm of x [..., cols] over its last dimension, with the rows' mean and
    rstd (float32) for the backward pass."""
    shape = x.shape
    if not shape:
        raise _mismatch("layer_norm")
    x = x.contiguous()
    lead, cols, dev, f32 = shape[:-1], shape[-1], x.device, torch.float32
    wp = bp = None
    if weight is not None:
        weight = _vector("layer_norm", x, weight, cols)
        wp = weight.data_ptr()
    if bias is not None:
        bias = _vector("layer_norm", x, bias, cols)
        bp = bias.data_ptr()
    y = torch.empty_like(x)
    mean = torch.empty(lead, dtype=f32, device=dev)
    rstd = torch.empty(lead, dtype=f32, device=dev)
    if cols == 0:  # the call is a no-op, and the mean of no elements 0 / 0
        mean.fill_(float("nan"))
        rstd.fill_(float("nan"))
    _call("qat_layer_norm", dev, _lib.lib().qat_layer_norm, _ptr(x), _dt(x), _leading(x, shape), cols,
          wp, bp, eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return LayerNorm(y, mean, rstd)


def _vector(what, x, v, cols):
    if v.dim() != 1 or v.numel() != cols:
        raise _mismatch(what)
    if v.dtype != x.dtype or v.device != x.device:
        _of_type(x, v)
    return v.contiguous()


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor],
                        mean: torch.Tensor, rstd: torch.Tensor, want_dx: bool = True,
                        want_dw: bool = True):
    """(dx, dweight, dbias) of layer_norm; None for what is not wanted."""
    shape = x.shape
    if not shape or dy.shape != shape:
        raise _mismatch("layer_norm_backward")
    cols = shape[-1]
    rows = _leading(x, shape)
    if mean.numel() != rows or rstd.numel() != rows:
        raise _mismatch("layer_norm_backward")
    if dy.dtype != x.dtype or dy.device != x.device:
        _of_type(x, dy)
    if mean.dtype != torch.float32 or rstd.dtype != torch.float32:
        raise TypeError("mean and rstd are float32")
    if mean.device != x.device or rstd.device != x.device:
        _on_device(x.device, mean, rstd)
    dy, x, mean, rstd = dy.contiguous(), x.contiguous(), mean.contiguous(), rstd.contiguous()
    wp = None
    if weight is not None:
        weight = _vector("layer_norm_backward", x, weight, cols)
        wp = weight.data_ptr()
    lib = _lib.lib()
    dx = torch.empty_like(x) if want_dx else None
    dw = db = ws = None
    n = 0
    if want_dw:
        dw = torch.empty(cols, dtype=x.dtype, device=x.device)
        db = torch.empty(cols, dtype=x.dtype, device=x.device)
        n = lib.qat_layer_norm_backward_workspace_bytes(rows, cols)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _call("qat_layer_norm_backward", x.device, lib.qat_layer_norm_backward, _ptr(dy), _ptr(x), _dt(x),
          rows, cols, wp, _ptr(mean), _ptr(rstd), dx.data_ptr() if want_dx else None,
          dw.data_ptr() if want_dw else None, db.data_ptr() if want_dw else None,
          ws.data_ptr() if n else None, n)
    return dx, dw, db


class LayerNormFunction(torch.autograd.Function):
    """layer_norm with its backward pass (first derivatives; a second one is an error)."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps=1e-5):
        r = layer_norm(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, r.mean, r.rstd)
        return r.y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd, want_dx=need[0],
                                         want_dw=need[1] or need[2])
        return dx, dw if need[1] else None, db if need[2] else None, None
