"""Attention operators (include/qat.h, "Attention operators"): the half of a layer
that reads a quantized key-value cache.

Norms of queries and keys for each head with the position rotation
(:func:`head_norm_rope`, :func:`head_norm_rope_backward`), a paged cache in the
library's formats that is quantized as it is written (:class:`KVCache`,
:func:`kv_cache`, :func:`kv_write`, :func:`kv_read`), and the attention of one new
token of each sequence over it (:func:`kv_attention`).  As in the layer operators
the ``qat_*`` functions mirror the C ABI, and the named ones check shapes, allocate
the outputs with torch and run on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import (AFFINE, CACHE_BF16, CACHE_E4M3, CACHE_E5M2, CACHE_INT4, CACHE_INT8, ROPE_HALF, ROPE_INTERLEAVED)
from .api import _DT, _SCHEME, _dt, _nbytes, _p, _s
from .layers import _call, _mismatch, _of_type, _on_device, _ptr, _vector

_LAYOUT = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED}
_CACHE = {"bf16": CACHE_BF16, "int8": CACHE_INT8, "int4": CACHE_INT4, "e4m3": CACHE_E4M3, "e5m2": CACHE_E5M2}


# ---------------------------------------------------------------------------
# norms of queries and keys with the position rotation
# ---------------------------------------------------------------------------
class HeadNormRope(NamedTuple):
    q: torch.Tensor
    k: Optional[torch.Tensor]


def rope_frequencies(rotary_dim: int, base: float = 10000.0, factor: float = 1.0,
                     original_length: Optional[int] = None, slow: float = 1.0,
                     fast: float = 32.0) -> torch.Tensor:
    """Radians a position of each pair, base^(-2j / rotary_dim), in float64 on the host.

    factor stretches them for contexts longer than the trained one: every
    frequency over factor (original_length None), or by parts, where a pair that
    turns at most `slow` times over original_length positions is divided by
    factor, one that turns `fast` times or more stays, and those between are mixed
    in proportion."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError(f"rotary_dim {rotary_dim} must be even")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    f = float(base) ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / max(1, rotary_dim))
    if original_length is None:
        return f / factor
    if not fast > slow:
        raise ValueError("fast must lie above slow")
    keep = ((f * original_length / math.tau - slow) / (fast - slow)).clamp(0.0, 1.0)
    return f * keep + f / factor * (1 - keep)


def rope_turns(frequencies: torch.Tensor, device=None) -> torch.Tensor:
    """The frequencies (radians a position) as the rotation takes them: int64 fractions
    of a turn in units of 2^-64, on `device` (the frequencies' own when None)."""
    f = frequencies.detach().to(device="cpu", dtype=torch.float64)
    if f.dim() != 1:
        raise _mismatch("rope_turns")
    if not bool(torch.isfinite(f).all()):
        raise ValueError("frequencies must be finite")
    turns = [int(math.fmod(x / math.tau, 1.0) * 2.0 ** 64) % (1 << 64) for x in f.tolist()]
    return torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64,
                        device=frequencies.device if device is None else device)


def qat_head_norm_rope(q, k, tokens, q_heads, k_heads, head_dim, q_strides, k_strides, positions, turns,
                       rotary_dim, layout, amplitude, norm, q_weight, k_weight, eps, q_out, k_out,
                       stream=None):
    st = _lib.lib().qat_head_norm_rope(
        _p(q), _p(k), _dt(q), tokens, q_heads, k_heads, head_dim, *q_strides, *k_strides, _p(positions),
        _p(turns), rotary_dim, _LAYOUT[layout], amplitude, int(norm), _p(q_weight), _p(k_weight), eps,
        _p(q_out), _p(k_out), _s(stream))
    _lib.check("qat_head_norm_rope", st)


def qat_head_norm_rope_backward_workspace_bytes(head_dim: int) -> int:
    return int(_lib.lib().qat_head_norm_rope_backward_workspace_bytes(head_dim))


def qat_head_norm_rope_backward(dq_out, dk_out, q, k, tokens, q_heads, k_heads, head_dim, q_strides,
                                k_strides, positions, turns, rotary_dim, layout, amplitude, norm,
                                q_weight, k_weight, eps, dq, dk, dq_weight, dk_weight, workspace,
                                stream=None):
    st = _lib.lib().qat_head_norm_rope_backward(
        _p(dq_out), _p(dk_out), _p(q), _p(k), _dt(q), tokens, q_heads, k_heads, head_dim, *q_strides,
        *k_strides, _p(positions), _p(turns), rotary_dim, _LAYOUT[layout], amplitude, int(norm),
        _p(q_weight), _p(k_weight), eps, _p(dq), _p(dk), _p(dq_weight), _p(dk_weight), _p(workspace),
        _nbytes(workspace), _s(stream))
    _lib.check("qat_head_norm_rope_backward", st)


def _heads(t: torch.Tensor) -> torch.Tensor:
    """t as [tokens, heads, head_dim] with a last stride of 1 (a copy where it has none)."""
    if t.dim() != 3:
        t = t.reshape(t.shape[:-2].numel(), *t.shape[-2:])
    return t if t.stride(2) == 1 or t.shape[2] <= 1 else t.contiguous()


_I64, _I32 = torch.int64, torch.int32


def _rope_inputs(what, q, k, positions, turns, q_weight, k_weight, norm, layout):
    """q and k as [tokens, heads, head_dim], then positions, turns and the weights, each
    as the kernels read it."""
    shape, dev, dtype = q.shape, q.device, q.dtype
    if len(shape) < 2 or turns.dim() != 1 or positions.numel() != (shape[0] if len(shape) == 3
                                                                  else shape[:-2].numel()):
        raise _mismatch(what)
    d = shape[-1]
    if positions.dtype is not _I64 or turns.dtype is not _I64:
        raise TypeError("positions and turns are int64")
    if layout not in _LAYOUT:
        raise ValueError(f"layout must be 'half' or 'interleaved', not {layout!r}")
    if positions.device != dev or turns.device != dev:
        _on_device(dev, positions, turns)
    if k is not None:
        ks = k.shape
        if len(ks) != len(shape) or ks[-1] != d or ks[:-2] != shape[:-2]:
            raise _mismatch(what)
        if k.dtype is not dtype or k.device != dev:
            _of_type(q, k)
        k = _heads(k)
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    if q_weight is not None or k_weight is not None:
        if not norm:
            raise ValueError("weights belong to the norm")
        if q_weight is not None:
            q_weight = _vector(what, q, q_weight, d)
        if k_weight is not None:
            k_weight = _vector(what, q, k_weight, d)
    return _heads(q), k, positions.contiguous(), turns.contiguous(), q_weight, k_weight


def head_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, turns: torch.Tensor,
                   q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                   eps: float = 1e-6, norm: bool = True, layout: str = "half",
                   amplitude: float = 1.0) -> HeadNormRope:
    """RMS norm of each head of q and k [..., heads, head_dim] and the rotation of its
    leading pairs by the token's position, in one pass.

    positions: int64, one for each token (q's leading dimensions); turns: the pairs'
    frequencies (:func:`rope_turns`; their number is half the rotated dimensions).
    norm=False rotates only.  amplitude scales the rotated part.  q and k may be
    views of one projection's output: only the last dimension has to be dense."""
    shape, k_shape = q.shape, None if k is None else k.shape
    q, k, positions, turns, wq, wk = _rope_inputs("head_norm_rope", q, k, positions, turns, q_weight, k_weight, norm,
                                                  layout)
    dev, dtype, qs = q.device, q.dtype, q.stride()
    qp, dt = _ptr(q), _dt(q)
    yq = torch.empty(shape, dtype=dtype, device=dev)
    yk = kp = ykp = None
    hk = ks0 = ks1 = 0
    if k is not None:
        hk, (ks0, ks1, _), kp = k.shape[1], k.stride(), k.data_ptr()
        yk = torch.empty(k_shape, dtype=dtype, device=dev)
        ykp = yk.data_ptr()
    _call("qat_head_norm_rope", dev, _lib.lib().qat_head_norm_rope, qp, kp, dt, q.shape[0], q.shape[1], hk,
          shape[-1], qs[0], qs[1], ks0, ks1, positions.data_ptr(), turns.data_ptr(), 2 * turns.numel(),
          _LAYOUT[layout], amplitude, 1 if norm else 0, None if wq is None else wq.data_ptr(),
          None if wk is None else wk.data_ptr(), eps, yq.data_ptr(), ykp)
    return HeadNormRope(yq, yk)


def head_norm_rope_backward(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], q: torch.Tensor,
                            k: Optional[torch.Tensor], positions: torch.Tensor, turns: torch.Tensor,
                            q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                            eps: float = 1e-6, norm: bool = True, layout: str = "half",
                            amplitude: float = 1.0, want_dx: bool = True, want_dw: bool = True):
    """(dq, dk, dq_weight, dk_weight) of head_norm_rope; None for what is not wanted and
    for weights that the call did not have."""
    what = "head_norm_rope_backward"
    shape, k_shape = q.shape, None if k is None else k.shape
    if dq_out.shape != shape or (k is None) != (dk_out is None) or (k is not None and dk_out.shape != k_shape):
        raise _mismatch(what)
    dtype, dev = q.dtype, q.device
    if dq_out.dtype is not dtype or dq_out.device != dev:
        _of_type(q, dq_out)
    if dk_out is not None and (dk_out.dtype is not dtype or dk_out.device != dev):
        _of_type(q, dk_out)
    q, k, positions, turns, wq, wk = _rope_inputs(what, q, k, positions, turns, q_weight, k_weight, norm, layout)
    dq_out = dq_out.contiguous()
    qs, d, gp, dt = q.stride(), shape[-1], _ptr(dq_out), _dt(q)
    dq = dk = dwq = dwk = ws = kp = gkp = dqp = dkp = wqp = wkp = dwqp = dwkp = wsp = None
    hk = ks0 = ks1 = n = 0
    if want_dx:
        dq = torch.empty(shape, dtype=dtype, device=dev)
        dqp = dq.data_ptr()
    if k is not None:
        dk_out = dk_out.contiguous()
        hk, (ks0, ks1, _), kp, gkp = k.shape[1], k.stride(), k.data_ptr(), dk_out.data_ptr()
        if want_dx:
            dk = torch.empty(k_shape, dtype=dtype, device=dev)
            dkp = dk.data_ptr()
    if wq is not None:
        wqp = wq.data_ptr()
        if want_dw:
            dwq = torch.empty(d, dtype=dtype, device=dev)
            dwqp = dwq.data_ptr()
    if wk is not None:
        wkp = wk.data_ptr()
        if want_dw:
            dwk = torch.empty(d, dtype=dtype, device=dev)
            dwkp = dwk.data_ptr()
    lib = _lib.lib()
    if dwq is not None or dwk is not None:
        n = lib.qat_head_norm_rope_backward_workspace_bytes(d)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        wsp = ws.data_ptr()
    _call("qat_head_norm_rope_backward", dev, lib.qat_head_norm_rope_backward, gp, gkp, q.data_ptr(), kp, dt,
          q.shape[0], q.shape[1], hk, d, qs[0], qs[1], ks0, ks1, positions.data_ptr(), turns.data_ptr(),
          2 * turns.numel(), _LAYOUT[layout], amplitude, 1 if norm else 0, wqp, wkp, eps, dqp, dkp, dwqp, dwkp,
          wsp, n)
    return dq, dk, dwq, dwk


class HeadNormRopeFunction(torch.autograd.Function):
    """head_norm_rope with its backward pass (first derivatives; a second one is an
    error): (q, k) of apply(q, k, positions, turns, q_weight, k_weight, eps, norm,
    layout, amplitude)."""

    @staticmethod
    def forward(ctx, q, k, positions, turns, q_weight=None, k_weight=None, eps=1e-6, norm=True, layout="half",
                amplitude=1.0):
        r = head_norm_rope(q, k, positions, turns, q_weight, k_weight, eps, norm, layout, amplitude)
        ctx.save_for_backward(q, k, positions, turns, q_weight, k_weight)
        ctx.options = (eps, norm, layout, amplitude)
        return r.q, r.k

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, positions, turns, wq, wk = ctx.saved_tensors
        need = (tuple(ctx.needs_input_grad) + (False,) * 6)[:6]  # (one for each argument that apply got)
        dq, dk, dwq, dwk = head_norm_rope_backward(dq_out, None if k is None else dk_out, q, k, positions, turns,
                                                   wq, wk, *ctx.options, want_dx=need[0] or need[1],
                                                   want_dw=need[4] or need[5])
        grads = (dq if need[0] else None, dk if need[1] else None, None, None, dwq if need[4] else None,
                 dwk if need[5] else None, None, None, None, None)
        return grads[:len(ctx.needs_input_grad)]


# ---------------------------------------------------------------------------
# the quantized key-value cache
# ---------------------------------------------------------------------------
class KVCache:
    """A paged cache of keys and values: its tensors, and the qat_kv_cache of their
    addresses (do not replace them).

    k, v: codes, uint8 [pages, heads, page_size, row bytes] ("int8", "int4", "e4m3",
    "e5m2"; a row is padded to 16 bytes), or bfloat16 [pages, heads, page_size,
    head_dim] ("bf16"); scales: float32 [pages, heads, page_size], and for affine
    integer codes zero points, int8, alike.  A position's slot is page * page_size +
    offset."""

    __slots__ = ("k", "v", "format", "head_dim", "k_scale", "v_scale", "k_zero_point", "v_zero_point", "pages",
                 "heads", "page_size", "device", "struct", "address", "workspace")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, format: str, head_dim: int,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 k_zero_point: Optional[torch.Tensor] = None, v_zero_point: Optional[torch.Tensor] = None):
        if format not in _CACHE:
            raise ValueError(f"format must be one of {', '.join(_CACHE)}, not {format!r}")
        if head_dim < 8 or head_dim > 256 or head_dim % 8:
            raise ValueError(f"head_dim {head_dim} must be a multiple of 8 up to 256")
        row = _row_elements(format, head_dim)
        if k.dim() != 4 or k.shape[3] != row or v.shape != k.shape:
            raise _mismatch("KVCache")
        dtype = torch.bfloat16 if format == "bf16" else torch.uint8
        if k.dtype != dtype or v.dtype != dtype:
            raise TypeError(f"a cache in {format} holds {dtype}")
        if k.shape[2] < 16 or k.shape[2] % 16:
            raise ValueError(f"page size {k.shape[2]} must be a multiple of 16")
        if not 1 <= k.shape[1] <= 32767 or k.shape[0] * k.shape[2] >= 1 << 31:
            raise ValueError("a cache has 1 to 32767 heads and less than 2^31 positions")
        if (k_scale is None) != (format == "bf16") or (v_scale is None) != (format == "bf16"):
            raise ValueError("quantized rows have scales, bf16 rows none")
        if (k_zero_point is None) != (v_zero_point is None) or (k_zero_point is not None
                                                                 and format not in ("int8", "int4")):
            raise ValueError("zero points belong to keys and values of the integer formats")
        for t, kind in ((k_scale, torch.float32), (v_scale, torch.float32), (k_zero_point, torch.int8),
                        (v_zero_point, torch.int8)):
            if t is None:
                continue
            if t.shape != k.shape[:3]:
                raise _mismatch("KVCache")
            if t.dtype != kind:
                raise TypeError("scales are float32, zero points int8")
        for t in (k, v, k_scale, v_scale, k_zero_point, v_zero_point):
            if t is not None and (not t.is_contiguous() or t.data_ptr() % 16):
                raise ValueError("the cache's tensors are contiguous and 16-byte aligned (they are written in place)")
        _on_device(k.device, v, k_scale, v_scale, k_zero_point, v_zero_point)
        self.k, self.v, self.format, self.head_dim = k, v, format, head_dim
        self.k_scale, self.v_scale = k_scale, v_scale
        self.k_zero_point, self.v_zero_point = k_zero_point, v_zero_point
        self.pages, self.heads, self.page_size = k.shape[0], k.shape[1], k.shape[2]
        self.device = k.device
        self.struct = _lib.KvCacheStruct(*(None if t is None else t.data_ptr() for t in (
            k, v, k_scale, v_scale, k_zero_point, v_zero_point)), self.pages, self.heads, self.page_size, head_dim,
            _CACHE[format])
        self.address = ctypes.addressof(self.struct)
        self.workspace = {}  # bytes that kv_attention needs, by the number of query heads


def _row_elements(format: str, head_dim: int) -> int:
    """The last dimension of a cache's codes."""
    if format == "bf16":
        return head_dim
    return ((head_dim // 2 if format == "int4" else head_dim) + 15) // 16 * 16


def kv_cache(pages: int, heads: int, page_size: int, head_dim: int, format: str = "int8",
             scheme="symmetric", device="cuda") -> KVCache:
    """An empty cache (zeros)."""
    if format not in _CACHE:
        raise ValueError(f"format must be one of {', '.join(_CACHE)}, not {format!r}")
    affine = _SCHEME[scheme] == AFFINE
    if affine and format not in ("int8", "int4"):
        raise ValueError("affine codes are int8 or int4")
    rows = (pages, heads, page_size)
    codes = torch.zeros((2,) + rows + (_row_elements(format, head_dim),), device=device,
                        dtype=torch.bfloat16 if format == "bf16" else torch.uint8)
    scales, zps = (None, None), (None, None)
    if format != "bf16":
        scales = torch.zeros((2,) + rows, device=device)
    if affine:
        zps = torch.zeros((2,) + rows, dtype=torch.int8, device=device)
    return KVCache(codes[0], codes[1], format, head_dim, scales[0], scales[1], zps[0], zps[1])


class KeysValues(NamedTuple):
    k: torch.Tensor
    v: torch.Tensor


def qat_kv_write(cache: KVCache, k, v, tokens, k_strides, v_strides, slots, stream=None):
    st = _lib.lib().qat_kv_write(cache.address, _p(k), _p(v), _dt(k), tokens, *k_strides, *v_strides, _p(slots),
                                 _s(stream))
    _lib.check("qat_kv_write", st)


def qat_kv_read(cache: KVCache, slots, tokens, k, v, stream=None):
    st = _lib.lib().qat_kv_read(cache.address, _p(slots), tokens, _p(k), _p(v), _dt(k), _s(stream))
    _lib.check("qat_kv_read", st)


def _slots(slots: torch.Tensor) -> torch.Tensor:
    if slots.dtype is not _I64:
        raise TypeError("slots are int64")
    return slots.contiguous()


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantizes k and v [..., heads, head_dim] (float32 or bfloat16) into the cache at
    `slots` (int64, one for each token).  Tokens whose slot lies outside the cache (-1
    in a padded batch) are not written.  Slots must differ: where one is given twice
    it is unspecified which token's codes and scales it holds."""
    what = "kv_write"
    shape, dev = k.shape, cache.device
    if len(shape) < 2 or v.shape != shape or shape[-2] != cache.heads or shape[-1] != cache.head_dim:
        raise _mismatch(what)
    tokens = shape[0] if len(shape) == 3 else shape[:-2].numel()
    if slots.numel() != tokens:
        raise _mismatch(what)
    if v.dtype is not k.dtype or v.device != k.device:
        _of_type(k, v)
    if k.device != dev or slots.device != dev:
        _on_device(dev, k, slots)
    slots, k, v = _slots(slots), _heads(k), _heads(v)
    ks, vs = k.stride(), v.stride()
    _call("qat_kv_write", dev, _lib.lib().qat_kv_write, cache.address, _ptr(k), v.data_ptr(), _dt(k), tokens,
          ks[0], ks[1], vs[0], vs[1], slots.data_ptr())


def kv_read(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> KeysValues:
    """The cached keys and values at `slots` (int64, any shape) as [..., heads, head_dim]
    in float32 or bfloat16; zeros for a slot outside the cache."""
    dev = cache.device
    if slots.device != dev:
        _on_device(dev, slots)
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    shape, slots = (*slots.shape, cache.heads, cache.head_dim), _slots(slots)
    sp = _ptr(slots)
    k = torch.empty(shape, dtype=dtype, device=dev)
    v = torch.empty(shape, dtype=dtype, device=dev)
    _call("qat_kv_read", dev, _lib.lib().qat_kv_read, cache.address, sp, slots.numel(), k.data_ptr(), v.data_ptr(),
          _DT[dtype])
    return KeysValues(k, v)


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------
class KvAttention(NamedTuple):
    y: torch.Tensor
    lse: Optional[torch.Tensor]   # float32 [batch, heads] (want_lse=True)


def qat_kv_attention_workspace_bytes(cache: KVCache, q_heads: int) -> int:
    return int(_lib.lib().qat_kv_attention_workspace_bytes(cache.address, q_heads))


def qat_kv_attention(q, batch, q_heads, q_strides, cache: KVCache, table, table_cols, table_stride, lengths,
                     scale, y, lse, workspace, stream=None):
    st = _lib.lib().qat_kv_attention(_p(q), _dt(q), batch, q_heads, *q_strides, cache.address, _p(table),
                                     table_cols, table_stride, _p(lengths), scale, _p(y), _p(lse),
                                     _p(workspace), _nbytes(workspace), _s(stream))
    _lib.check("qat_kv_attention", st)


def kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lengths: torch.Tensor,
                 scale: Optional[float] = None, want_lse: bool = False) -> KvAttention:
    """Attention of one new token of each sequence, q [batch, heads, head_dim] (heads a
    multiple of the cache's), over the first lengths[b] cached positions; position t of
    sequence b lies in page block_table[b, t // page_size] (both int32).

    scale defaults to head_dim^-0.5.  A length of 0 gives zeros (lse -inf).  Lengths
    that the table cannot hold and pages outside the cache make the sequence's outputs
    NaN; what lies behind a sequence's length has no effect.  For serving: the result
    has no gradient."""
    shape, table_shape, dev = q.shape, block_table.shape, q.device
    if len(shape) != 3 or shape[2] != cache.head_dim or shape[1] % cache.heads:
        raise _mismatch("kv_attention")
    batch, heads, d = shape
    if len(table_shape) != 2 or table_shape[0] != batch or lengths.dim() != 1 or lengths.shape[0] != batch:
        raise _mismatch("kv_attention")
    if block_table.dtype is not _I32 or lengths.dtype is not _I32:
        raise TypeError("block_table and lengths are int32")
    if cache.device != dev or block_table.device != dev or lengths.device != dev:
        _on_device(dev, cache, block_table, lengths)
    ts = block_table.stride()
    if ts[1] != 1 and table_shape[1] > 1:
        block_table = block_table.contiguous()
        ts = block_table.stride()
    lengths = lengths.contiguous()
    qs = q.stride()
    if qs[2] != 1:
        q = q.contiguous()
        qs = q.stride()
    qp, dt = _ptr(q), _dt(q)
    y = torch.empty(shape, dtype=q.dtype, device=dev)
    lse = torch.empty((batch, heads), dtype=torch.float32, device=dev) if want_lse else None
    if batch == 0 or heads == 0:
        return KvAttention(y, lse)
    lib = _lib.lib()
    n = cache.workspace.get(heads)
    if n is None:
        n = cache.workspace[heads] = lib.qat_kv_attention_workspace_bytes(cache.address, heads)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _call("qat_kv_attention", dev, lib.qat_kv_attention, qp, dt, batch, heads, qs[0], qs[1], cache.address,
          block_table.data_ptr(), table_shape[1], ts[0], lengths.data_ptr(), d ** -0.5 if scale is None else scale,
          y.data_ptr(), lse.data_ptr() if want_lse else None, ws.data_ptr(), n)
    return KvAttention(y, lse)
