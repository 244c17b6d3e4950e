"""Host-side refusals of the layer operators: every call fails its validation
before anything is enqueued (no GPU; the fake pointers are never read)."""
import ctypes

import pytest
import torch

import fake_quant_numerics_gb300 as fq
from fake_quant_numerics_gb300 import _lib as L

A = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    from fake_quant_numerics_gb300 import build

    build.build()
    return L.load(build_if_missing=False)


def w4(**kw):
    a = dict(codes=0x10000, scales=0x10000, zero_points=None, super_scales=None, rows=32, cols=128,
             group=64, layout=L.PER_GROUP)
    a.update(kw)
    return L.Weight4Struct(**a)


def lin(lib, x=A, dt=L.F32, tokens=2, y=A, ws=A, wsb=1 << 30, **kw):
    return lib.qat_linear4(x, dt, tokens, ctypes.byref(w4(**kw)), y, ws, wsb, None)


def test_linear4_refusals(lib):
    inv, uns, mis = L.QAT_ERR_INVALID_ARGUMENT, L.QAT_ERR_UNSUPPORTED, L.QAT_ERR_MISALIGNED
    assert lib.qat_linear4(A, L.F32, 2, None, A, A, 1 << 30, None) == inv
    assert lin(lib, dt=5) == uns
    assert lin(lib, layout=L.PER_COLUMN) == uns and lin(lib, layout=9) == uns
    assert lin(lib, tokens=-1) == inv and lin(lib, rows=-1) == inv and lin(lib, cols=-64) == inv
    assert lin(lib, group=48) == inv and lin(lib, group=0) == inv
    assert lin(lib, codes=None) == inv and lin(lib, scales=None) == inv
    assert lin(lib, x=None) == inv and lin(lib, y=None) == inv
    assert lin(lib, layout=L.W4_DOUBLE) == inv                       # no super scales
    assert lin(lib, layout=L.W4_DOUBLE, super_scales=0x10000, zero_points=0x10000) == inv
    assert lin(lib, rows=1 << 40, cols=1 << 20) == inv               # past the element limit
    assert lin(lib, codes=0x10004) == mis and lin(lib, scales=0x10002) == mis
    assert lin(lib, zero_points=0x10002) == mis and lin(lib, x=ODD) == mis and lin(lib, y=ODD) == mis
    need = lib.qat_linear4_workspace_bytes(L.F32, 2, 128)
    assert need >= 3 * 2 * 128 * 2
    assert lin(lib, ws=None) == L.QAT_ERR_WORKSPACE and lin(lib, wsb=need - 1) == L.QAT_ERR_WORKSPACE
    assert lin(lib, ws=ODD) == mis
    assert lin(lib, tokens=0, x=None, y=None) == L.QAT_OK
    assert lin(lib, rows=0, codes=None, scales=None, y=None) == L.QAT_OK


def test_gated4_refusals(lib):
    def call(act=L.SILU, y=A, up=None, down=None, ws=A, wsb=1 << 30, **kw):
        g, u = w4(**kw), up or w4(**kw)
        d = down or w4(rows=128, cols=32, layout=L.PER_ROW)
        return lib.qat_gated_ffn4(A, L.F32, 2, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), act,
                                  y, ws, wsb, None)

    assert call(act=7) == L.QAT_ERR_UNSUPPORTED
    assert call(y=None) == L.QAT_ERR_INVALID_ARGUMENT
    assert call(y=ODD) == L.QAT_ERR_MISALIGNED
    assert call(ws=None) == L.QAT_ERR_WORKSPACE
    need = lib.qat_gated_ffn4_workspace_bytes(L.F32, 2, 128, 32)
    assert call(wsb=need - 1) == L.QAT_ERR_WORKSPACE
    for other in (dict(rows=64), dict(cols=64), dict(group=32), dict(layout=L.PER_ROW),
                  dict(zero_points=0x10000)):
        assert call(up=w4(**other)) == L.QAT_ERR_DIMENSION_MISMATCH, other
    assert call(down=w4(rows=128, cols=64, layout=L.PER_ROW)) == L.QAT_ERR_DIMENSION_MISMATCH


def test_ffn_refusals(lib):
    def fwd(dt=L.BF16, t=4, d=16, f=32, act=L.SILU, **kw):
        a = dict(x=A, wg=A, wu=A, wd=A, h=A, g=None, u=None, y=A)
        a.update(kw)
        return lib.qat_gated_ffn(a["x"], dt, t, d, f, a["wg"], a["wu"], a["wd"], act, a["h"],
                                 a["g"], a["u"], a["y"], None, A, 1 << 40, None)

    inv, uns, mis = L.QAT_ERR_INVALID_ARGUMENT, L.QAT_ERR_UNSUPPORTED, L.QAT_ERR_MISALIGNED
    assert fwd(dt=9) == uns and fwd(act=3) == uns
    assert fwd(t=-1) == inv and fwd(d=-1) == inv and fwd(f=1 << 50, d=2) == inv
    assert all(fwd(**{k: None}) == inv for k in ("x", "wg", "wu", "wd", "h", "y"))
    assert fwd(g=A) == inv and fwd(u=A) == inv                        # both or neither
    assert all(fwd(**{k: ODD}) == mis for k in ("x", "wg", "wu", "wd", "h", "y"))
    assert fwd(t=0, x=None, y=None, h=None) == L.QAT_OK

    def bwd(dt=L.BF16, ws=A, wsb=1 << 40, **kw):
        a = dict(dy=A, x=A, wg=A, wu=A, wd=A, h=A, g=A, u=A, dx=A, dg=A, du=A, dd=A)
        a.update(kw)
        return lib.qat_gated_ffn_backward(a["dy"], a["x"], dt, 4, 16, 32, a["wg"], a["wu"], a["wd"],
                                          L.SILU, a["h"], a["g"], a["u"], a["dx"], a["dg"], a["du"],
                                          a["dd"], None, ws, wsb, None)

    assert bwd(dt=9) == uns
    assert all(bwd(**{k: None}) == inv for k in ("dy", "x", "wg", "wu", "wd", "h", "g", "u"))
    assert all(bwd(**{k: ODD}) == mis for k in ("dy", "x", "wg", "wu", "wd", "h", "g", "u", "dx", "dg"))
    need = lib.qat_gated_ffn_workspace_bytes(L.BF16, 4, 16, 32, 1)
    assert need > 0
    assert bwd(ws=None) == L.QAT_ERR_WORKSPACE and bwd(wsb=need - 1) == L.QAT_ERR_WORKSPACE
    assert bwd(ws=ODD) == mis
    assert lib.qat_gated_ffn_workspace_bytes(9, 4, 16, 32, 1) == 0


def test_layer_norm_refusals(lib):
    def fwd(dt=L.F32, rows=4, cols=64, eps=1e-5, x=A, y=A, w=A, mean=A):
        return lib.qat_layer_norm(x, dt, rows, cols, w, A, eps, y, mean, A, None)

    inv, uns, mis = L.QAT_ERR_INVALID_ARGUMENT, L.QAT_ERR_UNSUPPORTED, L.QAT_ERR_MISALIGNED
    assert fwd(dt=3) == uns and fwd(rows=-1) == inv and fwd(cols=-1) == inv
    for eps in (-1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == inv
    assert fwd(x=None) == inv and fwd(y=None) == inv
    assert fwd(x=ODD) == mis and fwd(w=ODD) == mis and fwd(mean=ctypes.c_void_p(0x10002)) == mis
    assert fwd(rows=0, x=None, y=None) == L.QAT_OK and fwd(cols=0, x=None, y=None) == L.QAT_OK

    def bwd(rows=4, ws=A, wsb=1 << 30, **kw):
        a = dict(dy=A, x=A, mean=A, rstd=A, dx=A, dw=A, db=A)
        a.update(kw)
        return lib.qat_layer_norm_backward(a["dy"], a["x"], L.F32, rows, 64, A, a["mean"], a["rstd"],
                                           a["dx"], a["dw"], a["db"], ws, wsb, None)

    assert all(bwd(**{k: None}) == inv for k in ("dy", "x", "mean", "rstd"))
    assert all(bwd(**{k: ODD}) == mis for k in ("dy", "x", "mean", "rstd", "dx", "dw", "db"))
    need = lib.qat_layer_norm_backward_workspace_bytes(4, 64)
    assert need > 0 and bwd(wsb=need - 1) == L.QAT_ERR_WORKSPACE and bwd(ws=None) == L.QAT_ERR_WORKSPACE
    assert bwd(ws=ODD) == mis
    assert bwd(rows=0, dw=None, db=None, dy=None, x=None, mean=None, rstd=None) == L.QAT_OK


def test_binding_refusals():
    """Shapes, types and host tensors, before any launch."""
    x = torch.zeros(3, 64)
    codes, scale = torch.zeros(64 * 16, dtype=torch.uint8), torch.ones(32)
    w = fq.weight4(codes, scale, 32, 64, "row")
    for bad in (lambda: fq.weight4(codes[1:], scale, 32, 64, "row"),
                lambda: fq.weight4(codes, scale[1:], 32, 64, "row"),
                lambda: fq.weight4(codes, scale, 32, 64, "row", zero_point=torch.zeros(3, dtype=torch.int32)),
                lambda: fq.linear4(torch.zeros(3, 63), w),
                lambda: fq.gated_ffn4(x, w, w, w),
                lambda: fq.gated_ffn(x, torch.zeros(8, 64), torch.zeros(8, 63), torch.zeros(64, 8)),
                lambda: fq.layer_norm(x, torch.zeros(63)),
                lambda: fq.layer_norm_backward(x, x, None, torch.zeros(2), torch.zeros(3))):
        with pytest.raises(fq.QatError) as e:
            bad()
        assert e.value.status == L.QAT_ERR_DIMENSION_MISMATCH
    with pytest.raises(ValueError):
        fq.weight4(codes, scale, 32, 64, "group", group=48)
    with pytest.raises(ValueError):
        fq.weight4(codes, scale, 32, 64, "column")
    for bad in (lambda: fq.weight4(codes.float(), scale, 32, 64, "row"),
                lambda: fq.weight4(codes, scale.double(), 32, 64, "row"),
                lambda: fq.layer_norm(x, torch.zeros(64, dtype=torch.bfloat16)),
                lambda: fq.gated_ffn(x, torch.zeros(8, 64).bfloat16(), torch.zeros(8, 64), torch.zeros(64, 8)),
                lambda: fq.linear4(x.half(), w)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for call in (lambda: fq.linear4(x, w), lambda: fq.layer_norm(x),
                 lambda: fq.gated_ffn(x, torch.zeros(8, 64), torch.zeros(8, 64), torch.zeros(64, 8))):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
