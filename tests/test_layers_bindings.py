"""What the layer bindings refuse or set up before anything reaches a kernel
(CPU; the meta device stands for another device)."""
import pytest
import torch

import fake_quant_numerics_gb300 as fq
from fake_quant_numerics_gb300 import _lib as L


def meta(t):
    return t.to("meta")


CODES, SCALE, ZP = torch.zeros(32 * 64 // 2, dtype=torch.uint8), torch.ones(32), torch.zeros(32, dtype=torch.int32)


@pytest.mark.parametrize("build", [
    lambda: fq.weight4(CODES, meta(SCALE), 32, 64, "row"),
    lambda: fq.weight4(meta(CODES), SCALE, 32, 64, "row"),
    lambda: fq.weight4(CODES, SCALE, 32, 64, "row", zero_point=meta(ZP)),
    lambda: fq.weight4_double(double(super_scales=meta(torch.ones(1))), 32, 64),
    lambda: fq.weight4_double(double(quantized_scales=meta(torch.zeros(32, dtype=torch.uint8))), 32, 64),
])
def test_weight_parts_share_a_device(build):
    """The kernels take raw addresses: a scale in host memory beside codes on the
    GPU must not reach them."""
    with pytest.raises(ValueError, match="tensors on (cpu|meta)"):
        build()


def double(n=32 * 64, **kw):
    blocks = -(-n // 64)
    a = dict(data=torch.zeros(-(-n // 2), dtype=torch.uint8), quantized_scales=torch.zeros(blocks, dtype=torch.uint8),
             super_scales=torch.ones(-(-blocks // 256)), len=n, y=None)
    a.update(kw)
    return fq.DoubleQuantized4Bit(**a)


def test_two_level_weight_checks_its_parts():
    assert fq.weight4_double(double(), 32, 64).rows == 32
    assert fq.weight4_double(double(3 * 5501), 3, 5501).super_scales.numel() == 2
    for short in (dict(data=torch.zeros(32 * 32 - 1, dtype=torch.uint8)),
                  dict(quantized_scales=torch.zeros(31, dtype=torch.uint8)), dict(super_scales=torch.ones(0))):
        with pytest.raises(fq.QatError) as e:
            fq.weight4_double(double(**short), 32, 64)
        assert e.value.status == L.QAT_ERR_DIMENSION_MISMATCH
    for other in (dict(data=torch.zeros(32 * 32)), dict(quantized_scales=torch.zeros(32)),
                  dict(super_scales=torch.ones(1).double())):
        with pytest.raises(TypeError):
            fq.weight4_double(double(**other), 32, 64)


def test_weights_are_where_x_is():
    w = fq.weight4(meta(CODES), meta(SCALE), 32, 64, "row")
    here = fq.weight4(CODES, SCALE, 32, 64, "row")
    down = fq.weight4(CODES, torch.ones(64), 64, 32, "row")
    x = torch.zeros(3, 64)
    for call in (lambda: fq.linear4(x, w), lambda: fq.gated_ffn4(x, w, here, down),
                 lambda: fq.gated_ffn4(x, here, w, down),
                 lambda: fq.gated_ffn4(x, here, here, fq.weight4(meta(CODES), meta(torch.ones(64)), 64, 32, "row"))):
        with pytest.raises(ValueError, match="tensors on (cpu|meta)"):
            call()


def test_saved_tensors_are_where_x_is():
    x, w, wd = torch.zeros(3, 64), torch.zeros(8, 64), torch.zeros(64, 8)
    kept = torch.zeros(3, 8)
    for g, u in ((meta(kept), kept), (kept, meta(kept))):
        with pytest.raises(ValueError, match="tensors on (cpu|meta)"):
            fq.gated_ffn_backward(x, x, w, w, wd, fq.GatedFfn(x, kept, g, u))
    row = torch.zeros(3)
    for mean, rstd in ((meta(row), row), (row, meta(row))):
        with pytest.raises(ValueError, match="tensors on (cpu|meta)"):
            fq.layer_norm_backward(x, x, None, mean, rstd)


# --- second derivatives --------------------------------------------------------
def test_layer_functions_refuse_second_derivatives(monkeypatch):
    """The backward passes fill tensors by address, so a gradient of a gradient
    would lose its terms without a word; it is an error instead.  Plain products
    stand for the kernels."""
    from fake_quant_numerics_gb300 import layers

    def norm(x, w, b, eps):
        return layers.LayerNorm(x.detach() * w.detach(), torch.zeros(len(x)), torch.ones(len(x)))

    def norm_back(dy, x, w, mean, rstd, want_dx, want_dw):
        return (dy * w).detach(), (dy * x).sum(0).detach(), dy.sum(0).detach()

    def ffn(x, wg, wu, wd, act, save):
        h = (x @ wg.T).detach()
        return layers.GatedFfn((h @ wd.T).detach(), h, h, h)

    def ffn_back(dy, x, wg, wu, wd, saved, act, want_dx, want_dw):
        return tuple(torch.ones_like(t) for t in (x, wg, wu, wd))

    for name, f in (("layer_norm", norm), ("layer_norm_backward", norm_back), ("gated_ffn", ffn),
                    ("gated_ffn_backward", ffn_back)):
        monkeypatch.setattr(layers, name, f)
    x, b = torch.randn(3, 4, requires_grad=True), torch.zeros(4, requires_grad=True)
    w = [torch.randn(4, 4, requires_grad=True) for _ in range(3)]
    for y in (fq.LayerNormFunction.apply(x, w[0][0], b, 1e-5), fq.GatedFfnFunction.apply(x, *w, "silu")):
        (dx,) = torch.autograd.grad((y * y).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            ((dx * dx).sum() + x.sum()).backward()


def test_ste_second_derivative(monkeypatch):
    """The estimator's backward pass is linear in the gradient: with a mask m,
    y = x (forward value kept) and L = sum y^3, dL/dx = 3 m y^2 and the gradient of
    sum (dL/dx) is 6 m y."""
    from fake_quant_numerics_gb300 import api

    m = torch.tensor([1.0, 0.0, 1.0])
    monkeypatch.setattr(api, "fake_quant_int", lambda x, *a, **k: api.FakeQuantInt(x.detach().clone(), None, m, None,
                                                                                 None, None))
    monkeypatch.setattr(api, "fake_quant_backward", lambda g, mask: (g * mask).detach())
    x = torch.tensor([2.0, 3.0, -1.0], requires_grad=True)
    y = fq.FakeQuantSTE.apply(x)
    (dx,) = torch.autograd.grad((y ** 3).sum(), x, create_graph=True)
    assert torch.equal(dx.detach(), 3 * m * x.detach() ** 2)
    (ddx,) = torch.autograd.grad(dx.sum(), x)
    assert torch.equal(ddx, 6 * m * x.detach())


# --- the current device ----------------------------------------------------------
@pytest.mark.parametrize("current,guarded", [(None, False), (1, True)])
def test_calls_launch_on_the_tensors_device(monkeypatch, current, guarded):
    """A launch goes to the current device, so tensors of another one make theirs
    current for the call (host tensors, whose device has no index, stand for them)."""
    from fake_quant_numerics_gb300 import layers

    entered, seen = [], []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *args):
            entered.pop()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 64
            return lambda *a: seen.append((name, bool(entered))) or 0

    monkeypatch.setattr(layers._lib, "lib", lambda: Lib())
    monkeypatch.setattr(layers, "_ptr", lambda t: t.data_ptr())
    monkeypatch.setattr(layers, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(layers, "_current_device", lambda: current, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    x, w, wd = torch.zeros(3, 64), torch.zeros(32, 64), torch.zeros(64, 32)
    w4, down = fq.weight4(CODES, SCALE, 32, 64, "row"), fq.weight4(CODES, torch.ones(64), 64, 32, "row")
    fq.linear4(x, w4)
    fq.gated_ffn4(x, w4, w4, down)
    r = fq.gated_ffn(x, w, w, wd, save=True)
    fq.gated_ffn_backward(x, x, w, w, wd, r)
    n = fq.layer_norm(x)
    fq.layer_norm_backward(x, x, None, n.mean, n.rstd)
    assert not entered
    names = ["linear4", "gated_ffn4", "gated_ffn", "gated_ffn_backward", "layer_norm", "layer_norm_backward"]
    assert seen == [("qat_" + name, guarded) for name in names]


def test_layer_norm_of_empty_rows_has_no_statistics(monkeypatch):
    """The library's call is a no-op for rows without elements: the binding gives
    their mean, 0 / 0, not the memory it allocated."""
    from fake_quant_numerics_gb300 import layers

    monkeypatch.setattr(layers, "_call", lambda *a: None)
    monkeypatch.setattr(layers, "_ptr", lambda t: t.data_ptr())
    monkeypatch.setattr(torch, "empty", lambda *s, **kw: torch.ones(*s, **kw))
    r = fq.layer_norm(torch.zeros(4, 0))
    assert torch.isnan(r.mean).all() and torch.isnan(r.rstd).all() and r.mean.shape == (4,)


def test_more_weight_rows_than_a_grid_holds_are_refused():
    """The kernel for any shape takes four rows a block: past 2^33 - 4 rows the number
    of blocks does not fit a launch, and past 2^34 it would wrap to a few."""
    import ctypes

    from fake_quant_numerics_gb300 import build

    build.build()
    lib = L.load(build_if_missing=False)
    at = ctypes.c_void_p(0x10000)

    def call(rows):
        w = L.Weight4Struct(0x10000, 0x10000, None, None, rows, 1, 0, L.PER_TENSOR)
        # (no tokens, no workspace: stops at the first check that fails)
        return (lib.qat_linear4(at, L.F32, 1, ctypes.byref(w), at, None, 0, None),
                lib.qat_linear4(at, L.F32, 0, ctypes.byref(w), at, None, 0, None))

    assert call((1 << 33) - 4) == (L.QAT_ERR_WORKSPACE, L.QAT_OK)
    for rows in ((1 << 33) - 3, 1 << 34, (1 << 34) + 8):
        assert call(rows) == (L.QAT_ERR_INVALID_ARGUMENT,) * 2
