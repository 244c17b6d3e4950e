"""GPU tests of the layer operators against their 64-bit definitions
(layer_reference.py, where the bounds are derived)."""
import numpy as np
import pytest
import torch

import fake_quant_numerics_gb300 as fq
import layer_reference as ref
from gpu_helpers import bits

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


def rnd(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def off_grid(t):
    """The same values one element past an aligned address."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


# --- products with 4-bit weights --------------------------------------------
LAYOUTS = [("tensor", 0, "symmetric"), ("row", 0, "affine"), ("group", 32, "symmetric"),
           ("group", 128, "affine"), ("group", 48, "affine"), ("double", 0, "")]


def quantized(rows, cols, granularity, group, scheme, seed=0):
    w = rnd(seed, rows, cols, scale=0.02)
    if granularity == "double":
        return fq.weight4_double(fq.quantize_4bit_double(w), rows, cols)
    r = fq.fake_quant_int(w, 4, scheme, granularity, group)
    return fq.weight4(r.codes, r.scale, rows, cols, granularity, group, r.zero_point)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("granularity,group,scheme", LAYOUTS)
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 1, 96), (1, 64, 384), (3, 33, 768), (8, 129, 96), (17, 40, 384), (33, 16, 1920),
    (70, 17, 96), (2, 1030, 4608)])
def test_linear4(dtype, granularity, group, scheme, tokens, rows, cols):
    if granularity == "group" and cols % group:
        cols = (cols // group + 1) * group
    w = quantized(rows, cols, granularity, group, scheme, seed=rows)
    x = rnd(tokens, tokens, cols, dtype=dtype)
    y = fq.linear4(x, w)
    assert y.dtype == dtype and y.shape == (tokens, rows)
    v, e = ref.product(ref.f64(x), ref.weight_values(w))
    ref.within(y, v, e + ref.half(dtype) * (np.abs(v) + e), "linear4")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("granularity", ["tensor", "row", "double"])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 3, 1), (5, 7, 31), (2, 65, 1001), (9, 31, 130),
                                              (4, 5, 16), (3, 1, 33), (6, 127, 250)])
def test_linear4_odd_rows(dtype, granularity, tokens, rows, cols):
    """Rows that start inside a byte and blocks that straddle rows."""
    w = quantized(rows, cols, granularity, 0, "affine", seed=cols)
    x = rnd(tokens + 1, tokens, cols, dtype=dtype)
    v, e = ref.product(ref.f64(x), ref.weight_values(w))
    ref.within(fq.linear4(x, w), v, e + ref.half(dtype) * (np.abs(v) + e), "linear4")


def test_linear4_views_and_strides():
    """x off its vector grid, x with a stride, leading dimensions."""
    w = quantized(96, 256, "group", 64, "affine")
    x = rnd(5, 2, 3, 256, dtype=torch.bfloat16)
    y = fq.linear4(x, w)
    assert y.shape == (2, 3, 96)
    assert torch.equal(fq.linear4(off_grid(x), w), y)
    wide = torch.zeros(2, 3, 512, dtype=torch.bfloat16, device="cuda")
    wide[..., ::2] = x
    assert torch.equal(fq.linear4(wide[..., ::2], w), y)
    out = off_grid(torch.zeros(6, 96, device="cuda"))
    ws = torch.empty(fq.qat_linear4_workspace_bytes(0, 6, 256), dtype=torch.uint8, device="cuda")
    fq.qat_linear4(x.float().contiguous(), 6, w, out, ws)
    assert torch.equal(out.to(torch.bfloat16).view(2, 3, 96), y)


def test_linear4_empty_sizes():
    w = quantized(16, 64, "row", 0, "symmetric")
    assert fq.linear4(torch.empty(0, 64, device="cuda"), w).shape == (0, 16)
    none = fq.weight4(torch.empty(0, dtype=torch.uint8, device="cuda"),
                      torch.ones(16, device="cuda"), 16, 0, "row")
    assert torch.equal(fq.linear4(torch.empty(3, 0, device="cuda"), none),
                       torch.zeros(3, 16, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear4_special_values(dtype):
    """A NaN or an infinity in one token stays in that token; large and
    small magnitudes keep their digits."""
    w = quantized(32, 256, "group", 128, "symmetric")
    v64 = ref.weight_values(w)
    x = rnd(1, 4, 256, dtype=dtype)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    y = ref.f64(fq.linear4(x, w))
    xs = ref.f64(x)
    assert np.isnan(y[1]).all()
    with np.errstate(invalid="ignore"):
        assert np.array_equal(y[2], np.where(v64[:, 9] == 0, np.nan, np.sign(v64[:, 9]) * np.inf),
                              equal_nan=True)
    v, e = ref.product(xs[[0, 3]], v64)
    ref.within(torch.from_numpy(y[[0, 3]]), v, e + ref.half(dtype) * (np.abs(v) + e), "clean tokens")
    for big in (1e35, 1e-30):
        xb = (rnd(2, 2, 256) * 0 + big).to(dtype)
        xb[:, 1::2] *= -1
        v, e = ref.product(ref.f64(xb), v64)
        ref.within(fq.linear4(xb, w), v, e + ref.half(dtype) * (np.abs(v) + e), f"x = {big}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("granularity,group,scheme", [("group", 32, "affine"), ("group", 128, "symmetric"),
                                                      ("row", 0, "affine"), ("double", 0, "")])
@pytest.mark.parametrize("tokens,dim,hidden", [(1, 256, 384), (5, 128, 1152), (9, 384, 128), (34, 128, 128)])
def test_gated_ffn4(dtype, act, granularity, group, scheme, tokens, dim, hidden):
    wg, wu = (quantized(hidden, dim, granularity, group, scheme, seed=s) for s in (1, 2))
    wd = quantized(dim, hidden, granularity, group, scheme, seed=3)
    x = rnd(4, tokens, dim, dtype=dtype, scale=4.0)
    y = fq.gated_ffn4(x, wg, wu, wd, activation=act)
    *_, h, eh = ref.gated(ref.f64(x), ref.weight_values(wg), ref.weight_values(wu), act)
    # h is kept in fp32; its products may take 16 of its bits when y is bf16
    eh = eh + (2.0 ** -16 if dtype == torch.bfloat16 else 4 * ref.U) * np.abs(h)
    d = ref.weight_values(wd)
    v, e = ref.product(h, d)
    e = e + eh @ np.abs(d).T
    ref.within(y, v, e + ref.half(dtype) * (np.abs(v) + e), "gated_ffn4")


def test_gated_ffn4_odd_sizes():
    wg, wu = (quantized(45, 77, "row", 0, "affine", seed=s) for s in (1, 2))
    wd = quantized(77, 45, "row", 0, "affine", seed=3)
    x = rnd(4, 3, 77, scale=4.0)
    *_, h, eh = ref.gated(ref.f64(x), ref.weight_values(wg), ref.weight_values(wu), "silu")
    d = ref.weight_values(wd)
    v, e = ref.product(h, d)
    e = e + (eh + 4 * ref.U * np.abs(h)) @ np.abs(d).T
    ref.within(fq.gated_ffn4(x, wg, wu, wd), v, e + 4 * ref.U * np.abs(v), "gated_ffn4")


# --- gated feed-forward block -----------------------------------------------
def ffn_case(tokens, dim, hidden, dtype, act, place=lambda t: t):
    x = place(rnd(1, tokens, dim, dtype=dtype))
    s = 2.0 / max(1, dim) ** 0.5
    wg, wu = (place(rnd(k, hidden, dim, dtype=dtype, scale=s)) for k in (2, 3))
    wd = place(rnd(4, dim, hidden, dtype=dtype, scale=1.0 / max(1, hidden) ** 0.5))
    dy = place(rnd(5, tokens, dim, dtype=dtype))
    r = fq.gated_ffn(x, wg, wu, wd, activation=act, save=True)
    grads = fq.gated_ffn_backward(dy, x, wg, wu, wd, r, activation=act)
    got = dict(zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (r.y, *grads)))
    want = ref.ffn(*(ref.f64(t) for t in (x, wg, wu, wd, dy)), act, dtype)
    for name, (v, e) in want.items():
        assert got[name].dtype == dtype
        ref.within(got[name], v, e + 1e-37, f"{name} {tokens}x{dim}x{hidden} {dtype} {act}")
    return r, grads


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("tokens,dim,hidden", [(1, 64, 128), (130, 128, 256), (257, 72, 136), (5, 264, 1032)])
def test_ffn(dtype, act, tokens, dim, hidden):
    ffn_case(tokens, dim, hidden, dtype, act)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim,hidden", [
    (1, 1, 1), (3, 5, 7), (129, 65, 127), (64, 100, 33), (31, 513, 260), (300, 130, 514),
    (1, 1024, 2048), (2, 2048, 520), (700, 384, 640), (1025, 256, 128), (16, 8, 4096), (33, 4096, 8)])
def test_ffn_sizes(dtype, tokens, dim, hidden):
    ffn_case(tokens, dim, hidden, dtype, "silu")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim,hidden", [
    (32, 640, 1032), (33, 648, 1032), (48, 1030, 320), (64, 1024, 520), (65, 640, 1032)])
def test_ffn_few_rows(dtype, tokens, dim, hidden):
    """Either side of the row counts at which a stage of the products changes size,
    over more steps than the stages hold."""
    ffn_case(tokens, dim, hidden, dtype, "gelu")


@pytest.mark.parametrize("dtype", DTYPES)
def test_ffn_odd_rows_in_many_tiles(dtype):
    """More tiles than clusters that split k: every output leaves from a tile's own
    sums, with rows off the vector grid."""
    ffn_case(1100, 517, 2051, dtype, "silu")


def test_ffn_few_rows_do_not_depend_on_what_else_is_staged():
    """The rows that a stage leaves out are read as whatever lies there: infinite
    weights of one output stay in that output."""
    x = rnd(1, 5, 1024, dtype=torch.bfloat16)
    w = [rnd(s, 300, 1024, dtype=torch.bfloat16, scale=0.05) for s in (2, 3)]
    wd = rnd(4, 1024, 300, dtype=torch.bfloat16, scale=0.05)
    clean = fq.gated_ffn(x, *w, wd)
    w[0][77] = float("inf")
    wd[500] = float("nan")
    r = fq.gated_ffn(x, *w, wd, save=True)
    keep = [i for i in range(300) if i != 77]
    assert torch.equal(r.h[:, keep], clean.h[:, keep])
    assert not torch.isfinite(r.gate_pre[:, 77]).any()
    assert torch.isfinite(r.gate_pre[:, keep]).all()
    assert torch.isnan(r.y[:, 500]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_ffn_views_off_the_vector_grid(dtype):
    ffn_case(70, 136, 264, dtype, "silu", place=off_grid)


@pytest.mark.parametrize("tokens,dim,hidden", [(0, 16, 32), (4, 0, 32), (4, 16, 0)])
def test_ffn_empty_sizes(tokens, dim, hidden):
    x, dy = torch.ones(tokens, dim, device="cuda"), torch.ones(tokens, dim, device="cuda")
    wg, wu = torch.ones(hidden, dim, device="cuda"), torch.ones(hidden, dim, device="cuda")
    wd = torch.ones(dim, hidden, device="cuda")
    r = fq.gated_ffn(x, wg, wu, wd, save=True)
    grads = fq.gated_ffn_backward(dy, x, wg, wu, wd, r)
    for t in (r.y, *grads):
        assert torch.equal(t, torch.zeros_like(t))


def test_ffn_saves_only_when_asked_and_gives_what_is_wanted():
    x, w = rnd(1, 40, 64, dtype=torch.bfloat16), [rnd(s, 96, 64, dtype=torch.bfloat16) for s in (2, 3)]
    wd, dy = rnd(4, 64, 96, dtype=torch.bfloat16), rnd(5, 40, 64, dtype=torch.bfloat16)
    plain, kept = fq.gated_ffn(x, *w, wd), fq.gated_ffn(x, *w, wd, save=True)
    assert plain.gate_pre is None and torch.equal(plain.y, kept.y) and torch.equal(plain.h, kept.h)
    with pytest.raises(ValueError):
        fq.gated_ffn_backward(dy, x, *w, wd, plain)
    both = fq.gated_ffn_backward(dy, x, *w, wd, kept)
    only_dx = fq.gated_ffn_backward(dy, x, *w, wd, kept, want_dw=False)
    only_dw = fq.gated_ffn_backward(dy, x, *w, wd, kept, want_dx=False)
    assert torch.equal(both[0], only_dx[0]) and only_dx[1:] == (None, None, None)
    assert only_dw[0] is None and all(torch.equal(a, b) for a, b in zip(both[1:], only_dw[1:]))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_gradients_against_differences(act):
    """<grad, v> against the central difference of <y, dy> along v, in fp32.  The
    step s leaves an error of s^2/6 of the third derivative (here within 2e-3 of
    the scale below: directions of size 1, weights of size 1/sqrt(n)) and
    rounding noise 2^-24 |y||dy| sqrt(n) / s, far below it."""
    t, d, f, step = 24, 40, 56, 2e-2
    x, dy = rnd(1, t, d), rnd(5, t, d)
    ws = [rnd(2, f, d, scale=d ** -0.5), rnd(3, f, d, scale=d ** -0.5), rnd(4, d, f, scale=f ** -0.5)]
    grads = fq.gated_ffn_backward(dy, x, *ws, fq.gated_ffn(x, *ws, act, save=True), act)
    args = [x, *ws]
    for k in range(4):
        v = rnd(10 + k, *args[k].shape)
        v = v / v.norm() * args[k].norm()

        def loss(s):
            moved = [a + s * v if j == k else a for j, a in enumerate(args)]
            return float((fq.gated_ffn(*moved, act).y.double() * dy.double()).sum())

        diff = (loss(step) - loss(-step)) / (2 * step)
        dot = float((grads[k].double() * v.double()).sum())
        scale = float(grads[k].double().norm() * v.double().norm())
        assert abs(diff - dot) <= 2e-3 * scale, (k, diff, dot, scale)


def test_ffn_nan_stays_in_its_rows():
    x = rnd(1, 200, 128, dtype=torch.bfloat16)
    w = [rnd(s, 256, 128, dtype=torch.bfloat16, scale=0.1) for s in (2, 3)]
    wd = rnd(4, 128, 256, dtype=torch.bfloat16, scale=0.1)
    clean = fq.gated_ffn(x, *w, wd).y
    x[131, 5] = float("nan")
    y = fq.gated_ffn(x, *w, wd).y
    assert torch.isnan(y[131]).all()
    keep = [i for i in range(200) if i != 131]
    assert torch.equal(y[keep], clean[keep])


def test_ffn_is_reproducible():
    x = rnd(1, 17, 1024, dtype=torch.bfloat16)
    w = [rnd(s, 2048, 1024, dtype=torch.bfloat16, scale=0.03) for s in (2, 3)]
    wd, dy = rnd(4, 1024, 2048, dtype=torch.bfloat16, scale=0.03), rnd(5, 17, 1024, dtype=torch.bfloat16)
    runs = []
    for _ in range(3):
        r = fq.gated_ffn(x, *w, wd, save=True)
        runs.append([r.y, *fq.gated_ffn_backward(dy, x, *w, wd, r)])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert np.array_equal(bits(a), bits(b))


def test_ffn_autograd():
    x = rnd(1, 2, 9, 48).requires_grad_()
    ws = [rnd(s, *shape, scale=0.2).requires_grad_() for s, shape in ((2, (80, 48)), (3, (80, 48)), (4, (48, 80)))]
    dy = rnd(5, 2, 9, 48)
    fq.GatedFfnFunction.apply(x, *ws, "silu").backward(dy)
    r = fq.gated_ffn(x.detach(), *(w.detach() for w in ws), save=True)
    want = fq.gated_ffn_backward(dy, x.detach(), *(w.detach() for w in ws), r)
    for t, g in zip((x, *ws), want):
        assert torch.equal(t.grad, g)


# --- layer norm --------------------------------------------------------------
def norm_case(rows, cols, dtype, affine=True, eps=1e-5, place=lambda t: t, shift=0.5):
    x = place(rnd(rows, rows, cols, dtype=dtype) + shift)
    w = place((1 + rnd(2, cols, scale=0.1)).to(dtype)) if affine else None
    b = place(rnd(3, cols, dtype=dtype)) if affine else None
    dy = place(rnd(4, rows, cols, dtype=dtype))
    r = fq.layer_norm(x, w, b, eps)
    dx, dw, db = fq.layer_norm_backward(dy, x, w, r.mean, r.rstd)
    got = {"y": r.y, "mean": r.mean, "rstd": r.rstd, "dx": dx, "dweight": dw, "dbias": db}
    n64 = [None if t is None else ref.f64(t) for t in (x, w, b)]
    for name, (v, e) in ref.norm(*n64, eps, ref.f64(dy), dtype).items():
        ref.within(got[name], v, e + 1e-37, f"{name} {rows}x{cols} {dtype}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [
    (1, 1), (7, 3), (1, 4096), (5, 31), (33, 256), (100, 264), (9, 520), (65, 1000), (400, 1024),
    (3, 1032), (17, 2048), (1000, 2056), (11, 4104), (330, 5003), (6, 8192), (5, 8200), (3, 16384),
    (2, 16392), (2, 20011), (3, 40000), (5000, 8)])
def test_layer_norm(dtype, rows, cols):
    norm_case(rows, cols, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [64, 1000, 4096, 9000])
def test_layer_norm_views_and_no_affine(dtype, cols):
    norm_case(37, cols, dtype, place=off_grid)
    norm_case(37, cols, dtype, affine=False)


def test_layer_norm_far_from_zero():
    """Deviations are summed around the mean: a mean a thousand times the spread."""
    norm_case(50, 1536, torch.float32, shift=1000.0)
    norm_case(50, 5003, torch.float32, shift=-1000.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_constant_and_special_rows(dtype):
    x = rnd(1, 6, 512, dtype=dtype)
    x[1] = 3.0
    x[3, 100] = float("nan")
    x[4, 0] = float("inf")
    r = fq.layer_norm(x, None, None, 1e-5)
    y = ref.f64(r.y)
    assert np.array_equal(y[1], np.zeros(512)) and abs(float(r.rstd[1]) - 1e5 ** 0.5) < 1e-3
    assert np.isnan(y[3]).all() and np.isnan(y[4]).all()
    clean = ref.norm(ref.f64(x[[0, 2, 5]]), None, None, 1e-5, None, dtype)["y"]
    ref.within(r.y[[0, 2, 5]], *clean, "clean rows")


def test_layer_norm_empty_sizes():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    r = fq.layer_norm(x, w, w)
    assert r.y.shape == (0, 64)
    dx, dw, db = fq.layer_norm_backward(x, x, w, r.mean, r.rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    assert fq.layer_norm(torch.empty(5, 0, device="cuda")).y.shape == (5, 0)


def test_layer_norm_gives_what_is_wanted_and_repeats():
    x, dy, w = rnd(1, 999, 768, dtype=torch.bfloat16), rnd(2, 999, 768, dtype=torch.bfloat16), None
    r = fq.layer_norm(x)
    both = fq.layer_norm_backward(dy, x, w, r.mean, r.rstd)
    for _ in range(3):
        again = fq.layer_norm_backward(dy, x, w, r.mean, r.rstd)
        assert all(np.array_equal(bits(a), bits(b)) for a, b in zip(both, again))
    only_dx = fq.layer_norm_backward(dy, x, w, r.mean, r.rstd, want_dw=False)
    only_dw = fq.layer_norm_backward(dy, x, w, r.mean, r.rstd, want_dx=False)
    assert torch.equal(only_dx[0], both[0]) and only_dx[1:] == (None, None)
    assert only_dw[0] is None and torch.equal(only_dw[1], both[1]) and torch.equal(only_dw[2], both[2])


def test_layer_norm_gradients_against_differences():
    """As for the block: central differences of <y, dy> in fp32, step 1e-2."""
    x, w, b, dy = rnd(1, 20, 96), 1 + rnd(2, 96, scale=0.1), rnd(3, 96), rnd(4, 20, 96)
    r = fq.layer_norm(x, w, b)
    grads = fq.layer_norm_backward(dy, x, w, r.mean, r.rstd)
    args = [x, w, b]
    for k in range(3):
        v = rnd(10 + k, *args[k].shape)

        def loss(s):
            moved = [a + s * v if j == k else a for j, a in enumerate(args)]
            return float((fq.layer_norm(*moved).y.double() * dy.double()).sum())

        diff = (loss(1e-2) - loss(-1e-2)) / 2e-2
        dot = float((grads[k].double() * v.double()).sum())
        scale = float(grads[k].double().norm() * v.double().norm())
        assert abs(diff - dot) <= 2e-3 * scale, (k, diff, dot, scale)


def test_layer_norm_autograd():
    x, w, b = rnd(1, 3, 5, 64).requires_grad_(), rnd(2, 64).requires_grad_(), rnd(3, 64).requires_grad_()
    dy = rnd(4, 3, 5, 64)
    fq.LayerNormFunction.apply(x, w, b, 1e-5).backward(dy)
    r = fq.layer_norm(x.detach(), w.detach(), b.detach())
    for t, g in zip((x, w, b), fq.layer_norm_backward(dy, x.detach(), w.detach(), r.mean, r.rstd)):
        assert torch.equal(t.grad, g)


# --- streams and graphs ------------------------------------------------------
def test_side_stream_and_graph_replay():
    """The calls run on the stream they are given and replay on new inputs."""
    x = rnd(1, 5, 256, dtype=torch.bfloat16)
    wg, wu = (quantized(384, 256, "group", 128, "affine", seed=s) for s in (1, 2))
    wd = quantized(256, 384, "group", 128, "affine", seed=3)
    fg, fu = (rnd(s, 384, 256, dtype=torch.bfloat16, scale=0.1) for s in (4, 5))
    fd = rnd(6, 256, 384, dtype=torch.bfloat16, scale=0.1)

    def step():
        n = fq.layer_norm(x)
        r = fq.gated_ffn(n.y, fg, fu, fd, save=True)
        return (fq.gated_ffn4(n.y, wg, wu, wd), r.y, *fq.gated_ffn_backward(x, n.y, fg, fu, fd, r),
                *fq.layer_norm_backward(x, x, None, n.mean, n.rstd))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (7, 8):
        x.copy_(rnd(seed, 5, 256, dtype=torch.bfloat16))
        graph.replay()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


# --- failure detection ---------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim,hidden", [(70, 1024, 256), (200, 128, 128), (2600, 256, 2048)])
def test_ffn_wait_that_runs_out_is_reported(dtype, tokens, dim, hidden):
    """With no polls allowed every bounded wait of the products gives up at once:
    the call returns, flags the time-out and leaves NaN, and the next call (with
    the default limit) is whole again."""
    x = rnd(1, tokens, dim, dtype=dtype)
    w = [rnd(s, hidden, dim, dtype=dtype, scale=0.1) for s in (2, 3)]
    wd = rnd(4, dim, hidden, dtype=dtype, scale=0.1)
    want = fq.gated_ffn(x, *w, wd)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, y = torch.zeros_like(want.h), torch.zeros_like(want.y)
    dt = 0 if dtype == torch.float32 else 1
    n = fq.qat_gated_ffn_workspace_bytes(dt, tokens, dim, hidden)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    lib = fq.load()
    try:
        lib.qat_debug_set_wait_limit(0)
        fq.qat_gated_ffn(x, tokens, dim, hidden, *w, wd, "silu", h, None, None, y, flags, ws)
        torch.cuda.synchronize()
    finally:
        lib.qat_debug_set_wait_limit(-1)
    assert int(flags.item()) & 16                      # QAT_FLAG_DEVICE_TIMEOUT
    assert torch.isnan(y).all() and torch.isnan(h).all()
    flags.zero_()
    fq.qat_gated_ffn(x, tokens, dim, hidden, *w, wd, "silu", h, None, None, y, flags, ws)
    assert int(flags.item()) == 0 and torch.equal(y, want.y) and torch.equal(h, want.h)


@pytest.mark.parametrize("tokens,dim,hidden", [(5, 1024, 256), (40, 1024, 256)])
def test_ffn_wait_that_runs_out_with_few_rows(tokens, dim, hidden):
    test_ffn_wait_that_runs_out_is_reported(torch.bfloat16, tokens, dim, hidden)


def test_example_trains_and_serves():
    """The example layer learns (the loss falls by half at least) and its 4-bit
    form stays near it: codes of 15 levels are off by 1/14 of a group's largest
    weight at most, about a tenth of the block's output, which is a part of y."""
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import qat_ffn_layer

    losses, off = qat_ffn_layer.main(steps=60)
    assert losses[-1] < 0.5 * losses[0]
    assert off < 0.15
