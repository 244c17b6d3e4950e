"""GPU tests of the layer operators at the edges of their ranges: empty sizes, time-outs
in the middle of a call, the tile shapes of the large products.  Bounds as in
layer_reference.py."""
import numpy as np
import pytest
import torch

import fake_quant_numerics_gb300 as fq
import layer_reference as ref
from test_gpu_layers import DTYPES, quantized, rnd

pytestmark = pytest.mark.gpu


def empty_weight(rows, cols):
    return fq.weight4(torch.empty(0, dtype=torch.uint8, device="cuda"), torch.ones(rows, device="cuda"), rows, cols,
                      "row")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim,hidden", [(3, 64, 0), (3, 0, 64), (3, 31, 0), (0, 64, 32), (600, 64, 0), (2, 0, 0)])
def test_gated_ffn4_empty_sizes(dtype, tokens, dim, hidden):
    """An empty sum is zero (act(0) * 0 too), no tokens are no output."""
    up = quantized(hidden, dim, "row", 0, "symmetric") if hidden and dim else empty_weight(hidden, dim)
    down = quantized(dim, hidden, "row", 0, "symmetric") if hidden and dim else empty_weight(dim, hidden)
    x = rnd(1, tokens, dim, dtype=dtype)
    y = fq.gated_ffn4(x, up, up, down)
    assert y.dtype == dtype and torch.equal(y, torch.zeros(tokens, dim, dtype=dtype, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_of_empty_rows(dtype):
    """The mean of no elements is 0 / 0, and so is what follows from it; memory that
    was freed before must not show through."""
    for _ in range(3):
        torch.full((4096,), 7.0, device="cuda")
    x = torch.empty(5, 3, 0, dtype=dtype, device="cuda")
    r = fq.layer_norm(x)
    assert r.y.shape == x.shape and r.mean.shape == r.rstd.shape == (5, 3)
    assert torch.isnan(r.mean).all() and torch.isnan(r.rstd).all()
    dx, dw, db = fq.layer_norm_backward(x, x, None, r.mean, r.rstd)
    assert dx.shape == x.shape and dw.shape == db.shape == (0,)


# --- bounded waits ---------------------------------------------------------------
class Timed:
    """One forward call of the gated block through the C ABI, with a limit on the
    polls of its device waits."""

    def __init__(self, tokens, dim, hidden, dtype):
        self.x, self.sizes = rnd(1, tokens, dim, dtype=dtype), (tokens, dim, hidden)
        self.w = [rnd(s, hidden, dim, dtype=dtype, scale=0.1) for s in (2, 3)]
        self.wd = rnd(4, dim, hidden, dtype=dtype, scale=0.1)
        n = fq.qat_gated_ffn_workspace_bytes(0 if dtype == torch.float32 else 1, *self.sizes)
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def run(self, limit):
        """(flags, h, g, u, y)"""
        tokens, dim, hidden = self.sizes
        h, y = self.x.new_zeros(tokens, hidden), torch.zeros_like(self.x)
        g, u = (torch.zeros(tokens, hidden, device="cuda") for _ in range(2))
        flags, lib = torch.zeros(1, dtype=torch.int32, device="cuda"), fq.load()
        try:
            lib.qat_debug_set_wait_limit(limit)
            fq.qat_gated_ffn(self.x, tokens, dim, hidden, *self.w, self.wd, "silu", h, g, u, y, flags, self.ws)
            torch.cuda.synchronize()
        finally:
            lib.qat_debug_set_wait_limit(-1)
        return int(flags.item()), h, g, u, y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim,hidden", [(70, 1024, 256), (200, 128, 128), (2600, 256, 2048)])
def test_wait_that_runs_out_leaves_no_stale_output(dtype, tokens, dim, hidden):
    """With no polls allowed nothing is computed: every output is NaN, both
    pre-activations among them."""
    call = Timed(tokens, dim, hidden, dtype)
    flags, *outs = call.run(0)
    assert flags & 16                                   # QAT_FLAG_DEVICE_TIMEOUT
    for name, t in zip(("h", "gate_pre", "up_pre", "y"), outs):
        assert torch.isnan(t).all(), name
    flags, *again = call.run(-1)
    assert flags == 0 and all(torch.isfinite(t).all() for t in again)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim,hidden", [(200, 128, 128), (1500, 192, 256)])
def test_wait_that_runs_out_in_the_middle(dtype, tokens, dim, hidden):
    """A limit that some waits pass and others may not: an output is either right or
    NaN, and without a flag all are right.  The block waits for the copies and
    products it has in flight before it ends, whichever warp gave up."""
    right_or_nan(dtype, tokens, dim, hidden)


def right_or_nan(dtype, tokens, dim, hidden):
    call = Timed(tokens, dim, hidden, dtype)
    flags, *whole = call.run(-1)
    assert flags == 0
    for limit in (1, 2, 3, 5, 9, 17, 40, 100):
        flags, *outs = call.run(limit)
        missing = 0
        for name, t, w in zip(("h", "gate_pre", "up_pre", "y"), outs, whole):
            nan = torch.isnan(t)
            missing += int(nan.sum())
            assert torch.equal(torch.where(nan, w, t), w), (limit, name)
        assert bool(flags & 16) or not missing, limit
    flags, *again = call.run(-1)
    assert flags == 0 and all(torch.equal(a, w) for a, w in zip(again, whole))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim,hidden", [(70, 1024, 256), (128, 2048, 640), (40, 384, 4096)])
def test_wait_that_runs_out_in_the_middle_of_split_sums(dtype, tokens, dim, hidden):
    """The CTAs of a cluster leave their sums where the copies land: no copy that is
    still in flight may put its data in the place of a NaN."""
    right_or_nan(dtype, tokens, dim, hidden)


# --- the large tiles -----------------------------------------------------------------
def sample(n, side, seed):
    """Indices on both sides of every tile edge and some between them."""
    at = {0, n - 1} | {i + d for i in range(side, n, side) for d in (-1, 0)}
    at |= set(np.random.default_rng(seed).integers(0, n, 48).tolist())
    return sorted(at)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim,hidden", [
    (5000, 1032, 1104), (5000, 1031, 1101),   # y, dx: tiles of 224 columns; gated, dh: of 256
    (4100, 2048, 1104), (4100, 2047, 1101),   # y, dx: tiles of 256 columns
    (192, 4096, 2304), (150, 4095, 2301),     # weight gradients: 256 columns, two of them at once
    (192, 2048, 2560), (150, 2049, 2563),     # weight gradients: 224 columns
])
def test_ffn_tiles_of_cta_pairs(dtype, tokens, dim, hidden):
    """Products large enough for pairs of CTAs with more than one tile each, in whole
    vectors and off them, on a sample of rows (of y and dx) and of hidden values (of
    the weights' gradients) with every tile edge in it."""
    x, dy = rnd(1, tokens, dim, dtype=dtype), rnd(5, tokens, dim, dtype=dtype)
    wg, wu = (rnd(s, hidden, dim, dtype=dtype, scale=2 * dim ** -0.5) for s in (2, 3))
    wd = rnd(4, dim, hidden, dtype=dtype, scale=hidden ** -0.5)
    r = fq.gated_ffn(x, wg, wu, wd, save=True)
    dx, dwg, dwu, dwd = fq.gated_ffn_backward(dy, x, wg, wu, wd, r)
    full = [ref.f64(t) for t in (x, wg, wu, wd, dy)]
    x64, wg64, wu64, wd64, dy64 = full
    rows = sample(tokens, 128, 1)
    want = ref.ffn(x64[rows], wg64, wu64, wd64, dy64[rows], "silu", dtype)
    for name, t in (("y", r.y), ("dx", dx)):
        v, e = want[name]
        ref.within(t[rows], v, e + 1e-37, f"{name} {dtype}")
    cols = sample(hidden, 16, 2)
    want = ref.ffn(x64, wg64[cols], wu64[cols], wd64[:, cols], dy64, "silu", dtype)
    for name, t in (("dw_gate", dwg[cols]), ("dw_up", dwu[cols]), ("dw_down", dwd[:, cols])):
        v, e = want[name]
        ref.within(t, v, e + 1e-37, f"{name} {dtype}")
