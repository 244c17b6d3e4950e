"""Attention operators on the GPU against their 64-bit definitions
(attention_reference.py, which derives every bound)."""
import math

import numpy as np
import pytest
import torch

import attention_reference as ref
from layer_reference import f64, within

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def randn(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


# --- head norm and rotation ------------------------------------------------------
ROPE = [
    # tokens, query heads, key heads, head_dim, rotary, layout, norm, amplitude, first position, type
    (1, 1, 1, 128, 128, "half", True, 1.0, 0, BF16),
    (5, 32, 8, 128, 128, "half", True, 1.0, 131000, BF16),
    (300, 32, 8, 128, 128, "half", True, 1.0, 7, BF16),       # several heads a group
    (7, 6, 2, 64, 32, "interleaved", True, 1.25, 100, F32),
    (9, 4, 4, 80, 40, "half", True, 1.0, 5, BF16),            # runs of four
    (9, 4, 1, 80, 20, "interleaved", True, 1.0, 5, F32),      # runs of two
    (3, 3, 2, 40, 10, "half", True, 0.5, -3, F32),            # single elements
    (3, 5, 1, 7, 4, "interleaved", True, 1.0, 1 << 40, BF16), # an odd head
    (4, 2, 2, 512, 512, "half", True, 1.0, 11, BF16),
    (4, 2, 2, 509, 254, "half", True, 1.0, 11, F32),          # eight runs a lane
    (4, 2, 1, 256, 0, "half", True, 1.0, 11, BF16),           # nothing turns
    (6, 3, 2, 96, 96, "interleaved", False, 1.0, 1 << 50, BF16),  # no norm
    (6, 3, 0, 64, 64, "half", False, 1.5, 9, F32),            # no keys
    (2, 1, 1, 1, 0, "half", True, 1.0, 0, F32),
    (70, 7, 7, 80, 40, "interleaved", True, 1.25, 4096, F32),
    (5, 3, 2, 127, 62, "half", True, 1.0, 77, BF16),          # two single elements a lane
    (5, 3, 2, 512, 24, "interleaved", True, 1.0, 77, BF16),   # two runs of four a lane
    (5, 3, 2, 500, 20, "half", True, 1.25, 77, F32),          # four runs of two a lane
    (2000, 9, 3, 64, 64, "half", True, 1.0, 50, BF16),        # more heads than the blocks hold at once
]


def rope_case(case, seed=0, weights=True, strided=True):
    t, hq, hk, d, rot, layout, norm, amplitude, first, dtype = case
    pad = 8 if strided else 0
    row = randn(seed, t, (hq + 2 * hk) * d + pad, dtype=dtype)
    q = row[:, :hq * d].view(t, hq, d)
    k = row[:, hq * d:(hq + hk) * d].view(t, hk, d) if hk else None
    return q, k


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(map(str, c[:6])))
@pytest.mark.parametrize("weights", [True, False])
def test_head_norm_rope(qat, case, weights):
    t, hq, hk, d, rot, layout, norm, amplitude, first, dtype = case
    q, k = rope_case(case)
    weights = weights and norm
    wq = 1 + randn(1, d, scale=0.3) if weights else None
    wk = 1 + randn(2, d, scale=0.3) if weights and hk else None
    wq, wk = (None if w is None else w.to(dtype) for w in (wq, wk))
    positions = torch.arange(first, first + t).cuda()
    turns = qat.rope_turns(qat.rope_frequencies(rot), "cuda")
    kw = dict(eps=1e-5, norm=norm, layout=layout, amplitude=amplitude)
    y = qat.head_norm_rope(q, k, positions, turns, wq, wk, **kw)
    dyq, dyk = randn(3, t, hq, d, dtype=dtype), randn(4, t, hk, d, dtype=dtype) if hk else None
    g = qat.head_norm_rope_backward(dyq, dyk, q, k, positions, turns, wq, wk, **kw)
    c, s = ref.angles(positions.tolist(), turns.tolist(), amplitude)
    for x, w, dy, got, dx, dw in ((q, wq, dyq, y.q, g[0], g[2]), (k, wk, dyk, y.k, g[1], g[3])):
        if x is None:
            assert got is None and dx is None and dw is None
            continue
        want = ref.rope(f64(x), None if w is None else f64(w), f64(dy), c, s, layout, 1e-5, norm, amplitude, dtype)
        assert got.dtype == dtype and got.is_contiguous()
        within(got, *want["y"], "y")
        within(dx, *want["dx"], "dx")
        if w is None:
            assert dw is None
        else:
            within(dw, *want["dw"], "dw")


def test_head_norm_rope_gradients_against_differences(qat):
    """dL/dx along a direction against the difference of the kernel's own fp32 outputs,
    L = sum c y.  Central differences at step h are off by h^2/6 |L'''|, outputs by
    rounding over 2 h."""
    t, hq, d, h = 5, 3, 64, 2.0 ** -7
    q, w = randn(0, t, hq, d), 1 + randn(1, d, scale=0.3)
    positions, turns = torch.arange(3, 3 + t).cuda(), qat.rope_turns(qat.rope_frequencies(32), "cuda")
    c, dirq, dirw = randn(2, t, hq, d), randn(3, t, hq, d), randn(4, d)

    def loss(e):
        y = qat.head_norm_rope(q + e * dirq, None, positions, turns, w + e * dirw).q
        return float((f64(y) * f64(c)).sum())

    dq, _, dw, _ = qat.head_norm_rope_backward(c, None, q, None, positions, turns, w)
    slope = float((f64(dq) * f64(dirq)).sum() + (f64(dw) * f64(dirw)).sum())
    d1 = (loss(h) - loss(-h)) / (2 * h)
    d2 = (loss(2 * h) - loss(-2 * h)) / (4 * h)
    # d1 and d2 bracket the h^2 term: slope = d1 + (d1 - d2) / 3 + O(h^4); the sums' rounding is
    # at most 960 terms of size about 4, each 2^-22 off, over 2 h
    assert abs(slope - (d1 + (d1 - d2) / 3)) <= abs(d1 - d2) + 960 * 4 * 2.0 ** -22 / (2 * h) / math.sqrt(960)


def test_head_norm_rope_of_views(qat):
    """Leading dimensions, views off the vector grid, expanded keys, no tokens."""
    turns = qat.rope_turns(qat.rope_frequencies(64), "cuda")
    flat = randn(0, 2 * 3 * 4 * 64 + 1)
    q = flat[1:].view(2, 3, 4, 64)
    positions = torch.arange(6).view(2, 3).cuda()
    c, s = ref.angles(range(6), turns.tolist(), 1.0)
    want = ref.rope(f64(q).reshape(6, 4, 64), None, None, c, s, "half", 1e-6, True, 1.0, F32)["y"]
    turned = q.transpose(2, 3).contiguous().transpose(2, 3)  # no dense last dimension
    for x in (q, q.clone(), turned):
        r = qat.head_norm_rope(x, x[:, :, :1].expand(2, 3, 2, 64), positions, turns)
        assert r.q.shape == q.shape and r.k.shape == (2, 3, 2, 64)
        within(r.q.view(6, 4, 64), *want, "q")
        for i in range(2):
            assert torch.equal(r.k[:, :, i], r.q[:, :, 0])
    none = qat.head_norm_rope(q[:0], q[:0], positions[:0], turns)
    assert none.q.shape == (0, 3, 4, 64)
    w = torch.ones(64, device="cuda")
    g = qat.head_norm_rope_backward(q[:0], q[:0], q[:0], q[:0], positions[:0], turns, w, w)
    assert not g[2].any() and not g[3].any() and g[0].numel() == 0
    e = randn(1, 3, 0, 64)
    g = qat.head_norm_rope_backward(e, e, e, e, positions[0], turns, w, w)
    assert not g[2].any() and not g[3].any()


def test_head_norm_rope_nonfinite_heads_stay_alone(qat):
    q = randn(0, 4, 8, 128, dtype=BF16)
    clean = qat.head_norm_rope(q, None, torch.arange(4).cuda(), qat.rope_turns(qat.rope_frequencies(128), "cuda")).q
    q[1, 3, 5], q[2, 0, 100] = float("nan"), float("inf")
    y = qat.head_norm_rope(q, None, torch.arange(4).cuda(), qat.rope_turns(qat.rope_frequencies(128), "cuda")).q
    assert torch.isnan(y[1, 3]).all() and torch.isnan(y[2, 0]).any()
    y[1, 3], y[2, 0] = clean[1, 3], clean[2, 0]
    assert torch.equal(y, clean)


def test_head_norm_rope_function(qat):
    """Gradients through autograd are the backward call's; one that is not asked for
    is None; a second derivative is refused."""
    turns, positions = qat.rope_turns(qat.rope_frequencies(64), "cuda"), torch.arange(6).cuda()
    q, k = randn(0, 6, 4, 64).requires_grad_(), randn(1, 6, 2, 64).requires_grad_()
    wq, wk = (1 + randn(2 + i, 64, scale=0.1) for i in range(2))
    wq.requires_grad_()
    cq, ck = randn(5, 6, 4, 64), randn(6, 6, 2, 64)
    yq, yk = qat.HeadNormRopeFunction.apply(q, k, positions, turns, wq, wk)
    ((yq * cq).sum() + (yk * ck).sum()).backward()
    want = qat.head_norm_rope_backward(cq, ck, q.detach(), k.detach(), positions, turns, wq.detach(), wk)
    assert torch.equal(q.grad, want[0]) and torch.equal(k.grad, want[1]) and torch.equal(wq.grad, want[2])
    assert wk.grad is None
    y, none = qat.HeadNormRopeFunction.apply(q, None, positions, turns)
    assert none is None
    (dq,) = torch.autograd.grad(y.square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((dq * dq).sum() + q.sum()).backward()


# --- the cache -------------------------------------------------------------------
FORMS = [("int8", "symmetric"), ("int8", "affine"), ("int4", "symmetric"), ("int4", "affine"), ("e4m3", "symmetric"),
         ("e5m2", "symmetric"), ("bf16", "symmetric")]


def special_rows(x):
    """Rows that the calibration has to treat apart."""
    x = x.clone()
    flat = x.view(-1, x.shape[-1])
    tiny = torch.finfo(torch.float32).tiny
    for i, v in enumerate((0.0, -0.0, 1.0, -2.5, float("nan"), float("inf"), -float("inf"), tiny / 1024, 3e38)):
        if i < len(flat):
            flat[i] = v if not math.isinf(v) and v == v else flat[i]
            if math.isinf(v) or v != v:
                flat[i, i % x.shape[-1]] = v
    if len(flat) > 12:
        flat[9] = flat[9].abs()      # no negative values
        flat[10] = -flat[10].abs()
        flat[11] = flat[11] * 1e-40  # subnormal
        flat[12, 0], flat[12, 1] = 3.3e38, -3.3e38  # an affine range that overflows
    return x


@pytest.mark.parametrize("form,scheme", FORMS)
@pytest.mark.parametrize("d,heads,page,dtype", [(128, 8, 16, BF16), (64, 3, 48, F32), (72, 2, 32, BF16), (8, 1, 16, F32),
                                               (256, 2, 256, F32), (40, 5, 16, BF16), (200, 1, 64, BF16)])
def test_kv_write_and_read(qat, form, scheme, d, heads, page, dtype):
    """Codes, scales and zero points bit for bit; what no slot names stays as it was."""
    pages, tokens = 5, 37
    cache = qat.kv_cache(pages, heads, page, d, form, scheme)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x5a)
    for t in (cache.k_scale, cache.v_scale):
        if t is not None:
            t.fill_(-7.0)
    g = torch.Generator().manual_seed(d)
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    slots[5], slots[6], slots[7] = -1, pages * page, 1 << 40
    # keys and values side by side, off the 16-byte grid
    both = special_rows(randn(1, tokens, 2 * heads, d)).to(dtype)
    flat = torch.empty(both.numel() + 1, dtype=dtype, device="cuda")
    flat[1:] = both.reshape(-1)
    both = flat[1:].view(tokens, 2 * heads, d) if page == 48 else both
    k, v = both[:, :heads], both[:, heads:]
    qat.kv_write(cache, k, v, slots.cuda())
    there = [i for i in range(tokens) if 0 <= slots[i] < pages * page]
    at = (slots[there] // page, slice(None), slots[there] % page)
    rest = torch.ones(pages, page, dtype=torch.bool)
    rest[at[0], at[2]] = False
    for name, x in (("k", k), ("v", v)):
        codes, rows = ref.codes_of(cache, name)[at], getattr(cache, name).cpu()
        x64 = f64(x)[there]
        if form == "bf16":
            assert torch.equal(rows[at].view(torch.int16), x.to(BF16).cpu()[there].view(torch.int16))
        else:
            q, scale, zp = ref.quantized(x64, form, scheme)
            np.testing.assert_array_equal(f64(getattr(cache, name + "_scale"))[at], scale)
            np.testing.assert_array_equal(codes, q)
            if scheme == "affine":
                np.testing.assert_array_equal(f64(getattr(cache, name + "_zero_point"))[at], zp)
            used = d // 2 if form == "int4" else d
            assert not rows[at][..., used:].any()  # padding
            left = getattr(cache, name + "_scale").cpu().permute(0, 2, 1)[rest]
            assert (left == -7.0).all()
        assert (rows.view(torch.uint8).permute(0, 2, 1, 3)[rest] == 0x5a).all()
    for out in (F32, BF16):
        r = qat.kv_read(cache, slots.cuda(), out)
        for name, got in (("k", r.k), ("v", r.v)):
            want = ref.values_of(cache, name)[at]
            want = torch.from_numpy(want).float() if out == F32 else torch.from_numpy(want).float().to(BF16)
            assert torch.equal(torch.nan_to_num(got.cpu()[there].float(), 12345.0),
                               torch.nan_to_num(want.float(), 12345.0))
            gone = [i for i in range(tokens) if i not in there]
            assert not got[gone].any()


@pytest.mark.parametrize("form,scheme,dtype", [("int8", "symmetric", BF16), ("int4", "affine", F32),
                                               ("e4m3", "symmetric", BF16), ("bf16", "symmetric", F32)])
def test_kv_many_tokens_are_each_as_alone(qat, form, scheme, dtype):
    """A long prompt, whose rows are taken several at a time, gives what short calls give."""
    t, heads, d = 27000, 7, 128  # (14 rows a token: no whole number of fours)
    pages = -(-t // 64)
    slots = torch.randperm(pages * 64, generator=torch.Generator().manual_seed(1))[:t].cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(t, heads, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k[77, 3] = 0
    k[78, 2, 5] = float("nan")
    once, parts = (qat.kv_cache(pages, heads, 64, d, form, scheme) for _ in range(2))
    qat.kv_write(once, k, v, slots)
    for a in range(0, t, 999):
        qat.kv_write(parts, k[a:a + 999], v[a:a + 999], slots[a:a + 999])
    for name in ("k", "v", "k_scale", "v_scale", "k_zero_point", "v_zero_point"):
        x, y = getattr(once, name), getattr(parts, name)
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name
    slots[5] = -1
    r = qat.kv_read(once, slots, dtype)
    for a in range(0, t, 999):
        p = qat.kv_read(once, slots[a:a + 999], dtype)
        for x, y in zip(r, p):
            assert torch.equal(x[a:a + 999].view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("form,scheme", FORMS[:6])
def test_kv_scales_of_every_size(qat, form, scheme):
    """Scales, zero points and codes are the rounded quotients bit for bit from subnormal
    rows to those near overflow (the division by a constant takes its reciprocal and two
    remainders only where nothing of them is lost)."""
    n, d = 1 << 16, 8
    g = torch.Generator().manual_seed(9)
    x = torch.randn(n, 1, d, generator=g) * 2.0 ** (torch.rand(n, 1, 1, generator=g) * 266 - 142)
    x[:4096] = x[:4096].to(BF16).float()
    cache = qat.kv_cache(n // 64, 1, 64, d, form, scheme)
    qat.kv_write(cache, x.cuda(), x.flip(0).cuda(), torch.arange(n).cuda())
    for name, y in (("k", x), ("v", x.flip(0))):
        q, scale, zp = ref.quantized(f64(y)[:, 0], form, scheme)
        np.testing.assert_array_equal(f64(getattr(cache, name + "_scale")).reshape(-1), scale)
        np.testing.assert_array_equal(ref.codes_of(cache, name).reshape(n, d), q)
        if scheme == "affine":
            np.testing.assert_array_equal(f64(getattr(cache, name + "_zero_point")).reshape(-1), zp)


@pytest.mark.parametrize("form,scheme", FORMS[:4])
def test_kv_rows_are_the_fake_quant_view(qat, form, scheme):
    """A cached row reads back as the per-row fake-quant view of the same row."""
    cache = qat.kv_cache(4, 2, 16, 128, form, scheme)
    k, v = randn(0, 64, 2, 128, dtype=BF16), randn(1, 64, 2, 128, dtype=BF16)
    slots = torch.randperm(64, generator=torch.Generator().manual_seed(0)).cuda()
    qat.kv_write(cache, k, v, slots)
    r = qat.kv_read(cache, slots)
    for got, x in ((r.k, k), (r.v, v)):
        view = qat.fake_quant_int(x.reshape(-1, 128), 8 if form == "int8" else 4, scheme, "row").y
        assert torch.equal(got.view(-1, 128), view)


def test_kv_calls_of_nothing(qat):
    cache = qat.kv_cache(2, 2, 16, 64, "int8")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    qat.kv_write(cache, randn(0, 0, 2, 64), randn(0, 0, 2, 64), none)
    assert not cache.k.any()
    assert qat.kv_read(cache, none).k.shape == (0, 2, 64)
    empty = qat.kv_cache(0, 2, 16, 64, "int4")
    slots = torch.arange(3).cuda()
    qat.kv_write(empty, randn(0, 3, 2, 64), randn(0, 3, 2, 64), slots)
    r = qat.kv_read(empty, slots.view(3, 1), F32)
    assert r.k.shape == (3, 1, 2, 64) and not r.k.any() and not r.v.any()
    y = qat.kv_attention(randn(0, 2, 2, 64), empty, torch.zeros(2, 1, dtype=torch.int32, device="cuda"),
                         torch.tensor([0, 1], dtype=torch.int32, device="cuda"), want_lse=True)
    assert not y.y[0].any() and torch.isnan(y.y[1]).all() and torch.isnan(y.lse[1]).all()
    y = qat.kv_attention(randn(0, 2, 2, 64), cache, torch.zeros(2, 0, dtype=torch.int32, device="cuda"),
                         torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    assert not y.y[0].any() and torch.isnan(y.y[1]).all()
    assert qat.kv_attention(randn(0, 0, 2, 64), cache, torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                            torch.zeros(0, dtype=torch.int32, device="cuda")).y.shape == (0, 2, 64)


# --- attention ----------------------------------------------------------------------
def filled(qat, seed, lengths, kv_heads, d, page, form, scheme, spare=3, poison=True):
    """A cache that holds the sequences on scattered pages, and their table.  What no
    sequence owns - spare pages, the rest of last pages - holds NaN scales (NaN
    values in bf16), and the table's unused entries pages that do not exist."""
    need = [-(-max(0, n) // page) for n in lengths]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lengths), max(1, max(need)) + 1), -1, dtype=torch.int32)
    table[:, 1::2] = 1 << 30
    cache = qat.kv_cache(pages, kv_heads, page, d, form, scheme)
    if poison:
        for t in (cache.k, cache.v) if form == "bf16" else (cache.k_scale, cache.v_scale):
            t.fill_(float("nan"))
        if form != "bf16":
            cache.k.fill_(0x7f), cache.v.fill_(0x7f)
    at = 0
    for b, n in enumerate(lengths):
        table[b, :need[b]] = order[at:at + need[b]].int()
        at += need[b]
        if n > 0:
            t = torch.arange(n)
            slots = table[b].long()[t // page] * page + t % page
            k = randn(seed + 7 * b, n, kv_heads, d, dtype=BF16) * 1.5
            k[:, :, ::17] *= 3
            qat.kv_write(cache, k, randn(seed + 7 * b + 1, n, kv_heads, d, dtype=BF16) + 0.25, slots.cuda())
    return cache, table


def check_attention(qat, seed, lengths, heads, kv_heads, d, page, form, scheme, dtype, scale=None, q=None):
    cache, table = filled(qat, seed, lengths, kv_heads, d, page, form, scheme)
    q = randn(seed + 1000, len(lengths), heads, d, dtype=dtype) if q is None else q
    r = qat.kv_attention(q, cache, table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), scale, want_lse=True)
    y, ey, lse, el = ref.attention(f64(q), cache, table.numpy(), lengths, d ** -0.5 if scale is None else scale, dtype)
    assert r.y.dtype == dtype and r.lse.dtype == F32
    empty = np.array([n <= 0 for n in lengths])
    assert not r.y.cpu()[empty].any() and (r.lse.cpu()[empty] == -math.inf).all()
    full = ~empty
    within(r.y.cpu()[full], y[full], ey[full], "y")
    within(r.lse.cpu()[full], lse[full], el[full], "lse")
    return cache, table, q, r


@pytest.mark.parametrize("form,scheme", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_kv_attention_formats(qat, form, scheme, dtype):
    check_attention(qat, 3, [1, 0, 15, 16, 17, 100, 257, 513], 8, 2, 128, 16, form, scheme, dtype)


@pytest.mark.parametrize("d,page", [(8, 16), (40, 16), (64, 48), (72, 32), (80, 16), (96, 64), (120, 16), (192, 128),
                                    (200, 16), (256, 64)])
@pytest.mark.parametrize("form,scheme", [("int8", "symmetric"), ("int4", "affine"), ("bf16", "symmetric")])
def test_kv_attention_head_dims(qat, d, page, form, scheme):
    check_attention(qat, d, [33, 1, 150], 4, 2, d, page, form, scheme, BF16)
    check_attention(qat, d, [70, 31], 3, 1, d, page, form, scheme, F32)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (6, 2), (5, 1), (7, 1), (9, 1), (16, 1), (17, 1), (24, 3),
                                            (40, 1), (64, 2)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_kv_attention_head_groups(qat, heads, kv_heads, dtype):
    check_attention(qat, heads, [45, 200, 3], heads, kv_heads, 64, 16, "int8", "affine", dtype)


@pytest.mark.parametrize("lengths", [[5000], [1] * 300, [0] * 5, [0, 0, 4097, 0], [4000, 1, 1, 1, 4000, 17, 0],
                                     [16 * i for i in range(20)], [-5, 20], [2047, 2048, 2049, 64, 63, 65]])
def test_kv_attention_lengths(qat, lengths):
    """Long, short, empty and mixed sequences: every way a batch is cut into pieces."""
    check_attention(qat, 11, lengths, 4, 2, 64, 64, "int8", "symmetric", BF16)


@pytest.mark.parametrize("heads,kv_heads,d,form,scheme", [(16, 1, 128, "int4", "affine"), (12, 1, 96, "e4m3", "symmetric"),
                                                          (11, 1, 128, "bf16", "symmetric"), (20, 2, 40, "int8", "affine")])
def test_kv_attention_wide_groups(qat, heads, kv_heads, d, form, scheme):
    check_attention(qat, 21, [90, 0, 333, 16], heads, kv_heads, d, 32, form, scheme, BF16)


@pytest.mark.parametrize("form,scheme", FORMS[:6])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_kv_attention_of_values_far_apart(qat, form, scheme, dtype, order):
    """Values whose scales differ by 2^60, growing, falling and mixed; tiny ones, and rows of
    zeros."""
    n, d = 400, 64
    cache = qat.kv_cache(30, 2, 16, d, form, scheme)
    table = torch.randperm(30, generator=torch.Generator().manual_seed(0)).int()[:25].view(1, 25)
    e = torch.linspace(-30, 30, n)
    e = {"up": e, "down": e.flip(0), "mixed": e[torch.randperm(n, generator=torch.Generator().manual_seed(1))]}[order]
    k, v = randn(1, n, 2, d), randn(2, n, 2, d) * (2.0 ** e).cuda()[:, None, None]
    v[50:60] = 0
    v[70] = 1e-40
    v[:, 1] *= 2.0 ** -90
    t = torch.arange(n)
    slots = table[0].long()[t // 16] * 16 + t % 16
    qat.kv_write(cache, k, v, slots.cuda())
    q = randn(3, 1, 4, d, dtype=dtype)
    r = qat.kv_attention(q, cache, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    y, ey, _, _ = ref.attention(f64(q), cache, table.numpy(), [n], d ** -0.5, dtype)
    within(r.y, y, ey, "y")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", ["int8", "bf16"])
def test_kv_attention_of_large_and_small_queries(qat, form, dtype):
    """Query heads of very different sizes share a read of the cache."""
    q = randn(4, 2, 4, 64, dtype=dtype)
    q = q * torch.tensor([1e-30, 1.0, 1e-4, 30.0]).cuda().to(dtype)[None, :, None]
    q[1, 0] = 0
    check_attention(qat, 4, [100, 33], 4, 1, 64, 16, form, "symmetric", dtype, None, q)


def test_kv_attention_of_many_sequences(qat):
    """More sequences than a block has threads, some empty: each as in a small batch."""
    g = torch.Generator().manual_seed(5)
    lengths = torch.randint(0, 70, (1100,), generator=g).tolist()
    lengths[500], lengths[1099] = 3000, 0
    cache, table = filled(qat, 31, lengths, 2, 64, 16, "int8", "symmetric")
    q, n = randn(7, 1100, 4, 64, dtype=BF16), torch.tensor(lengths, dtype=torch.int32)
    r = qat.kv_attention(q, cache, table.cuda(), n.cuda(), want_lse=True)
    for part in (slice(0, 8), slice(496, 504), slice(1092, 1100)):
        y, ey, lse, el = ref.attention(f64(q[part]), cache, table[part].numpy(), lengths[part], 0.125, BF16)
        within(r.y[part], y, ey, "y")
        full = np.isfinite(lse)
        within(r.lse[part].cpu()[full], lse[full], el[full], "lse")
    empty = [i for i, x in enumerate(lengths) if x == 0]
    assert not r.y[empty].any() and torch.isinf(r.lse[empty]).all()
    assert torch.isfinite(r.y).all()


@pytest.mark.parametrize("form,pages,d", [("bf16", 70000, 256), ("int8", 140000, 256)])
def test_cache_offsets_past_32_bits(qat, form, pages, d):
    """Slots whose rows lie more than 2^32 bytes into the cache: what a small cache gives."""
    heads, page, n = 8, 16, 200
    k, v, q = (randn(i, n, heads, d, dtype=BF16) for i in range(3))
    q = q[:1].repeat(1, 2, 1)[:, :2 * heads].contiguous()
    lengths = torch.tensor([n], dtype=torch.int32).cuda()
    t = torch.arange(n)
    out = []
    for total, first in ((16, 0), (pages, pages - 13)):
        cache = qat.kv_cache(total, heads, page, d, form)
        table = torch.arange(first, first + 13, dtype=torch.int32).flip(0).view(1, 13)
        slots = (table[0].long()[t // page] * page + t % page).cuda()
        qat.kv_write(cache, k, v, slots)
        r = qat.kv_read(cache, slots)
        out.append((r.k, r.v, qat.kv_attention(q, cache, table.cuda(), lengths).y))
        assert cache.k.numel() * cache.k.element_size() > 1 << 32 or total == 16
        del cache
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_kv_attention_on_two_streams_at_once(qat):
    """Calls that overlap on the GPU have workspaces of their own."""
    lengths = [3000, 1, 2500]
    cache, table, q, r = check_attention(qat, 12, lengths, 8, 2, 128, 16, "int8", "symmetric", BF16)
    n, tab = torch.tensor(lengths, dtype=torch.int32).cuda(), table.cuda()
    q2 = (q.float() * -0.5).to(BF16)
    r2 = qat.kv_attention(q2, cache, tab, n).y
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    out = []
    for _ in range(20):
        for s, x in zip(streams, (q, q2)):
            with torch.cuda.stream(s):
                out.append(qat.kv_attention(x, cache, tab, n).y)
    torch.cuda.synchronize()
    for i, y in enumerate(out):
        assert torch.equal(y, r2 if i % 2 else r.y)


def test_kv_write_of_a_slot_twice_spares_the_others(qat):
    cache = qat.kv_cache(4, 2, 16, 64, "int8")
    k, v = randn(0, 40, 2, 64), randn(1, 40, 2, 64)
    slots = torch.arange(40).cuda()
    qat.kv_write(cache, k, v, slots)
    want = qat.kv_read(cache, slots, F32)
    slots[7] = 8
    qat.kv_write(cache, k, v, slots)
    got = qat.kv_read(cache, torch.arange(40).cuda(), F32)
    keep = [i for i in range(40) if i not in (7, 8)]
    assert torch.equal(got.k[keep], want.k[keep]) and torch.equal(got.v[keep], want.v[keep])
    assert torch.equal(got.k[7], want.k[7])  # (as the first call left it)


def test_kv_attention_sharp_and_flat_scores(qat):
    """Scores far apart (one weight takes all), equal scores, a negative scale, scale 0."""
    lengths = [300, 40]
    q = randn(5, 2, 4, 128, dtype=BF16)
    for scale in (0.0, -0.2, 3.0):
        check_attention(qat, 5, lengths, 4, 2, 128, 16, "e4m3", "symmetric", BF16, scale, q)
    check_attention(qat, 5, lengths, 4, 2, 128, 16, "int8", "symmetric", F32, 1.0, q.float() * 30)


def test_kv_attention_refused_sequences_stay_alone(qat):
    """Pages outside the cache and lengths that the table cannot hold make NaN of their
    own sequence only."""
    lengths = [40, 90, 50, 64]
    cache, table, q, good = check_attention(qat, 2, lengths, 4, 2, 64, 16, "int8", "symmetric", BF16)
    for bad in (-1, cache.pages, -(1 << 31), (1 << 31) - 1):
        t = table.clone()
        t[1, 3] = bad
        r = qat.kv_attention(q, cache, t.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), want_lse=True)
        assert torch.isnan(r.y[1]).all() and torch.isnan(r.lse[1]).all()
        for b in (0, 2, 3):
            assert torch.equal(r.y[b], good.y[b]) and torch.equal(r.lse[b], good.lse[b])
    far = list(lengths)
    for n in (table.shape[1] * 16 + 1, (1 << 31) - 1):
        far[2] = n
        r = qat.kv_attention(q, cache, table.cuda(), torch.tensor(far, dtype=torch.int32).cuda(), want_lse=True)
        assert torch.isnan(r.y[2]).all() and torch.isnan(r.lse[2]).all()
        for b in (0, 1, 3):
            assert not torch.isnan(r.y[b]).any()


@pytest.mark.parametrize("form", ["int8", "bf16"])
def test_kv_attention_nonfinite_rows(qat, form):
    """A NaN key or value inside the length reaches its own sequence and key head only."""
    lengths = [100, 100]
    for name in ("k", "v"):
        cache, table = filled(qat, 4, lengths, 2, 64, 16, form, "symmetric")
        q = randn(9, 2, 4, 64, dtype=BF16)
        n = torch.tensor(lengths, dtype=torch.int32).cuda()
        clean = qat.kv_attention(q, cache, table.cuda(), n).y
        x = getattr(cache, name if form == "bf16" else name + "_scale")
        x[int(table[1, 2]), 1, 5] = float("nan")
        y = qat.kv_attention(q, cache, table.cuda(), n).y
        assert torch.isnan(y[1, 2:]).all()
        y[1, 2:] = clean[1, 2:]
        assert torch.equal(y, clean)


def test_kv_attention_views_and_repeats(qat):
    """Strided queries and tables give the same bits; so does every call."""
    lengths = [700, 20, 333]
    cache, table, q, r = check_attention(qat, 6, lengths, 8, 2, 128, 16, "int4", "affine", BF16)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    row = torch.zeros(3, 12 * 128 + 1, dtype=BF16, device="cuda")
    row[:, 1:8 * 128 + 1] = q.reshape(3, -1)
    wide = torch.full((3, 2 * table.shape[1]), -9, dtype=torch.int32).cuda()
    wide[:, :table.shape[1]] = table.cuda()
    for view in (q, row[:, 1:8 * 128 + 1].view(3, 8, 128), q.transpose(0, 1).contiguous().transpose(0, 1)):
        for tab in (table.cuda(), wide[:, :table.shape[1]], table.t().contiguous().cuda().t()):
            got = qat.kv_attention(view, cache, tab, n, want_lse=True)
            assert torch.equal(got.y, r.y) and torch.equal(got.lse, r.lse)


def test_kv_attention_shared_pages(qat):
    """Sequences may share pages (a common prefix)."""
    cache, table, q, r = check_attention(qat, 8, [64, 64], 4, 2, 64, 16, "int8", "symmetric", BF16)
    table[1] = table[0]
    n = torch.tensor([64, 50], dtype=torch.int32)
    got = qat.kv_attention(q, cache, table.cuda(), n.cuda())
    y, ey, _, _ = ref.attention(f64(q), cache, table.numpy(), n.tolist(), 64 ** -0.5, BF16)
    within(got.y, y, ey, "y")


# --- as they are used -----------------------------------------------------------------
def test_decoding_steps_in_a_graph(qat):
    """A step of the attention half - rotate, write, attend - captured once and
    replayed on two streams' worth of inputs: each replay gives what direct calls
    give, and the workspaces of two graphs do not meet."""
    batch, hq, hk, d, page = 3, 8, 2, 64, 16
    turns = qat.rope_turns(qat.rope_frequencies(d), "cuda")
    wq, wk = (1 + randn(i, d, scale=0.1) for i in range(2))
    wq, wk = wq.to(BF16), wk.to(BF16)
    start = [37, 0, 130]

    class Program:
        def __init__(self, seed):
            self.cache, table = filled(qat, seed, [n + 4 * page for n in start], hk, d, page, "int8", "symmetric",
                                       poison=False)
            self.table = table.cuda()
            self.qkv = torch.zeros(batch, (hq + 2 * hk) * d, dtype=BF16, device="cuda")
            self.positions = torch.tensor(start).cuda()

        def step(self):
            q = self.qkv[:, :hq * d].view(batch, hq, d)
            k = self.qkv[:, hq * d:(hq + hk) * d].view(batch, hk, d)
            v = self.qkv[:, (hq + hk) * d:].view(batch, hk, d)
            r = qat.head_norm_rope(q, k, self.positions, turns, wq, wk)
            pages = self.table.long().gather(1, (self.positions // page)[:, None])[:, 0]
            qat.kv_write(self.cache, r.k, v, pages * page + self.positions % page)
            y = qat.kv_attention(r.q, self.cache, self.table, (self.positions + 1).int()).y
            self.positions += 1
            return y

    graphs, direct = [], []
    for seed in (1, 2):
        p = Program(seed)
        p.step()  # warm-up
        p.positions -= 1
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                y = p.step()
        graphs.append((p, g, y))
        direct.append(Program(seed))
    torch.cuda.synchronize()
    for t in range(4):
        for i, (p, g, y) in enumerate(graphs):
            x = randn(100 + 10 * t + i, batch, (hq + 2 * hk) * d, dtype=BF16)
            p.qkv.copy_(x)
            g.replay()
            direct[i].qkv.copy_(x)
            want = direct[i].step()
            assert torch.equal(y, want)
    for i, (p, _, _) in enumerate(graphs):
        assert torch.equal(p.cache.k, direct[i].cache.k) and torch.equal(p.cache.v_scale, direct[i].cache.v_scale)


def test_calls_on_another_stream(qat):
    """Each call runs on the current stream, in order with what the stream holds."""
    lengths = [500, 20]
    cache, table, q, r = check_attention(qat, 6, lengths, 4, 2, 64, 16, "int8", "symmetric", BF16)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    tab, late = table.cuda(), torch.zeros_like(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
        y = qat.kv_attention(late, cache, tab, n).y
    s.synchronize()
    assert torch.equal(y, r.y)


def test_captured_backward(qat):
    """A backward pass captured into a graph gives the direct call's gradients."""
    turns, positions = qat.rope_turns(qat.rope_frequencies(64), "cuda"), torch.arange(40).cuda()
    w = (1 + randn(2, 64, scale=0.1)).requires_grad_()
    q = randn(0, 40, 4, 64).requires_grad_()
    c = randn(1, 40, 4, 64)

    def step():
        y, _ = qat.HeadNormRopeFunction.apply(q, None, positions, turns, w)
        return torch.autograd.grad((y * c).sum(), (q, w))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = step()
    torch.cuda.current_stream().wait_stream(s)
    with torch.no_grad():
        q.copy_(randn(7, 40, 4, 64))
        w.mul_(1.5)
    g.replay()
    torch.cuda.synchronize()
    dq, _, dw, _ = qat.head_norm_rope_backward(c, None, q.detach(), None, positions, turns, w.detach())
    assert torch.equal(got[0], dq) and torch.equal(got[1], dw)


def test_example_serves_from_every_cache(qat):
    """The example's layer runs, and its outputs are numbers of the layer's shape."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "qat_attention_layer.py")
    spec = importlib.util.spec_from_file_location("qat_attention_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    want, off = example.main(steps=20, dim=256)
    assert want.shape == (20, 3, 256) and torch.isfinite(want).all()
    assert set(off) == {"int8", "e4m3", "int4"} and all(math.isfinite(v) for v in off.values())
