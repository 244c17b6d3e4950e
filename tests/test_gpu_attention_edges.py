"""Attention operators on the GPU where a plain call does not lead.  Bounds are those of
attention_reference.py unless a test derives its own."""
import math

import numpy as np
import pytest
import torch

import attention_reference as ref
from layer_reference import U, f64, within

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def randn(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


# --- norms without an epsilon ------------------------------------------------------
@pytest.mark.parametrize("tokens,hq,hk,d,layout,dtype", [
    (1, 1, 1, 128, "half", BF16),            # groups without a head
    (5, 5, 2, 64, "half", BF16),
    (37, 3, 0, 80, "interleaved", F32),
    (2000, 9, 3, 128, "half", BF16),         # two heads a group, an odd number of both
    (700, 31, 9, 128, "interleaved", F32),
    (1300, 31, 9, 128, "half", BF16),        # four a group
])
def test_head_norm_rope_backward_without_epsilon(qat, tokens, hq, hk, d, layout, dtype):
    """eps = 0 and heads that are not zero: no head is missing a norm, so every gradient is
    the formula's.  (Steps of a group that has no head see zeros, whose norm is 0 / 0.)"""
    q, k = randn(0, tokens, hq, d, dtype=dtype), randn(1, tokens, hk, d, dtype=dtype) if hk else None
    wq, wk = (1 + randn(2 + i, d, scale=0.3) for i in range(2))
    wq, wk = wq.to(dtype), wk.to(dtype) if hk else None
    gq, gk = randn(4, tokens, hq, d, dtype=dtype), randn(5, tokens, hk, d, dtype=dtype) if hk else None
    positions, turns = torch.arange(tokens).cuda(), qat.rope_turns(qat.rope_frequencies(d), "cuda")
    dq, dk, dwq, dwk = qat.head_norm_rope_backward(gq, gk, q, k, positions, turns, wq, wk, 0.0, True, layout)
    c, s = ref.angles(positions.tolist(), turns.tolist(), 1.0)
    for x, w, g, dx, dw in ((q, wq, gq, dq, dwq), (k, wk, gk, dk, dwk)):
        if x is None:
            continue
        want = ref.rope(f64(x), f64(w), f64(g), c, s, layout, 0.0, True, 1.0, dtype)
        within(dx, *want["dx"], "dx")
        within(dw, *want["dw"], "dw")


# --- several heads a group -----------------------------------------------------------
# Once the heads fill the GPU twice, a group takes 2, 4 or 8 of a token's (the launchers'
# rule: forward from 2 sms 2048 / lanes heads, backward from 2 * 304 * 256 / lanes), the
# last group of the queries, and of the keys, what is left of them.
WALKS = [
    # tokens, query heads, key heads, head_dim, rotary, layout, norm, type; heads a group on 152 SMs
    (600, 31, 9, 128, 128, "half", True, BF16),           # 1, backward 2
    (1100, 31, 9, 128, 64, "half", True, BF16),           # 1, 4
    (2100, 31, 9, 128, 128, "interleaved", True, BF16),   # 2, 8
    (4100, 31, 9, 128, 128, "half", True, BF16),          # 4, 8
    (8200, 31, 9, 128, 128, "interleaved", False, BF16),  # 8, 8
    (8200, 9, 3, 128, 128, "half", True, F32),            # 2, 8
    (8200, 21, 0, 128, 32, "interleaved", True, F32),     # 4, 8 (no keys)
    (8100, 7, 3, 40, 10, "half", True, F32),              # 8, 8 (single elements)
    (8100, 7, 7, 80, 20, "interleaved", True, BF16),      # 8, 8 (runs of two)
    (13000, 9, 3, 72, 72, "half", True, BF16),            # 8, 8 (runs of four)
]


@pytest.mark.parametrize("case", WALKS, ids=lambda c: "-".join(map(str, c[:6])))
def test_head_norm_rope_several_heads_a_group(qat, case):
    """A large call gives each token what a call of few tokens gives it, which is the
    formula's; weight gradients are the formula's sums."""
    t, hq, hk, d, rot, layout, norm, dtype = case
    row = randn(0, t, (hq + 2 * hk) * d + 8, dtype=dtype)  # (queries, keys and values side by side)
    q = row[:, :hq * d].view(t, hq, d)
    k = row[:, hq * d:(hq + hk) * d].view(t, hk, d) if hk else None
    gq, gk = randn(1, t, hq, d, dtype=dtype), randn(2, t, hk, d, dtype=dtype) if hk else None
    wq = wk = None
    if norm:
        wq, wk = ((1 + randn(3 + i, d, scale=0.3)).to(dtype) for i in range(2))
        wk = wk if hk else None
    positions, turns = torch.arange(900, 900 + t).cuda(), qat.rope_turns(qat.rope_frequencies(rot), "cuda")
    kw = dict(eps=1e-5, norm=norm, layout=layout, amplitude=1.25)
    y = qat.head_norm_rope(q, k, positions, turns, wq, wk, **kw)
    dq, dk, dwq, dwk = qat.head_norm_rope_backward(gq, gk, q, k, positions, turns, wq, wk, **kw)

    def few(x, a):
        return None if x is None else x[a:a + 64]

    for a in range(0, t, 64):
        args = few(q, a), few(k, a), positions[a:a + 64], turns, wq, wk
        y1 = qat.head_norm_rope(*args, **kw)
        g1 = qat.head_norm_rope_backward(few(gq, a), few(gk, a), *args, **kw)
        for got, want in ((y.q, y1.q), (y.k, y1.k), (dq, g1[0]), (dk, g1[1])):
            assert got is None and want is None or torch.equal(got[a:a + 64], want)
    some = torch.tensor([0, 1, t // 2, t - 2, t - 1])
    c, s = ref.angles(positions[some].tolist(), turns.tolist(), 1.25)
    for x, w, g, got, dx in ((q, wq, gq, y.q, dq), (k, wk, gk, y.k, dk)):
        if x is not None:
            want = ref.rope(f64(x[some]), None if w is None else f64(w), f64(g[some]), c, s, layout, 1e-5, norm, 1.25,
                            dtype)
            within(got[some], *want["y"], "y")
            within(dx[some], *want["dx"], "dx")
    # dw = sum g' z in 64 bits (the angle's integer product wraps as the definition does)
    a = (positions[:, None] * turns[None]).double() * (2 * math.pi * 2.0 ** -64)
    c, s = a.cos()[:, None] * 1.25, a.sin()[:, None] * 1.25
    i = torch.arange(rot // 2).cuda()
    at, bt = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    for x, w, g, dw in ((q, wq, gq, dwq), (k, wk, gk, dwk)):
        if w is None:
            assert dw is None
            continue
        x, g = x.double(), g.double()
        z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)
        gb, both = g.clone(), g.abs()
        gb[..., at], gb[..., bt] = g[..., at] * c + g[..., bt] * s, g[..., bt] * c - g[..., at] * s
        both[..., at] = both[..., bt] = g[..., at].abs() + g[..., bt].abs()
        # ref.rope's bound: the sum, z's norm, and the turned gradient's angle
        rel = (8 * math.sqrt(d) + 6) * U
        err = (8 * math.sqrt(x.shape[0] * x.shape[1] + 16) * U + rel + 4 * U) * (gb * z).abs().sum((0, 1)) \
            + (6 * 1.25 + 4 * 1.25) * U * (both * z.abs()).sum((0, 1))
        want = (gb * z).sum((0, 1))
        within(dw, f64(want), f64(err + ref.step(dtype) * (want.abs() + err)), "dw")


# --- infinities in a bf16 cache --------------------------------------------------------
def bf16_sequences(qat, seed, lengths, kv_heads, d, page):
    """A bf16 cache that holds the sequences on scattered pages, and their table."""
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(lengths), max(need)), -1, dtype=torch.int32)
    cache, at = qat.kv_cache(sum(need), kv_heads, page, d, "bf16"), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache.k.copy_(randn(seed, *cache.k.shape, dtype=BF16))
    cache.v.copy_(randn(seed + 1, *cache.v.shape, dtype=BF16))
    return cache, table


def queries(kind, seed, *shape):
    """bf16 queries; fp32 ones of 24 bits, and of the 8 or 16 that one or two bf16 parts hold."""
    q = randn(seed, *shape)
    if kind == "bf16":
        return q.to(BF16)
    if kind == "fp32 of 8 bits":
        return q.to(BF16).float()
    return (q.to(BF16).float() * 1.0078125).contiguous() if kind == "fp32 of 16 bits" else q


KINDS = ["bf16", "fp32", "fp32 of 8 bits", "fp32 of 16 bits"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 72, 256])
def test_kv_attention_infinite_values(qat, kind, d):
    """An infinite value makes its element of its key head's outputs infinite, two of both
    signs NaN; the other elements keep their bits."""
    lengths, page = [1, 40, 300, 6000], 16
    cache, table = bf16_sequences(qat, 3, lengths, 2, d, page)
    q, n, tab = queries(kind, 9, 4, 4, d), torch.tensor(lengths, dtype=torch.int32).cuda(), table.cuda()
    want = qat.kv_attention(q, cache, tab, n).y.clone()
    inf = float("inf")
    # sequence, position, element, value
    for b, t, e, x in ((0, 0, 3, inf), (0, 0, 5, -inf), (1, 39, 0, inf), (1, 7, d - 1, -inf), (2, 0, 8, inf),
                       (2, 299, 9, -inf), (3, 3000, 17, inf), (3, 3001, 17, inf), (3, 5999, 40, -inf)):
        cache.v[int(table[b, t // page]), 1, t % page, e] = x
        want[b, 2:, e] = x
    for b, t, u, e in ((1, 3, 20, 11), (2, 10, 11, 12), (3, 1, 5000, 13)):
        cache.v[int(table[b, t // page]), 1, t % page, e] = inf
        cache.v[int(table[b, u // page]), 1, u % page, e] = -inf
        want[b, 2:, e] = float("nan")
    got = qat.kv_attention(q, cache, tab, n).y
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, 0.0, inf, -inf), torch.nan_to_num(want, 0.0, inf, -inf))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 72, 256])
def test_kv_attention_infinite_keys(qat, kind, d):
    """A key whose score is -inf has weight 0: the outputs are those of the sequence without
    it.  One whose score is inf makes NaN, as inf - inf does."""
    lengths, page, e = [2, 40, 300, 6000], 16, 5
    dtype = BF16 if kind == "bf16" else F32
    cache, table = bf16_sequences(qat, 5, lengths, 2, d, page)
    q, tab = queries(kind, 9, 4, 4, d), table.cuda()
    q[:, 0, e], q[:, 1, e], q[:, 2, e], q[:, 3, e] = 1.5, -1.5, q[:, 2, e].abs() + q[0, 0, 0].abs(), -2.0
    if kind == "fp32 of 8 bits":
        q = q.to(BF16).float()
    without = qat.kv_cache(cache.pages, 2, page, d, "bf16")
    without.k.copy_(cache.k), without.v.copy_(cache.v)
    for b, t, x in ((0, 0, math.inf), (1, 39, -math.inf), (2, 0, math.inf), (3, 4000, -math.inf)):
        n = lengths[b]
        # heads 0, 1 read key head 0, which keeps its keys
        cache.k[int(table[b, t // page]), 1, t % page, e] = x
        for c in (without.k, without.v):  # the last position takes the place of position t
            last = c[int(table[b, (n - 1) // page]), :, (n - 1) % page].clone()
            c[int(table[b, t // page]), :, t % page] = last
    n = torch.tensor(lengths, dtype=torch.int32)
    r = qat.kv_attention(q, cache, tab, n.cuda(), want_lse=True)
    y, ey, lse, el = ref.attention(f64(q), without, table.numpy(), (n - 1).tolist(), d ** -0.5, dtype)
    for b, up in ((0, True), (1, False), (2, True), (3, False)):
        good, bad = (3, 2) if up else (2, 3)  # (q's sign times the infinity's)
        within(r.y[b, good], y[b, good], ey[b, good], "y")
        within(r.lse[b, good], lse[b, good], el[b, good], "lse")
        assert torch.isnan(r.y[b, bad]).all() and not torch.isnan(r.y[b, :2]).any()
    # nothing but such keys
    cache.k[int(table[0, 0]), 1, :2, e] = math.inf
    r = qat.kv_attention(q, cache, tab, n.cuda(), want_lse=True)
    assert not r.y[0, 3].any() and r.lse[0, 3] == -math.inf


def test_kv_attention_weights_of_bf16_rows(qat):
    """Weighted values that cancel to 2^-16 of their size show a weight's last bits under a
    bf16 output too.  Queries of one element make scores exact products: a weight is off by
    the rounding of score * log2 e (3 U of up to 2) and of the hardware exponential (2^-22),
    its sum by 3 U; the nine products of a sum by 2 U each.  That is below 40 U of the
    values' size; weights of 16 bits were off by up to 2^-17 of it."""
    batch, heads, d, page = 32, 3, 64, 16
    cache = qat.kv_cache(batch, heads, page, d, "bf16")
    g = torch.Generator().manual_seed(7)
    q = torch.zeros(batch, heads, d)
    q[..., 9] = 1.0
    k0 = (torch.rand(batch, heads, 3, generator=g) * 2 - 1).to(BF16).double()
    w = torch.softmax(k0, -1)[..., None]
    v = torch.zeros(batch, heads, 3, d, dtype=torch.float64)
    v[:, :, 0] = (1 + torch.rand(batch, heads, d, generator=g)).to(BF16).double()
    v[:, :, 1] = (-v[:, :, 0] * w[:, :, 0] / w[:, :, 1]).to(BF16).double()
    v[:, :, 2] = (-(v[:, :, :2] * w[:, :, :2]).sum(2) / w[:, :, 2]).to(BF16).double()
    want, size = (v * w).sum(2), (v.abs() * w).sum(2)
    cache.k[:, :, :3, 9] = k0.to(BF16).cuda()
    cache.v[:, :, :3] = v.to(BF16).cuda()
    table = torch.arange(batch, dtype=torch.int32).view(batch, 1).cuda()
    n = torch.full((batch,), 3, dtype=torch.int32).cuda()
    for dtype in (BF16, F32):
        y = qat.kv_attention(q.to(dtype).cuda(), cache, table, n, 1.0).y
        within(y, f64(want), f64(40 * U * size + ref.step(dtype) * (want.abs() + 40 * U * size)), "y")


# --- long runs -------------------------------------------------------------------------
@pytest.mark.parametrize("form", ["int8", "int4", "e4m3", "bf16"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_kv_attention_sums_of_long_runs(qat, form, dtype):
    """More sequences of 2^20 positions than warps, so that one warp adds up tens of thousands
    of tiles.  Values are positive: each of N = n / 16 additions rounds by at most U of the
    sum so far, of either sign, U sqrt(N) / 3 in all and 8 sqrt(N) U far above it.  (The
    sequences share their pages.  Queries of one element make scores exact: 10 U a weight.)"""
    n, d, page, batch = 1 << 20, 64, 1 << 13, 2000
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = qat.kv_cache(n // page, 1, page, d, form)
    k = torch.rand(n, 1, d, generator=g, device="cuda") * 2 - 1
    v = torch.rand(n, 1, d, generator=g, device="cuda") + 0.5
    slots = torch.arange(n, device="cuda")
    qat.kv_write(cache, k, v, slots)
    r = qat.kv_read(cache, slots, F32)
    q = torch.zeros(1, 1, d, device="cuda")
    q[..., 9] = 2.0
    s = r.k[:, 0].double() @ q[0, 0].double()
    want, lse = torch.softmax(s, 0) @ r.v[:, 0].double(), torch.logsumexp(s, 0)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").view(1, -1).expand(batch, -1)
    got = qat.kv_attention(q.to(dtype).expand(batch, 1, d), cache, table,
                           torch.full((batch,), n, dtype=torch.int32, device="cuda"), 1.0, want_lse=True)
    err = (8 * math.sqrt(n / 16) + 40) * U * want.abs()
    for i in (0, 1, 777, batch - 1):
        within(got.y[i, 0], f64(want), f64(err + ref.step(dtype) * (want.abs() + err)), "y")
        assert abs(float(got.lse[i, 0]) - float(lse)) <= (8 * math.sqrt(n / 16) + 40) * U + 4 * U * float(lse)


# --- value scales under unequal weights --------------------------------------------------
FORMS = [("int8", "symmetric"), ("int8", "affine"), ("int4", "symmetric"), ("int4", "affine"), ("e4m3", "symmetric"),
         ("e5m2", "symmetric"), ("bf16", "symmetric")]


def unequal(kind, n, g):
    """Scores [n, 2] of two heads that share a key head (nats), and exponents of the values' sizes."""
    s, e = torch.rand(n, 2, generator=g) * 6 - 3, torch.zeros(n)
    if kind.startswith("far"):    # one row, far larger than the others, that no head attends to
        _, at, e_far = kind.split()
        s[int(at) % n], e[int(at) % n] = -1000.0, float(e_far)
    elif kind == "tiny":          # all of them near the end of binary32's range
        e[:] = -112
    elif kind == "two heads":     # one head attends to small values, the other to large ones
        e[::2] = -40
        s[::2, 1] -= 200
        s[1::2, 0] -= 200
    elif kind == "fall":          # large values first, whose weights fade
        e = torch.linspace(60, -60, n)
        s = torch.linspace(-20, 20, n)[:, None].repeat(1, 2)
    elif kind == "records":       # scores that keep growing over rows of zeros
        e[16:] = -math.inf
        s = torch.linspace(0, 40, n)[:, None] * torch.tensor([1.0, 0.7])
    else:
        s, e = torch.rand(n, 2, generator=g) * 60 - 30, torch.rand(n, generator=g) * 80 - 40
    return s, e


@pytest.mark.parametrize("form,scheme", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["far 0 24", "far 200 40", "far -1 80", "far 17 -80", "two heads", "fall", "records",
                                  "random", "tiny"])
def test_kv_attention_scales_under_unequal_weights(qat, form, scheme, dtype, kind):
    """What fp16 parts of a weight times its value's scale lose is 2^-33 of the largest such
    product of the head: rows that it does not attend to, and other heads, cost it nothing.

    Each head's queries have one element, a power of two, so that products with the codes are
    exact; a score is off by 4 U of itself (its scale, log2 e and the two products).  Moving
    the maximum rounds what is summed by 6 U (exponential and product); it moves by 2^4 or for
    a product 2^6 times the largest."""
    n, d, page = 1000, 64, 16
    g = torch.Generator().manual_seed(len(kind))
    s, e = unequal(kind, n, g)
    cache = qat.kv_cache(-(-n // page), 1, page, d, form, scheme)
    table = torch.randperm(cache.pages, generator=g).int().view(1, -1)
    t = torch.arange(n)
    pages = table[0].long()[t // page]
    k = torch.zeros(n, 1, d)
    k[:, 0, :2] = s / 4
    v = torch.randn(n, 1, d, generator=g) * (2.0 ** e)[:, None, None]
    qat.kv_write(cache, k.cuda(), v.cuda(), (pages * page + t % page).cuda())
    q = torch.zeros(1, 2, d)
    q[0, 0, 0] = q[0, 1, 1] = 4.0
    r = qat.kv_attention(q.to(dtype).cuda(), cache, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), 1.0,
                         want_lse=True)
    at = pages, 0, t % page
    kv, vv, codes = ref.values_of(cache, "k")[at], ref.values_of(cache, "v")[at], np.abs(ref.codes_of(cache, "v")[at])
    vs = np.zeros(n) if form == "bf16" else np.abs(f64(cache.v_scale)[at])
    zp = ref.extra_codes(cache, pages.numpy(), 0, t.numpy())[:, None]
    zv = ref.extra_values(cache, pages.numpy(), 0, t.numpy())[:, None]
    bits = 1.45 * f64(s.max(0).values - s.min(0).values).sum()  # (of both heads' scores)
    moves = 4 + bits / 4 + float(e[e > -math.inf].max() - e[e > -math.inf].min()) / 6
    for h in range(2):
        x = kv[:, h] * 4
        w = np.exp(x - x.max())
        total = w.sum()
        w /= total
        want = w @ vv
        # (the part's bits: 8 U, or 2^-22 under a bf16 output)
        rel = (8 * np.abs(x) + 8 * np.abs(x - x.max()) + 16 + 6 * moves) * U
        size = np.abs(vv) + np.abs(want) + zv
        err = (w * rel) @ size + (8 * math.sqrt(n) + 16) * U * (w @ size) + n * (2.0 ** -126 * np.abs(vv).max(0) + 2.0 ** -148)
        err = err + 2.0 ** -33 * (w * vs).max() * (codes + zp).sum(0)
        within(r.y[0, h], want, err + ref.step(dtype) * (np.abs(want) + err), "y")
        lse = x.max() + math.log(total)
        assert abs(float(r.lse[0, h]) - lse) <= (w * rel).sum() + (8 * math.sqrt(n) + 16) * U + 4 * U * abs(lse)


# --- every kernel of the attention -------------------------------------------------------
@pytest.mark.parametrize("form,scheme", [f for f in FORMS if f != ("int8", "symmetric") and f != ("int4", "symmetric")])
@pytest.mark.parametrize("d", [16, 64, 104, 128, 232, 256])
def test_kv_attention_every_kernel(qat, form, scheme, d):
    """Both output types, whole and partial head sizes, groups of one to eight and of more
    query heads, in sequences within a block and across blocks."""
    page, lengths = 32, [5, 0, 800, 33]
    g = torch.Generator().manual_seed(d)
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(need) + 1, generator=g).int()
    table, at = torch.full((4, max(need)), -1, dtype=torch.int32), 0
    cache = qat.kv_cache(sum(need) + 1, 2, page, d, form, scheme)
    for b, n in enumerate(lengths):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        if n:
            t = torch.arange(n)
            slots = table[b].long()[t // page] * page + t % page
            qat.kv_write(cache, randn(b, n, 2, d, dtype=BF16), randn(9 + b, n, 2, d, dtype=BF16), slots.cuda())
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    for dtype in (BF16, F32):
        for heads in (2, 6, 22):
            q = randn(heads, 4, heads, d, dtype=dtype)
            r = qat.kv_attention(q, cache, table.cuda(), n, want_lse=True)
            y, ey, lse, el = ref.attention(f64(q), cache, table.numpy(), lengths, d ** -0.5, dtype)
            within(r.y, y, ey, "y")
            full = [0, 2, 3]
            within(r.lse[full], lse[full], el[full], "lse")
            assert not r.y[1].any() and (r.lse[1] == -math.inf).all()


# --- the calls that mirror the C entry points ----------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_calls_with_the_users_own_buffers(qat, dtype):
    """The qat_* calls, into outputs and workspaces that the caller has, on a stream of the
    caller's: what the named functions give; the workspace that a call needs is checked."""
    t, hq, hk, d, page = 50, 6, 2, 64, 16
    row = randn(0, t, (hq + 2 * hk) * d, dtype=dtype).view(t, hq + 2 * hk, d)
    q, k, v = row[:, :hq], row[:, hq:hq + hk], row[:, hq + hk:]
    wq, wk = ((1 + randn(1 + i, d, scale=0.3)).to(dtype) for i in range(2))
    positions, turns = torch.arange(t).cuda(), qat.rope_turns(qat.rope_frequencies(32), "cuda")
    gq, gk = randn(5, t, hq, d, dtype=dtype), randn(6, t, hk, d, dtype=dtype)
    want = qat.head_norm_rope(q, k, positions, turns, wq, wk, 1e-5, True, "interleaved", 1.25)
    grads = qat.head_norm_rope_backward(gq, gk, q, k, positions, turns, wq, wk, 1e-5, True, "interleaved", 1.25)
    cache, same = (qat.kv_cache(-(-t // page), hk, page, d, "int8", "affine") for _ in range(2))
    slots = torch.arange(t).cuda()
    qat.kv_write(same, want.k, v, slots)
    rows = qat.kv_read(same, slots, dtype)
    table = torch.arange(cache.pages, dtype=torch.int32).view(1, -1).cuda().expand(3, -1).contiguous()
    n = torch.tensor([t, 7, 0], dtype=torch.int32).cuda()
    attended = qat.kv_attention(want.q[:3], same, table, n, 0.2, want_lse=True)
    torch.cuda.synchronize()

    s = torch.cuda.Stream()
    yq, yk, dq, dk = (torch.empty(t, h, d, dtype=dtype, device="cuda") for h in (hq, hk, hq, hk))
    dwq, dwk = (torch.empty(d, dtype=dtype, device="cuda") for _ in range(2))
    rk, rv = torch.empty_like(yk), torch.empty_like(yk)
    y, lse = torch.empty(3, hq, d, dtype=dtype, device="cuda"), torch.empty(3, hq, device="cuda")
    rope = t, hq, hk, d, q.stride()[:2], k.stride()[:2], positions, turns, 32, "interleaved", 1.25, True, wq, wk, 1e-5
    ws = torch.empty(qat.qat_head_norm_rope_backward_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    ws_attn = torch.empty(qat.qat_kv_attention_workspace_bytes(cache, hq), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    qat.qat_head_norm_rope(q, k, *rope, yq, yk, s)
    qat.qat_head_norm_rope_backward(gq, gk, q, k, *rope, dq, dk, dwq, dwk, ws, s)
    qat.qat_kv_write(cache, yk, v, t, yk.stride()[:2], v.stride()[:2], slots, s)
    qat.qat_kv_read(cache, slots, t, rk, rv, s)
    attn = yq, 3, hq, yq.stride()[:2], cache, table, table.shape[1], table.stride(0), n, 0.2, y, lse
    qat.qat_kv_attention(*attn, ws_attn, s)
    s.synchronize()
    for a, b in ((yq, want.q), (yk, want.k), (dq, grads[0]), (dk, grads[1]), (dwq, grads[2]), (dwk, grads[3]),
                 (cache.k, same.k), (cache.v_scale, same.v_scale), (rk, rows.k), (rv, rows.v), (y, attended.y),
                 (lse, attended.lse)):
        assert torch.equal(a, b)
    with pytest.raises(qat.QatError):
        qat.qat_kv_attention(*attn, ws_attn[:-16], s)
    with pytest.raises(qat.QatError):
        qat.qat_head_norm_rope_backward(gq, gk, q, k, *rope, dq, dk, dwq, dwk, ws[:-16], s)


# --- the largest calls -------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_kv_attention_longest_sequence(qat, dtype):
    """2^31 - 1025 positions (of pages that repeat) are the most a sequence may have: one more
    is NaN, and the sequence beside it is as alone.  A warp adds up 74 000 tiles."""
    n, d, page = (1 << 31) - 1025, 16, 1 << 20
    cache = qat.kv_cache(1, 1, page, d, "int8")
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = torch.rand(page, 1, d, generator=g, device="cuda") * 2 - 1, torch.rand(page, 1, d, generator=g, device="cuda")
    v[page - 1025:] += 3  # (what the last page's end leaves out would show)
    slots = torch.arange(page, device="cuda")
    qat.kv_write(cache, k, v, slots)
    r = qat.kv_read(cache, slots, F32)
    q = torch.zeros(3, 1, d, device="cuda")
    q[..., 9] = 2.0
    table = torch.zeros(1, 2048, dtype=torch.int32, device="cuda").expand(3, -1)
    got = qat.kv_attention(q.to(dtype), cache, table, torch.tensor([5, n, n + 1], dtype=torch.int32, device="cuda"), 1.0,
                           want_lse=True)
    times = torch.full((page,), 2048.0, device="cuda", dtype=torch.float64)
    times[n % page:] -= 1
    s = r.k[:, 0].double() @ q[0, 0].double()
    w = times * s.exp()
    for b, w in ((0, s[:5].exp()), (1, w)):
        want, lse, steps = (w @ r.v[:len(w), 0].double()) / w.sum(), float(w.sum().log()), 8 * math.sqrt(80000)
        err = (steps + 40) * U * want.abs()
        within(got.y[b, 0], f64(want), f64(err + ref.step(dtype) * (want.abs() + err)), "y")
        assert abs(float(got.lse[b, 0]) - lse) <= (steps + 40) * U + 4 * U * lse
    assert torch.isnan(got.y[2]).all() and torch.isnan(got.lse[2]).all()


def test_kv_attention_largest_batch(qat):
    """65535 sequences, every other one empty, and one more is refused."""
    batch, d = 65535, 16
    cache = qat.kv_cache(64, 2, 16, d, "bf16")
    cache.k.copy_(randn(0, *cache.k.shape, dtype=BF16)), cache.v.copy_(randn(1, *cache.v.shape, dtype=BF16))
    q = randn(2, 64, 4, d, dtype=BF16).repeat(1024, 1, 1)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(64, 1).repeat(1024, 1)
    n = (torch.arange(64, dtype=torch.int32, device="cuda") % 17).repeat(1024)
    n[1::2] = 0
    few = qat.kv_attention(q[:64], cache, table[:64], n[:64], want_lse=True)
    got = qat.kv_attention(q[:batch], cache, table[:batch], n[:batch], want_lse=True)
    want = few.y.repeat(1024, 1, 1)[:batch], few.lse.repeat(1024, 1)[:batch]
    assert torch.equal(got.y, want[0]) and torch.equal(got.lse, want[1])
    with pytest.raises(qat.QatError):
        qat.kv_attention(q, cache, table, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_operators_of_most_heads(qat, dtype):
    """32767 heads are each as one of a few; so are 100000 query heads of one cache head."""
    heads, few, d, t = 32767, 31, 8, 3
    q, k, v = (randn(i, t, few, d, dtype=dtype).repeat(1, 1057, 1) for i in range(3))
    assert q.shape[1] == heads
    positions, turns = torch.arange(5, 5 + t).cuda(), qat.rope_turns(qat.rope_frequencies(4), "cuda")
    w = torch.ones(d, dtype=dtype, device="cuda")
    r = qat.head_norm_rope(q, k, positions, turns, w, w)
    dq, dk, _, dw = qat.head_norm_rope_backward(v, v, q, k, positions, turns, w, w)
    cache, small = (qat.kv_cache(1, h, 16, d, "int8", "affine") for h in (heads, few))
    slots = torch.arange(t).cuda()
    qat.kv_write(cache, k, v, slots)
    rows = qat.kv_read(cache, slots, dtype)
    table, n = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([t], dtype=torch.int32, device="cuda")
    y = qat.kv_attention(q[:1], cache, table, n).y
    q1, k1, v1 = (x[:, :few].contiguous() for x in (q, k, v))
    r1 = qat.head_norm_rope(q1, k1, positions, turns, w, w)
    g1 = qat.head_norm_rope_backward(v1, v1, q1, k1, positions, turns, w, w)
    qat.kv_write(small, k1, v1, slots)
    rows1 = qat.kv_read(small, slots, dtype)
    y1 = qat.kv_attention(q1[:1], small, table, n).y
    for got, want in ((r.q, r1.q), (r.k, r1.k), (dq, g1[0]), (dk, g1[1]), (rows.k, rows1.k), (rows.v, rows1.v), (y, y1)):
        assert torch.equal(got, want.repeat(1, 1057, 1))
    # the gradient of the keys' weight: 1057 times the few heads' sum, of products of up to 6 in size
    c, s = ref.angles(positions.tolist(), turns.tolist(), 1.0)
    one = ref.rope(f64(k1), np.ones(d), f64(v1), c, s, "half", 1e-6, True, 1.0, F32)["dw"]
    size = np.abs(one[0]) * 1057
    err = (8 * math.sqrt(heads * t) + 40) * U * 1057 * few * t * 6 + 1057 * one[1]
    within(dw, one[0] * 1057, err + ref.step(dtype) * (size + err), "dw")
    # one cache head
    lone = qat.kv_cache(4, 1, 16, 64, "int8")
    slots = torch.arange(50).cuda()
    qat.kv_write(lone, randn(4, 50, 1, 64, dtype=dtype), randn(5, 50, 1, 64, dtype=dtype), slots)
    q = randn(6, 1, 10, 64, dtype=dtype)
    table, n = torch.arange(4, dtype=torch.int32).view(1, 4).cuda(), torch.tensor([50], dtype=torch.int32, device="cuda")
    got = qat.kv_attention(q.repeat(1, 10000, 1), lone, table, n).y.view(10000, 10, 64)
    y, ey, _, _ = ref.attention(f64(q), lone, table.cpu().numpy(), [50], 0.125, dtype)
    for i in (0, 1, 4999, 9999):
        within(got[i], y[0], ey[0], "y")
    assert (got - got[:1]).abs().max() <= 2 * float(ey.max())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_head_norm_rope_cosines_and_sines(qat, layout):
    """The pair (1, 0) turns to (cos, sin).  The reduced angle x, at most pi / 4, is off by 3 U
    of itself (its integer, the constant and their product) and by 2^-32 of a turn: 1.7 U of
    either.  The cosine's series leaves out less than 0.5 U, and rounds in its last step (U),
    the one before (0.6 U) and the square (0.3 U); the sine's rounds by less; the amplitude's
    product by U: 5.1 U, and 6 U is the bound that the rotation's tests take."""
    t, d = 4001, 64
    g = torch.Generator().manual_seed(5)
    positions = torch.cat([torch.arange(2000), torch.randint(-(1 << 62), 1 << 62, (2001,), generator=g)]).cuda()
    turns = qat.rope_turns(qat.rope_frequencies(d), "cuda")
    q = torch.zeros(t, 1, d, device="cuda")
    i = torch.arange(d // 2)
    a, b = (i, i + d // 2) if layout == "half" else (2 * i, 2 * i + 1)
    q[..., a] = 1.0
    for amplitude in (1.0, 0.75):
        y = qat.head_norm_rope(q, None, positions, turns, norm=False, layout=layout, amplitude=amplitude).q[:, 0]
        c, s = ref.angles(positions.tolist(), turns.tolist(), amplitude)
        within(y[:, a], c, 6 * U * amplitude + np.zeros_like(c), "cos")
        within(y[:, b], s, 6 * U * amplitude + np.zeros_like(s), "sin")
