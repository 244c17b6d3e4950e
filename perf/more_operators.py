"""Measured cases of the attention operators that serve a layer from a quantized key-value cache.

Four operators, in the order in which a decoding step uses them:

* ``rope``: the norm of queries and keys for each head with the position rotation in the same pass, forward and as a
  training step (gradients of queries, keys and both norm weights);
* ``write``: keys and values quantized (int8, int4, E4M3, E5M2) as they are written to the paged cache, and read back;
* ``read``: cached positions gathered and dequantized;
* ``attention``: one new token of each sequence over its pages of the cache.

Where ``own`` is false the operators are computed in their plain form, in 32 bits with elementary torch operations (in
64 for angles and for the quotients that decide a code).
"""
import math
import random

import torch

own = False

F32, BF16 = "fp32", "bf16"
_DTYPES = {F32: torch.float32, BF16: torch.bfloat16}
_FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
_INT = {"int8": 8, "int4": 4}

# The most work of each range (the listed cases reach it).
_MAX_ROPE = 8192 * 40 * 128
_MAX_ROWS = 65536 * 8 * 128
_MAX_CACHE = 2 * 131072 * 8 * 128
_MAX_SCORES = 4 * _MAX_CACHE


def _rope(name, tokens, heads, kv_heads, dim, rotary, train, norm=True, layout="half", amplitude=1.0, far=131072,
          dtype=BF16):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "train": train, "norm": norm, "layout": layout, "amplitude": amplitude, "far": far,
            "dtype": dtype}


def _rows(name, op, tokens, kv_heads, dim, page, form, scheme="symmetric", dtype=BF16):
    return {"name": name, "op": op, "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page, "format": form,
            "scheme": scheme, "dtype": dtype}


def _attention(name, batch, longest, ragged, heads, kv_heads, dim, page, form, scheme="symmetric", dtype=BF16):
    return {"name": name, "op": "attention", "batch": batch, "longest": longest, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "format": form, "scheme": scheme, "dtype": dtype}


def listed():
    return [
        # the new tokens of a few sequences: launch latency
        _rope("rope-tokens", 8, 32, 8, 128, 128, False),
        # a training step's queries and keys at full size
        _rope("rope-train", 8192, 32, 8, 128, 128, True),
        # a training step of a small odd-sized layer: part of the head turns, interleaved pairs, a long-context factor
        _rope("rope-train-odd-fp32", 1021, 7, 7, 80, 40, True, layout="interleaved", amplitude=1.25, dtype=F32),
        # the new token of each of a batch's sequences into the cache
        _rows("write-tokens", "write", 16, 8, 128, 16, "int8"),
        # a prompt into the smallest cache: affine 4-bit codes
        _rows("write-prompt-int4", "write", 16384, 8, 128, 64, "int4", "affine"),
        # a cached prefix read back for a prompt that goes on from it: the largest gather
        _rows("read-prefix", "read", 65536, 8, 128, 64, "int8"),
        # the same for a small odd-sized layer in fp32
        _rows("read-odd-fp32", "read", 1003, 5, 72, 48, "e4m3", dtype=F32),
        # one sequence, a short context: latency
        _attention("attention-token", 1, 700, False, 32, 8, 128, 16, "int8"),
        # a batch of requests of different lengths, one of them empty and one of a single token
        _attention("attention-batch-int4", 64, 8192, True, 32, 8, 128, 64, "int4", "affine"),
        # two long contexts: the largest cache
        _attention("attention-long-e4m3", 2, 131072, False, 32, 8, 128, 256, "e4m3"),
        # as many key heads as query heads, short heads, no quantization
        _attention("attention-heads-bf16", 32, 2048, True, 16, 16, 64, 32, "bf16"),
        # a ragged batch of a small odd-sized layer in fp32
        _attention("attention-odd-fp32", 13, 1500, True, 10, 2, 80, 16, "int8", dtype=F32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "rope", "write", "read", "attention", "attention", "attention"))
    dtype = rng.choice((BF16, BF16, BF16, F32))
    kv = rng.choice((1, 2, 3, 4, 5, 8, 8, 8, 16))
    group = rng.choice((1, 1, 2, 3, 4, 4, 5, 8, 16))
    dim = rng.choice((64, 64, 80, 96, 128, 128, 128, 192, 256, 40))
    form = rng.choice(("int8", "int8", "int4", "int4", "e4m3", "e4m3", "e5m2", "bf16"))
    scheme = rng.choice(("symmetric", "affine")) if form in _INT else "symmetric"
    page = rng.choice((16, 16, 32, 48, 64, 128, 256))
    if op == "rope":
        tokens = max(1, min(_log_int(rng, 1, 8192), _MAX_ROPE // (kv * (group + 1) * dim)))
        rotary = rng.choice((dim, dim, dim // 2, dim // 4))
        norm = rng.random() < 0.8
        case = _rope("", tokens, kv * group, kv, dim, rotary, rng.random() < 0.5, norm,
                     rng.choice(("half", "half", "interleaved")), rng.choice((1.0, 1.0, 1.25)),
                     _log_int(rng, tokens, 131072), dtype)
    elif op == "attention":
        batch = _log_int(rng, 1, 128)
        most = min(_MAX_CACHE // (kv * dim), _MAX_SCORES // (kv * group * dim)) // batch
        case = _attention("", batch, min(_log_int(rng, 1, 131072), most), rng.random() < 0.7, kv * group, kv, dim, page,
                          form, scheme, dtype)
    else:
        tokens = min(_log_int(rng, 1, 65536), _MAX_ROWS // (kv * dim))
        case = _rows("", op, tokens, kv, dim, page, form, scheme, dtype)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _frequencies(rotary):
    """Radians a position for each pair, in 64 bits."""
    return 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)


def _lengths(case):
    """The lengths of a batch's sequences: a plain function of the case."""
    batch, longest = case["batch"], case["longest"]
    if not case["ragged"]:
        return [longest] * batch
    rng = random.Random(batch * 1000003 + longest)
    out = [longest] + [_log_int(rng, max(1, longest // 16), longest) for _ in range(batch - 1)]
    out[1:3] = [0, 1][: max(0, batch - 1)]
    rng.shuffle(out)
    return out


def _keys_values(gen, *shape):
    """Keys with a few channels far out, as they are behind a norm and its weight; values."""
    far = torch.where(torch.rand(shape[-1], generator=gen, device="cuda") < 0.03, 6.0, 1.0)
    return _randn(gen, *shape) * far, _randn(gen, *shape)


def _empty_cache(case, pages):
    h, p, d, form = case["kv_heads"], case["page"], case["dim"], case["format"]
    cache = {"k_scale": None, "v_scale": None, "k_zero_point": None, "v_zero_point": None}
    for name in ("k", "v"):
        if form == "bf16":
            cache[name] = torch.zeros(pages, h, p, d, dtype=torch.bfloat16, device="cuda")
            continue
        row = d // 2 if form == "int4" else d
        cache[name] = torch.zeros(pages, h, p, (row + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
        cache[name + "_scale"] = torch.zeros(pages, h, p, device="cuda")
        if case["scheme"] == "affine":
            cache[name + "_zero_point"] = torch.zeros(pages, h, p, dtype=torch.int8, device="cuda")
    return cache


def _fill(gen, case, cache):
    """Every position of a cache, some pages at a time."""
    pages, h, p = cache["k"].shape[:3]
    step = max(1, (1 << 25) // (h * p * case["dim"]))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for name, x in zip(("k", "v"), _keys_values(gen, n, h, p, case["dim"])):
            _put(cache, name, slice(a, a + n), x, case)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, d = _DTYPES[case["dtype"]], case["dim"]
    state = {"case": case}
    if case["op"] == "rope":
        t, hq, hk = case["tokens"], case["heads"], case["kv_heads"]
        # queries and keys lie side by side, as a layer's one projection leaves them
        qkv = (_randn(gen, t, hq + 2 * hk, d) * _randn(gen, t, 1, 1).mul(0.3).exp()).to(dtype)
        state["q"], state["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        start = int(torch.randint(case["far"] - t + 1, (1,), generator=gen, device="cuda"))
        state["positions"] = torch.arange(start, start + t, device="cuda")
        state["frequencies"] = _frequencies(case["rotary"])
        state["wq"] = state["wk"] = None
        if case["norm"]:
            state["wq"], state["wk"] = ((1 + 0.2 * _randn(gen, d)).to(dtype) for _ in range(2))
        if case["train"]:
            state["dq"], state["dk"] = (_randn(gen, t, h, d).mul(1e-2).to(dtype) for h in (hq, hk))
        if own:
            import fake_quant_numerics_gb300 as fq

            state["turns"] = fq.rope_turns(state["frequencies"])
        return state
    if case["op"] == "attention":
        lengths = _lengths(case)
        need = [-(-n // case["page"]) for n in lengths]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        state["table"] = table
        state["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        state["q"] = _randn(gen, case["batch"], case["heads"], d).to(dtype)
        state["cache"] = _empty_cache(case, pages)
        _fill(gen, case, state["cache"])
    else:
        t, h = case["tokens"], case["kv_heads"]
        pages = -(-t // case["page"]) + 3
        # whole pages in any order, their positions in theirs
        order = torch.randperm(pages, generator=gen, device="cuda")
        slots = (order[:, None] * case["page"] + torch.arange(case["page"], device="cuda")).reshape(-1)
        state["slots"] = slots[:t].contiguous()
        state["cache"] = _empty_cache(case, pages)
        if case["op"] == "write":
            k, v = _keys_values(gen, t, h, d)
            state["k"], state["v"] = k.to(dtype), v.to(dtype)
        else:
            _fill(gen, case, state["cache"])
    if own:
        import fake_quant_numerics_gb300 as fq

        c = state["cache"]
        state["handle"] = fq.KVCache(c["k"], c["v"], case["format"], d, c["k_scale"], c["v_scale"], c["k_zero_point"],
                                     c["v_zero_point"])
    return state


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _over(a, b):
    """The quotient in binary32 (in 64 bits first: a quotient decides a code)."""
    return (a.double() / b).float()


def _codes(x, form, scheme):
    """Codes of the rows of x with their scale and zero point; the library's calibration, a row of D each."""
    x = x.float()
    if form in _FP8:
        kind, top = _FP8[form]
        scale = _over(x.abs().amax(-1), top)
        t = _over(x, scale[..., None].double())
        t = torch.where(scale[..., None] > 0, t, torch.zeros_like(t)).clamp(-top, top)
        return t.to(kind).view(torch.uint8), scale, None
    high = 2 ** (_INT[form] - 1) - 1
    low = -high if scheme == "symmetric" else -high - 1
    if scheme == "symmetric":
        zp = None
        scale = _over(x.abs().amax(-1), float(high))
    else:
        lo, hi = x.amin(-1).clamp_max(0), x.amax(-1).clamp_min(0)
        scale = _over(hi - lo, float(high - low))
        zp = torch.where(scale > 0, low - _over(lo, scale.double()), torch.zeros_like(scale)).round().clamp(low, high)
    q = _over(x, scale[..., None].double()).round()
    q = torch.where(scale[..., None] > 0, q, torch.zeros_like(q))
    if zp is not None:
        q = q + zp[..., None]
        zp = zp.to(torch.int8)
    q = q.clamp(low, high).to(torch.int8).view(torch.uint8)
    if form == "int4":
        q = (q[..., 0::2] << 4) | (q[..., 1::2] & 15)
    return q, scale, zp


def _put(cache, name, at, x, case):
    """The rows of x at an index of the cache's [pages, heads, page] positions."""
    if case["format"] == "bf16":
        cache[name][at] = x.to(torch.bfloat16)
        return
    q, scale, zp = _codes(x, case["format"], case["scheme"])
    cache[name][at] = torch.nn.functional.pad(q, (0, cache[name].shape[-1] - q.shape[-1]))
    cache[name + "_scale"][at] = scale
    if zp is not None:
        cache[name + "_zero_point"][at] = zp


def _get(cache, name, at, case):
    """The values of the cache's rows at an index, in 32 bits."""
    form, d = case["format"], case["dim"]
    rows = cache[name][at]
    if form == "bf16":
        return rows.float()
    if form in _FP8:
        q = rows[..., :d].contiguous().view(_FP8[form][0]).float()
    elif form == "int8":
        q = rows[..., :d].view(torch.int8).float()
    else:
        q = torch.stack([rows >> 4, rows & 15], -1).flatten(-2)[..., :d].float()
        q = torch.where(q > 7, q - 16, q)
    if case["scheme"] == "affine":
        q = q - cache[name + "_zero_point"][at].float()[..., None]
    return q * cache[name + "_scale"][at][..., None]


def _spread(slots, case):
    """Index of the positions `slots` of every head in the cache: [tokens, heads]."""
    heads = torch.arange(case["kv_heads"], device="cuda")
    return (slots // case["page"])[:, None], heads[None, :], (slots % case["page"])[:, None]


def _turn(x, cos, sin, layout):
    """The rotation of the leading pairs of x [tokens, heads, dim]; the rest as it is."""
    r = 2 * cos.shape[-1]
    if layout == "half":
        a, b = x[..., : r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rope(state):
    case = state["case"]
    angle = state["positions"].double()[:, None] * state["frequencies"][None]
    cos = (angle.cos() * case["amplitude"]).float()[:, None]
    sin = (angle.sin() * case["amplitude"]).float()[:, None]
    out = {}
    for name, weight in (("q", "wq"), ("k", "wk")):
        x = state[name].float()
        w = state[weight].float() if case["norm"] else None
        rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) if case["norm"] else None
        z = x * rstd if case["norm"] else x
        out[name] = _turn(z * w if case["norm"] else z, cos, sin, case["layout"]).to(state[name].dtype)
        if not case["train"]:
            continue
        g = _turn(state["d" + name].float(), cos, -sin, case["layout"])
        if case["norm"]:
            out["d" + weight] = (g * z).sum((0, 1)).to(state[name].dtype)
            g = g * w
            g = rstd * (g - z * (g * z).mean(-1, keepdim=True))
        out["d" + name] = g.to(state[name].dtype)
    return out


def _plain_attention(state):
    case, q, cache, lengths = state["case"], state["q"], state["cache"], state["lengths"]
    batch, heads, d = q.shape
    kv = case["kv_heads"]
    table = state["table"].long().clamp_min(0)

    def gather(name):  # [batch, kv heads, positions, dim]
        x = _get(cache, name, table, case)
        return x.transpose(1, 2).reshape(batch, kv, -1, d)

    s = (q.float().view(batch, kv, heads // kv, d) @ gather("k").transpose(-1, -2)) * d ** -0.5
    there = torch.arange(s.shape[-1], device="cuda") < lengths[:, None]
    s = torch.where(there[:, None, None], s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    y = (p @ gather("v")) / torch.where(total > 0, total, torch.ones_like(total))
    return y.reshape(batch, heads, d).to(q.dtype)


def _plain(state):
    case = state["case"]
    if case["op"] == "rope":
        return _plain_rope(state)
    if case["op"] == "attention":
        return _plain_attention(state)
    at = _spread(state["slots"], case)
    if case["op"] == "write":
        for name in ("k", "v"):
            _put(state["cache"], name, at, state[name], case)
    return {name: _get(state["cache"], name, at, case).to(_DTYPES[case["dtype"]]) for name in ("k", "v")}


def _own(state):
    import fake_quant_numerics_gb300 as fq

    case = state["case"]
    if case["op"] == "rope":
        more = {"layout": case["layout"], "amplitude": case["amplitude"]}
        if not case["norm"]:
            more["norm"] = False
        q, k, positions, turns, wq, wk = (state[n] for n in ("q", "k", "positions", "turns", "wq", "wk"))
        r = fq.head_norm_rope(q, k, positions, turns, wq, wk, **more)
        out = {"q": r.q, "k": r.k}
        if case["train"]:
            g = fq.head_norm_rope_backward(state["dq"], state["dk"], q, k, positions, turns, wq, wk, **more)
            out["dq"], out["dk"] = g[0], g[1]
            if case["norm"]:
                out["dwq"], out["dwk"] = g[2], g[3]
        return out
    if case["op"] == "attention":
        return fq.kv_attention(state["q"], state["handle"], state["table"], state["lengths"]).y
    if case["op"] == "write":
        fq.kv_write(state["handle"], state["k"], state["v"], state["slots"])
    r = fq.kv_read(state["handle"], state["slots"], _DTYPES[case["dtype"]])
    return {"k": r.k, "v": r.v}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the least work, and the definition in 64 bits
# ---------------------------------------------------------------------------
def _row_bytes(case):
    """A cached key or value: its codes and parameters."""
    d, form = case["dim"], case["format"]
    if form == "bf16":
        return 2 * d
    return (d // 2 if form == "int4" else d) + 4 + (case["scheme"] == "affine")


def work(case):
    e, d, kv = (4 if case["dtype"] == F32 else 2), case["dim"], case["kv_heads"]
    if case["op"] == "rope":
        t, h = case["tokens"], case["heads"] + kv
        weights = 2 * d * e if case["norm"] else 0
        small = 8 * t + 8 * (case["rotary"] // 2) + weights
        if case["train"]:  # x and the gradients read, the outputs and the gradients' gradients written
            return {"bytes": 4 * t * h * d * e + small + weights, "flops": 24 * t * h * d}
        return {"bytes": 2 * t * h * d * e + small, "flops": 9 * t * h * d}
    if case["op"] == "attention":
        n = sum(_lengths(case))
        table = sum(4 * -(-x // case["page"]) for x in _lengths(case)) + 4 * case["batch"]
        return {"bytes": 2 * n * kv * _row_bytes(case) + 2 * case["batch"] * case["heads"] * d * e + table,
                "flops": 4 * n * case["heads"] * d}
    rows = 2 * case["tokens"] * kv
    if case["op"] == "write":  # the rows in, their codes out, the values that they stand for out
        return {"bytes": rows * (2 * d * e + _row_bytes(case)) + 8 * case["tokens"], "flops": 8 * rows * d}
    return {"bytes": rows * (d * e + _row_bytes(case)) + 8 * case["tokens"], "flops": 2 * rows * d}


def _exact_fp8(byte, form):
    """The value of an FP8 code from its fields, in 64 bits."""
    mant, bias = (3, 7) if form == "e4m3" else (2, 15)
    b = byte.long()
    exponent, fraction = (b & 127) >> mant, (b & ((1 << mant) - 1)).double() / (1 << mant)
    small = fraction * 2.0 ** (1 - bias)
    value = torch.where(exponent == 0, small, (1 + fraction) * torch.exp2((exponent - bias).double()))
    return torch.where(b > 127, -value, value)


def _exact_rows(state, name, index):
    """The cache's rows at flat positions ((page * heads + head) * page size + offset), in 64 bits."""
    case, cache = state["case"], state["cache"]
    form, d = case["format"], case["dim"]
    rows = cache[name].flatten(0, 2)[index]
    if form == "bf16":
        return rows.double()
    if form in _FP8:
        value = _exact_fp8(rows[:, :d], form)
    elif form == "int8":
        value = rows[:, :d].double()
        value -= 256.0 * (value > 127)
    else:
        i = torch.arange(d, device="cuda")
        value = ((rows[:, i // 2] >> (4 * (1 - i % 2)).to(torch.uint8)) & 15).double()
        value -= 16.0 * (value > 7)
    if case["scheme"] == "affine":
        value -= cache[name + "_zero_point"].flatten()[index].double()[:, None]
    return value * cache[name + "_scale"].flatten()[index].double()[:, None]


def _exact_round_trip(x, case):
    """What a written row reads back as: its scale and quotients are binary32 numbers, the rest is in 64 bits."""
    form, r = case["format"], (lambda t: t.float().double())
    x = x.double()
    if form == "bf16":
        return x.to(torch.bfloat16).double()
    if form in _FP8:
        mant, least, top = (3, -6, 448.0) if form == "e4m3" else (2, -14, 57344.0)
        scale = r(x.abs().max(-1, keepdim=True).values / top)
        t = r(x / scale)
        exponent = torch.frexp(t).exponent.sub(1).clamp_min(least).double()
        unit = torch.exp2(exponent - mant)
        return (torch.round(t / unit) * unit).clamp(-top, top) * scale
    levels = 2 ** _INT[form]
    if case["scheme"] == "symmetric":
        scale = r(x.abs().max(-1, keepdim=True).values / (levels // 2 - 1))
        return torch.clamp(torch.round(r(x / scale)), 1 - levels // 2, levels // 2 - 1) * scale
    least, most = x.min(-1, keepdim=True).values.clamp(max=0), x.max(-1, keepdim=True).values.clamp(min=0)
    scale = r(r(most - least) / (levels - 1))
    zero = torch.clamp(torch.round(r(-levels // 2 - r(least / scale))), -levels // 2, levels // 2 - 1)
    code = torch.clamp(torch.round(r(x / scale)) + zero, -levels // 2, levels // 2 - 1)
    return (code - zero) * scale


def _exact_rope(state):
    """Rotations as products of complex numbers."""
    case = state["case"]
    d, half = case["dim"], case["rotary"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (i, i + half) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    phase = torch.outer(state["positions"].double(), state["frequencies"])
    unit = torch.polar(torch.full_like(phase, case["amplitude"]), phase)[:, None, :]

    def rotated(x, by):
        y = x.clone()
        pairs = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * by
        y[..., first], y[..., second] = pairs.real, pairs.imag
        return y

    out = {}
    for name, weight in (("q", "wq"), ("k", "wk")):
        x = state[name].double()
        w, size = torch.ones(d, dtype=torch.float64, device="cuda"), 1.0
        if case["norm"]:
            w = state[weight].double()
            size = ((x ** 2).sum(-1, keepdim=True) / d + 1e-6) ** 0.5
        out[name] = rotated(x / size * w, unit)
        if case["train"]:
            g = rotated(state["d" + name].double(), unit.conj())
            out["d" + name] = g
            if case["norm"]:
                out["d" + weight] = torch.einsum("thd,thd->d", g, x / size)
                dot = torch.einsum("thd,d,thd->th", g, w, x)[..., None]
                out["d" + name] = g * w / size - x * dot / (d * size ** 3)
    return out


def _exact_attention(state):
    case = state["case"]
    q = state["q"].double()
    batch, heads, d = q.shape
    kv, page = case["kv_heads"], case["page"]
    y = torch.zeros_like(q)
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        i = torch.arange(n, device="cuda")
        pages = state["table"][b].long()[i // page]
        for h in range(kv):
            index = (pages * kv + h) * page + i % page
            group = slice(h * (heads // kv), (h + 1) * (heads // kv))
            scores = torch.einsum("gd,nd->gn", q[b, group], _exact_rows(state, "k", index)) / math.sqrt(d)
            weights = torch.exp(scores - torch.logsumexp(scores, -1, keepdim=True))
            y[b, group] = torch.einsum("gn,nd->gd", weights, _exact_rows(state, "v", index))
    return y


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(state)
    if case["op"] == "attention":
        return _exact_attention(state)
    if case["op"] == "write":
        return {name: _exact_round_trip(state[name], case) for name in ("k", "v")}
    page, kv, slots = case["page"], case["kv_heads"], state["slots"]
    index = (slots[:, None] // page * kv + torch.arange(kv, device="cuda")) * page + slots[:, None] % page
    return {name: _exact_rows(state, name, index.reshape(-1)).view(-1, kv, case["dim"]) for name in ("k", "v")}
