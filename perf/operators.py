"""Measured cases of the transformer-layer operators that stand next to the fake-quant calls.

Three operators, the feed-forward half of a layer whose weights are trained through fake quantization and served
from their 4-bit codes:

* ``linear4``: products of a few tokens with a 4-bit weight, in the code layouts the library writes (integer codes
  with a scale per group, row or tensor, symmetric or affine; the two-level format with blocks of 64);
* ``ffn``: the gated feed-forward block (both projections, the activation and the product, then the projection
  back), forward, as a training step (forward and backward), and from 4-bit codes for single tokens (``ffn4``);
* ``layernorm``: layer norm, forward and as a training step (gradients of the input, the weight and the bias).

Where ``own`` is false the operators are computed in their plain form, in 32 bits with elementary torch operations.
"""
import math

import torch

own = False

F32, BF16 = "fp32", "bf16"
_DTYPES = {F32: torch.float32, BF16: torch.bfloat16}

# The largest sizes of each range (the listed cases reach them).
_MAX_TOKENS4 = 32
_MAX_FFN = 4096 * 4096 * 14336
_MAX_NORM = 16384 * 4096


def _linear4(name, tokens, out, inner, granularity="group", group=128, scheme="symmetric", dtype=BF16):
    return {"name": name, "op": "linear4", "tokens": tokens, "out": out, "in": inner, "granularity": granularity,
            "group": group, "scheme": scheme, "dtype": dtype}


def _ffn4(name, tokens, dim, hidden, granularity="group", group=128, scheme="symmetric", dtype=BF16,
          activation="silu"):
    return {"name": name, "op": "ffn4", "tokens": tokens, "dim": dim, "hidden": hidden, "granularity": granularity,
            "group": group, "scheme": scheme, "dtype": dtype, "activation": activation}


def _ffn(name, tokens, dim, hidden, train, dtype=BF16, activation="silu"):
    return {"name": name, "op": "ffn", "tokens": tokens, "dim": dim, "hidden": hidden, "train": train,
            "dtype": dtype, "activation": activation}


def _norm(name, rows, cols, train, dtype=BF16):
    return {"name": name, "op": "layernorm", "rows": rows, "cols": cols, "train": train, "dtype": dtype}


def listed():
    return [
        # one token through a small projection: launch latency
        _linear4("linear4-token-small", 1, 1024, 1024),
        # one token through the library's per-group weight workload [14336, 4096], groups of 128
        _linear4("linear4-token", 1, 14336, 4096),
        # a batch of decoding requests through the projection back, affine codes in small groups
        _linear4("linear4-batch-affine", 16, 4096, 14336, group=64, scheme="affine"),
        # a ragged batch in fp32 on the two-level format; an odd number of outputs (a vocabulary or adapter head)
        _linear4("linear4-double-odd", 5, 4099, 4096, granularity="double", dtype=F32),
        # decoding one token: the whole gated block from 4-bit codes
        _ffn4("ffn4-token", 1, 4096, 14336),
        # decoding a batch: affine codes in the smallest groups
        _ffn4("ffn4-batch-affine", 8, 4096, 8192, group=32, scheme="affine", activation="gelu"),
        # a ragged prompt through the block
        _ffn("ffn-forward-ragged", 1001, 4096, 14336, False),
        # a training step at full size: the largest case
        _ffn("ffn-train", 4096, 4096, 14336, True),
        # a training step of a small odd-sized block in fp32 (gradient checks, small experiments)
        _ffn("ffn-train-odd-fp32", 300, 510, 1363, True, dtype=F32, activation="gelu"),
        # the norm of a few decoding tokens: launch latency
        _norm("layernorm-tokens", 4, 4096, False),
        # the norm of a training step's tokens
        _norm("layernorm-train", 16384, 4096, True),
        # odd rows in fp32
        _norm("layernorm-train-odd-fp32", 2053, 5003, True, dtype=F32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer's width: mostly multiples of 128, some of 8, some of neither."""
    n = _log_int(rng, lo, hi)
    step = rng.choice((128, 128, 128, 8, 1))
    return max(step, n // step * step)


def _codes_of(rng, inner):
    """Granularity, group and inner length of a 4-bit weight near `inner` wide."""
    granularity = rng.choice(("group", "group", "group", "row", "tensor", "double"))
    group = rng.choice((32, 64, 128)) if granularity == "group" else 128
    if granularity == "group":
        inner = max(group, inner // group * group)
    return granularity, group, inner


def draw(rng):
    op = rng.choice(("linear4", "linear4", "ffn4", "ffn", "ffn", "layernorm", "layernorm"))
    dtype = rng.choice((BF16, BF16, BF16, F32))
    scheme = rng.choice(("symmetric", "affine"))
    activation = rng.choice(("silu", "gelu", "relu"))
    if op == "linear4":
        granularity, group, inner = _codes_of(rng, _width(rng, 64, 14336))
        case = _linear4("", _log_int(rng, 1, _MAX_TOKENS4), _width(rng, 64, 14336), inner, granularity, group, scheme,
                        dtype)
    elif op == "ffn4":
        granularity, group, dim = _codes_of(rng, _width(rng, 64, 4096))
        hidden = _width(rng, 64, 14336)
        if granularity == "group":
            hidden = max(group, hidden // group * group)
        case = _ffn4("", _log_int(rng, 1, _MAX_TOKENS4), dim, hidden, granularity, group, scheme, dtype, activation)
    elif op == "ffn":
        case = _ffn("", _log_int(rng, 1, 4096), _width(rng, 64, 4096), _width(rng, 64, 14336),
                    rng.random() < 0.6, dtype, activation)
    else:
        rows, cols = _log_int(rng, 1, 16384), _width(rng, 8, 16384)
        rows = max(1, min(rows, _MAX_NORM // cols))
        case = _norm("", rows, cols, rng.random() < 0.6, dtype)
    del case["name"]
    # the listed widths stand for this repository's workloads; this one is none of them
    return draw(rng) if 3 << 10 in case.values() else case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _pack(q):
    """Codes two per byte, element 2j in the high nibble (flat order)."""
    q = (q.reshape(-1) & 15).to(torch.uint8)
    if q.numel() % 2:
        q = torch.cat([q, q.new_zeros(1)])
    return (q[0::2] << 4) | q[1::2]


def _quantized(gen, rows, cols, granularity, group, scheme):
    """A weight ~ N(0, 0.02^2) as 4-bit codes with their parameters (what a user's program keeps)."""
    w = _randn(gen, rows, cols) * 0.02
    if granularity == "double":
        n = w.numel()
        pad = torch.nn.functional.pad(w.reshape(-1), (0, -n % 64)).reshape(-1, 64)
        s = pad.abs().amax(1) / 7
        q = (pad / s.clamp_min(1e-30)[:, None]).round().clamp(-8, 7).to(torch.int32).reshape(-1)[:n]
        blocks = torch.nn.functional.pad(s, (0, -s.numel() % 256)).reshape(-1, 256)
        sup = blocks.amax(1).clamp_min(1e-8)
        qs = (blocks / sup[:, None] * 255).round().clamp(0, 255).to(torch.uint8).reshape(-1)[: s.numel()]
        return {"codes": _pack(q), "scale": qs.contiguous(), "super": sup, "zp": None, "rows": rows, "cols": cols,
                "granularity": granularity, "group": 64}
    units = w.reshape({"group": (-1, group), "row": (rows, cols), "tensor": (1, -1)}[granularity])
    if scheme == "symmetric":
        s = units.abs().amax(1) / 7
        zp, low = None, -7
        q = (units / s[:, None]).round().clamp(low, 7)
    else:
        lo, hi = units.amin(1).clamp_max(0), units.amax(1).clamp_min(0)
        s = (hi - lo) / 15
        zp = (-8 - lo / s).round().clamp(-8, 7)
        q = ((units / s[:, None]).round() + zp[:, None]).clamp(-8, 7)
        zp = zp.to(torch.int32)
    return {"codes": _pack(q.to(torch.int32)), "scale": s.contiguous(), "super": None, "zp": zp, "rows": rows,
            "cols": cols, "granularity": granularity, "group": group}


def _view(gen, rows, cols, dtype):
    """The fake-quant view of a weight: int8 grid values per row, in the layer's type."""
    w = _randn(gen, rows, cols) * 0.02
    s = w.abs().amax(1, keepdim=True) / 127
    return ((w / s).round() * s).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "linear4":
        state["w"] = _quantized(gen, case["out"], case["in"], case["granularity"], case["group"], case["scheme"])
        state["x"] = _randn(gen, case["tokens"], case["in"]).to(dtype)
    elif case["op"] == "ffn4":
        d, f = case["dim"], case["hidden"]
        for name, rows, cols in (("gate", f, d), ("up", f, d), ("down", d, f)):
            state[name] = _quantized(gen, rows, cols, case["granularity"], case["group"], case["scheme"])
        state["x"] = _randn(gen, case["tokens"], d).to(dtype)
    elif case["op"] == "ffn":
        t, d, f = case["tokens"], case["dim"], case["hidden"]
        state["gate"], state["up"] = _view(gen, f, d, dtype), _view(gen, f, d, dtype)
        state["down"] = _view(gen, d, f, dtype)
        state["x"] = _randn(gen, t, d).to(dtype)
        state["dy"] = (_randn(gen, t, d) * 1e-2).to(dtype) if case["train"] else None
    else:
        r, c = case["rows"], case["cols"]
        # residual-stream rows: their own spread and offset, a few channels far out
        x = _randn(gen, r, c) * _randn(gen, r, 1).mul(0.5).exp() + 0.1 * _randn(gen, r, 1)
        x = torch.where(torch.rand(c, generator=gen, device="cuda") < 0.01, x * 20, x)
        state["x"] = x.to(dtype)
        state["weight"] = (1 + 0.1 * _randn(gen, c)).to(dtype)
        state["bias"] = (0.1 * _randn(gen, c)).to(dtype)
        state["dy"] = (_randn(gen, r, c) * 1e-2).to(dtype) if case["train"] else None
    return state


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_weight(w):
    """The codes' values in 32 bits: (q - zp) * scale."""
    rows, cols, n = w["rows"], w["cols"], w["rows"] * w["cols"]
    c = w["codes"]
    q = torch.stack([c >> 4, c & 15], 1).reshape(-1)[:n].to(torch.int32)
    q = torch.where(q > 7, q - 16, q).float()
    if w["granularity"] == "double":
        scale = w["scale"].float() / 255 * w["super"].repeat_interleave(256)[: w["scale"].numel()]
        return (q * scale.repeat_interleave(64)[:n]).reshape(rows, cols)
    units = q.reshape(w["scale"].numel(), -1)
    if w["zp"] is not None:
        units = units - w["zp"].float()[:, None]
    return (units * w["scale"][:, None]).reshape(rows, cols)


def _plain_act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        phi = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    return g.clamp_min(0), (g > 0).float()


def _plain(state):
    case = state["case"]
    x = state["x"].float()
    dtype = state["x"].dtype
    if case["op"] == "linear4":
        return (x @ _plain_weight(state["w"]).T).to(dtype)
    if case["op"] in ("ffn4", "ffn"):
        names = ("gate", "up", "down")
        wg, wu, wd = (_plain_weight(state[k]) if case["op"] == "ffn4" else state[k].float() for k in names)
        g, u = x @ wg.T, x @ wu.T
        a, da = _plain_act(g, case["activation"])
        h = a * u
        y = (h @ wd.T).to(dtype)
        if case["op"] == "ffn4" or not case["train"]:
            return y
        dy = state["dy"].float()
        dh = dy @ wd
        dg, du = dh * u * da, dh * a
        dx = dg @ wg + du @ wu
        return {"y": y, "dx": dx.to(dtype), "dw_gate": (dg.T @ x).to(dtype), "dw_up": (du.T @ x).to(dtype),
                "dw_down": (dy.T @ h).to(dtype)}
    w, b = state["weight"].float(), state["bias"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + 1e-5)
    xhat = xc * rstd
    y = (xhat * w + b).to(dtype)
    if not case["train"]:
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy = state["dy"].float()
    wdy = dy * w
    dx = rstd * (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True))
    return {"y": y, "dx": dx.to(dtype), "dweight": (dy * xhat).sum(0).to(dtype), "dbias": dy.sum(0).to(dtype)}


def _own_weight(fq, w):
    if w["granularity"] == "double":
        dq = fq.DoubleQuantized4Bit(w["codes"], w["scale"], w["super"], w["rows"] * w["cols"], None)
        return fq.weight4_double(dq, w["rows"], w["cols"])
    return fq.weight4(w["codes"], w["scale"], w["rows"], w["cols"], w["granularity"], w["group"], w["zp"])


def _own(state):
    import fake_quant_numerics_gb300 as fq

    case, x = state["case"], state["x"]
    if case["op"] == "linear4":
        return fq.linear4(x, _own_weight(fq, state["w"]))
    if case["op"] == "ffn4":
        gate, up, down = (_own_weight(fq, state[k]) for k in ("gate", "up", "down"))
        return fq.gated_ffn4(x, gate, up, down, activation=case["activation"])
    if case["op"] == "ffn":
        weights = state["gate"], state["up"], state["down"]
        if not case["train"]:
            return fq.gated_ffn(x, *weights, activation=case["activation"]).y
        r = fq.gated_ffn(x, *weights, activation=case["activation"], save=True)
        dx, dg, du, dd = fq.gated_ffn_backward(state["dy"], x, *weights, r, activation=case["activation"])
        return {"y": r.y, "dx": dx, "dw_gate": dg, "dw_up": du, "dw_down": dd}
    r = fq.layer_norm(x, state["weight"], state["bias"], eps=1e-5)
    if not case["train"]:
        return {"y": r.y, "mean": r.mean, "rstd": r.rstd}
    dx, dw, db = fq.layer_norm_backward(state["dy"], x, state["weight"], r.mean, r.rstd)
    return {"y": r.y, "dx": dx, "dweight": dw, "dbias": db}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the least work, and the definition in 64 bits
# ---------------------------------------------------------------------------
def _weight_bytes(rows, cols, granularity, group, scheme):
    n = rows * cols
    if granularity == "double":
        blocks = -(-n // 64)
        return -(-n // 2) + blocks + 4 * -(-blocks // 256)
    units = {"group": n // group, "row": rows, "tensor": 1}[granularity]
    return -(-n // 2) + units * (8 if scheme == "affine" else 4)


def work(case):
    e = 4 if case["dtype"] == F32 else 2
    if case["op"] == "linear4":
        t, n, k = case["tokens"], case["out"], case["in"]
        return {"bytes": _weight_bytes(n, k, case["granularity"], case["group"], case["scheme"]) + e * t * (n + k),
                "flops": 2 * t * n * k}
    if case["op"] == "ffn4":
        t, d, f = case["tokens"], case["dim"], case["hidden"]
        each = (case["granularity"], case["group"], case["scheme"])
        return {"bytes": 2 * _weight_bytes(f, d, *each) + _weight_bytes(d, f, *each) + 2 * e * t * d,
                "flops": 6 * t * d * f}
    if case["op"] == "ffn":
        t, d, f = case["tokens"], case["dim"], case["hidden"]
        if case["train"]:
            return {"bytes": e * (4 * t * d + 6 * d * f), "flops": 18 * t * d * f}
        return {"bytes": e * (2 * t * d + 3 * d * f), "flops": 6 * t * d * f}
    r, c = case["rows"], case["cols"]
    if case["train"]:
        return {"bytes": e * (4 * r * c + 4 * c), "flops": 20 * r * c}
    return {"bytes": e * (2 * r * c + 2 * c) + 8 * r, "flops": 8 * r * c}


def _exact_weight(w):
    """One table lookup per nibble, then each unit's parameters, in binary64."""
    table = torch.tensor([v - 16 if v > 7 else v for v in range(16)], dtype=torch.float64, device="cuda")
    n = w["rows"] * w["cols"]
    byte = w["codes"].long()
    value = torch.empty(2 * byte.numel(), dtype=torch.float64, device="cuda")
    value[0::2], value[1::2] = table[byte // 16], table[byte % 16]
    value = value[:n]
    i = torch.arange(n, device="cuda")
    if w["granularity"] == "double":
        unit = i // 64
        value *= (w["scale"].double() / 255.0)[unit] * w["super"].double()[unit // 256]
        return value.view(w["rows"], w["cols"])
    unit = i // (n // w["scale"].numel())
    if w["zp"] is not None:
        value -= w["zp"].double()[unit]
    return (value * w["scale"].double()[unit]).view(w["rows"], w["cols"])


def _exact_act(g, kind):
    if kind == "silu":
        e = torch.exp(-g)
        return g / (1 + e), (1 + e + g * e) / (1 + e) ** 2
    if kind == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(-(g ** 2) / 2) / math.sqrt(math.tau)
    return torch.where(g > 0, g, torch.zeros_like(g)), torch.where(g > 0, 1.0, 0.0).double()


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "linear4":
        return torch.einsum("tk,nk->tn", x, _exact_weight(s["w"]))
    if case["op"] in ("ffn4", "ffn"):
        if case["tokens"] * case["dim"] * case["hidden"] > _MAX_FFN:
            return None
        get = _exact_weight if case["op"] == "ffn4" else torch.Tensor.double
        gate = torch.einsum("td,fd->tf", x, get(s["gate"]))
        up = torch.einsum("td,fd->tf", x, get(s["up"]))
        act, slope = _exact_act(gate, case["activation"])
        y = torch.einsum("tf,df->td", act * up, get(s["down"]))
        if case["op"] == "ffn4" or not case["train"]:
            return y
        dy = s["dy"].double()
        back = torch.einsum("td,df->tf", dy, s["down"].double())
        d_gate, d_up = back * up * slope, back * act
        dx = torch.einsum("tf,fd->td", d_gate, s["gate"].double())
        dx += torch.einsum("tf,fd->td", d_up, s["up"].double())
        return {"y": y, "dx": dx, "dw_gate": torch.einsum("tf,td->fd", d_gate, x),
                "dw_up": torch.einsum("tf,td->fd", d_up, x), "dw_down": torch.einsum("td,tf->df", dy, act * up)}
    w, b = s["weight"].double(), s["bias"].double()
    n = case["cols"]
    mean = x.sum(1) / n
    var = ((x - mean[:, None]) ** 2).sum(1) / n
    rstd = (var + 1e-5) ** -0.5
    z = (x - mean[:, None]) * rstd[:, None]
    y = z * w + b
    if not case["train"]:
        return {"y": y, "mean": mean, "rstd": rstd}
    dz = s["dy"].double() * w
    m1, m2 = dz.sum(1) / n, (dz * z).sum(1) / n
    dx = (dz - m1[:, None] - z * m2[:, None]) * rstd[:, None]
    return {"y": y, "dx": dx, "dweight": torch.einsum("rc,rc->c", s["dy"].double(), z),
            "dbias": s["dy"].double().sum(0)}
