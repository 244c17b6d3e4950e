"""Plain 64-bit definitions of the attention operators, with the bounds their
outputs are held to (CPU, numpy).

U = 2^-24 is half an ulp of 1 in binary32.  A binary32 sum of n terms with absolute
sum S is taken to be within 8 sqrt(n) U S of its value (rounding errors of either
sign add like a random walk; sums on the tensor cores, which round toward zero, stay
inside it because partial sums of mixed sign grow like S / sqrt(n), and their
measured bias is 1e-9 of the sum a term: below 8 sqrt(n) U up to 10^5 terms).  An
output's own rounding is half a step: 2^-8 of a bf16 value, U of a binary32 one.
"""
import math

import numpy as np
import torch

from layer_reference import U, f64

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
BITS = {"int8": 8, "int4": 4}


def step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2 * U


# --- head norm and rotation --------------------------------------------------
def angles(positions, turns, amplitude):
    """Cosines and sines [tokens, pairs] of position * turns modulo 2^64, in units of
    2^-64 of a turn (exact integers; the angle is then rounded to 64 bits once)."""
    a = np.array([[((int(p) * int(t)) % (1 << 64)) / 2.0 ** 64 for t in turns] for p in positions])
    a = 2 * math.pi * a.reshape(len(positions), len(turns))
    return np.cos(a) * amplitude, np.sin(a) * amplitude


def turn(x, c, s, layout):
    """The leading pairs of x [tokens, heads, dim] turned."""
    r = 2 * c.shape[-1]
    y = x.copy()
    i = np.arange(r // 2)
    a, b = (i, i + r // 2) if layout == "half" else (2 * i, 2 * i + 1)
    c, s = c[:, None], s[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rope(x, w, g, c, s, layout, eps, norm, amplitude, dtype):
    """{name: (value, bound)} of y, and with a gradient g of dx and dw."""
    d = x.shape[-1]
    r = step(dtype)
    ec = 6 * U * amplitude  # the hardware angle's cosine and sine are a few ulp of 1 off
    w = np.ones(d) if w is None else w
    size = np.sqrt((x * x).mean(-1, keepdims=True) + eps) if norm else np.ones(x.shape[:-1] + (1,))
    rel = (8 * math.sqrt(d) + 6) * U if norm else 0.0  # of 1 / size
    z = x / size
    p = z * w
    ep = (rel + 4 * U) * np.abs(p)

    def turned(v, ev, back):
        y = turn(v, c, -s if back else s, layout)
        n = 2 * c.shape[-1]
        both = np.abs(v).copy()
        if n:
            i = np.arange(n // 2)
            a, b = (i, i + n // 2) if layout == "half" else (2 * i, 2 * i + 1)
            both[..., a] = both[..., b] = np.abs(v[..., a]) + np.abs(v[..., b])
            ev = ev.copy()
            ev[..., a] = ev[..., b] = ev[..., a] + ev[..., b]
        return y, max(1.0, amplitude) * ev + (ec + 4 * U * max(1.0, amplitude)) * both

    y, ey = turned(p, ep, False)
    out = {"y": (y, ey + r * (np.abs(y) + ey))}
    if g is None:
        return out
    gb, egb = turned(g, np.zeros_like(g), True)
    gw = gb * w
    egw = egb * np.abs(w) + 2 * U * np.abs(gw)
    if not norm:
        out["dx"] = (gw, egw + r * (np.abs(gw) + egw))
        return out
    mean = (gw * z).mean(-1, keepdims=True)
    emean = ((8 * math.sqrt(d) + 8) * U + rel) * np.abs(gw * z).mean(-1, keepdims=True) \
        + (egw * np.abs(z)).mean(-1, keepdims=True)
    inner = gw - z * mean
    einner = egw + np.abs(z) * (emean + (rel + 6 * U) * np.abs(mean)) + 4 * U * np.abs(gw)
    dx = inner / size
    edx = (einner + (rel + 4 * U) * np.abs(inner)) / size
    out["dx"] = (dx, edx + r * (np.abs(dx) + edx))
    n = x.shape[0] * x.shape[1]
    dw = (gb * z).sum((0, 1))
    edw = (8 * math.sqrt(n + 16) * U + rel + 4 * U) * np.abs(gb * z).sum((0, 1)) + (egb * np.abs(z)).sum((0, 1))
    out["dw"] = (dw, edw + r * (np.abs(dw) + edw))
    return out


# --- the cache's rows ----------------------------------------------------------
def r32(x):
    return np.asarray(x, dtype=np.float32).astype(float)


def fp8_round(t, form):
    """Round to nearest even on the format's grid, saturating."""
    mant, least = (3, -6) if form == "e4m3" else (2, -14)
    e = np.floor(np.log2(np.maximum(np.abs(t), 1e-300)))
    e = np.maximum(np.where(2.0 ** (e + 1) <= np.abs(t), e + 1, np.where(2.0 ** e > np.abs(t), e - 1, e)), least)
    unit = 2.0 ** (e - mant)
    return np.clip(np.rint(t / unit) * unit, -TOP[form], TOP[form])


def quantized(x, form, scheme="symmetric"):
    """(codes or code values, scale, zero point) of the rows of x (binary32 values as
    float64).  Scales, quotients and the affine range are binary32 numbers: each is
    the 64-bit result rounded once (a 53-bit quotient of 24-bit numbers rounds to the
    24 bits that one rounding gives)."""
    with np.errstate(all="ignore"):
        fine = np.isfinite(x).all(-1)
        x = np.where(fine[..., None], x, 0.0)
        top = np.abs(x).max(-1) if x.shape[-1] else np.zeros(x.shape[:-1])
        zp = np.zeros_like(top)
        if form in TOP:
            scale = r32(top / TOP[form])
            q = fp8_round(np.where(scale[..., None] > 0, r32(x / scale[..., None]), 0.0), form)
        else:
            high = 2 ** (BITS[form] - 1) - 1
            low = -high if scheme == "symmetric" else -high - 1
            if scheme == "symmetric":
                scale = r32(top / high)
            else:
                lo, hi = np.minimum(x.min(-1), 0.0), np.maximum(x.max(-1), 0.0)
                scale = r32(r32(hi - lo) / (high - low))
                zp = np.clip(np.rint(r32(low - r32(lo / scale))), low, high)
                zp = np.where((scale > 0) & np.isfinite(scale), zp, 0.0)
            q = np.clip(np.rint(r32(x / scale[..., None])) + zp[..., None], low, high)
            q = np.where((scale[..., None] > 0) & np.isfinite(scale[..., None]), q, 0.0)
        scale = np.where(fine & np.isfinite(scale), scale, np.nan)
        q = np.where(np.isnan(scale)[..., None], 0.0, q)
        zp = np.where(np.isnan(scale), 0.0, zp)
    return q, scale, zp


def fp8_values(byte, form):
    mant, bias = (3, 7) if form == "e4m3" else (2, 15)
    b = byte.astype(int)
    e, f = (b & 127) >> mant, (b & ((1 << mant) - 1)) / (1 << mant)
    v = np.where(e == 0, f * 2.0 ** (1 - bias), (1 + f) * 2.0 ** (e - bias))
    return np.where(b > 127, -v, v)


def codes_of(cache, name):
    """Code values [pages, heads, page_size, head_dim] of a cache, in 64 bits."""
    rows = getattr(cache, name).cpu()
    d = cache.head_dim
    if cache.format == "bf16":
        return rows.double().numpy()
    b = rows.numpy()
    if cache.format in TOP:
        return fp8_values(b[..., :d], cache.format)
    if cache.format == "int8":
        return b.view(np.int8)[..., :d].astype(float)
    q = np.stack([b >> 4, b & 15], -1).reshape(b.shape[:-1] + (-1,))[..., :d].astype(int)
    return np.where(q > 7, q - 16, q).astype(float)


def values_of(cache, name):
    """The values that a cache's rows stand for, exactly, in 64 bits."""
    q = codes_of(cache, name)
    if cache.format == "bf16":
        return q
    zp = getattr(cache, name + "_zero_point")
    if zp is not None:
        q = q - f64(zp)[..., None]
    return q * f64(getattr(cache, name + "_scale"))[..., None]


# --- attention -------------------------------------------------------------------
def attention(q, cache, table, lengths, scale, dtype):
    """(y, bound, lse, bound) of the definition, sequence by sequence."""
    kv, vv = values_of(cache, "k"), values_of(cache, "v")
    batch, heads, d = q.shape
    group = heads // cache.heads
    y, ey = np.zeros(q.shape), np.zeros(q.shape)
    lse, elv = np.full((batch, heads), -np.inf), np.zeros((batch, heads))
    for b in range(batch):
        n = int(lengths[b])
        if n <= 0:
            continue
        t = np.arange(n)
        pages = np.asarray(table[b])[t // cache.page_size] if n <= len(table[b]) * cache.page_size else None
        if pages is None or (pages < 0).any() or (pages >= cache.pages).any():
            y[b], lse[b] = np.nan, np.nan
            continue
        for h in range(heads):
            k, v = kv[pages, h // group, t % cache.page_size], vv[pages, h // group, t % cache.page_size]
            s = k @ q[b, h] * scale
            es = ((8 * math.sqrt(d) + 12) * U * (np.abs(k) @ np.abs(q[b, h])) * abs(scale)) + 8 * U * np.abs(s)
            # affine codes: products with the codes, then with the zero point
            es = es + extra_affine(cache, pages, h // group, t, q[b, h]) * abs(scale) * (8 * math.sqrt(d) + 4) * U
            top = s.max()
            e = np.exp(s - top)
            w = e / e.sum()
            y[b, h] = w @ v
            lse[b, h] = top + math.log(e.sum())
            # weights: their exponent's error, the hardware exponential (2^-21) and, under a bf16
            # output, their two 16-bit parts
            rel = 2 * es + 2.0 ** -21 + 8 * U * np.abs(s - top) + (2.0 ** -16 if dtype == torch.bfloat16 else 8 * U)
            size = np.abs(v) + np.abs(y[b, h]) + extra_values(cache, pages, h // group, t)[:, None]
            err = (w * rel) @ size + (8 * math.sqrt(n) + 16) * U * (w @ size)
            # weights, and their products with values, below the normal range of binary32 may
            # be lost: each less than 2^-126 times 1 + |v| (the sum of weights is at least 1)
            err = err + n * 2.0 ** -126 * (1 + np.abs(v).max(0))
            if cache.format != "bf16":
                # fp16's last bit (half of 2^-24) where a weight times its scale is a number of up
                # to 2^8 times the largest scale or more: 2^-33 of that scale, a code each
                vs = np.abs(f64(cache.v_scale)[pages, h // group, t % cache.page_size])
                code = np.abs(v) / np.where(vs > 0, vs, 1.0)[:, None]
                err = err + 2.0 ** -33 * vs.max() * (code + extra_codes(cache, pages, h // group, t)[:, None]).sum(0)
            ey[b, h] = err + step(dtype) * (np.abs(y[b, h]) + err)
            elv[b, h] = (w * rel).sum() + es.max() + (8 * math.sqrt(n) + 16) * U + 4 * U * abs(lse[b, h])
    return y, ey, lse, elv


def extra_affine(cache, pages, head, t, q):
    """|zero point * scale| sum |q|: what the subtraction of the zero points may cancel."""
    if cache.k_zero_point is None:
        return np.zeros(len(t))
    z, s = f64(cache.k_zero_point)[pages, head, t % cache.page_size], f64(cache.k_scale)[pages, head, t % cache.page_size]
    return np.abs(z * s) * np.abs(q).sum()


def extra_values(cache, pages, head, t):
    if cache.v_zero_point is None:
        return np.zeros(len(t))
    return np.abs(f64(cache.v_zero_point)[pages, head, t % cache.page_size]
                  * f64(cache.v_scale)[pages, head, t % cache.page_size])


def extra_codes(cache, pages, head, t):
    if cache.v_zero_point is None:
        return np.zeros(len(t))
    return np.abs(f64(cache.v_zero_point)[pages, head, t % cache.page_size])
