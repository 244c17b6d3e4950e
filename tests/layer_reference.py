"""Plain 64-bit definitions of the layer operators, with the bounds their
outputs are held to (CPU, numpy).

The bounds follow the kernels' arithmetic, elementwise.  U = 2^-24 is half an
ulp of 1 in binary32.  A binary32 sum of n products with absolute sum S is
within 8 sqrt(n) U S of its value: rounding errors of either sign add like a
random walk, and sums that always round toward zero stay within the same bound
because their partial sums grow like S / sqrt(n) for data of mixed sign.  A
bfloat16 rounding is within 2^-8 of the value (half an ulp is 2^-9; the factor
covers the neighbour's binade).
"""
import math

import numpy as np
import torch

U = 2.0 ** -24


def half(dtype):
    """Relative rounding of an output of this type."""
    return 2.0 ** -8 if dtype == torch.bfloat16 else 4 * U


def f64(t):
    return t.detach().cpu().double().numpy()


def within(got, ref, tol, what):
    got = f64(got)
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst "
                           f"{np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} of the bound")


# --- 4-bit weights ---------------------------------------------------------
def codes_of(packed, n):
    c = packed.cpu().numpy().astype(np.int64)
    q = np.stack([c >> 4, c & 15], 1).reshape(-1)[:n]
    return np.where(q > 7, q - 16, q).astype(np.float64)


def weight_values(w):
    """[rows, cols] values of a Weight4 (layout 0 tensor, 1 row, 2 group, 16 two-level)."""
    n = w.rows * w.cols
    q = codes_of(w.codes, n)
    i = np.arange(n)
    if w.layout == 16:
        s = f64(w.scale) / 255.0
        q = q * s[i // 64] * f64(w.super_scales)[i // 64 // 256]
    else:
        unit = i // max(1, n // max(1, w.scale.numel()))
        if w.zero_point is not None:
            q = q - f64(w.zero_point)[unit]
        q = q * f64(w.scale)[unit]
    return q.reshape(w.rows, w.cols)


def product(x, w):
    """x w^T and the bound of its binary32 sum."""
    s = np.abs(x) @ np.abs(w).T
    return x @ w.T, 8 * math.sqrt(max(1, w.shape[1]) + 16) * U * s


# --- activations -----------------------------------------------------------
_erf = np.vectorize(math.erf, otypes=[float])


def act(kind, g):
    """act(g), act'(g)."""
    if kind == "silu":
        s = 1 / (1 + np.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        phi = 0.5 * (1 + _erf(g / math.sqrt(2))) if g.size else g
        return g * phi, phi + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    return np.maximum(g, 0), (g > 0).astype(float)


def act_bounds(kind, g, eg):
    """Bounds of act and act' when g is off by eg: the slopes of silu and gelu are
    at most 1.13 and those of their derivatives at most 0.8; relu' jumps at 0."""
    a, _ = act(kind, g)
    ea = 1.2 * eg + 8 * U * (np.abs(a) + 1e-30)
    if kind == "relu":
        return ea, (np.abs(g) <= eg).astype(float)
    return ea, 0.8 * eg + 16 * U


def gated(x, wg, wu, kind):
    """g, u, h and their bounds before h is rounded."""
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a, _ = act(kind, g)
    ea, _ = act_bounds(kind, g, eg)
    h = a * u
    return g, eg, u, eu, h, ea * (np.abs(u) + eu) + np.abs(a) * eu + 4 * U * np.abs(h)


def ffn(x, wg, wu, wd, dy, kind, dtype):
    """{name: (value, bound)} of the gated block's outputs; dy may be None."""
    r = half(dtype)
    g, eg, u, eu, h, eh = gated(x, wg, wu, kind)
    eh = eh + r * (np.abs(h) + eh)
    y, ey = product(h, wd)
    ey = ey + eh @ np.abs(wd).T
    out = {"y": (y, ey + r * (np.abs(y) + ey))}
    if dy is None:
        return out
    a, da = act(kind, g)
    ea, eda = act_bounds(kind, g, eg)
    dh, edh = product(dy, wd.T)
    dg, du = dh * u * da, dh * a
    edg = edh * np.abs(u * da) + (np.abs(dh) + edh) * (eu * (np.abs(da) + eda) + np.abs(u) * eda)
    edu = edh * np.abs(a) + (np.abs(dh) + edh) * ea
    edg += (r + 8 * U) * (np.abs(dg) + edg)
    edu += (r + 8 * U) * (np.abs(du) + edu)

    def put(name, terms):
        v = sum(p @ q for p, _, q, _ in terms)
        n = sum(p.shape[1] for p, _, _, _ in terms)
        s = sum(np.abs(p) @ np.abs(q) for p, _, q, _ in terms)
        e = 8 * math.sqrt(n + 16) * U * s
        e = e + sum(ep @ (np.abs(q) + eq) + np.abs(p) @ eq for p, ep, q, eq in terms)
        out[name] = (v, e + r * (np.abs(v) + e))

    z = np.zeros_like
    put("dx", [(dg, edg, wg, z(wg)), (du, edu, wu, z(wu))])
    put("dw_gate", [(dg.T, edg.T, x, z(x))])
    put("dw_up", [(du.T, edu.T, x, z(x))])
    put("dw_down", [(dy.T, z(dy.T), h, eh)])
    return out


# --- layer norm ------------------------------------------------------------
def norm(x, w, b, eps, dy, dtype):
    """{name: (value, bound)}; w, b, dy may be None."""
    rows, cols = x.shape
    r = half(dtype)
    w = np.ones(cols) if w is None else w
    b = np.zeros(cols) if b is None else b
    mean = x.mean(1, keepdims=True)
    xc = x - mean
    var = (xc * xc).mean(1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    z = xc * rstd
    n = 8 * math.sqrt(cols + 16) * U
    em = n * np.abs(x).mean(1, keepdims=True)
    exc = em + 2 * U * np.abs(x)
    # a mean that is off by em adds em^2 to the variance, the rounded x - mean 2 U |x| each
    evar = n * var + em * em + 2 * (np.abs(xc) * exc).mean(1, keepdims=True)
    ers = rstd * np.minimum(1.0, 0.5 * evar / (var + eps) + 8 * U)
    ez = exc * rstd + np.abs(xc) * ers + exc * ers + 4 * U * np.abs(z)
    y = z * w + b
    ey = ez * np.abs(w) + 4 * U * (np.abs(z * w) + np.abs(b))
    out = {"y": (y, ey + r * (np.abs(y) + ey)), "mean": (mean[:, 0], em[:, 0] + 4 * U * np.abs(mean[:, 0])),
           "rstd": (rstd[:, 0], ers[:, 0] + 4 * U * rstd[:, 0])}
    if dy is None:
        return out
    p = dy * w
    m1, m2 = p.mean(1, keepdims=True), (p * z).mean(1, keepdims=True)
    am1 = np.abs(p).mean(1, keepdims=True)
    am2 = np.abs(p * z).mean(1, keepdims=True)
    em1 = (n + 4 * U) * am1
    em2 = (n + 4 * U) * am2 + (np.abs(p) * ez).mean(1, keepdims=True)
    d = p - m1 - z * m2
    ed = 8 * U * (np.abs(p) + am1 + np.abs(z) * am2) + em1 + np.abs(z) * em2 + ez * (np.abs(m2) + em2)
    dx = rstd * d
    edx = (rstd + ers) * ed + ers * np.abs(d)
    out["dx"] = (dx, edx + r * (np.abs(dx) + edx))
    k = 8 * math.sqrt(rows + 16) * U
    dw, db = (dy * z).sum(0), dy.sum(0)
    edw = k * np.abs(dy * z).sum(0) + (np.abs(dy) * ez).sum(0)
    edb = k * np.abs(dy).sum(0)
    out["dweight"] = (dw, edw + r * (np.abs(dw) + edw))
    out["dbias"] = (db, edb + r * (np.abs(db) + edb))
    return out
