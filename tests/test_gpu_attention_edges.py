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
