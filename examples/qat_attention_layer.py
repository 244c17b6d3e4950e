"""The attention half of a layer served from codes: 4-bit projections and a quantized
paged key-value cache.

    q, k, v = split(qkv(x));  q, k = rotate(norm(q), norm(k));  cache <- k, v
    y = x + out(attention(q, cache))

Every decoding step runs a batch of sequences one token further; the whole step is
captured into a CUDA graph once and replayed.  The same tokens are served from a cache
in each format, and the outputs compared with those of the bf16 cache.

    python examples/qat_attention_layer.py [--steps 64]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fake_quant_numerics_gb300 as fq  # noqa: E402


class Layer:
    """Projections as 4-bit codes, norm weights, and one cache with its page table."""

    def __init__(self, dim, heads, kv_heads, head_dim, batch, longest, form, scheme="symmetric", page=16, group=64,
                 seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def codes(rows, cols):
            w = (torch.randn(rows, cols, generator=g) * cols ** -0.5).to(device)
            r = fq.fake_quant_int(w, 4, "symmetric", "group", group)
            return fq.weight4(r.codes, r.scale, rows, cols, "group", group)

        self.heads, self.kv_heads, self.head_dim, self.page = heads, kv_heads, head_dim, page
        self.qkv = codes((heads + 2 * kv_heads) * head_dim, dim)
        self.out = codes(dim, heads * head_dim)
        self.q_norm, self.k_norm = (torch.ones(head_dim, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.turns = fq.rope_turns(fq.rope_frequencies(head_dim), device)
        pages = -(-longest // page)
        self.cache = fq.kv_cache(batch * pages, kv_heads, page, head_dim, form, scheme, device)
        # any page may hold any part of any sequence
        order = torch.randperm(batch * pages, generator=g).to(torch.int32)
        self.table = order.view(batch, pages).to(device)
        self.positions = torch.zeros(batch, dtype=torch.int64, device=device)

    def step(self, x):
        """One token of each sequence, x [batch, dim]."""
        batch, hq, hk, d = len(x), self.heads, self.kv_heads, self.head_dim
        qkv = fq.linear4(x, self.qkv).view(batch, hq + 2 * hk, d)
        r = fq.head_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], self.positions, self.turns, self.q_norm, self.k_norm)
        page = self.table.gather(1, (self.positions // self.page)[:, None])[:, 0].long()
        fq.kv_write(self.cache, r.k, qkv[:, hq + hk:], page * self.page + self.positions % self.page)
        self.positions += 1
        y = fq.kv_attention(r.q, self.cache, self.table, self.positions.int()).y
        return x + fq.linear4(y.view(batch, hq * d), self.out)


def serve(xs, form, scheme="symmetric", **sizes):
    """The layer's outputs for xs [steps, batch, dim], each step a replay of one graph."""
    layer = Layer(xs.shape[2], batch=xs.shape[1], longest=len(xs), form=form, scheme=scheme, **sizes)
    x = xs[0].clone()
    layer.step(x)  # first use outside the graph
    layer.positions.zero_()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = layer.step(x)
    torch.cuda.current_stream().wait_stream(stream)
    layer.positions.zero_()
    out = []
    for t in xs:
        x.copy_(t)
        graph.replay()
        out.append(y.clone())
    return torch.stack(out)


def main(steps=64, dim=512, heads=8, kv_heads=2, head_dim=64, batch=3):
    g = torch.Generator().manual_seed(3)
    xs = torch.randn(steps, batch, dim, generator=g).cuda().to(torch.bfloat16)
    sizes = dict(heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    want = serve(xs, "bf16", **sizes).float()
    off = {}
    for form, scheme in (("int8", "symmetric"), ("e4m3", "symmetric"), ("int4", "affine")):
        got = serve(xs, form, scheme, **sizes).float()
        off[form] = float((got - want).norm() / want.norm())
        print(f"{form:5s} cache: outputs within {off[form]:.4f} of the bf16 cache's")
    return want, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=64)
    main(ap.parse_args().steps)
