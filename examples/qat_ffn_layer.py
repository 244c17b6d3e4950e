"""A pre-norm gated feed-forward layer trained through fake quantization, then
served from 4-bit codes:

    y = x + down(act(gate(n)) * up(n)),  n = layer_norm(x)

Training keeps float32 masters.  Each step runs the layer on their int8 fake-quant
views (bfloat16), takes the gradients of the block and of the norm, passes the
weights' through the straight-through estimator and updates masters and views with
the fused optimizer step.  Serving quantizes the masters to 4-bit groups once and
runs single tokens from the codes.

    python examples/qat_ffn_layer.py [--steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fake_quant_numerics_gb300 as fq  # noqa: E402


class Layer:
    """The layer's masters, their views and the optimizer state."""

    def __init__(self, dim, hidden, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) * cols ** -0.5).to(device)

        self.masters = [weight(hidden, dim), weight(hidden, dim), weight(dim, hidden)]
        self.moments = [(torch.zeros_like(w), torch.zeros_like(w)) for w in self.masters]
        self.norm = [torch.ones(dim, device=device), torch.zeros(dim, device=device)]
        self.views, self.masks, self.t = [], [], 0
        for w in self.masters:
            r = fq.fake_quant_int(w, 8, "symmetric", "tensor")
            self.views.append(r.y.to(torch.bfloat16))
            self.masks.append(r.mask)

    def step(self, x, target, lr=2e-3):
        """One training step on the mean squared error; returns the loss."""
        self.t += 1
        nw, nb = (t.to(torch.bfloat16) for t in self.norm)
        n = fq.layer_norm(x, nw, nb)
        r = fq.gated_ffn(n.y, *self.views, activation="silu", save=True)
        diff = x.float() + r.y.float() - target.float()
        dy = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        dn, *grads = fq.gated_ffn_backward(dy, n.y, *self.views, r, activation="silu")
        _, dnw, dnb = fq.layer_norm_backward(dn, x, nw, n.mean, n.rstd)
        for i, grad in enumerate(grads):
            grad = fq.fake_quant_backward(grad.float(), self.masks[i])
            view = fq.optimizer_step(self.masters[i], grad, *self.moments[i], self.t, lr,
                                     target="int8", want_mask=True)
            self.views[i], self.masks[i] = view.view.to(torch.bfloat16), view.mask
        for p, grad in zip(self.norm, (dnw, dnb)):
            p -= lr * grad.float()
        return float((diff * diff).mean())

    def forward(self, x):
        """The layer on the training views."""
        n = fq.layer_norm(x, *(t.to(x.dtype) for t in self.norm))
        return x + fq.gated_ffn(n.y, *self.views, activation="silu").y

    def quantize(self, group=32):
        """The masters as 4-bit codes with a scale per group."""
        out = []
        for w in self.masters:
            r = fq.fake_quant_int(w, 4, "symmetric", "group", group)
            out.append(fq.weight4(r.codes, r.scale, *w.shape, "group", group))
        return out

    def serve(self, x, codes):
        """The layer from 4-bit codes, for a few tokens."""
        n = fq.layer_norm(x, *(t.to(x.dtype) for t in self.norm))
        return x + fq.gated_ffn4(n.y, *codes, activation="silu")


def main(steps=60, dim=256, hidden=768, tokens=512):
    layer = Layer(dim, hidden)
    teacher = Layer(dim, hidden, seed=1)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(tokens, dim, generator=g).cuda().to(torch.bfloat16)
    target = teacher.forward(x)
    losses = [layer.step(x, target) for _ in range(steps)]
    codes = layer.quantize()
    trained, served = layer.forward(x[:4]).float(), layer.serve(x[:4], codes).float()
    off = float((served - trained).norm() / trained.norm())
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps; "
          f"served from 4-bit codes within {off:.3f} of the trained layer")
    return losses, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    main(ap.parse_args().steps)
