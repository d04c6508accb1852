"""Training steps of a pre-norm attention block over a feature map, with the
library's layer norm, attention gradient and orthogonalised updates.

    y = x + attention(layer_norm(x) Wqkv) Wo

on the 26x26 positions of a 512-channel map.  The forward's products and its
softmax are plain torch (the library starts from forward outputs, as it does for
convolutions); every gradient between the loss and the weights' products, and the
update of the weights, is the library's.

    python examples/attention_block.py [--steps 20]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from activation_backward_gb300 import transformer as tr  # noqa: E402


class AttentionBlock:
    """The block's fp32 weights, their momenta, and its passes in 16 bits."""

    def __init__(self, channels, heads, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = dict(wqkv=(channels, 3 * channels), wo=(channels, channels))
        self.w = {n: torch.randn(s, generator=g, device="cuda") / math.sqrt(channels) for n, s in w.items()}
        self.m = {n: torch.zeros_like(t) for n, t in self.w.items()}
        self.gamma, self.beta = torch.ones(channels, device="cuda"), torch.zeros(channels, device="cuda")
        self.channels, self.heads, self.dim, self.dtype = channels, heads, channels // heads, dtype

    def forward(self, x):
        """y, and what the backward pass needs.  x [batch, positions, channels]."""
        b, n, c = x.shape
        h, mean, rstd = tr.layer_norm(x, self.gamma, self.beta)
        qkv = (h @ self.w["wqkv"].to(self.dtype)).view(b, n, 3, self.heads, self.dim)
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]  # views: the library takes their strides
        s = torch.einsum("bihd,bjhd->bhij", q.float(), k.float()) / math.sqrt(self.dim)
        lse = torch.logsumexp(s, -1)
        o = torch.einsum("bhij,bjhd->bihd", torch.exp(s - lse[..., None]), v.float()).to(self.dtype)
        y = x + (o.reshape(b, n, c) @ self.w["wo"].to(self.dtype))
        return y, (x, h, mean, rstd, q, k, v, o, lse)

    def backward(self, dy, saved):
        """dx and the gradients of wqkv, wo, gamma and beta."""
        x, h, mean, rstd, q, k, v, o, lse = saved
        b, n, c = x.shape
        rows = lambda t: t.reshape(b * n, -1)  # noqa: E731
        do = (dy @ self.w["wo"].to(self.dtype).t()).view(b, n, self.heads, self.dim)
        g = {"wo": (rows(o).t() @ rows(dy)).float()}
        dqkv = torch.stack(tr.attention_backward(q, k, v, o, lse, do), 2).reshape(b, n, 3 * c)
        g["wqkv"] = (rows(h).t() @ rows(dqkv)).float()
        dh = dqkv @ self.w["wqkv"].to(self.dtype).t()
        # the shortcut's delta joins the norm's in one pass
        dx, g["gamma"], g["beta"] = tr.layer_norm_backward(x, dh, self.gamma, mean, rstd, residual=dy)
        return dx, g

    def update(self, g, lr, momentum=0.95):
        """Muon: the matrices move along their orthogonalised momentum."""
        for name, w in self.w.items():
            m = self.m[name].mul_(momentum).add_(g[name])
            scale = math.sqrt(max(1.0, w.shape[0] / w.shape[1]))
            w.sub_(tr.orthogonalize(g[name] + momentum * m, scale=scale).float(), alpha=lr)
        self.gamma.sub_(g["gamma"], alpha=lr)
        self.beta.sub_(g["beta"], alpha=lr)


def train(steps, batch=8, side=26, channels=512, heads=8, lr=0.02, seed=0, dtype=torch.bfloat16):
    """The losses of `steps` steps towards the outputs of another block."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((batch, side * side, channels), generator=g, device="cuda").to(dtype)
    target = AttentionBlock(channels, heads, dtype, seed + 2).forward(x)[0]
    block, losses = AttentionBlock(channels, heads, dtype, seed), []
    for _ in range(steps):
        y, saved = block.forward(x)
        d = y.float() - target.float()
        losses.append(float(d.square().mean()))
        block.update(block.backward((2 * d / d.numel()).to(dtype), saved)[1], lr)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    for i, loss in enumerate(train(ap.parse_args().steps)):
        print(f"step {i}: loss {loss:.5f}")
