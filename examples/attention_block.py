"""Training steps of a pre-norm attention block over a feature map, with the
library's layer norm, attention, query/key norms with rotation, dropout and
orthogonalised updates.

    y = x + dropout(attention(layer_norm(x) Wqkv) Wo)

on the 26x26 positions of a 512-channel map.  The products with the weights are plain
torch; everything between them, every gradient and the update of the weights is the
library's.  With --qk-norm the heads' queries and keys are normed and turned by their
positions first; with --dropout P a share of the block's output is dropped.

    python examples/attention_block.py [--steps 20] [--qk-norm] [--dropout 0.1]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from activation_backward_gb300 import transformer as tr  # noqa: E402


def rotary_table(positions, dim, base=10000.0):
    """cos and sin of every position's dim / 2 angles, fp32 [positions, dim / 2, 2]; the angles in fp64, as
    those of far positions need."""
    freq = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], -1).float().cuda()


class AttentionBlock:
    """The block's fp32 weights, their momenta, and its passes in 16 bits."""

    def __init__(self, channels, heads, dtype=torch.bfloat16, seed=0, causal=False, qk_norm=False, p=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = dict(wqkv=(channels, 3 * channels), wo=(channels, channels))
        self.w = {n: torch.randn(s, generator=g, device="cuda") / math.sqrt(channels) for n, s in w.items()}
        self.m = {n: torch.zeros_like(t) for n, t in self.w.items()}
        self.gamma, self.beta = torch.ones(channels, device="cuda"), torch.zeros(channels, device="cuda")
        self.channels, self.heads, self.dim, self.dtype = channels, heads, channels // heads, dtype
        self.causal, self.qk_norm, self.p, self.seed, self.drawn = causal, qk_norm, p, seed, 0
        self.gq, self.gk = (torch.ones(self.dim, device="cuda") for _ in range(2))
        self.table = None

    def forward(self, x):
        """y, and what the backward pass needs.  x [batch, positions, channels]."""
        b, n, c = x.shape
        h, mean, rstd = tr.layer_norm(x, self.gamma, self.beta)
        qkv = (h @ self.w["wqkv"].to(self.dtype)).view(b, n, 3, self.heads, self.dim)
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]  # views: the library takes their strides
        heads = q, k
        if self.qk_norm:
            if self.table is None or self.table.shape[0] < n:
                self.table = rotary_table(n, self.dim)
            q, k = tr.qk_norm_rope(q, k, self.gq, self.gk, self.table)
        o, lse = tr.attention(q, k, v, causal=self.causal)
        z = o.reshape(b, n, c) @ self.w["wo"].to(self.dtype)
        offset = self.drawn
        if self.p > 0:
            self.drawn += (z.numel() + 3) // 4  # the next step's counters begin behind this one's
            y = tr.dropout(z, self.p, self.seed, offset, residual=x)
        else:
            y = x + z
        return y, (x, h, mean, rstd, heads, q, k, v, o, lse, offset)

    def backward(self, dy, saved):
        """dx and the gradients of wqkv, wo, gamma and beta (and gq and gk)."""
        x, h, mean, rstd, heads, q, k, v, o, lse, offset = saved
        b, n, c = x.shape
        rows = lambda t: t.reshape(b * n, -1)  # noqa: E731
        dz = tr.dropout(dy, self.p, self.seed, offset) if self.p > 0 else dy  # the same mask again
        do = (dz @ self.w["wo"].to(self.dtype).t()).view(b, n, self.heads, self.dim)
        g = {"wo": (rows(o).t() @ rows(dz)).float()}
        dq, dk, dv = tr.attention_backward(q, k, v, o, lse, do, causal=self.causal)
        if self.qk_norm:
            dq, dk, g["gq"], g["gk"] = tr.qk_norm_rope_backward(*heads, dq, dk, self.gq, self.gk, self.table)
        dqkv = torch.stack([dq, dk, dv], 2).reshape(b, n, 3 * c)
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
        for name in ("gamma", "beta", "gq", "gk"):
            if name in g:
                getattr(self, name).sub_(g[name], alpha=lr)


def train(steps, batch=8, side=26, channels=512, heads=8, lr=0.02, seed=0, dtype=torch.bfloat16, **kw):
    """The losses of `steps` steps towards the outputs of another block."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((batch, side * side, channels), generator=g, device="cuda").to(dtype)
    target = AttentionBlock(channels, heads, dtype, seed + 2).forward(x)[0]
    block, losses = AttentionBlock(channels, heads, dtype, seed, **kw), []
    for _ in range(steps):
        y, saved = block.forward(x)
        d = y.float() - target.float()
        losses.append(float(d.square().mean()))
        block.update(block.backward((2 * d / d.numel()).to(dtype), saved)[1], lr)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description="Training steps of an attention block.")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--qk-norm", action="store_true")
    ap.add_argument("--dropout", type=float, default=0.0)
    args = ap.parse_args()
    for i, loss in enumerate(train(args.steps, qk_norm=args.qk_norm, p=args.dropout)):
        print(f"step {i}: loss {loss:.5f}")
