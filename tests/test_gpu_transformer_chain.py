"""Layer norm, query/key norms with rotation, attention and dropout run together as a block does, forward and backward:
against autograd in fp64, captured into a graph, and on packed documents."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

from activation_backward_gb300 import transformer as tr
from oracle import transformer as T

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rotated(x, table):
    """x [b, n, h, d] turned in pairs (j, j + d / 2), in its own type."""
    d = x.shape[-1] // 2
    cos, sin = (table[: x.shape[1], :, i].to(x.dtype)[None, :, None] for i in (0, 1))
    a, b = x[..., :d], x[..., d:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


@pytest.mark.parametrize("causal", [False, True])
def test_block_gradients_match_autograd(cuda_lib, causal):
    """f16 gradients of the whole block against fp64 autograd of the same formulas, with the oracle's mask.  Between loss
    and gradient lie about sixteen roundings (norm, projection, heads' norm, P, o, projection, dropout, and their
    gradients) of 2^-11 relatively, of unrelated signs: 24 of them cover any one gradient's 2-norm."""
    ex = example()
    blk = ex.AttentionBlock(128, 4, torch.float16, seed=3, causal=causal, qk_norm=True, p=0.25)
    blk.gq, blk.gk = (torch.rand(32, device="cuda") + 0.5 for _ in range(2))
    blk.drawn = 1000
    x = torch.randn(2, 49, 128, device="cuda").half()
    y, saved = blk.forward(x)
    assert blk.drawn == 1000 + 2 * 49 * 128 // 4
    dy = torch.randn_like(y)
    dx, g = blk.backward(dy, saved)
    p = {n: t.half().double().requires_grad_() for n, t in blk.w.items()}
    for n in ("gamma", "beta", "gq", "gk"):
        p[n] = getattr(blk, n).double().requires_grad_()
    xd = x.double().requires_grad_()
    mu = xd.mean(-1, keepdim=True)
    h = (xd - mu) / torch.sqrt(((xd - mu) ** 2).mean(-1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
    q, k, v = (h @ p["wqkv"]).view(2, 49, 3, 4, 32).unbind(2)
    q, k = (rotated(t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * p[n], blk.table) for t, n in ((q, "gq"), (k, "gk")))
    s = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(32)
    if causal:
        s = s.masked_fill(~torch.ones(49, 49, device="cuda").bool().tril(), -math.inf)
    z = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v).reshape(2, 49, 128) @ p["wo"]
    keep = torch.from_numpy(T.dropout_keep((2, 49, 128), 0.25, 3, 1000)).cuda()
    want = xd + torch.where(keep, z / 0.75, 0.0)
    assert (y.double() - want).norm() <= 24 * 2.0 ** -11 * want.norm()
    want.backward(dy.double())
    for name, got, w in [("dx", dx, xd.grad)] + [(n, g[n], p[n].grad) for n in p]:
        assert (got.double() - w).norm() <= 24 * 2.0 ** -11 * w.norm(), name


def test_block_runs_with_everything_on(cuda_lib):
    losses = example().train(3, batch=2, side=13, qk_norm=True, p=0.1)
    assert all(math.isfinite(v) for v in losses)


def chain(x, gamma, qkv_of, gq, gk, table, step, cu=None):
    """A block's forward and backward by the library's calls alone (no products with weights)."""
    h, mean, rstd = tr.layer_norm(x, gamma)
    q, k, v = qkv_of(h)
    yq, yk = tr.qk_norm_rope(q, k, gq, gk, table)
    o, lse = tr.attention(yq, yk, v, causal=True, cu_q=cu)
    y = tr.dropout(o, 0.25, 9, offset=64, residual=q.contiguous(), step=step)
    do = tr.dropout(y, 0.25, 9, offset=64, step=step)
    dq, dk, dv = tr.attention_backward(yq, yk, v, o, lse, do, causal=True, cu_q=cu)
    dq, dk, dgq, dgk = tr.qk_norm_rope_backward(q, k, dq, dk, gq, gk, table)
    dh = torch.cat([dq, dk, dv], -2).reshape(x.shape)
    dx, dg, _ = tr.layer_norm_backward(x, dh, gamma, mean, rstd)
    return y, o, lse, dx, dg, dgq, dgk


def inputs(shape, dtype=torch.bfloat16):
    x = torch.randn(*shape, 4 * 64, device="cuda").to(dtype)
    qkv_of = lambda h: (lambda t: (t[..., :2, :], t[..., 2:3, :], t[..., 3:, :]))(h.view(*shape, 4, 64))  # noqa: E731
    gamma = torch.rand(256, device="cuda") + 0.5
    gq, gk = (torch.rand(64, device="cuda") + 0.5 for _ in range(2))
    return x, gamma, qkv_of, gq, gk, example().rotary_table(400, 64), torch.zeros(1, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("packed", [False, True])
def test_captured_and_replayed(cuda_lib, packed):
    """A graph of the whole chain, while its eager results live, on new inputs and a moved step, on another stream."""
    shape = (300,) if packed else (2, 150)
    a = inputs(shape)
    cu = torch.tensor([0, 120, 120, 300], dtype=torch.int32, device="cuda") if packed else None
    chain(*a, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(*a, cu)
        a[-1].add_(300 * 2 * 64 // 4)
    a[-1].zero_()
    side = torch.cuda.Stream()
    for turn in range(2):
        a[0].copy_(torch.randn_like(a[0].float()).to(a[0].dtype))
        before = a[-1].clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        got = [t.clone() for t in out]
        for g, w in zip(got, chain(*a[:-1], before, cu)):
            assert torch.equal(g, w)


def test_packed_documents_are_the_documents_alone(cuda_lib):
    """Each document of a packed row gives what it gives by itself (positions begin anew: by `pos`)."""
    x, gamma, qkv_of, gq, gk, table, _ = inputs((300,))
    cu = torch.tensor([0, 120, 300], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(120), torch.arange(180)]).int().cuda()
    q, k, v = qkv_of(tr.layer_norm(x, gamma)[0])
    yq, yk = tr.qk_norm_rope(q, k, gq, gk, table, pos)
    o, lse = tr.attention(yq, yk, v, causal=True, cu_q=cu, max_q=180, max_k=180)
    for s, e in ((0, 120), (120, 300)):
        aq, ak = tr.qk_norm_rope(q[s:e], k[s:e], gq, gk, table)
        assert torch.equal(aq, yq[s:e]) and torch.equal(ak, yk[s:e])
        ao, al = tr.attention(aq[None], ak[None], v[None, s:e], causal=True)
        w = np.abs(ao.double().cpu().numpy()[0])
        assert (np.abs((ao[0].double() - o[s:e].double()).cpu().numpy()) <= 2.0 ** -7 * w + 2.0 ** -7 * np.abs(v[s:e].double().cpu().numpy()).max()).all()
        assert torch.allclose(al[0], lse[:, s:e], atol=1e-4)
