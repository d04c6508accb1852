"""Transformer operators on tensors of more than 2^31 elements: what lies past 32-bit offsets comes out as it would alone."""
import numpy as np
import pytest
import torch

from activation_backward_gb300 import transformer as tr
from oracle import transformer as T

from .test_gpu_attention import compare, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_layer_norm(cuda_lib):
    rows, cols = 1_100_000, 2048
    x = torch.randn(rows, cols, device="cuda", dtype=BF)
    dy = torch.randn(rows, cols, device="cuda", dtype=BF)
    gamma = torch.rand(cols, device="cuda") + 0.5
    y, mean, rstd = tr.layer_norm(x, gamma)
    dx, dgamma, dbeta = tr.layer_norm_backward(x, dy, gamma, mean, rstd, residual=dy)
    for part in (slice(0, 3000), slice(rows - 3000, rows)):
        a, b = x[part].contiguous(), dy[part].contiguous()
        y2, mean2, rstd2 = tr.layer_norm(a, gamma)
        assert torch.equal(y[part], y2) and torch.equal(mean[part], mean2) and torch.equal(rstd[part], rstd2)
        assert torch.equal(dx[part], tr.layer_norm_backward(a, b, gamma, mean2, rstd2, residual=b)[0])
    # sums of 1.1 million terms of order 1: fp32 partial sums over rows, each within 2^-24 of the absolute terms' sum times
    # their number in a chain (at most 4096 rows, then 304 partial sums)
    db, dg, size = (torch.zeros(cols, device="cuda", dtype=torch.float64) for _ in range(3))
    for i in range(0, rows, 50_000):
        d = dy[i:i + 50_000].double()
        h = (x[i:i + 50_000].double() - mean[i:i + 50_000, None]) * rstd[i:i + 50_000, None]
        db += d.sum(0)
        dg += (d * h).sum(0)
        size += torch.maximum(d.abs(), (d * h).abs()).sum(0)
    bar = 4400 * 2.0 ** -24 * size
    assert torch.all((dbeta.double() - db).abs() <= bar) and torch.all((dgamma.double() - dg).abs() <= bar)


def test_attention(cuda_lib):
    """Packed sequences, the last ones at the end of 2.3e9 elements."""
    heads, dim, length, n = 16, 128, 64, 17_500
    total = length * n
    q, k, v, o, do = (torch.zeros(total, heads, dim, device="cuda", dtype=BF) for _ in range(5))
    lse = torch.zeros(heads, total, device="cuda")
    cu = torch.arange(0, total + 1, length, device="cuda", dtype=torch.int32)
    rng, kept = np.random.default_rng(5), {}
    for s in (0, n // 2, n - 1):
        kept[s] = make(rng, 1, length, length, heads, heads, dim, BF, "bshd", 0.1, True)
        at = slice(s * length, (s + 1) * length)
        for t, own in zip((q, k, v, o, do), (kept[s][i] for i in (0, 1, 2, 3, 5))):
            t[at] = own[0]
        lse[:, at] = kept[s][4][0]
    assert q.numel() > 1 << 31
    outs = tr.attention_backward(q, k, v, o, lse, do, causal=True, scale=0.1, cu_q=cu, check=True)
    for s, args in kept.items():
        compare(args, [g[None, s * length:(s + 1) * length] for g in outs], 0.1, True, BF)
    for g in outs:  # everything else had do = 0
        assert torch.count_nonzero(g[length:n // 2 * length]) == 0 and torch.count_nonzero(g[(n // 2 + 1) * length:-length]) == 0


def test_orthogonalize(cuda_lib):
    batch, rows, cols = 1100, 1000, 2000
    G = torch.zeros(batch, rows, cols, device="cuda", dtype=BF)
    for i in (0, batch // 2, batch - 1):
        G[i] = torch.randn(rows, cols, device="cuda").to(BF)
    assert G.numel() > 1 << 31
    out = tr.orthogonalize(G, check=True)
    for i in (0, batch - 1):
        want = T.orthogonalize(G[i].double().cpu().numpy())
        assert np.linalg.norm(out[i].double().cpu().numpy() - want) <= (8e-3 + 2.0 ** -9) * np.linalg.norm(want)
    assert torch.count_nonzero(out[1:batch // 2]) == 0 and torch.count_nonzero(out[batch // 2 + 1:-1]) == 0
    # the same matrix alone takes other tiles: its bits may differ, its values not
    one = tr.orthogonalize(G[batch // 2], check=True)
    assert (one.float() - out[batch // 2].float()).norm() <= 8e-3 * one.float().norm()
