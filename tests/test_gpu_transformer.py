"""The torch-tensor calls of the transformer-layer operators, and the example that runs them together, against
autograd in fp64."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

from activation_backward_gb300 import transformer as tr
from activation_backward_gb300 import inputs
from activation_backward_gb300.layer import DeviceLayer
from oracle import transformer as T

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_layer_norm_round_trip_on_views(cuda_lib):
    big = torch.randn(6, 10, 3, 96, device="cuda", dtype=torch.bfloat16)
    x = big[:, :, 1]  # rows 288 apart
    gamma, beta = torch.rand(96, device="cuda") + 0.5, torch.randn(96, device="cuda")
    y, mean, rstd = tr.layer_norm(x, gamma, beta)
    want = T.layernorm_forward(x.double().cpu().numpy().reshape(60, 96), gamma.cpu(), beta.cpu(), 1e-5)
    assert y.shape == x.shape and np.allclose(y.double().cpu().numpy().reshape(60, 96), want[0], rtol=2.0 ** -8, atol=1e-5)
    dy, res = torch.randn_like(y), torch.randn_like(y)
    dx, dg, db = tr.layer_norm_backward(x, dy, gamma, mean, rstd, residual=res)
    a = [t.double().cpu().numpy().reshape(60, 96) for t in (x, dy, res)]
    w = T.layernorm_backward(a[0], a[1], gamma.cpu(), mean.cpu(), rstd.cpu(), a[2])
    assert np.allclose(dx.double().cpu().numpy().reshape(60, 96), w[0], rtol=2.0 ** -8, atol=1e-4)
    dg2, db2 = dg.clone(), db.clone()
    tr.layer_norm_backward(x, dy, gamma, mean, rstd, dgamma=dg2, dbeta=db2)
    assert np.allclose(dg2.double().cpu().numpy(), 2 * w[1], atol=1e-3) and np.allclose(db2.cpu().numpy(), 2 * w[2], atol=1e-3)
    with pytest.raises(ValueError):
        tr.layer_norm(big.transpose(2, 3))
    with pytest.raises(ValueError):
        tr.layer_norm_backward(x, dy[:5], gamma, mean, rstd)


def test_attention_backward_refuses_what_it_cannot_read(cuda_lib):
    q = torch.randn(1, 8, 2, 64, device="cuda", dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 8, device="cuda")
    with pytest.raises(ValueError):
        tr.attention_backward(q, q, q, q, lse.transpose(1, 2), q)
    with pytest.raises(ValueError):
        tr.attention_backward(q[0], q[0], q[0], q[0], lse[0], q[0])  # packed without starts
    with pytest.raises(ValueError):
        tr.attention_backward(q[0], q[0], q[0], q[0], lse[0], q[0], cu_q=torch.tensor([0, 8], device="cuda"))
    with pytest.raises(tr.B.CbaError):
        x = torch.randn(1, 8, 2, 60, device="cuda", dtype=torch.bfloat16)
        tr.attention_backward(x, x, x, x, lse, x)


def test_a_convolutions_weight_gradient_orthogonalised(cuda_lib):
    """The conv backward's dW, as the update of its weights."""
    dl = DeviceLayer(inputs.make_config(2, batch=2)[0])
    dl.run()
    dW = dl.dW.view(dl.geom.K, -1)
    O = tr.orthogonalize(dW, out_dtype=torch.float32)
    want = T.orthogonalize(dW.double().cpu().numpy())
    assert np.linalg.norm(O.double().cpu().numpy() - want) <= 8e-3 * np.linalg.norm(want)
    s = torch.linalg.svdvals(O.double())
    assert s.max() < 1.3 and s.median() > 0.6


def test_block_gradients_match_autograd(cuda_lib):
    """f16 gradients of the whole block against fp64 autograd of the same formulas: each of the about ten roundings
    between loss and gradient is 2^-11 relatively, of unrelated signs: 16 of them cover any one gradient's 2-norm."""
    ex = example()
    blk = ex.AttentionBlock(128, 4, torch.float16, seed=3)
    x = torch.randn(2, 49, 128, device="cuda").half()
    y, saved = blk.forward(x)
    dy = torch.randn_like(y)
    dx, g = blk.backward(dy, saved)
    p = {n: t.half().double().requires_grad_() for n, t in blk.w.items()}
    p["gamma"], p["beta"] = (t.double().requires_grad_() for t in (blk.gamma, blk.beta))
    xd = x.double().requires_grad_()
    mu = xd.mean(-1, keepdim=True)
    h = (xd - mu) / torch.sqrt(((xd - mu) ** 2).mean(-1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
    q, k, v = (h @ p["wqkv"]).view(2, 49, 3, 4, 32).unbind(2)
    a = torch.softmax(torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(32), -1)
    (xd + torch.einsum("bhij,bjhd->bihd", a, v).reshape(2, 49, 128) @ p["wo"]).backward(dy.double())
    for name, got, want in [("dx", dx, xd.grad)] + [(n, g[n], p[n].grad) for n in p]:
        assert (got.double() - want).norm() <= 16 * 2.0 ** -11 * want.norm(), name


def test_block_trains(cuda_lib):
    losses = example().train(12, batch=2, side=13)
    assert all(math.isfinite(v) for v in losses) and losses[-1] < 0.5 * losses[0]
