"""Query/key norms on the GPU for heads at the ends of the elements' range, against the 64-bit oracle.

Bars as of heads of order 1 (u = 2^-24, w the elements' unit roundoff): an output of the forward by (dim / 2 + 16) u of its
absolute terms, in which r counts dim / 2 + 4.  Here r may be as small as 2^-128, a number below fp32's normal ones that is
rounded to 2^-150: another 2^-22 = 4 u, which the 16 have room for (rsqrtf 4, the products by 1 / dim, r, gamma and the
angle 4, their sum 1).  dx by (2 dim + 32) u of its absolute terms, dgamma by (N + 2 dim + 32) u of N terms.  Outputs below
the normal numbers are rounded to half of the type's smallest one.
"""
import math

import numpy as np
import pytest
import torch

from activation_backward_gb300 import transformer as tr
from oracle import transformer as T

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF = torch.float32, torch.bfloat16
W, SMALLEST = {F32: U, BF: 2.0 ** -8}, {F32: 2.0 ** -149, BF: 2.0 ** -133}
# halves of a multiple of 16; of no multiple; part of a head; pairs (2j, 2j + 1); no rotation
KINDS = [(64, 64, False), (128, 128, False), (256, 256, False), (8, 8, False), (40, 40, False), (128, 64, False), (96, 96, True), (24, 0, False)]


def f8(t):
    return t.double().cpu().numpy()


def within(got, want, bar, what):
    bad = ~(np.abs(got - want) <= bar)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size}, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def turned(x, table, interleaved):
    """The sums of the absolute terms of the rotation, either way."""
    if table is None:
        return x
    n, i = table.shape[1], np.arange(table.shape[1])
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y, cos, sin = x.copy(), np.abs(table[:, None, :, 0]), np.abs(table[:, None, :, 1])
    y[..., a] = x[..., a] * cos + x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def check(q, dy, rot, interleaved, eps):
    """Both directions of q [tokens, heads, dim]."""
    n, _, dim = q.shape
    angle = np.random.default_rng(dim).uniform(-math.pi, math.pi, (n, rot // 2))
    table = torch.from_numpy(np.stack([np.cos(angle), np.sin(angle)], -1)).float().cuda() if rot else None
    gamma = torch.rand(dim, device="cuda") + 0.5
    w, low, at = W[q.dtype], SMALLEST[q.dtype], np.arange(n)
    x, t, gm = f8(q), None if table is None else f8(table), f8(gamma)
    kw = dict(gamma_q=gamma, table=table, interleaved=interleaved, eps=eps)

    def bar(terms, want, c):
        return c * U * terms * (1 + 2 * w) + 1.01 * w * np.abs(want) + low

    want = T.norm_rope_forward(x, gm, t, at, eps, True, interleaved)
    h = np.abs(T.norm_rope_forward(x, gm, None, None, eps))
    within(f8(tr.qk_norm_rope(q, None, **kw)[0]), want, bar(turned(h, t, interleaved), want, dim / 2 + 16), "y")

    dx, _, dgamma, _ = tr.qk_norm_rope_backward(q, None, dy, None, **kw)
    want, wg = T.norm_rope_backward(x, f8(dy), gm, t, at, eps, True, interleaved)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    norm, g = np.abs(x * r), turned(np.abs(f8(dy)), t, interleaved)
    terms = r * (g * gm + norm * (g * gm * norm).mean(-1, keepdims=True))
    assert np.abs(want).max() < 1e38  # no infinities asked for
    within(f8(dx), want, bar(terms, want, 2 * dim + 32), "dx")
    within(f8(dgamma), wg, (x.shape[0] * x.shape[1] + 2 * dim + 32) * U * (g * norm).sum((0, 1)) + 1e-30, "dgamma")


@pytest.mark.parametrize("dtype,big", [(F32, 3.3e38), (F32, 1e38), (F32, 2e19), (BF, 3.3e38), (BF, 1e38)])
@pytest.mark.parametrize("dim,rot,interleaved", KINDS)
def test_heads_near_the_largest_number(cuda_lib, dim, rot, interleaved, dtype, big):
    """Elements of either sign between a quarter of `big` and `big`; beside them heads of order 1.  The gradients are
    large enough for dx to be normal numbers."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    q = torch.rand((9, 3, dim), generator=g, device="cuda") * 0.75 + 0.25
    q = q * torch.where(torch.rand(q.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    q[:, :2] *= big
    q = q.to(dtype)
    assert torch.isfinite(q).all()
    dy = (torch.randn(q.shape, generator=g, device="cuda") * 1e6).to(dtype)
    check(q, dy, rot, interleaved, 1e-6)
