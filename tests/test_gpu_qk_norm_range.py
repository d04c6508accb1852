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
    eps = float(np.float32(eps))
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
    assert np.abs(want).max() < 1e38  # no infinities asked for, but where r itself is past fp32's numbers
    got, past = f8(dx), np.broadcast_to(r > 3.4e38, want.shape)
    assert not np.isfinite(got[past]).any()
    within(np.where(past, want, got), want, bar(terms, want, 2 * dim + 32), "dx")
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


@pytest.mark.parametrize("dtype,size,eps", [(F32, 1e-18, 0.0), (F32, 1e-25, 0.0), (F32, 1e-38, 0.0), (F32, 1e-42, 0.0), (F32, 3e-45, 0.0),
                                            (F32, 1e-20, 1e-40), (F32, 1e-25, 1e-45), (F32, 1e-17, 1e-31), (F32, 1e-40, 1e-30),
                                            (BF, 1e-25, 0.0), (BF, 1e-37, 0.0), (BF, 1e-39, 0.0), (BF, 1e-20, 1e-38)])
@pytest.mark.parametrize("dim,rot,interleaved", KINDS)
def test_heads_of_small_numbers(cuda_lib, dim, rot, interleaved, dtype, size, eps):
    """Squares that vanish in fp32, with no eps or one as small; heads of order 1 in the same warps.  The gradients are small
    enough for dx, 1 / size times as large, to stay below 1e38; where 1 / size does not, dx has no finite value."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    q, dy = (torch.randn((9, 3, dim), generator=g, device="cuda") for _ in range(2))
    q[..., 0] = 2.0  # (no head of zeros alone)
    q[:, 1:], dy[:, 1:] = q[:, 1:] * size, dy[:, 1:] * min(1.0, size * 1e36)
    check(q.to(dtype), dy.to(dtype), rot, interleaved, eps)


def test_heads_of_zeros_without_eps_are_0_over_0(cuda_lib):
    """NaN, as by the formula, in their own rows alone."""
    q, dy = (torch.randn((5, 4, 64), device="cuda") for _ in range(2))
    y, dx = tr.qk_norm_rope(q, None, eps=0.0)[0], tr.qk_norm_rope_backward(q, None, dy, None, eps=0.0)[0]
    p = q.clone()
    p[2, 1] = 0
    y2, dx2 = tr.qk_norm_rope(p, None, eps=0.0)[0], tr.qk_norm_rope_backward(p, None, dy, None, eps=0.0)[0]
    keep = torch.ones(5, 4, dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.isnan(y2[2, 1]).all() and torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
