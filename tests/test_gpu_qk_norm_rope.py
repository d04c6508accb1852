"""Query/key norms with rotation on the GPU against the 64-bit oracle, element by element.

Bars, from the arithmetic.  u = 2^-24 of fp32, w: unit roundoff of the elements (u, 2^-11 f16, 2^-8 bf16).  r is off by
(dim / 2 + 4) u relatively (a sum of dim squares under a root), a product or sum by u: an output of the forward, (x_a cos -
x_b sin) r gamma, by C u (|x_a cos| + |x_b sin|) r |gamma| with C = dim / 2 + 16, and its rounding w.  In the backward g =
R^T dy is off by 2 u of its absolute terms G, dx = r (w - n mean(w n)) by C' u r (|W| + |n| mean |W n|) with W = G |gamma|
and C' = 2 dim + 32 (the mean's dim terms, r twice).  dgamma sums N = tokens x heads terms: (N + C') u of sum G |n|.
"""
import math

import numpy as np
import pytest
import torch

import activation_backward_gb300 as cba
from activation_backward_gb300 import transformer as tr
from oracle import transformer as T

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF = torch.float32, torch.float16, torch.bfloat16
W = {F32: U, F16: 2.0 ** -11, BF: 2.0 ** -8}
EPS = 1e-6


def f8(t):
    return None if t is None else t.double().cpu().numpy()


def absolute(x, table, pos, interleaved):
    """The sums of the absolute terms of the rotation, either way."""
    return np.abs(x) if table is None else _abs_rotate(np.abs(x), np.abs(table), pos, interleaved)


def _abs_rotate(x, table, pos, interleaved):
    n = table.shape[1]
    row = table[np.clip(pos, 0, table.shape[0] - 1)][:, None]
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y = x.copy()
    y[..., a] = x[..., a] * row[..., 0] + x[..., b] * row[..., 1]
    y[..., b] = x[..., a] * row[..., 1] + x[..., b] * row[..., 0]
    return y


def check(got, want, bar, what):
    got = f8(got).reshape(want.shape)
    bad = ~(np.abs(got - want) <= bar)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} past the bar, worst "
                           f"{np.max((np.abs(got - want) / np.maximum(bar, 1e-300))[bad]):.3g}, first at {np.argwhere(bad)[0]}")


def own_rounding(y, dtype):
    return 1.01 * W[dtype] * np.abs(y) + (2.0 ** -25 if dtype == F16 else 2.0 ** -149)


def flat(t):
    return f8(t).reshape(-1, *t.shape[-2:])


def check_forward(x, y, gamma, table, pos, norm, interleaved, what):
    a = flat(x)
    dim = a.shape[-1]
    want = T.norm_rope_forward(a, f8(gamma), f8(table), pos, EPS, norm, interleaved)
    h = np.abs(T.norm_rope_forward(a, f8(gamma), None, None, EPS, norm))
    bar = (dim / 2 + 16) * U * absolute(h, f8(table), pos, interleaved)
    check(y, want, bar * (1 + 2 * W[x.dtype]) + own_rounding(want, x.dtype), what)


def check_backward(x, dy, dx, dgamma, gamma, table, pos, norm, interleaved, what):
    a, b = flat(x), flat(dy)
    dim = a.shape[-1]
    want, wg = T.norm_rope_backward(a, b, f8(gamma), f8(table), pos, EPS, norm, interleaved)
    G = absolute(b, f8(table), pos, interleaved)
    if not norm:
        check(dx, want, 4 * U * G + own_rounding(want, x.dtype), what)
        return
    r = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + EPS)
    n, gw = np.abs(a * r), G * (1 if gamma is None else np.abs(f8(gamma)))
    bar = (2 * dim + 32) * U * r * (gw + n * (gw * n).mean(-1, keepdims=True))
    check(dx, want, bar * (1 + 2 * W[x.dtype]) + own_rounding(want, x.dtype), what)
    if dgamma is not None:
        terms = a.shape[0] * a.shape[1]
        check(dgamma, wg, (terms + 2 * dim + 32) * U * (G * n).sum((0, 1)) + 1e-30, what + " gamma")


def make_table(positions, rot, seed=0):
    a = np.random.default_rng(seed).uniform(-math.pi, math.pi, (positions, rot // 2))
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1)).float().cuda()


def place(rng, shape, layout, dtype, scale=1.0):
    t = torch.from_numpy(rng.normal(size=shape) * scale).to("cuda", dtype)
    if layout == "bhsd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "wide":
        big = torch.full((*shape[:2], shape[2] + 2, shape[3] + 8), math.nan, device="cuda", dtype=dtype)
        big[:, :, 1:-1, 8:] = t
        return big[:, :, 1:-1, 8:]
    return t


def both(batch, n, hq, hk, dim, rot, dtype, param, interleaved=False, norm=True, layout="bshd", positions=None, with_pos=True, seed=0,
         gammas=True):
    rng = np.random.default_rng(seed)
    q, k, dyq, dyk = (place(rng, (batch, n, h, dim), layout, dtype, s) for h, s in ((hq, 1), (hk, 2), (hq, 0.1), (hk, 0.1)))
    gq, gk = ((torch.rand(dim, device="cuda") + 0.5).to(param) if norm and gammas else None for _ in range(2))
    positions = positions or n + 5
    table = make_table(positions, rot) if rot else None
    pos = torch.from_numpy(rng.integers(-3, positions + 3, (batch, n))).int().cuda() if with_pos else None
    at = f8(pos).astype(int).reshape(-1) if with_pos else np.tile(np.arange(n), batch)
    kw = dict(gamma_q=gq, gamma_k=gk, table=table, pos=pos, norm=norm, interleaved=interleaved, eps=EPS)
    yq, yk = tr.qk_norm_rope(q, k, **kw)
    check_forward(q, yq, gq, table, at, norm, interleaved, "q")
    check_forward(k, yk, gk, table, at, norm, interleaved, "k")
    dq, dk, dgq, dgk = tr.qk_norm_rope_backward(q, k, dyq, dyk, **kw)
    check_backward(q, dyq, dq, dgq, gq, table, at, norm, interleaved, "dq")
    check_backward(k, dyk, dk, dgk, gk, table, at, norm, interleaved, "dk")


@pytest.mark.parametrize("dtype,param", [(F32, F32), (BF, BF), (BF, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("dim,rot", [(8, 8), (16, 16), (40, 40), (64, 64), (64, 32), (96, 96), (128, 128), (128, 64), (256, 256), (136, 30)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_dims_pairs(cuda_lib, dtype, param, dim, rot, interleaved):
    both(2, 9, 4, 2, dim, rot, dtype, param, interleaved, seed=dim + rot)


@pytest.mark.parametrize("batch,n,hq,hk", [(1, 1, 1, 1), (3, 1, 8, 2), (1, 33, 32, 8), (2, 169, 8, 8), (1, 7, 40, 1), (1, 700, 3, 3),
                                           (1, 5, 100, 7), (5, 1000, 1, 1)])
@pytest.mark.parametrize("dim", [24, 64, 128])
def test_sizes(cuda_lib, batch, n, hq, hk, dim):
    both(batch, n, hq, hk, dim, dim, BF, BF, seed=n, with_pos=n % 2 == 0)


@pytest.mark.parametrize("layout", ["bshd", "bhsd", "wide"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_layouts(cuda_lib, layout, dtype):
    both(3, 20, 4, 2, 64, 64, dtype, F32, layout=layout)
    both(3, 20, 4, 2, 72, 24, dtype, F32, layout=layout, interleaved=True)


@pytest.mark.parametrize("norm,rot", [(False, 64), (True, 0), (False, 0), (False, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_or_rotation_alone(cuda_lib, norm, rot, interleaved):
    both(2, 30, 4, 2, 64, rot, BF, F32, interleaved, norm)
    both(2, 30, 4, 2, 64, rot, F32, F32, interleaved, norm, gammas=False)


@pytest.mark.parametrize("dim,rot", [(24, 16), (40, 16), (96, 48), (256, 144), (72, 46), (256, 250)])
def test_part_of_a_head_turned(cuda_lib, dim, rot):
    for dtype, param in ((F32, F32), (BF, F32), (F16, F16)):
        both(2, 150, 5, 2, dim, rot, dtype, param)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [32, 30, 0])
def test_elements_past_the_turned_ones_stay(cuda_lib, rot, interleaved):
    """Bit by bit, infinities and the sign of a zero among them, and NaN as some NaN (IEEE 754 leaves open which one an
    operation gives); the turned ones stay finite."""
    q = torch.randn(7, 4, 64, device="cuda", dtype=BF)
    q[:, 1, rot], q[:, 2, 40], q[:, 3, 63], q[:, 0, 50] = math.inf, math.nan, -math.inf, -0.0
    for sign in (1, -1):
        kw = dict(table=make_table(7, rot) if rot else None, norm=False, interleaved=interleaved)
        y = tr.qk_norm_rope(q, None, **kw)[0] if sign > 0 else tr.qk_norm_rope_backward(q, None, q, None, **kw)[0]
        got, want = (t[..., rot:].contiguous() for t in (y, q))
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        number = ~torch.isnan(want)
        assert torch.equal(got.view(torch.int16)[number], want.view(torch.int16)[number])
        assert torch.isfinite(y[..., :rot]).all()


@pytest.mark.parametrize("batch,n", [(1, 1), (8, 1), (2, 9), (1, 75), (1, 77), (1, 152), (1, 305), (2, 304)])
@pytest.mark.parametrize("hq,hk", [(32, 8), (20, 0), (71, 5)])
def test_few_tokens_of_many_heads(cuda_lib, batch, n, hq, hk):
    """A token's heads shared by one to eight warps, some of them without any."""
    for dim, rot, interleaved in ((128, 128, False), (64, 32, False), (256, 256, True), (40, 40, False)):
        if hk:
            both(batch, n, hq, hk, dim, rot, BF, F32, interleaved)
        else:
            rng = np.random.default_rng(n)
            q, dy = (torch.from_numpy(rng.normal(size=(batch, n, hq, dim))).to("cuda", BF) for _ in range(2))
            gamma, table = torch.rand(dim, device="cuda") + 0.5, make_table(n, rot)
            kw = dict(gamma_q=gamma, table=table, interleaved=interleaved, eps=EPS)
            at = np.tile(np.arange(n), batch)
            y, _ = tr.qk_norm_rope(q, None, **kw)
            check_forward(q, y, gamma, table, at, True, interleaved, "q")
            dq, _, dg, _ = tr.qk_norm_rope_backward(q, None, dy, None, **kw)
            check_backward(q, dy, dq, dg, gamma, table, at, True, interleaved, "dq")


def test_queries_alone(cuda_lib):
    q, dy = torch.randn(2, 10, 3, 64, device="cuda"), torch.randn(2, 10, 3, 64, device="cuda")
    table = make_table(10, 64)
    y, none = tr.qk_norm_rope(q, None, table=table)
    assert none is None
    at = np.tile(np.arange(10), 2)
    check_forward(q, y, None, table, at, True, False, "q")
    dq, dk, dg, none = tr.qk_norm_rope_backward(q, None, dy, None, table=table)
    assert dk is None and none is None
    check_backward(q, dy, dq, dg, None, table, at, True, False, "dq")


def test_no_tokens(cuda_lib):
    q, k = torch.empty(2, 0, 4, 64, device="cuda"), torch.empty(2, 0, 2, 64, device="cuda")
    tr.qk_norm_rope(q, k, table=make_table(3, 64))
    dq, dk, gq, gk = tr.qk_norm_rope_backward(q, k, q, k, table=make_table(3, 64))
    assert (gq == 0).all() and (gk == 0).all()
    gq, gk = torch.full((64,), 2.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    tr.qk_norm_rope_backward(q, k, q, k, dgamma_q=gq, dgamma_k=gk)
    assert (gq == 2).all() and (gk == 3).all()


def test_dgamma_is_added_to(cuda_lib):
    q, k = torch.randn(40, 4, 64, device="cuda").to(BF), torch.randn(40, 2, 64, device="cuda").to(BF)
    _, _, gq, gk = tr.qk_norm_rope_backward(q, k, q, k)
    hq, hk = torch.full_like(gq, 5.0), torch.full_like(gk, -7.0)
    tr.qk_norm_rope_backward(q, k, q, k, dgamma_q=hq, dgamma_k=hk)
    assert torch.equal(hq, gq + 5.0) and torch.equal(hk, gk - 7.0)


@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (32, False)])
def test_in_place_and_one_side_of_dgamma(cuda_lib, rot, interleaved):
    q, k = torch.randn(30, 4, 64, device="cuda").to(BF), torch.randn(30, 2, 64, device="cuda").to(BF)
    table = make_table(30, rot)
    kw = dict(table=table, interleaved=interleaved)
    yq, yk = tr.qk_norm_rope(q, k, **kw)
    q2, k2 = q.clone(), k.clone()
    d = cba.make_qk_norm_rope_desc(q2, k2, yq=q2, yk=k2, rot_dim=rot, interleaved=interleaved, positions=30)
    cba.cba_qk_norm_rope_forward(d, q2, k2, None, None, table, None, q2, k2)
    assert torch.equal(q2, yq) and torch.equal(k2, yk)
    want = tr.qk_norm_rope_backward(q, k, yq, yk, **kw)
    d = cba.make_qk_norm_rope_desc(q, k, dyq=yq, dyk=yk, dq=yq, dk=yk, rot_dim=rot, interleaved=interleaved, positions=30)
    ws = torch.full((cba.cba_qk_norm_rope_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    gk = torch.empty(64, device="cuda")
    cba.cba_qk_norm_rope_backward(d, q, k, None, None, table, None, yq, yk, yq, yk, None, gk, ws)
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1]) and torch.equal(gk, want[3])


@pytest.mark.parametrize("dtype,big", [(F32, 1e30), (BF, 1e30), (F32, 1e19), (F16, 60000.0), (F32, 1e-25)])
def test_magnitudes(cuda_lib, dtype, big):
    """Squares that overflow fp32 (or vanish beside eps) still give the formula's values: of the large ones, the same as of
    heads of order 1, and gradients `big` times smaller."""
    x = torch.randn(20, 2, 64, device="cuda")
    q = (x * big).to(dtype) if big < 6e4 or dtype != F16 else (x.clamp(-1, 1) * big).to(dtype)
    assert torch.isfinite(q).all()
    table, at = make_table(20, 64), np.arange(20)
    y, _ = tr.qk_norm_rope(q, None, table=table, eps=EPS)
    check_forward(q, y, None, table, at, True, False, "y")
    dy = torch.randn(20, 2, 64, device="cuda").to(dtype)
    dq, _, dg, _ = tr.qk_norm_rope_backward(q, None, dy, None, table=table, eps=EPS)
    check_backward(q, dy, dq, dg, None, table, at, True, False, "dq")  # (of order 1e-30: fp32's normal numbers)


def test_nan_stays_in_its_head(cuda_lib):
    for bad in (math.nan, math.inf):
        q, k = torch.randn(6, 4, 64, device="cuda"), torch.randn(6, 2, 64, device="cuda")
        base = tr.qk_norm_rope(q, k, table=make_table(6, 64))
        q2 = q.clone()
        q2[2, 1, 5] = bad
        got = tr.qk_norm_rope(q2, k, table=make_table(6, 64))
        keep = torch.ones(6, 4, dtype=torch.bool, device="cuda")
        keep[2, 1] = False
        assert torch.equal(got[0][keep], base[0][keep]) and torch.equal(got[1], base[1]) and torch.isnan(got[0][2, 1]).any()


def test_heads_of_zeros(cuda_lib):
    q = torch.zeros(3, 2, 64, device="cuda")
    y, _ = tr.qk_norm_rope(q, None)
    dq, _, dg, _ = tr.qk_norm_rope_backward(q, None, torch.ones_like(q), None)
    assert (y == 0).all() and (dg == 0).all() and torch.allclose(dq, torch.full_like(dq, EPS ** -0.5), rtol=1e-6)


def test_gradient_against_differences(cuda_lib):
    """The kernels' own forward in fp32: central differences of step 2^-6 have a truncation of step^2 / 6 times the third
    derivative (of order 10 here: 4e-4) and a rounding of 16 u sum |y dy| / step (2e-3 of it)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q, dy = (torch.randn(4, 1, 32, generator=g, device="cuda") for _ in range(2))
    gamma, table = torch.rand(32, generator=g, device="cuda") + 0.5, make_table(4, 32)
    kw = dict(gamma_q=gamma, table=table)
    dq = tr.qk_norm_rope_backward(q, None, dy, None, **kw)[0]
    step = 2.0 ** -6
    for i in range(0, 128, 7):
        hi, lo = q.clone(), q.clone()
        hi.view(-1)[i] += step
        lo.view(-1)[i] -= step
        d = ((tr.qk_norm_rope(hi, None, **kw)[0].double() - tr.qk_norm_rope(lo, None, **kw)[0].double()) * dy.double()).sum()
        assert abs(float(d) / (2 * step) - float(dq.view(-1)[i])) < 5e-3


def test_same_bits_graphs_and_streams(cuda_lib):
    q, k = torch.randn(2, 500, 8, 64, device="cuda").to(BF), torch.randn(2, 500, 2, 64, device="cuda").to(BF)
    dyq, dyk = torch.randn_like(q.float()).to(BF), torch.randn_like(k.float()).to(BF)
    table = make_table(500, 64)
    d = cba.make_qk_norm_rope_desc(q, k, dyq=dyq, dyk=dyk, dq=q, dk=k, positions=500)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    gq, gk = (torch.empty(64, device="cuda") for _ in range(2))
    ws = torch.empty(cba.cba_qk_norm_rope_workspace_bytes(d), dtype=torch.uint8, device="cuda")

    def call():
        cba.cba_qk_norm_rope_backward(d, q, k, None, None, table, None, dyq, dyk, dq, dk, gq, gk, ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    dyq.mul_(0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    got = [t.clone() for t in (dq, dk, gq, gk)]
    want = tr.qk_norm_rope_backward(q, k, dyq, dyk, table=table)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits(cuda_lib):
    """Tokens that lie 2^16 elements apart: offsets past 2^31 elements, loads and stores."""
    n, gap = 40000, 1 << 16
    big = torch.empty(n * gap, dtype=BF, device="cuda")
    q = big.as_strided((n, 2, 64), (gap, 64, 1))
    y = big.as_strided((n, 2, 64), (gap, 64, 1), 4096)
    q.copy_(torch.randn(n, 2, 64, device="cuda").to(BF))
    table, gamma = make_table(n, 64), torch.rand(64, device="cuda") + 0.5
    want, _ = tr.qk_norm_rope(q.contiguous(), None, gamma_q=gamma, table=table)
    d = cba.make_qk_norm_rope_desc(q, None, yq=y, positions=n)
    cba.cba_qk_norm_rope_forward(d, q, None, gamma, None, table, None, y, None)
    assert torch.equal(y, want)
    got = tr.qk_norm_rope_backward(q, None, y, None, gamma_q=gamma, table=table)
    want = tr.qk_norm_rope_backward(q.contiguous(), None, y.contiguous(), None, gamma_q=gamma, table=table)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("heads_q,heads_k", [(1, 606), (1, 607), (1, 700), (700, 1), (2, 1300)])
def test_one_side_with_nearly_all_heads(cuda_lib, heads_q, heads_k):
    """More tokens than warps and so many heads on one side that the other's share of the blocks is less than one."""
    n, dim, rot = 2500, 136, 30
    table, gamma = make_table(n, rot), torch.rand(dim, device="cuda") + 0.5
    q, k, dyq, dyk = (torch.randn(n, h, dim, device="cuda").to(BF) for h in (heads_q, heads_k) * 2)
    kw = dict(gamma_q=gamma, table=table, eps=EPS)
    yq, yk = tr.qk_norm_rope(q, k, gamma_k=gamma, **kw)
    dq, dk, gq, gk = tr.qk_norm_rope_backward(q, k, dyq, dyk, gamma_k=gamma, **kw)
    few, many = ((q, dyq, yq, dq, gq), (k, dyk, yk, dk, gk))[:: 1 if heads_q < heads_k else -1]
    x, dy, y, dx, dg = few
    check_forward(x, y, gamma, table, np.arange(n), True, False, "the few heads")
    check_backward(x, dy, dx, dg, gamma, table, np.arange(n), True, False, "the few heads' gradient")
    x, dy, y, dx, dg = many  # the same bits as by themselves
    assert torch.equal(y, tr.qk_norm_rope(x, None, **kw)[0])
    want = tr.qk_norm_rope_backward(x, None, dy, None, **kw)
    assert torch.equal(dx, want[0])
    # sums of the same terms by other blocks: each off by (terms + 4) u of the sum of absolute terms
    n2 = tr.qk_norm_rope(x, None, eps=EPS)[0]
    g2 = tr.qk_norm_rope_backward(x, None, dy, None, table=table, norm=False)[0]
    terms = (n2.double() * g2.double()).abs().sum((0, 1)) * 1.02  # (n2 and g2 are rounded to bf16)
    assert ((dg.double() - want[2].double()).abs() <= 2 * (n * x.shape[1] + 4) * U * terms).all() and (dg != 0).any()
