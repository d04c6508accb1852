"""Layer norm on the GPU against the 64-bit oracle, element by element.

Bars, from the arithmetic: u = 2^-24 is fp32's unit roundoff, w the output
type's (0 for fp32, 2^-11 for f16, 2^-8 for bf16: round to nearest).  A sum of
n terms along a chain of c additions is off by at most c u sum|terms|; every
chain here (a thread's own elements, the shuffles, the partial rows) is shorter
than 96 additions for the sizes below, so C = 128 covers it with the few
roundings of each term.  The inputs are converted exactly.
"""
import numpy as np
import pytest
import torch

import activation_backward_gb300 as cba
from oracle import transformer as T

pytestmark = pytest.mark.gpu

U, C = 2.0 ** -24, 128
W = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # f16's subnormal step
EPS = 1e-5

TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
         (torch.float16, torch.float16), (torch.float16, torch.float32)]
# one row and one column, odd rows, each row width class of the kernels, one past each, and rows too long for registers
SIZES = [(1, 1), (3, 1), (5, 7), (169, 255), (33, 256), (130, 260), (700, 512), (65, 520), (41, 1024), (9, 1032), (17, 2048),
         (5, 2056), (11, 4096), (3, 4104), (400, 333), (7, 8192), (3, 8200), (2, 12345), (5, 16392),
         # enough rows for the kernels that run ahead of them
         (9800, 8), (5003, 264), (4900, 520), (2467, 1024), (1301, 2056), (620, 4096), (613, 8192)]


def f8(t):
    return t.double().cpu().numpy()


def rows_of(rng, rows, cols, dtype, pad, shift=0.0, scale=1.0):
    a = torch.from_numpy(rng.normal(size=(rows, cols + pad)) * scale + shift)
    return a.to(device="cuda", dtype=dtype)[:, :cols]


def desc_of(x, param, **more):
    return cba.make_layernorm_desc(x.shape[0], x.shape[1], type=cba.dtype_code(x.dtype),
                                   param_type=cba.dtype_code(param), eps=EPS, ld_x=x.stride(0), **more)


def ws_of(d):
    return torch.empty(cba.cba_layernorm_workspace_bytes(d), dtype=torch.uint8, device="cuda")


def check(got, want, bar, dtype, what):
    got, bar = f8(got), bar + W[dtype] * np.abs(want) + TINY[dtype]
    bad = ~(np.abs(got - want) <= bar)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} past the bar, worst "
                           f"{np.max(np.abs(got - want) / np.maximum(bar, 1e-300)):.3g}")


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,param", TYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_forward(cuda_lib, rows, cols, dtype, param, pad):
    rng = np.random.default_rng(rows + cols)
    x = rows_of(rng, rows, cols, dtype, pad, shift=0.3)
    ga, be = rows_of(rng, 1, cols, param, 0, 1.0, 0.3)[0], rows_of(rng, 1, cols, param, 0)[0]
    y = torch.empty((rows, cols + pad), dtype=dtype, device="cuda").fill_(7)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    cba.cba_layernorm_forward(desc_of(x, param, ld_y=cols + pad), x, ga, be, y, mean, rstd)
    assert torch.all(y[:, cols:] == 7)  # the padding is not written
    wy, wm, wr = T.layernorm_forward(f8(x), f8(ga), f8(be), EPS)
    xa = np.abs(f8(x)).mean(1)
    check(mean, wm, C * U * xa, torch.float32, "mean")
    # the mean's error moves the centred sum by its square only; the rest is C u of var
    dm = (C * U * xa) ** 2
    check(rstd, wr, C * U * wr + wr ** 3 * dm, torch.float32, "rstd")
    h = np.abs(f8(x) - wm[:, None]) * wr[:, None]
    eh = C * U * (1 + h) + (C * U * xa * wr)[:, None] + h * (wr ** 2 * dm)[:, None]
    check(y[:, :cols], wy, eh * np.abs(f8(ga)) + 4 * U * np.abs(f8(be)), dtype, "y")


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,param", TYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("pad,residual,accumulate", [(0, True, 0), (8, False, 1), (3, True, 1)])
def test_backward(cuda_lib, rows, cols, dtype, param, pad, residual, accumulate):
    rng = np.random.default_rng(rows * 3 + cols)
    x, dy = rows_of(rng, rows, cols, dtype, pad, 0.3), rows_of(rng, rows, cols, dtype, pad)
    res = rows_of(rng, rows, cols, dtype, pad) if residual else None
    ga = rows_of(rng, 1, cols, param, 0, 1.0, 0.3)[0]
    _, m, r = T.layernorm_forward(f8(x), None, None, EPS)
    mean, rstd = (torch.from_numpy(a).float().cuda() for a in (m, r))
    d = desc_of(x, param, accumulate=accumulate, ld_dy=cols + pad, ld_dx=cols + pad, ld_residual=cols + pad)
    dx = torch.empty((rows, cols + pad), dtype=dtype, device="cuda").fill_(7)
    old = rng.normal(size=(2, cols)).astype(np.float32)
    dgamma, dbeta = torch.from_numpy(old).cuda()
    ws = ws_of(d)
    cba.cba_layernorm_backward(d, x, dy, ga, mean, rstd, res, dx, dgamma, dbeta, ws)
    assert torch.all(dx[:, cols:] == 7)
    wx, wg, wb = T.layernorm_backward(f8(x), f8(dy), f8(ga), f8(mean), f8(rstd), None if res is None else f8(res))
    h = (f8(x) - f8(mean)[:, None]) * f8(rstd)[:, None]
    g = np.abs(f8(dy) * f8(ga))
    rs = f8(rstd)[:, None]
    bar = rs * U * (8 * g + C * g.mean(1, keepdims=True) + np.abs(h) * C * (g * np.abs(h)).mean(1, keepdims=True))
    check(dx[:, :cols], wx, bar + 8 * U * np.abs(wx) + (8 * U * np.abs(f8(res)) if residual else 0), dtype, "dx")
    o = old.astype(np.float64) if accumulate else np.zeros((2, cols))
    check(dgamma, wg + o[0], C * U * ((np.abs(f8(dy) * h)).sum(0) + np.abs(o[0])), torch.float32, "dgamma")
    check(dbeta, wb + o[1], C * U * (np.abs(f8(dy)).sum(0) + np.abs(o[1])), torch.float32, "dbeta")


def test_no_affine_parameters_and_nullable_outputs(cuda_lib):
    rng = np.random.default_rng(1)
    x, dy = rows_of(rng, 19, 70, torch.float32, 0), rows_of(rng, 19, 70, torch.float32, 0)
    d = desc_of(x, torch.float32)
    y = torch.empty_like(x)
    cba.cba_layernorm_forward(d, x, None, None, y)
    wy, m, r = T.layernorm_forward(f8(x), None, None, EPS)
    assert np.allclose(f8(y), wy, rtol=0, atol=C * U * 8)
    mean, rstd = (torch.from_numpy(a).float().cuda() for a in (m, r))
    dx, dgamma = torch.empty_like(x), torch.zeros(70, device="cuda")
    cba.cba_layernorm_backward(d, x, dy, None, mean, rstd, None, dx, dgamma, None, ws_of(d))
    wx, wg, _ = T.layernorm_backward(f8(x), f8(dy), None, f8(mean), f8(rstd))
    assert np.allclose(f8(dx), wx, rtol=0, atol=C * U * 40) and np.allclose(f8(dgamma), wg, rtol=0, atol=C * U * 40)
    cba.cba_layernorm_backward(d, x, dy, None, mean, rstd, None, dx, None, None, ws_of(d))


def test_constant_rows_and_a_row_of_infinities(cuda_lib):
    """A constant row has variance 0: y = beta, rstd = 1/sqrt(eps).  A row that
    holds an infinity or a NaN is NaN throughout; its neighbours are not touched."""
    x = torch.randn(6, 640, device="cuda")
    x[1] = 3.0
    x[2, 5] = float("inf")
    x[4, 600] = float("nan")
    d = desc_of(x, torch.float32)
    ga, be = torch.ones(640, device="cuda"), torch.full((640,), 0.25, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    cba.cba_layernorm_forward(d, x, ga, be, y, mean, rstd)
    assert torch.all(y[1] == 0.25) and abs(rstd[1].item() * EPS ** 0.5 - 1) < 1e-6
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    good = torch.isfinite(y).all(1)
    assert good.tolist() == [True, True, False, True, False, True]


def test_no_rows(cuda_lib):
    d = cba.make_layernorm_desc(0, 100)
    assert cba.cba_layernorm_forward(d, None, None, None, None) == cba.CBA_OK
    dgamma, dbeta = torch.full((100,), 3.0, device="cuda"), torch.full((100,), 4.0, device="cuda")
    cba.cba_layernorm_backward(d, None, None, None, None, None, None, None, dgamma, dbeta, ws_of(d))
    assert torch.all(dgamma == 0) and torch.all(dbeta == 0)
    d = cba.make_layernorm_desc(0, 100, accumulate=1)
    dgamma.fill_(2)
    cba.cba_layernorm_backward(d, None, None, None, None, None, None, None, dgamma, None, ws_of(d))
    assert torch.all(dgamma == 2)


@pytest.mark.parametrize("cols", [96, 9000])
def test_in_place_same_bits_and_side_stream(cuda_lib, cols):
    rng = np.random.default_rng(cols)
    x, dy = (rows_of(rng, 300, cols, torch.bfloat16, 0) for _ in range(2))
    ga = torch.ones(cols, device="cuda")
    d = desc_of(x, torch.float32)
    y, mean, rstd = torch.empty_like(x), torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    cba.cba_layernorm_forward(d, x, ga, None, y, mean, rstd)
    first = None
    for target in ("fresh", "dy", "residual", "x"):
        a, b, c = x.clone(), dy.clone(), dy.clone()
        dx = {"fresh": torch.empty_like(x), "dy": b, "residual": c, "x": a}[target]
        dgamma, dbeta, ws = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda"), ws_of(d)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        cba.cba_layernorm_backward(d, a, b, ga, mean, rstd, c, dx, dgamma, dbeta, ws, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        got = (dx.clone(), dgamma, dbeta)
        first = got if first is None else first
        assert all(torch.equal(p, q) for p, q in zip(got, first)), target
    z = x.clone()
    cba.cba_layernorm_forward(d, z, ga, None, z)
    assert torch.equal(z, y)


def test_many_rows_of_few_columns(cuda_lib):
    """Row indices past 2^31 / cols elements stay exact: the last row of a tensor of more than 2^31 elements."""
    rows, cols = 1 << 20, 2112
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(cols, device="cuda").to(torch.bfloat16)
    y = torch.empty_like(x)
    cba.cba_layernorm_forward(desc_of(x, torch.float32), x, None, None, y)
    want = T.layernorm_forward(f8(x[-1:]), None, None, EPS)[0]
    assert np.max(np.abs(f8(y[-1:]) - want)) <= 2.0 ** -8 * 1.8 and torch.all(y[:5] == 0)
