"""Dropout on the GPU against the 64-bit oracle: the mask exactly, the values to their roundings (u = 2^-24 for the scale,
for the product and for the sum, w for the element type)."""
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


def f8(t):
    return t.double().cpu().numpy()


def check(x, residual, y, p, seed, offset):
    a, b = f8(x), 0.0 if residual is None else f8(residual)
    want = T.dropout(a, p, seed, offset, None if residual is None else b)
    scaled = np.abs(T.dropout(a, p, seed, offset))
    bar = 2 * U * scaled + U * np.abs(want)
    bar = bar * (1 + 2 * W[x.dtype]) + 1.01 * W[x.dtype] * np.abs(want) + (2.0 ** -25 if x.dtype == F16 else 0)
    assert (np.abs(f8(y) - want) <= bar).all()
    if residual is None:  # x has no zeros: the mask itself
        assert np.array_equal(f8(y) != 0, T.dropout_keep(a.shape, p, seed, offset) if p < 1 else np.zeros(a.shape, bool))


def rows(shape, dtype, pad, at=0):
    """A tensor without zeros whose rows lie `pad` elements apart, `at` elements into its memory."""
    r, c = shape
    big = torch.full((r * (c + pad) + at,), math.nan, device="cuda", dtype=dtype)
    t = big[at:].as_strided((r, c), (c + pad, 1))
    t.copy_((torch.rand(shape, device="cuda") + 0.25) * torch.where(torch.rand(shape, device="cuda") < 0.5, -1.0, 1.0))
    return t


@pytest.mark.parametrize("dtype", [F32, F16, BF])
@pytest.mark.parametrize("shape", [(1, 1), (1, 3), (1, 4), (3, 5), (7, 8), (169, 255), (64, 512), (33, 1000), (5, 4099), (1, 100001)])
@pytest.mark.parametrize("residual", [True, False])
def test_sizes(cuda_lib, dtype, shape, residual):
    x, r = rows(shape, dtype, 0), rows(shape, dtype, 0) if residual else None
    check(x, r, tr.dropout(x, 0.25, 77, 5, r), 0.25, 77, 5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("cols", [1, 24, 255, 256])
@pytest.mark.parametrize("pad_x,pad_r", [(0, 8), (8, 8), (3, 0), (1, 5), (8, 3)])
def test_strides(cuda_lib, dtype, cols, pad_x, pad_r):
    x, r = rows((37, cols), dtype, pad_x), rows((37, cols), dtype, pad_r)
    check(x, r, tr.dropout(x, 0.5, 3, 9, r), 0.5, 3, 9)
    check(x, None, tr.dropout(x, 0.5, 3, 9), 0.5, 3, 9)


@pytest.mark.parametrize("dtype", [F32, F16])
def test_bases_off_16_bytes(cuda_lib, dtype):
    x, r = rows((40, 64), dtype, 0, at=1), rows((40, 64), dtype, 0, at=3)
    check(x, r, tr.dropout(x, 0.1, 3, 0, r), 0.1, 3, 0)


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.05, 0.1, 0.3333, 0.9, 0.9999, 1.0])
def test_probabilities(cuda_lib, p):
    x, r = rows((50, 333), F32, 0), rows((50, 333), F32, 0)
    check(x, None, tr.dropout(x, p, 123, 0), p, 123, 0)
    check(x, r, tr.dropout(x, p, 123, 0, r), p, 123, 0)
    if p in (0.0, 1.0):
        assert torch.equal(tr.dropout(x, p, 9), x * (1 - p))


@pytest.mark.parametrize("seed,offset", [(0, 0), (1 << 63, 7), ((1 << 64) - 1, 1 << 32), (5, (1 << 32) - 3), (5, (1 << 64) - 10)])
def test_seeds_and_counters(cuda_lib, seed, offset):
    """All bits of both count; the counter runs over 2^32 and over 2^64."""
    x = rows((9, 40), BF, 0)
    keep = T.philox(seed, (np.uint64(offset) + np.arange(90, dtype=np.uint64))).reshape(9, 40) >= np.uint64(1 << 31)
    assert np.array_equal(f8(tr.dropout(x, 0.5, seed, offset)) != 0, keep)


def test_the_gradient_uses_the_same_mask(cuda_lib):
    x, dy = rows((100, 96), F32, 0), rows((100, 96), F32, 0)
    y, dx = tr.dropout(x, 0.3, 42, 1000, residual=None), tr.dropout(dy, 0.3, 42, 1000)
    assert torch.equal(y != 0, dx != 0)
    # y is linear in x: the directional derivative is the difference itself
    want = (f8(dx) * f8(x)).sum()
    assert abs(want - (f8(dy) * f8(y)).sum()) <= 4 * U * np.abs(f8(dx) * f8(x)).sum()


def test_dropped_elements_count_as_zero_whatever_they_hold(cuda_lib):
    x = torch.full((64, 64), math.nan, device="cuda")
    keep = torch.from_numpy(T.dropout_keep((64, 64), 0.5, 1, 0)).cuda()
    y = tr.dropout(x, 0.5, 1)
    assert (y[~keep] == 0).all() and torch.isnan(y[keep]).all()
    assert (tr.dropout(x * math.inf, 1.0, 1) == 0).all()


def test_in_place_and_status(cuda_lib):
    for dtype, cols in ((F32, 64), (BF, 31)):
        x, r = rows((20, cols), dtype, 0), rows((20, cols), dtype, 0)
        want = tr.dropout(x, 0.25, 6, 2, r)
        d = cba.make_dropout_desc(20, cols, type=cba.dtype_code(dtype), p=0.25, seed=6, offset=2)
        a, b = x.clone(), r.clone()
        cba.cba_dropout(d, a, r, None, a)
        cba.cba_dropout(d, x, b, None, b)
        assert torch.equal(a, want) and torch.equal(b, want)


def test_nothing_past_the_rows_is_written(cuda_lib):
    out = torch.full((10, 40), 7.0, device="cuda")
    x = rows((10, 33), F32, 0)
    d = cba.make_dropout_desc(10, 33, p=0.5, seed=6, ld_y=40)
    cba.cba_dropout(d, x, None, None, out)
    assert (out[:, 33:] == 7).all() and torch.equal(out[:, :33], tr.dropout(x, 0.5, 6))


def test_a_replayed_graph_draws_anew(cuda_lib):
    """The step lies on the device: a graph that moves it on has another mask each time, the one of a call at that offset."""
    x = rows((30, 100), BF, 0)
    step, y = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.empty_like(x)
    d = cba.make_dropout_desc(30, 100, type=cba.CBA_BF16, p=0.5, seed=8, offset=100)
    cba.cba_dropout(d, x, None, step, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cba.cba_dropout(d, x, None, step, y)
        step.add_(750)
    step.zero_()
    seen = []
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tr.dropout(x, 0.5, 8, 100 + 750 * i))
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])
    assert torch.equal(tr.dropout(x, 0.5, 8, 100, step=torch.full((1,), 750, dtype=torch.int64, device="cuda")), seen[1])


def test_empty(cuda_lib):
    assert tr.dropout(torch.empty(0, 16, device="cuda"), 0.5, 1).shape == (0, 16)


def test_more_than_2_to_the_31_elements(cuda_lib):
    """Past 2^32 elements, with and without gaps between rows: the ends against the oracle."""
    cols = 4099
    rows_n = (1 << 32) // cols + 3
    x = torch.ones(rows_n, cols + 1, dtype=F16, device="cuda")
    for t in (x[:, :cols], x.view(-1)[: rows_n * cols].view(rows_n, cols)):
        y = tr.dropout(t, 0.5, 21, 7)
        for r in (0, rows_n // 2, rows_n - 1):
            first = r * cols // 4 * 4
            words = T.philox(21, np.uint64(7) + np.arange(first // 4, (r * cols + cols + 3) // 4, dtype=np.uint64)).reshape(-1)
            keep = words[r * cols - first:][:cols] >= np.uint64(1 << 31)
            assert np.array_equal(f8(y[r]), np.where(keep, 2.0, 0.0))
        del y
