"""Newton-Schulz orthogonalisation on the GPU against the 64-bit oracle.

Bar, from the arithmetic.  Rounding to f16 is a relative error of 2.1e-4 in the
2-norm of a matrix of unrelated elements (2^-11 at worst each, the mean square of a
uniform rounding).  A step rounds X (1 part), S (|b| + 2 |c| |S| parts, through b S
X and c S S X) and B = b S + c S^2 (2.8 parts at most); while S is small beside 1
only X's counts.  In the last three of five steps S is of order 1: 3 steps of 2.1e-4 (1
+ 4.8 + 4.1 + 2.8) = 8e-3 if all point the same way, and less the steps there are.
Single elements: six times that of the root mean square, plus the output's rounding.
"""
import numpy as np
import pytest
import torch

import activation_backward_gb300 as cba
from oracle import transformer as T

pytestmark = pytest.mark.gpu

BAR = 8e-3
W = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def call(G, out, **kw):
    kw.setdefault("ld_in", G.stride(1) if G.shape[1] > 1 else 0)
    d = cba.make_orthogonalize_desc(*G.shape, in_type=cba.dtype_code(G.dtype), out_type=cba.dtype_code(out.dtype), **kw)
    ws = torch.empty(cba.cba_orthogonalize_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    cba.cba_orthogonalize(d, G, out, ws)
    assert cba.cba_get_status(ws) == cba.CBA_OK
    return out


def check(got, G, bar=BAR, **kw):
    for g, x in zip(got, G):
        want = T.orthogonalize(x.double().cpu().numpy(), **kw)
        err = g.double().cpu().numpy() - want
        w = W[g.dtype]
        norm = np.linalg.norm(want)
        assert np.linalg.norm(err) <= (bar + w / 2) * norm, np.linalg.norm(err) / norm
        rms = norm / np.sqrt(want.size)
        assert np.all(np.abs(err) <= 6 * bar * rms + w * np.abs(want)), np.max(np.abs(err)) / rms


def draw(seed, *shape, scale=1e-3, dtype=torch.float32):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=shape) * scale).to("cuda", dtype)


SHAPES = [(1, 1, 1), (1, 1, 9), (1, 9, 1), (2, 7, 5), (1, 50, 500), (1, 500, 50), (3, 64, 64), (1, 128, 576), (1, 130, 260),
          (2, 255, 1024), (1, 1024, 255), (1, 129, 129), (1, 512, 2304), (5, 300, 200), (1, 260, 1100), (1, 1280, 1280),
          # one block per matrix: the largest that fit, with an odd number of 64-column boxes, and the first that do not
          (2, 64, 1600), (1, 1, 1601), (3, 128, 640), (2, 65, 320), (1, 630, 127), (2, 128, 641), (1, 1290, 33),
          # enough tiles for pairs of blocks and for the symmetric products' triangle, with ragged edges
          (3, 900, 1300), (5, 1300, 1000),
          # contractions shared by clusters of 2, 4 and 8 blocks, with ragged tiles, from either side
          (1, 385, 4099), (2, 260, 5000), (6, 300, 1023), (1, 3001, 391), (8, 200, 2000), (1, 1100, 1300)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(cuda_lib, shape):
    G = draw(shape[1] * 7 + shape[2], *shape)
    check(call(G, torch.full(shape, 9.0, device="cuda", dtype=torch.bfloat16)), G)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("out", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("scale", [1e-4, 1.0, 50.0])
def test_types_and_magnitudes(cuda_lib, dtype, out, scale):
    G = draw(3, 2, 96, 200, scale=scale, dtype=dtype)
    check(call(G, torch.empty(G.shape, device="cuda", dtype=out)), G)


@pytest.mark.parametrize("scale", [1e-15, 1e15])
def test_extreme_magnitudes(cuda_lib, scale):
    G = draw(4, 1, 40, 60, scale=scale)
    check(call(G, torch.empty_like(G), eps=0.0), G, eps=0.0)


@pytest.mark.parametrize("rows,cols", [(70, 150), (150, 70)])
def test_strides_and_in_place(cuda_lib, rows, cols):
    wide = draw(5, 3, rows, cols + 5)
    G = wide[:, :, 2:cols + 2]  # rows of an odd pitch, at an odd offset
    buf = torch.full((3, rows + 1, cols + 3), 9.0, device="cuda", dtype=torch.bfloat16)
    d = cba.make_orthogonalize_desc(3, rows, cols, ld_in=cols + 5, batch_in=rows * (cols + 5), ld_out=cols + 3,
                                    batch_out=(rows + 1) * (cols + 3))
    ws = torch.empty(cba.cba_orthogonalize_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    cba.cba_orthogonalize(d, G, buf, ws)
    check(buf[:, :rows, :cols], G)
    assert torch.all(buf[:, rows:] == 9) and torch.all(buf[:, :, cols:] == 9)
    same = G.contiguous()
    keep = same.clone()
    check(call(same, same), keep)


@pytest.mark.parametrize("steps,coef,scale", [(1, cba.NEWTON_SCHULZ, 1.0), (3, cba.NEWTON_SCHULZ, 0.2), (10, (1.875, -1.25, 0.375), 1.0)])
def test_steps_coefficients_and_scale(cuda_lib, steps, coef, scale):
    G = draw(6, 1, 60, 320)
    bar = BAR if steps <= 5 else 2 * BAR  # ten steps: S is of order 1 in more of them, and the map contracts there
    check(call(G, torch.empty_like(G), steps=steps, coefficients=coef, scale=scale), G, bar, steps=steps, coefficients=coef, scale=scale)


def test_a_low_rank_gradient(cuda_lib):
    """Eight directions a hundred times the rest: all of them come out near 1."""
    rng = np.random.default_rng(7)
    G = rng.normal(size=(200, 8)) @ rng.normal(size=(8, 640)) * 10 + rng.normal(size=(200, 640))
    t = torch.from_numpy(G).float().cuda()[None]
    out = call(t, torch.empty_like(t))[0].double().cpu().numpy()
    want = T.orthogonalize(t[0].double().cpu().numpy())
    # f16's 2.1e-4 of the eight large directions is noise of 2.1e-4 * 30 of the others' elements
    assert np.linalg.norm(out - want) <= (BAR + 30 * 2.1e-4 * 4) * np.linalg.norm(want)


def test_zeros_infinities_and_neighbours(cuda_lib):
    G = draw(8, 4, 80, 90)
    G[1] = 0
    G[2, 3, 4] = float("inf")
    out = call(G, torch.full(G.shape, 9.0, device="cuda", dtype=torch.bfloat16))
    assert torch.all(out[1] == 0) and torch.isnan(out[2]).all()
    check(out[[0, 3]], G[[0, 3]])


def test_same_bits_and_graph(cuda_lib):
    from activation_backward_gb300.layer import capture_graph
    G = draw(9, 2, 300, 700)
    first = call(G, torch.empty(G.shape, device="cuda", dtype=torch.bfloat16)).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = call(G, torch.empty_like(first))
    side.synchronize()
    assert torch.equal(first, again)
    d = cba.make_orthogonalize_desc(2, 300, 700)
    ws = torch.empty(cba.cba_orthogonalize_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(first)
    g = capture_graph(lambda: cba.cba_orthogonalize(d, G, out, ws))
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)


@pytest.mark.parametrize("shape", [
    # clusters of two blocks on a long contraction; tiles of 128 columns beside pairs of blocks; both sides tall
    (6, 300, 3201), (8, 1000, 1010), (3, 5000, 300), (1, 1999, 2050),
    # one block per matrix, from one chunk of columns to seven, in rows that are and are not whole vectors
    (2, 64, 256), (2, 40, 260), (1, 77, 513), (2, 513, 77), (2, 33, 1030), (1, 128, 600),
], ids=str)
def test_tiles_and_chunks(cuda_lib, shape):
    G = draw(sum(shape), *shape)
    first = call(G, torch.full(shape, 9.0, device="cuda", dtype=torch.float16)).clone()
    check(first, G)
    assert torch.equal(first, call(G, torch.empty_like(first)))
