"""How far fp32 results of the Newton-Schulz iteration, whose operands are f16, are from the 64-bit iteration.

Bars, Frobenius norms relative to O's, from the arithmetic.  r = 2.1e-4 is an f16 rounding of a matrix of unrelated elements.
Where the singular values of X are of order 1 (S between 0.5 and 1.4), a step adds the roundings of X (1 part), of S, through b S
+ c S^2 with S as rounded in both (|b + 2 c S| of it, 2.7 at most), and of C (1 part): 4.7 r.  Four such steps, all errors in the
same direction: 4e-3.  Directions far below the leading ones grow by a = 3.4445 a step, and so does the rounding error in them: a
rounding of X of norm 1, as at the start, becomes a^5 r, and each later one as much, unrelated: sqrt(5) a^5 r, beside an O of norm
sqrt(m).
"""
import numpy as np
import pytest
import torch

from oracle import transformer as T

from .test_gpu_ortho import call

pytestmark = pytest.mark.gpu
R, FLAT = 2.1e-4, 4e-3
SHAPES = [(1, 300), (7, 9), (50, 500), (500, 50), (64, 64), (128, 576), (129, 129), (300, 301), (200, 2000), (1000, 600), (24, 4096)]


def relative_error(A):
    G = torch.from_numpy(np.asarray(A)).float().cuda()[None]
    want = T.orthogonalize(G[0].double().cpu().numpy())
    got = call(G, torch.empty_like(G))[0].double().cpu().numpy()
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("kind", ["noise", "low rank", "equal"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_flat_spectra(cuda_lib, shape, kind):
    rng = np.random.default_rng(shape[0] + 3 * shape[1])
    A = rng.normal(size=shape)
    if kind == "low rank":
        k = max(1, min(shape) // 16)
        A += rng.normal(size=(shape[0], k)) @ rng.normal(size=(k, shape[1])) / np.sqrt(k)
    if kind == "equal":
        u, _, v = np.linalg.svd(A, full_matrices=False)
        A = u @ v
    assert relative_error(A) <= FLAT


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_singular_values_over_four_decades(cuda_lib, shape):
    rng = np.random.default_rng(shape[0] + 5 * shape[1])
    m = min(shape)
    u, _, v = np.linalg.svd(rng.normal(size=shape), full_matrices=False)
    assert relative_error((u * np.logspace(0, -4, m)) @ v) <= FLAT + np.sqrt(5 / m) * 3.4445 ** 5 * R
