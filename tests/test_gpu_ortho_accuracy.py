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


def steep_bar(G):
    """The few singular values of a matrix of few rows may all meet the polynomial where it is steep.  An error e of X becomes at
    most D e, D the largest of |p'(s)| and p(s) / s between the smallest and the largest singular value; to it come the roundings
    of S, |b + 2 c t| r |S| sigma at most, of C, r |C| sigma, and of the new X."""
    a, b, c = 3.4445, -4.7750, 2.0315
    X = G if G.shape[0] <= G.shape[1] else G.T
    X = X / np.linalg.norm(X)
    e = R * np.linalg.norm(X)
    for _ in range(5):
        s = np.linalg.svd(X, compute_uv=False)
        grid = np.linspace(s.min(), s.max(), 200)
        t = grid ** 2
        D = max(np.abs(a + 3 * b * t + 5 * c * t * t).max(), np.abs(a + b * t + c * t * t).max())
        S = X @ X.T
        C = a * np.eye(len(S)) + b * S + c * S @ S
        X = C @ X
        e = D * e + R * (s.max() * (np.abs(b + 2 * c * t).max() * np.linalg.norm(S) + np.linalg.norm(C)) + np.linalg.norm(X))
    return e / np.linalg.norm(X)


@pytest.mark.parametrize("shape", [(2, 9), (3, 31), (3, 104), (4, 1419), (1134, 4), (105, 3)], ids=str)
def test_few_rows(cuda_lib, shape):
    rng = np.random.default_rng(shape[0] + shape[1])
    for _ in range(10):
        A = rng.normal(size=shape).astype(np.float32)
        assert relative_error(A) <= steep_bar(A.astype(np.float64))
