"""Newton-Schulz with coefficients whose polynomial leaves the usual range: singular values up to 2 before every step, C = a I +
b S + c S^2 up to whatever the coefficients make it.

Bar, Frobenius norms, from the arithmetic.  An f16 rounding of a matrix of unrelated elements is r = 2.1e-4 of its norm (the
mean square of a uniform relative rounding of 2^-11 at worst).  With sigma the largest singular value of X before a step and t =
sigma^2, the step takes an error e of X to at most (|a| + 3 |b| t + 5 |c| t^2) e, and adds the roundings of S, (|b| + 2 |c| t) r
|S| sigma, of C, r |C| sigma, and of the new X, r |X'|.
"""
import numpy as np
import pytest
import torch

from oracle import transformer as T

from .test_gpu_ortho import call

pytestmark = pytest.mark.gpu
R = 2.1e-4


def bar_of(G, steps, coefficients, eps):
    a, b, c = coefficients
    X = G if G.shape[0] <= G.shape[1] else G.T
    X = X / (np.linalg.norm(X) + eps)
    e = R * np.linalg.norm(X)
    for _ in range(steps):
        sigma = np.linalg.norm(X, 2)
        t, S = sigma ** 2, X @ X.T
        C = a * np.eye(len(S)) + b * S + c * S @ S
        X = C @ X
        e = ((abs(a) + 3 * abs(b) * t + 5 * abs(c) * t * t) * e + R * sigma * ((abs(b) + 2 * abs(c) * t) * np.linalg.norm(S)
             + np.linalg.norm(C)) + R * np.linalg.norm(X))
    return e


def matrix(seed, rows, cols, lead):
    """A random matrix with `lead` as the part of its norm that lies in one direction."""
    rng = np.random.default_rng(seed)
    noise = rng.normal(size=(rows, cols))
    one = np.outer(rng.normal(size=rows), rng.normal(size=cols))
    G = lead * one / np.linalg.norm(one) + np.sqrt(1 - lead ** 2) * noise / np.linalg.norm(noise)
    return torch.from_numpy(G).float().cuda()[None]


SHAPES = [(40, 70), (70, 40), (128, 300), (200, 330), (330, 200), (700, 900), (260, 4100)]


@pytest.mark.parametrize("steps,coefficients", [(1, (20.0, -30.0, 12.0)), (1, (1000.0, -1.0, 0.0)), (2, (8.2, -23.6, 17.4)),
                                                (1, (-17.0, 3.0, 40.0)), (1, (1e-3, 2e-3, -1e-3))], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_coefficients_of_any_size(cuda_lib, shape, steps, coefficients):
    G = matrix(shape[0], *shape, 0.5)
    g = G[0].double().cpu().numpy()
    want = T.orthogonalize(g, steps, coefficients)
    got = call(G, torch.empty_like(G), steps=steps, coefficients=coefficients)[0].double().cpu().numpy()
    assert np.linalg.norm(got - want) <= bar_of(g, steps, coefficients, 1e-7)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_singular_values_of_two(cuda_lib, shape):
    """p(1) = 2: the second step starts from 2, where the polynomial's factor is 45.8."""
    coefficients = (2.9, -4.775, 3.875)
    G = matrix(shape[1], *shape, 0.999)
    g = G[0].double().cpu().numpy()
    want = T.orthogonalize(g, 2, coefficients)
    assert 70 < np.linalg.norm(want, 2) < 95
    got = call(G, torch.empty_like(G), steps=2, coefficients=coefficients)[0].double().cpu().numpy()
    assert np.isfinite(got).all() and np.linalg.norm(got - want) <= bar_of(g, 2, coefficients, 1e-7)
