"""Pins of the 64-bit reference of the transformer-layer operators: central
differences of the forward formulas (fp64), closed forms and identities."""
import numpy as np
import pytest

from oracle import transformer as T

STEP = 1e-5
# central differences in fp64 of functions of order 1: truncation ~STEP^2,
# rounding ~1e-16 / STEP; 1e-7 leaves two orders of room
BAR = 1e-7


def diff(f, x, pick):
    """Central difference of the scalar f with respect to the entries `pick` of x."""
    out = []
    for i in pick:
        keep = x[i]
        x[i] = keep + STEP
        hi = f()
        x[i] = keep - STEP
        lo = f()
        x[i] = keep
        out.append((hi - lo) / (2 * STEP))
    return np.array(out)


def some(rng, shape, n=25):
    return [tuple(int(rng.integers(d)) for d in shape) for _ in range(n)]


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (5, 12), (3, 33)])
@pytest.mark.parametrize("affine", [True, False])
def test_layernorm_backward_is_the_derivative_of_the_forward(rows, cols, affine):
    rng = np.random.default_rng(rows * 100 + cols)
    x, dy = rng.normal(size=(rows, cols)) + 0.5, rng.normal(size=(rows, cols))
    gamma, beta = (rng.uniform(0.5, 1.5, cols), rng.normal(size=cols)) if affine else (None, None)
    eps = 1e-2
    _, mean, rstd = T.layernorm_forward(x, gamma, beta, eps)
    dx, dgamma, dbeta = T.layernorm_backward(x, dy, gamma, mean, rstd)

    def loss():
        return float((T.layernorm_forward(x, gamma, beta, eps)[0] * dy).sum())

    at = some(rng, x.shape)
    assert np.allclose(diff(loss, x, at), [dx[i] for i in at], rtol=0, atol=BAR * 100)
    if affine:
        cols_at = [(int(c),) for c in rng.integers(cols, size=10)]
        assert np.allclose(diff(loss, gamma, cols_at), [dgamma[i] for i in cols_at], rtol=0, atol=BAR * 100)
        assert np.allclose(diff(loss, beta, cols_at), [dbeta[i] for i in cols_at], rtol=0, atol=BAR * 100)


def test_layernorm_residual_adds_and_dx_sums_to_zero():
    rng = np.random.default_rng(3)
    x, dy, res = (rng.normal(size=(4, 9)) for _ in range(3))
    _, mean, rstd = T.layernorm_forward(x, None, None, 1e-5)
    dx = T.layernorm_backward(x, dy, None, mean, rstd)[0]
    assert np.allclose(dx.sum(1), 0, atol=1e-12)
    assert np.array_equal(T.layernorm_backward(x, dy, None, mean, rstd, res)[0], dx + res)


@pytest.mark.parametrize("len_q,len_k,hq,hk,causal", [
    (1, 1, 1, 1, False), (5, 7, 2, 1, False), (6, 6, 4, 2, True), (3, 8, 2, 2, True),
    (8, 3, 2, 1, True),  # the first queries see no key
])
def test_attention_backward_is_the_derivative_of_the_forward(len_q, len_k, hq, hk, causal):
    rng = np.random.default_rng(len_q * 10 + len_k)
    d, scale = 4, 0.6
    q = rng.normal(size=(len_q, hq, d))
    k, v = rng.normal(size=(len_k, hk, d)), rng.normal(size=(len_k, hk, d))
    do = rng.normal(size=q.shape)
    o, lse = T.attention_forward(q, k, v, scale, causal)
    grads = T.attention_backward(q, k, v, o, lse, do, scale, causal)

    def loss():
        return float((T.attention_forward(q, k, v, scale, causal)[0] * do).sum())

    for x, g in zip((q, k, v), grads):
        at = some(rng, x.shape)
        assert np.allclose(diff(loss, x, at), [g[i] for i in at], rtol=0, atol=BAR * 100)
    if causal and len_q > len_k:
        assert np.all(grads[0][:len_q - len_k] == 0) and np.all(np.isneginf(lse[:, :len_q - len_k]))


def test_attention_forward_is_a_weighted_mean():
    rng = np.random.default_rng(9)
    q, k = rng.normal(size=(4, 2, 8)), rng.normal(size=(6, 1, 8))
    o, lse = T.attention_forward(q, k, np.ones((6, 1, 8)), 0.3)
    assert np.allclose(o, 1.0) and lse.shape == (2, 4)


@pytest.mark.parametrize("rows,cols", [(4, 9), (9, 4), (6, 6)])
def test_orthogonalize_maps_the_singular_values(rows, cols):
    """The iteration keeps the singular vectors and applies the odd polynomial
    p(s) = a s + b s^3 + c s^5 to each singular value of G / |G|, `steps` times."""
    rng = np.random.default_rng(rows)
    G = rng.normal(size=(rows, cols))
    a, b, c = coef = (3.4445, -4.7750, 2.0315)
    u, s, vt = np.linalg.svd(G, full_matrices=False)
    s = s / (np.linalg.norm(G) + 1e-7)
    for steps in (1, 3, 5):
        t = s.copy()
        for _ in range(steps):
            t = a * t + b * t ** 3 + c * t ** 5
        got = T.orthogonalize(G, steps, coef, scale=0.5)
        assert np.allclose(got, 0.5 * (u * t) @ vt, atol=1e-10)
    assert np.all(np.abs(t - 0.95) < 0.35)  # near the nearest orthogonal matrix's values


def test_orthogonalize_of_zeros_is_zero():
    assert np.all(T.orthogonalize(np.zeros((3, 5))) == 0)
