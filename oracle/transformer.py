"""64-bit reference of the transformer-layer operators (plain numpy): layer
norm, attention's backward pass and Newton-Schulz orthogonalisation.  Test
infrastructure only; written from the formulas, sharing nothing with the CUDA
library, and pinned to central differences and closed forms."""
import numpy as np

f8 = np.float64


def layernorm_forward(x, gamma, beta, eps):
    """(y, mean, rstd) of x [rows, cols]; gamma and beta may be None."""
    x = np.asarray(x, f8)
    mean = x.sum(1) / x.shape[1]
    var = ((x - mean[:, None]) ** 2).sum(1) / x.shape[1]
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, f8)
    if beta is not None:
        y = y + np.asarray(beta, f8)
    return y, mean, rstd


def layernorm_backward(x, dy, gamma, mean, rstd, residual=None):
    """(dx, dgamma, dbeta) for given row statistics."""
    x, dy, mean, rstd = (np.asarray(a, f8) for a in (x, dy, mean, rstd))
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * np.asarray(gamma, f8)
    n = x.shape[1]
    dx = rstd[:, None] * (g - g.sum(1, keepdims=True) / n - h * ((g * h).sum(1, keepdims=True) / n))
    if residual is not None:
        dx = dx + np.asarray(residual, f8)
    return dx, (dy * h).sum(0), dy.sum(0)


def causal_mask(len_q, len_k):
    """Query i sees the keys j <= i + len_k - len_q (aligned at the last ones)."""
    return np.arange(len_k)[None, :] <= np.arange(len_q)[:, None] + (len_k - len_q)


def attention_forward(q, k, v, scale, causal=False):
    """(o, lse) of one sequence: q [len_q, heads_q, dim], k and v [len_k,
    heads_kv, dim]; o like q, lse [heads_q, len_q] (-inf for a row without keys,
    whose o is 0)."""
    q, k, v = (np.asarray(a, f8) for a in (q, k, v))
    group = q.shape[1] // k.shape[1]
    o, lse = np.zeros_like(q), np.full((q.shape[1], q.shape[0]), -np.inf)
    ok = causal_mask(q.shape[0], k.shape[0]) if causal else np.ones((q.shape[0], k.shape[0]), bool)
    for h in range(q.shape[1]):
        s = np.where(ok, scale * q[:, h] @ k[:, h // group].T, -np.inf)
        for i in range(q.shape[0]):
            if ok[i].any():
                m = s[i].max()
                e = np.exp(s[i] - m)
                lse[h, i] = m + np.log(e.sum())
                o[i, h] = e @ v[:, h // group] / e.sum()
    return o, lse


def attention_backward(q, k, v, o, lse, do, scale, causal=False):
    """(dq, dk, dv) of one sequence, from the given o and lse."""
    q, k, v, o, lse, do = (np.asarray(a, f8) for a in (q, k, v, o, lse, do))
    group = q.shape[1] // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    ok = causal_mask(q.shape[0], k.shape[0]) if causal else np.ones((q.shape[0], k.shape[0]), bool)
    for h in range(q.shape[1]):
        j = h // group
        s = scale * q[:, h] @ k[:, j].T
        p = np.zeros_like(s)
        live = ok & np.isfinite(lse[h])[:, None]
        p[live] = np.exp((s - np.where(np.isfinite(lse[h]), lse[h], 0.0)[:, None])[live])
        dp = do[:, h] @ v[:, j].T
        ds = p * (dp - (do[:, h] * o[:, h]).sum(1, keepdims=True))
        dq[:, h] = scale * ds @ k[:, j]
        dk[:, j] += scale * ds.T @ q[:, h]
        dv[:, j] += p.T @ do[:, h]
    return dq, dk, dv


def orthogonalize(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0):
    """Newton-Schulz iteration of one matrix from either side: X <- aX + (bS +
    cS^2) X with S = X X^T (rows <= cols), or the transposed form."""
    a, b, c = coefficients
    X = np.asarray(G, f8)
    X = X / (np.sqrt((X * X).sum()) + eps)
    for _ in range(steps):
        if X.shape[0] <= X.shape[1]:
            S = X @ X.T
            X = a * X + (b * S + c * S @ S) @ X
        else:
            S = X.T @ X
            X = a * X + X @ (b * S + c * S @ S)
    return scale * X
