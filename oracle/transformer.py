"""64-bit reference of the transformer-layer operators (plain numpy): layer
norm, attention, query and key norms with rotation, dropout and Newton-Schulz
orthogonalisation.  Test
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


def rotate(x, table, pos, interleaved, back=False):
    """x [tokens, heads, dim] with the pairs of its first 2 * table.shape[1] elements turned
    by the angles of table [positions, pairs, 2] at the tokens' pos (taken into its range)."""
    x, table = np.array(x, f8), np.asarray(table, f8)
    n = table.shape[1]
    row = table[np.clip(np.asarray(pos), 0, table.shape[0] - 1)][:, None]
    cos, sin = row[..., 0], -row[..., 1] if back else row[..., 1]
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y = x.copy()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def norm_rope_forward(x, gamma, table, pos, eps, norm=True, interleaved=False):
    """Each head of x [tokens, heads, dim] normed, scaled and turned (table None: not)."""
    x = np.asarray(x, f8)
    if norm:
        x = x / np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + eps)
        if gamma is not None:
            x = x * np.asarray(gamma, f8)
    return x if table is None else rotate(x, table, pos, interleaved)


def norm_rope_backward(x, dy, gamma, table, pos, eps, norm=True, interleaved=False):
    """(dx, dgamma); dgamma is None without the norm."""
    x, dy = np.asarray(x, f8), np.asarray(dy, f8)
    g = dy if table is None else rotate(dy, table, pos, interleaved, back=True)
    if not norm:
        return g, None
    rms = np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + eps)
    n = x / rms
    w = g if gamma is None else g * np.asarray(gamma, f8)
    return (w - n * ((w * n).sum(-1, keepdims=True) / x.shape[-1])) / rms, (g * n).sum((0, 1))


def philox(seed, counters):
    """The four 32-bit words (uint64 [n, 4]) of Philox4x32-10 at 64-bit counters."""
    low, u = np.uint64(0xFFFFFFFF), np.uint64
    c = np.asarray(counters, np.uint64)
    x = [c & low, c >> u(32), np.zeros_like(c), np.zeros_like(c)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(q >> u(32)) ^ x[1] ^ u(k[0]), q & low, (p >> u(32)) ^ x[3] ^ u(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(x, 1)


def dropout_keep(shape, p, seed, offset):
    """Which elements are kept; p as the fp32 number that it is given as."""
    n = int(np.prod(shape))
    counters = np.uint64(offset) + np.arange((n + 3) // 4, dtype=np.uint64)
    words = philox(seed, counters).reshape(-1)[:n]
    return (words >= np.uint64(np.rint(f8(np.float32(p)) * 2.0 ** 32))).reshape(shape)


def dropout(x, p, seed, offset=0, residual=None):
    x = np.asarray(x, f8)
    keep = dropout_keep(x.shape, p, seed, offset)
    scaled = np.where(keep, x, 0.0) / (1.0 - f8(np.float32(p)) if keep.any() else 1.0)
    return scaled if residual is None else scaled + np.asarray(residual, f8)
