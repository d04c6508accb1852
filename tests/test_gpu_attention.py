"""Attention's backward pass on the GPU against the 64-bit oracle's formulas,
element by element.

Bars, from the arithmetic.  w: unit roundoff of the 16-bit type (2^-8 bf16,
2^-11 f16), u = 2^-24 of fp32.  P carries a relative error e from its fp32
exponent (a dot product of `dim` terms, the subtraction of lse, the power of
two): e <= C u (1 + scale max |q|.|k| + max |lse|), C = 2 dim + 64, plus w when it is
rounded for P^T do.  dS carries w + e relatively, plus P times the errors C u
|do|.|v| and C u |do|.|o| of dP and D.  The long sums are fp32 (C' u of the sum of
absolute terms, C' = 4096 at the lengths below), and the result is rounded once
(w).  f16 holds dS times a power of two that puts 2 max|do| max|v| at 2^15 or half of
it, so values under 2^-14 of that unit round to 2^-25 of it: b 2^-39 each.
"""
import numpy as np
import pytest
import torch

import activation_backward_gb300 as cba
from oracle import transformer as T

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
W = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
BF, F16 = torch.bfloat16, torch.float16


def f8(t):
    return t.double().cpu().numpy()


def bars(q, k, v, o, lse, do, scale, causal, dtype):
    """(want, bar) of dq, dk, dv for one sequence, all fp64 arrays."""
    want = T.attention_backward(q, k, v, o, lse, do, scale, causal)
    bar = [np.zeros_like(g) for g in want]
    w, dim, group = W[dtype], q.shape[2], q.shape[1] // k.shape[1]
    if not q.size or not k.size:
        return want, bar
    C, C2 = 2 * dim + 64, 4096
    ok = T.causal_mask(q.shape[0], k.shape[0]) if causal else np.ones((q.shape[0], k.shape[0]), bool)
    b = 2 * np.sqrt((do ** 2).sum(-1).max()) * np.sqrt((v ** 2).sum(-1).max()) if dtype == F16 else 0.0
    for h in range(q.shape[1]):
        j = h // group
        m = np.where(np.isfinite(lse[h]), lse[h], 0.0)
        p = np.where(ok & np.isfinite(lse[h])[:, None], np.exp(np.minimum(scale * q[:, h] @ k[:, j].T - m[:, None], 50)), 0.0)
        e = C * U * (1 + scale * (np.abs(q[:, h]) @ np.abs(k[:, j]).T).max() + np.abs(m).max())
        dd = (do[:, h] * o[:, h]).sum(1, keepdims=True)
        ds = np.abs(p * (do[:, h] @ v[:, j].T - dd))
        dp = C * U * (np.abs(do[:, h]) @ np.abs(v[:, j]).T + (np.abs(do[:, h]) * np.abs(o[:, h])).sum(1, keepdims=True))
        eds = (w + e + C2 * U) * ds + p * dp + b * 2.0 ** -39
        bar[0][:, h] = scale * eds @ np.abs(k[:, j])
        bar[1][:, j] += scale * eds.T @ np.abs(q[:, h])
        bar[2][:, j] += ((w + e + C2 * U) * p + (2.0 ** -37 if dtype == F16 else 0)).T @ np.abs(do[:, h])
    tiny = 2.0 ** -25 if dtype == F16 else 0.0
    # the result's own rounding acts on the value with its error
    return want, [x * (1 + 2 * w) + 1.01 * w * np.abs(g) + tiny for x, g in zip(bar, want)]


def check(got, want, bar, what):
    got = f8(got)
    bad = ~(np.abs(got - want) <= bar)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} past the bar, worst "
                           f"{np.max(np.abs(got - want) / np.maximum(bar, 1e-300)):.3g}")


def place(a, layout, dtype):
    """a [batch, len, heads, dim] on the GPU in the given memory order, as that view."""
    t = torch.from_numpy(a).to("cuda", dtype)
    if layout == "bhsd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "wide":  # a slice of a wider projection
        big = torch.full((*t.shape[:2], t.shape[2] + 3, t.shape[3] + 8), 5.0, device="cuda", dtype=dtype)
        big[:, :, 1:1 + t.shape[2], 8:] = t
        return big[:, :, 1:1 + t.shape[2], 8:]
    return t.contiguous()


def make(rng, batch, len_q, len_k, hq, hk, dim, dtype, layout, scale, causal, do_scale=0.05):
    shape_q, shape_k = (batch, len_q, hq, dim), (batch, len_k, hk, dim)
    q, k, v, do = (place(rng.normal(size=s) * f, layout, dtype)
                   for s, f in ((shape_q, 1), (shape_k, 1), (shape_k, 1), (shape_q, do_scale)))
    o, lse = np.zeros(shape_q), np.zeros((batch, hq, len_q))
    for b in range(batch):
        o[b], lse[b] = T.attention_forward(f8(q[b]), f8(k[b]), f8(v[b]), scale, causal)
    return q, k, v, place(o, layout, dtype), torch.from_numpy(lse).float().cuda(), do


def run(q, k, v, o, lse, do, scale, causal, layout="bshd", cu_q=None, cu_k=None, **packed):
    outs = []
    for t in (q, k, v):
        z = torch.full(t.shape, 9.0, device="cuda", dtype=t.dtype)
        outs.append(z.transpose(-3, -2).contiguous().transpose(-3, -2) if layout == "bhsd" else z)
    d = cba.make_attention_desc(q, k, v, o, do, *outs, causal=causal, scale=scale, **packed)
    ws = torch.empty(cba.cba_attention_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    cba.cba_attention_backward(d, q, k, v, o, lse, do, cu_q, cu_k, *outs, ws)
    assert cba.cba_get_status(ws) == cba.CBA_OK
    return outs


def compare(args, outs, scale, causal, dtype):
    q, k, v, o, lse, do = (f8(a) for a in args)
    for b in range(q.shape[0]):
        want, bar = bars(q[b], k[b], v[b], o[b], lse[b], do[b], scale, causal, dtype)
        for name, g, x, y in zip(("dq", "dk", "dv"), outs, want, bar):
            check(g[b], x, y, f"{name} of sequence {b}")


LENGTHS = [(1, 1), (1, 5), (5, 1), (7, 9), (64, 64), (127, 129), (128, 128), (129, 127), (169, 169), (300, 200), (200, 300),
           (1, 700), (700, 1), (385, 640)]


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("len_q,len_k", LENGTHS)
@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, BF), (64, F16), (128, F16)], ids=str)
def test_lengths(cuda_lib, len_q, len_k, dim, dtype, causal):
    rng = np.random.default_rng(len_q * 1000 + len_k)
    args = make(rng, 2, len_q, len_k, 4, 2, dim, dtype, "bshd", dim ** -0.5, causal)
    compare(args, run(*args, dim ** -0.5, causal), dim ** -0.5, causal, dtype)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, BF), (64, F16), (128, F16)], ids=str)
def test_more_tiles_than_blocks(cuda_lib, dim, dtype, causal):
    """Several tiles per block, of unlike work: 320 of keys, 640 of queries, ragged, repeated."""
    rng = np.random.default_rng(dim)
    args = make(rng, 32, 330, 200, 10, 5, dim, dtype, "bshd", 0.1, causal)
    first = [t.clone() for t in run(*args, 0.1, causal)]
    compare(args, first, 0.1, causal, dtype)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, run(*args, 0.1, causal)))


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF)], ids=str)
@pytest.mark.parametrize("len_q,len_k,hq,hk", [(1100, 1500, 4, 1), (3, 2700, 2, 1), (2700, 3, 2, 2), (1500, 1100, 8, 1)])
def test_few_tiles_cut_into_items(cuda_lib, len_q, len_k, hq, hk, dim, dtype, causal):
    """Too few tiles for the SMs: their steps are shared out and the sums joined, with the same bits every time."""
    rng = np.random.default_rng(len_q + hq)
    args = make(rng, 1, len_q, len_k, hq, hk, dim, dtype, "bshd", 0.1, causal)
    first = [t.clone() for t in run(*args, 0.1, causal)]
    compare(args, first, 0.1, causal, dtype)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run(*args, 0.1, causal)))


def test_packed_tiles_cut_into_items(cuda_lib):
    rng = np.random.default_rng(11)
    lens = [0, 1700, 5, 900, 130]
    parts, args, cu = pack(rng, lens, lens, 4, 1, 128, BF, 0.1, True)
    outs = run(*args, 0.1, True, cu_q=cu[0], cu_k=cu[1], sequences=5, max_q=1700, max_k=1700)
    at = 0
    for p, n in zip(parts, lens):
        compare(p, [g[None, at:at + n] for g in outs], 0.1, True, BF)
        at += n


@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, F16)], ids=str)
def test_many_packed_sequences(cuda_lib, dim, dtype):
    rng = np.random.default_rng(dim)
    lens = [int(x) for x in rng.integers(0, 420, size=60)]
    parts, args, cu = pack(rng, lens, lens, 4, 2, dim, dtype, 0.1, True)
    outs = run(*args, 0.1, True, cu_q=cu[0], cu_k=cu[1], sequences=60, max_q=max(lens), max_k=max(lens))
    at = 0
    for p, n in zip(parts, lens):
        compare(p, [g[None, at:at + n] for g in outs], 0.1, True, dtype)
        at += n


@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
@pytest.mark.parametrize("dim", [8, 16, 40, 72, 80, 96, 120])
def test_head_dimensions(cuda_lib, dim, dtype):
    rng = np.random.default_rng(dim)
    args = make(rng, 1, 150, 170, 2, 1, dim, dtype, "bshd", 0.2, True)
    compare(args, run(*args, 0.2, True), 0.2, True, dtype)


@pytest.mark.parametrize("layout", ["bhsd", "wide"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (6, 2), (8, 1)])
def test_layouts_and_shared_heads(cuda_lib, layout, hq, hk):
    rng = np.random.default_rng(hq * 10 + hk)
    args = make(rng, 3, 140, 260, hq, hk, 64, BF, layout, 0.125, True)
    compare(args, run(*args, 0.125, True, layout), 0.125, True, BF)


@pytest.mark.parametrize("dtype,do_scale", [(BF, 1e-12), (BF, 1e12), (F16, 1e-4), (F16, 300.0)], ids=str)
def test_small_and_large_gradients(cuda_lib, dtype, do_scale):
    rng = np.random.default_rng(5)
    args = make(rng, 1, 200, 500, 2, 2, 64, dtype, "bshd", 0.125, False, do_scale)
    compare(args, run(*args, 0.125, False), 0.125, False, dtype)


def pack(rng, lens_q, lens_k, hq, hk, dim, dtype, scale, causal):
    parts = [make(rng, 1, a, b, hq, hk, dim, dtype, "bshd", scale, causal) for a, b in zip(lens_q, lens_k)]
    q, k, v, o, do = (torch.cat([p[i][0] for p in parts]) for i in (0, 1, 2, 3, 5))
    lse = torch.cat([p[4][0] for p in parts], 1).contiguous()
    cu = [torch.tensor(np.cumsum([0] + list(x)), dtype=torch.int32, device="cuda") for x in (lens_q, lens_k)]
    return parts, (q, k, v, o, lse, do), cu


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
@pytest.mark.parametrize("lens_q,lens_k", [
    ((1,), (1,)), ((130, 1, 0, 257, 64), (130, 1, 0, 257, 64)), ((40, 0, 200, 5), (0, 90, 129, 300)), ((128, 128), (128, 256)),
    ((0, 0), (3, 200)), ((70, 130), (0, 0)),
])
def test_packed(cuda_lib, lens_q, lens_k, dtype, causal):
    rng = np.random.default_rng(sum(lens_q) + len(lens_k))
    parts, args, cu = pack(rng, lens_q, lens_k, 4, 2, 72, dtype, 0.15, causal)
    outs = run(*args, 0.15, causal, cu_q=cu[0], cu_k=cu[1], sequences=len(lens_q), max_q=max(lens_q), max_k=max(lens_k))
    at = [0, 0]
    for p, a, b in zip(parts, lens_q, lens_k):
        own = [outs[0][None, at[0]:at[0] + a], outs[1][None, at[1]:at[1] + b], outs[2][None, at[1]:at[1] + b]]
        compare(p, own, 0.15, causal, dtype)
        at = [at[0] + a, at[1] + b]


@pytest.mark.parametrize("dim", [64, 128])
def test_a_neighbour_full_of_infinities(cuda_lib, dim):
    """Sequences 1 and 3 hold nothing but NaN and infinities; 0, 2 and 4 get the bits they get without them."""
    rng = np.random.default_rng(dim)
    lens = (100, 60, 200, 130, 77)
    parts, args, cu = pack(rng, lens, lens, 2, 1, dim, BF, 0.1, True)
    clean = [t.clone() for t in run(*args, 0.1, True, cu_q=cu[0], cu_k=cu[1], sequences=5, max_q=200, max_k=200)]
    ends = np.cumsum((0,) + lens)
    for i, bad in ((1, float("nan")), (3, float("inf"))):
        for t in (args[0], args[1], args[2], args[3], args[5]):
            t[ends[i]:ends[i + 1]] = bad
        args[4][:, ends[i]:ends[i + 1]] = bad
    dirty = run(*args, 0.1, True, cu_q=cu[0], cu_k=cu[1], sequences=5, max_q=200, max_k=200)
    for x, y in zip(clean, dirty):
        for i in (0, 2, 4):
            assert torch.equal(x[ends[i]:ends[i + 1]], y[ends[i]:ends[i + 1]])


def test_rows_without_keys_are_zero(cuda_lib):
    rng = np.random.default_rng(2)
    args = make(rng, 1, 300, 40, 2, 2, 64, BF, "bshd", 0.125, True)
    dq, dk, dv = run(*args, 0.125, True)
    assert torch.all(dq[:, :260] == 0) and torch.isfinite(dk.float()).all() and torch.isfinite(dv.float()).all()
    assert torch.isneginf(args[4][:, :, :260]).all()
    # a row that the caller's own mask emptied: lse = -infinity
    args = make(rng, 1, 30, 40, 1, 1, 64, BF, "bshd", 0.125, False)
    args[4][:, :, 7] = -float("inf")
    compare(args, run(*args, 0.125, False), 0.125, False, BF)


def test_no_queries_or_no_keys(cuda_lib):
    rng = np.random.default_rng(4)
    for len_q, len_k in ((0, 200), (200, 0), (0, 0)):
        args = make(rng, 2, len_q, len_k, 2, 1, 64, BF, "bshd", 0.1, False)
        for g in run(*args, 0.1, False):
            assert torch.all(g == 0)


def test_same_bits_on_another_stream_and_in_a_graph(cuda_lib):
    from activation_backward_gb300.layer import capture_graph
    rng = np.random.default_rng(6)
    args = make(rng, 2, 400, 400, 4, 2, 128, BF, "bshd", 0.09, True)
    first = run(*args, 0.09, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run(*args, 0.09, True)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    q, k, v, o, lse, do = args
    outs = [torch.zeros_like(t) for t in (q, k, v)]
    d = cba.make_attention_desc(q, k, v, o, do, *outs, causal=True, scale=0.09)
    ws = torch.empty(cba.cba_attention_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    g = capture_graph(lambda: cba.cba_attention_backward(d, q, k, v, o, lse, do, None, None, *outs, ws))
    for t in outs:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_gradients_match_differences_of_the_forward(cuda_lib):
    """Central differences of the 64-bit forward loss along random directions, against the GPU's gradients."""
    rng = np.random.default_rng(8)
    args = make(rng, 1, 70, 90, 2, 1, 64, F16, "bshd", 0.125, True, 1.0)
    got = [f8(g[0]) for g in run(*args, 0.125, True)]
    q, k, v, _, _, do = (f8(a[0]) for a in args)
    for i, g in enumerate(got):
        x = [q, k, v]
        step = rng.normal(size=x[i].shape)
        val = []
        for sgn in (1, -1):
            y = list(x)
            y[i] = x[i] + sgn * 1e-5 * step
            val.append((T.attention_forward(*y, 0.125, True)[0] * do).sum())
        want = (val[0] - val[1]) / 2e-5
        # f16 roundings of o (in D), P, dS and the result, each w relatively and independent across elements: 16 w of the
        # directional sum's 2-norm
        bar = 16 * 2.0 ** -11 * np.sqrt(((g * step) ** 2).sum()) + 16 * 2.0 ** -11 * np.abs(g).max() * np.sqrt(g.size) / 8
        assert abs((g * step).sum() - want) <= bar, (i, (g * step).sum(), want, bar)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF)], ids=str)
@pytest.mark.parametrize("len_q,len_k,hq,hk", [(2100, 3900, 2, 1), (1900, 300, 8, 1), (2050, 2050, 4, 4)])
def test_many_items_of_a_tile(cuda_lib, len_q, len_k, hq, hk, dim, dtype, causal):
    """Both sides cut, tiles of up to 15 items, and tiles that stay whole although some SMs go without."""
    rng = np.random.default_rng(len_q + hq)
    args = make(rng, 1, len_q, len_k, hq, hk, dim, dtype, "bshd", 0.1, causal)
    first = [t.clone() for t in run(*args, 0.1, causal)]
    compare(args, first, 0.1, causal, dtype)
    assert all(torch.equal(a, b) for a, b in zip(first, run(*args, 0.1, causal)))


@pytest.mark.parametrize("hk,len_k", [(1, 3), (3, 700), (7, 129)])
def test_the_row_of_v_that_sets_the_scale(cuda_lib, hk, len_k):
    """f16: one row of v a thousand times the rest, the last of all rows; nothing overflows."""
    rng = np.random.default_rng(hk)
    q, k, v, o, lse, do = make(rng, 3, 140, len_k, 2 * hk, hk, 64, F16, "bshd", 0.1, False)
    v[-1, -1, -1] *= 1000.0
    o2, lse2 = T.attention_forward(f8(q[-1]), f8(k[-1]), f8(v[-1]), 0.1, False)
    o[-1] = torch.from_numpy(o2).to("cuda", F16)
    args = (q, k, v, o, lse, do)
    compare(args, run(*args, 0.1, False), 0.1, False, F16)
