"""Attention's forward pass on the GPU against the 64-bit oracle, element by element.

Bars, from the arithmetic.  w: unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 f16: half a step is half of eps, eps
2^-7 and 2^-10), u = 2^-24 of fp32.  exp(S - m) carries a relative error e from its fp32 exponent (a dot product of `dim`
terms, the subtraction of the maximum, the power of two): e <= C u (1 + |scale| max |q|.|k| + max |lse|), C = 2 dim + 64,
plus w when it is rounded for its product with v.  Numerator and sum are fp32 (C2 u of the sum of absolute terms each, C2 =
4096 at the lengths below), so o is off by (w + 2 e + 2 C2 u) sum_j p_j |v_j| and its own rounding w.  f16 holds p times
2^7 at the row's largest or more, so values under 2^-14 of that unit round to 2^-25 of it: 2^-32 of the largest p each.
lse is off by e + C2 u and its own rounding.
"""
import math

import numpy as np
import pytest
import torch

import activation_backward_gb300 as cba
from activation_backward_gb300 import transformer as tr
from oracle import transformer as T

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
W = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
BF, F16 = torch.bfloat16, torch.float16
C2 = 4096


def f8(t):
    return t.double().cpu().numpy()


def bars(q, k, v, scale, causal, dtype):
    """(o, lse, bar of o, bar of lse) of one sequence, all fp64 arrays; -inf where a row sees no key."""
    o, lse = T.attention_forward(q, k, v, scale, causal)
    bo, bl = np.zeros_like(o), np.zeros_like(lse)
    w, dim, group = W[dtype], q.shape[2], q.shape[1] // k.shape[1]
    if not q.size or not k.size:
        return o, lse, bo, bl
    ok = T.causal_mask(q.shape[0], k.shape[0]) if causal else np.ones((q.shape[0], k.shape[0]), bool)
    for h in range(q.shape[1]):
        j = h // group
        m = np.where(np.isfinite(lse[h]), lse[h], 0.0)
        p = np.where(ok, np.exp(np.minimum(scale * q[:, h] @ k[:, j].T - m[:, None], 0.0)), 0.0)
        e = (2 * dim + 64) * U * (1 + abs(scale) * (np.abs(q[:, h]) @ np.abs(k[:, j]).T).max() + np.abs(m).max())
        small = 2.0 ** -32 * p.max(1, keepdims=True) * ok if dtype == F16 else 0.0
        bo[:, h] = ((w + 2 * e + 2 * C2 * U) * p + small) @ np.abs(v[:, j])
        bl[h] = e + C2 * U + 4 * U * np.abs(m)
    return o, lse, bo * (1 + 2 * w) + 1.01 * w * np.abs(o) + (2.0 ** -25 if dtype == F16 else 0.0), bl


def check(got, want, bar, what):
    got = f8(got)
    with np.errstate(invalid="ignore"):  # -inf - -inf
        bad = ~((np.abs(got - want) <= bar) | (got == want))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} past the bar, worst "
                           f"{np.nanmax(np.abs(got - want)[bad] / np.maximum(bar[bad], 1e-300)):.3g}, first at {np.argwhere(bad)[0]}")


def place(a, layout, dtype):
    """a [batch, len, heads, dim] on the GPU in the given memory order, as that view."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)
    if layout == "bhsd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "wide":  # a slice of a wider projection
        big = torch.full((*t.shape[:2], t.shape[2] + 3, t.shape[3] + 8), math.nan, device="cuda", dtype=dtype)
        big[:, :, 1:1 + t.shape[2], 8:] = t
        return big[:, :, 1:1 + t.shape[2], 8:]
    return t


def run(q, k, v, scale, causal, layout="bshd", cu_q=None, cu_k=None, want_lse=True, **packed):
    o = torch.full(q.shape, 9.0, device="cuda", dtype=q.dtype)
    if layout == "bhsd":
        o = o.transpose(-3, -2).contiguous().transpose(-3, -2)
    lse = torch.full((*q.shape[:-3], q.shape[-2], q.shape[-3]), 9.0, device="cuda") if want_lse else None
    d = cba.make_attention_desc(q, k, v, o, causal=causal, scale=scale, **packed)
    ws = torch.full((cba.cba_attention_forward_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    cba.cba_attention_forward(d, q, k, v, cu_q, cu_k, o, lse, ws)
    assert cba.cba_get_status(ws) == cba.CBA_OK
    return o, lse


def compare(q, k, v, o, lse, scale, causal):
    for b in range(q.shape[0]):
        wo, wl, bo, bl = bars(f8(q[b]), f8(k[b]), f8(v[b]), scale, causal, q.dtype)
        check(o[b], wo, bo, f"o of sequence {b}")
        check(lse[b], wl, bl, f"lse of sequence {b}")


def one(seed, batch, len_q, len_k, hq, hk, dim, dtype, layout, causal, scale=None, q_scale=1.0):
    rng = np.random.default_rng(seed)
    scale = dim ** -0.5 if scale is None else scale
    q = place(rng.normal(size=(batch, len_q, hq, dim)) * q_scale, layout, dtype)
    k, v = (place(rng.normal(size=(batch, len_k, hk, dim)), layout, dtype) for _ in range(2))
    o, lse = run(q, k, v, scale, causal, layout)
    compare(q, k, v, o, lse, scale, causal)


LENGTHS = [(1, 1), (1, 5), (5, 1), (7, 9), (64, 64), (127, 129), (128, 128), (129, 127), (169, 169), (300, 200), (200, 300),
           (1, 700), (700, 1), (257, 640), (513, 513), (640, 255)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("len_q,len_k", LENGTHS)
def test_lengths(cuda_lib, len_q, len_k, causal):
    one(len_q * 1000 + len_k, 2, len_q, len_k, 2, 1, 64, BF, "bshd", causal)
    one(len_q * 1000 + len_k, 1, len_q, len_k, 3, 3, 128, F16, "bhsd", causal)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("dim", [8, 16, 24, 40, 56, 64, 72, 80, 96, 120, 128])
def test_head_dims(cuda_lib, dim, dtype):
    one(dim, 2, 150, 170, 2, 1, dim, dtype, "wide", True)
    one(dim, 1, 3, 400, 4, 2, dim, dtype, "bshd", False)


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (3, 1), (4, 2), (5, 1), (6, 2), (7, 1), (8, 1), (12, 4), (16, 1), (24, 2), (48, 1),
                                   (130, 1), (9, 9)])
@pytest.mark.parametrize("len_q,len_k", [(1, 200), (37, 61), (150, 150)])
def test_shared_heads(cuda_lib, hq, hk, len_q, len_k):
    one(hq * 10 + hk, 1, len_q, len_k, hq, hk, 64, BF, "bhsd", True)


@pytest.mark.parametrize("layout", ["bshd", "bhsd", "wide"])
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("dim", [64, 128])
def test_layouts(cuda_lib, layout, dtype, dim):
    one(5, 3, 140, 140, 4, 2, dim, dtype, layout, True)


def test_slices_of_one_projection(cuda_lib):
    rng = np.random.default_rng(8)
    qkv = torch.from_numpy(rng.normal(size=(2, 169, 3, 4, 64))).to("cuda", BF)
    q, k, v = qkv.unbind(2)
    o, lse = tr.attention(q, k, v, check=True)
    compare(q, k, v, o, lse, 0.125, False)


@pytest.mark.parametrize("batch,len_q,len_k,hq,hk,causal", [
    (1, 1, 5000, 4, 1, True), (1, 1, 5000, 1, 1, False), (3, 2, 3001, 8, 2, True), (1, 17, 4097, 2, 2, True), (2, 129, 2500, 1, 1, True),
    (1, 2500, 2500, 1, 1, True), (1, 1500, 2100, 2, 1, False), (1, 3000, 40, 1, 1, True)])
@pytest.mark.parametrize("dim,dtype", [(128, BF), (64, F16)])
def test_few_rows_over_many_keys(cuda_lib, batch, len_q, len_k, hq, hk, causal, dim, dtype):
    """Too few tiles of queries for the card: the keys are cut and joined."""
    one(len_q + len_k, batch, len_q, len_k, hq, hk, dim, dtype, "bshd", causal)


@pytest.mark.parametrize("len_k", [640, 900, 1300, 1700, 2900, 20000, 33000])
@pytest.mark.parametrize("len_q,hq,hk,causal", [(1, 8, 1, False), (3, 2, 2, True), (300, 2, 1, True)])
def test_numbers_of_items_joined(cuda_lib, len_k, len_q, hq, hk, causal):
    """From two items of a pair of tiles to more than fifty, some of them without keys under the mask."""
    one(len_k, 1, len_q, len_k, hq, hk, 72, BF, "bshd", causal)


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0, 1e-3, 20.0])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_scales(cuda_lib, scale, dtype):
    one(3, 1, 150, 300, 2, 1, 64, dtype, "bshd", True, scale=scale)


@pytest.mark.parametrize("how", ["rising", "falling", "last", "equal"])
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("dim", [64, 128])
def test_maxima_that_move(cuda_lib, how, dtype, dim):
    """Logits that grow (or fall) by 100 and more from one tile of keys to the next: each brings a new maximum."""
    rng = np.random.default_rng(4)
    n = 900
    q, v = rng.normal(size=(1, 200, 2, dim)) * 0.1, rng.normal(size=(1, n, 1, dim))
    k = rng.normal(size=(1, n, 1, dim)) * 0.1
    q[..., 0] = 1.0
    k[..., 0] = {"rising": np.arange(n), "falling": -np.arange(n), "last": np.where(np.arange(n) == n - 1, 300, 0),
                 "equal": np.zeros(n)}[how][None, :, None]
    if how == "equal":
        k[:], q[:] = 1.0, 1.0
    q, k, v = (place(t, "bshd", dtype) for t in (q, k, v))
    for scale in (1.0, 0.25):
        o, lse = run(q, k, v, scale, False)
        compare(q, k, v, o, lse, scale, False)


def test_without_lse(cuda_lib):
    rng = np.random.default_rng(0)
    q, k, v = (place(rng.normal(size=(1, 300, 2, 64)), "bshd", BF) for _ in range(3))
    a, _ = run(q, k, v, 0.125, True)
    b, _ = run(q, k, v, 0.125, True, want_lse=False)
    assert torch.equal(a, b)
    q1 = q[:, :1]
    a, _ = run(q1, k, v, 0.125, False)
    b, _ = run(q1, k, v, 0.125, False, want_lse=False)
    assert torch.equal(a, b)


@pytest.mark.parametrize("causal", [False, True])
def test_no_keys_and_no_queries(cuda_lib, causal):
    q, k = torch.randn(2, 130, 2, 64, device="cuda").to(BF), torch.randn(2, 0, 1, 64, device="cuda").to(BF)
    o, lse = run(q, k, k, 0.125, causal)
    assert (o == 0).all() and torch.isneginf(lse).all()
    q = torch.randn(2, 0, 2, 64, device="cuda").to(BF)
    k = torch.randn(2, 9, 1, 64, device="cuda").to(BF)
    run(q, k, k, 0.125, causal)


def test_rows_without_keys(cuda_lib):
    """Causal with more queries than keys: the first rows see none, in whole tiles of them and in part of one."""
    for len_q, len_k, dim in ((300, 10, 64), (600, 200, 128), (129, 128, 64)):
        q = torch.randn(1, len_q, 2, dim, device="cuda").to(BF)
        k, v = (torch.randn(1, len_k, 2, dim, device="cuda").to(BF) for _ in range(2))
        o, lse = run(q, k, v, 0.1, True)
        n = len_q - len_k
        assert (o[:, :n] == 0).all() and torch.isneginf(lse[..., :n]).all() and torch.isfinite(lse[..., n:]).all()
        compare(q, k, v, o, lse, 0.1, True)


# ---- packed sequences

def packed_case(lens_q, lens_k, hq, hk, dim, dtype, causal, tight=True, before=0, after=0, seed=0):
    """Sequences between NaN rows of neighbours: `before` and `after` tokens belong to none."""
    rng = np.random.default_rng(seed)
    cu = [np.cumsum([before] + list(x)) for x in (lens_q, lens_k)]
    total = [int(c[-1]) + after for c in cu]
    q = place(rng.normal(size=(1, total[0], hq, dim)), "bshd", dtype)[0]
    k, v = (place(rng.normal(size=(1, total[1], hk, dim)), "bshd", dtype)[0] for _ in range(2))
    for t, c in ((q, cu[0]), (k, cu[1]), (v, cu[1])):
        t[:before] = math.nan
        t[int(c[-1]):] = math.nan
    cq, ck = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in cu)
    bound = dict(max_q=max(lens_q), max_k=max(lens_k)) if tight else {}
    o, lse = run(q, k, v, dim ** -0.5, causal, cu_q=cq, cu_k=ck, sequences=len(lens_q), **bound)
    for b in range(len(lens_q)):
        s, t = slice(cu[0][b], cu[0][b + 1]), slice(cu[1][b], cu[1][b + 1])
        wo, wl, bo, bl = bars(f8(q[s]), f8(k[t]), f8(v[t]), dim ** -0.5, causal, dtype)
        check(o[s], wo, bo, f"o of sequence {b}")
        check(lse[:, s], wl, bl, f"lse of sequence {b}")
    for s in (slice(0, before), slice(int(cu[0][-1]), total[0])):  # nobody's rows stay as they were
        assert (o[s] == 9).all() and (lse[:, s] == 9).all()


@pytest.mark.parametrize("tight", [True, False])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([5, 130, 1, 64], None), ([0, 300, 0, 0, 7], None), ([128, 128], None), ([257], None), ([1] * 40, None),
    ([20, 150, 3], [150, 20, 400]), ([1, 1, 1], [700, 0, 3]), ([90, 0], [0, 50])])
def test_packed(cuda_lib, lens_q, lens_k, causal, tight):
    packed_case(lens_q, lens_k or lens_q, 4, 2, 64, BF, causal, tight, before=3, after=70)
    packed_case(lens_q, lens_k or lens_q, 2, 2, 128, F16, causal, tight)


def test_packed_one_long_among_short(cuda_lib):
    packed_case([10, 1900, 30, 5], [10, 1900, 30, 5], 1, 1, 128, BF, True)
    packed_case([1, 1, 1, 1], [2000, 5, 0, 1300], 4, 1, 64, F16, True, tight=True)


def test_packed_neighbours_do_not_leak(cuda_lib):
    """Infinities and NaN of one sequence do not reach another's rows, tile by tile."""
    rng = np.random.default_rng(6)
    lens = [100, 60, 200]
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    q, k, v = (place(rng.normal(size=(1, 360, 2, 64)), "bshd", BF)[0] for _ in range(3))
    o, lse = run(q, k, v, 0.125, False, cu_q=cu, cu_k=cu, sequences=3)
    for bad in (math.nan, math.inf, -math.inf):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for t in (q2, k2, v2):
            t[100:160] = bad
        o2, lse2 = run(q2, k2, v2, 0.125, False, cu_q=cu, cu_k=cu, sequences=3)
        keep = [i for i in range(360) if not 100 <= i < 160]
        assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[:, keep], lse[:, keep])


def test_packed_lengths_past_their_bounds(cuda_lib):
    """Tokens past max_q and max_k are not computed, and nothing past them is written."""
    q, k, v = (torch.randn(300, 2, 64, device="cuda").to(BF) for _ in range(3))
    cu = torch.tensor([0, 200, 300], dtype=torch.int32, device="cuda")
    o, lse = run(q, k, v, 0.125, False, cu_q=cu, cu_k=cu, sequences=2, max_q=150, max_k=120)
    for b, (s, e) in enumerate(((0, 200), (200, 300))):
        n, m = min(e - s, 150), min(e - s, 120)
        wo, wl, bo, bl = bars(f8(q[s:s + n]), f8(k[s:s + m]), f8(v[s:s + m]), 0.125, False, BF)
        check(o[s:s + n], wo, bo, f"o of sequence {b}")
        check(lse[:, s:s + n], wl, bl, f"lse of sequence {b}")
    assert (o[150:200] == 9).all() and (lse[:, 150:200] == 9).all()


# ---- values

def test_nan_and_infinities_spread_in_their_rows(cuda_lib):
    """A NaN in a query row spoils that row alone; in a key or value, every row that sees it."""
    q, k, v = (torch.randn(1, 200, 1, 64, device="cuda").to(BF) for _ in range(3))
    base, _ = run(q, k, v, 0.125, True)
    q2 = q.clone()
    q2[0, 50, 0, 3] = math.nan
    o, lse = run(q2, k, v, 0.125, True)
    assert torch.isnan(o[0, 50]).all() and torch.isnan(lse[0, 0, 50])
    rest = [i for i in range(200) if i != 50]
    assert torch.equal(o[0, rest], base[0, rest])
    k2 = k.clone()
    k2[0, 130, 0, 0] = math.nan
    o, lse = run(q, k2, v, 0.125, True)
    assert torch.isnan(o[0, 130:]).all() and torch.equal(o[0, :130], base[0, :130])  # masked before they are used
    v2 = v.clone()
    v2[0, 130, 0, 7] = math.inf
    o, lse = run(q, k, v2, 0.125, True)
    assert torch.isinf(o[0, 130:, 0, 7]).all() and torch.equal(o[0, :128], base[0, :128])
    assert torch.equal(o[0, 130:, 0, 8:], base[0, 130:, 0, 8:]) and torch.isfinite(lse).all()


def test_large_logits_and_minus_infinity(cuda_lib):
    """Rows whose logits are the fp32 range's: shares of one key; logits of -inf on all keys are a row without keys."""
    q = torch.zeros(1, 4, 1, 64, device="cuda", dtype=BF)
    k, v = torch.zeros(1, 300, 1, 64, device="cuda", dtype=BF), torch.randn(1, 300, 1, 64, device="cuda").to(BF)
    q[0, :, 0, 0] = torch.tensor([1e15, -1e15, 1.0, 0.0])
    k[0, :, 0, 0] = torch.arange(300, device="cuda")
    o, lse = run(q, k, v, 1.0, False)
    kf = k[0, :, 0, 0].double()
    top = (kf == kf.max()).nonzero()[:, 0]
    want = v[0, top, 0].double().mean(0)
    assert (o[0, 0, 0].double() - want).abs().max() <= 2.0 ** -7 * v[0, top, 0].double().abs().max()
    assert torch.equal(o[0, 1, 0], v[0, 0, 0]) and (o[0, 3, 0].double() - v[0, :, 0].double().mean(0)).abs().max() <= 2.0 ** -7
    assert abs(float(lse[0, 0, 3]) - math.log(300)) < 1e-4
    k[0, :, 0, 1] = -math.inf
    q[0, 2, 0, 1] = 1.0
    q[0, [0, 1, 3], 0, 1] = 0.0  # 0 * inf: NaN
    o, lse = run(q, k, v, 1.0, False)
    assert (o[0, 2] == 0).all() and torch.isneginf(lse[0, 0, 2]) and torch.isnan(o[0, [0, 1, 3]]).all()


# ---- runs

def test_same_bits_every_time_and_the_backward_reads_it(cuda_lib):
    for shape in ((1, 1, 4000), (2, 300, 300), (1, 1800, 1800)):
        b, n, m = shape
        q, k, v = (torch.randn(b, i, 2, 64, device="cuda").to(F16) for i in (n, m, m))
        a, la = tr.attention(q, k, v, causal=True, check=True)
        for _ in range(3):
            o, lse = tr.attention(q, k, v, causal=True)
            assert torch.equal(a, o) and torch.equal(la, lse)


def test_gradients_of_its_own_outputs(cuda_lib):
    """attention and attention_backward together against fp64 autograd of the same inputs.  do is 16-bit and exact; o is
    rounded once (w) before D reads it, P and dS once for their products: 8 w of each gradient's norm covers them."""
    for dtype in (BF, F16):
        q, k, v, do = (torch.randn(2, 150, h, 64, device="cuda").to(dtype) for h in (4, 2, 2, 4))
        o, lse = tr.attention(q, k, v, causal=True)
        grads = tr.attention_backward(q, k, v, o, lse, do, causal=True, check=True)
        p = [t.double().requires_grad_() for t in (q, k, v)]
        s = torch.einsum("bihd,bjhd->bhij", p[0], p[1].repeat_interleave(2, 2)) / 8
        s = s.masked_fill(~torch.ones(150, 150, device="cuda").bool().tril(), -math.inf)
        torch.einsum("bhij,bjhd->bihd", s.softmax(-1), p[2].repeat_interleave(2, 2)).backward(do.double())
        for got, x in zip(grads, p):
            assert (got.double() - x.grad).norm() <= 8 * W[dtype] * x.grad.norm()


def test_streams_and_graphs(cuda_lib):
    """Captured and replayed on new inputs, on a stream of its own, with a workspace that two graphs share in turn."""
    shapes = [((1, 1, 3000), True), ((2, 260, 260), False)]
    runs = []
    for (b, n, m), causal in shapes:
        q, k, v = (torch.randn(b, i, 2, 64, device="cuda").to(BF) for i in (n, m, m))
        o, lse = torch.empty_like(q), torch.empty(b, 2, n, device="cuda")
        runs.append((cba.make_attention_desc(q, k, v, o, causal=causal), q, k, v, o, lse))
    ws = torch.empty(max(cba.cba_attention_forward_workspace_bytes(r[0]) for r in runs), dtype=torch.uint8, device="cuda")

    def call(r):
        d, q, k, v, o, lse = r
        cba.cba_attention_forward(d, q, k, v, None, None, o, lse, ws)

    for r in runs:
        call(r)
    torch.cuda.synchronize()
    graphs = []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(r)
        graphs.append(g)
    side = torch.cuda.Stream()
    for r in runs:
        for t in r[1:4]:
            t.copy_(torch.randn_like(t.float()).to(t.dtype))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(2):
            for g in graphs:
                g.replay()
    side.synchronize()
    got = [(r[4].clone(), r[5].clone()) for r in runs]
    for r, (o, lse) in zip(runs, got):
        call(r)
        torch.cuda.synchronize()
        assert torch.equal(r[4], o) and torch.equal(r[5], lse)
        compare(r[1], r[2], r[3], o, lse, 0.125, r[0].causal == 1)


def test_two_streams_at_once(cuda_lib):
    """Two calls with workspaces of their own, in flight at the same time."""
    args = [[torch.randn(2, n, 4, 128, device="cuda").to(BF) for _ in range(3)] for n in (700, 500)]
    want = [tr.attention(*a, causal=True) for a in args]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in args], []
    for s, a in zip(streams, args):
        with torch.cuda.stream(s):
            got.append([tr.attention(*a, causal=True) for _ in range(4)])
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


# ---- ends of the ranges

def test_no_tokens_at_all(cuda_lib):
    """Packed calls without queries, or with bounds of 0, write nothing and leave a status that says so."""
    k = torch.randn(20, 1, 64, device="cuda").to(BF)
    cu = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")
    ck = torch.tensor([0, 9, 20], dtype=torch.int32, device="cuda")
    run(k[:0], k, k, 0.125, True, cu_q=cu, cu_k=ck, sequences=2)
    o, lse = run(k, k, k, 0.125, True, cu_q=ck, cu_k=ck, sequences=2, max_q=0, max_k=0)
    assert (o == 9).all() and (lse == 9).all()
    o, lse = run(k, k[:0], k[:0], 0.125, False, cu_q=ck, cu_k=cu, sequences=2)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_starts_that_are_wrong_stay_in_the_tensors(cuda_lib):
    """Values of cu past the tensors, negative or falling give some result, and rows of one good sequence its own."""
    q = torch.randn(300, 2, 64, device="cuda").to(BF)
    for starts in ([0, 1 << 30, 300], [-5, 200, 100, 1 << 31 - 1], [300, 0, 300]):
        cu = torch.tensor(starts, dtype=torch.int64).clamp(max=2 ** 31 - 1).int().cuda()
        for bound in ({}, dict(max_q=40, max_k=40)):
            run(q, q, q, 0.125, True, cu_q=cu, cu_k=cu, sequences=len(starts) - 1, **bound)


@pytest.mark.parametrize("scale", [3e38, -3e38, 1e-42])
def test_scales_at_the_ends_of_fp32(cuda_lib, scale):
    """Logits that overflow are infinite, equal or none: a row of zeros keeps equal shares."""
    q, k = torch.zeros(1, 3, 1, 64, device="cuda", dtype=BF), torch.zeros(1, 200, 1, 64, device="cuda", dtype=BF)
    v = torch.randn(1, 200, 1, 64, device="cuda").to(BF)
    o, lse = run(q, k, v, scale, False)
    assert torch.allclose(o[0, :, 0].double(), v[0, :, 0].double().mean(0).expand(3, 64), atol=2.0 ** -8)
    assert torch.allclose(lse.double(), torch.full_like(lse.double(), math.log(200)), atol=1e-5)


def test_many_sequences_of_one_token(cuda_lib):
    """4000 packed sequences of a token each, and one long one: slots and search past a warp's width."""
    lens = [1] * 4000 + [700] + [0] * 30 + [1] * 70
    rng = np.random.default_rng(1)
    cu = np.cumsum([0] + lens)
    q, k, v = (place(rng.normal(size=(1, int(cu[-1]), 1, 64)), "bshd", BF)[0] for _ in range(3))
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for bound in ({}, dict(max_q=700, max_k=700)):
        o, lse = run(q, k, v, 0.125, True, cu_q=c, cu_k=c, sequences=len(lens), **bound)
        ones = [i for i in range(4000)] + list(range(4700, 4770))
        assert torch.equal(o[ones], v[ones])
        wo, wl, bo, bl = bars(f8(q[4000:4700]), f8(k[4000:4700]), f8(v[4000:4700]), 0.125, True, BF)
        check(o[4000:4700], wo, bo, "o")
        check(lse[:, 4000:4700], wl, bl, "lse")


def test_offsets_past_32_bits(cuda_lib):
    """Keys and values of a cache whose tokens lie 2^16 elements apart: offsets past 2^31 elements."""
    n, gap = 40000, 1 << 16
    big = torch.empty(n * gap, dtype=BF, device="cuda")
    k = big.as_strided((1, n, 1, 64), (n * gap, gap, 64, 1))
    v = big.as_strided((1, n, 1, 64), (n * gap, gap, 64, 1), 4096)
    k.copy_(torch.randn(1, n, 1, 64, device="cuda").to(BF))
    v.copy_(torch.randn(1, n, 1, 64, device="cuda").to(BF))
    q = torch.randn(1, 5, 1, 64, device="cuda").to(BF)
    a, la = run(q, k, v, 0.125, True)
    b, lb = run(q, k.contiguous(), v.contiguous(), 0.125, True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    del k, v, big
    # o and q the same way
    big = torch.empty(n * gap, dtype=BF, device="cuda")
    q = big.as_strided((1, n, 1, 64), (n * gap, gap, 64, 1))
    o = big.as_strided((1, n, 1, 64), (n * gap, gap, 64, 1), 4096)
    q.copy_(torch.randn(1, n, 1, 64, device="cuda").to(BF))
    kv = torch.randn(1, 50, 1, 64, device="cuda").to(BF)
    d = cba.make_attention_desc(q, kv, kv, o, scale=0.125)
    ws = torch.empty(cba.cba_attention_forward_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    cba.cba_attention_forward(d, q, kv, kv, None, None, o, None, ws)
    want, _ = run(q.contiguous(), kv, kv, 0.125, False)
    assert cba.cba_get_status(ws) == cba.CBA_OK and torch.equal(o, want)


@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, BF), (64, F16)])
@pytest.mark.parametrize("causal", [False, True])
def test_packed_results_do_not_depend_on_the_neighbours_queries(cuda_lib, dim, dtype, causal):
    """A tile's rows behind a sequence hold the next one's queries: whatever their logits, the sequence keeps its bits, over
    several steps of keys."""
    rng = np.random.default_rng(dim)
    lens = [500, 60, 700, 33]
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    n = sum(lens)
    for hq, hk in ((2, 2), (6, 2)):
        q = place(rng.normal(size=(1, n, hq, dim)), "bshd", dtype)[0]
        k, v = (place(rng.normal(size=(1, n, hk, dim)), "bshd", dtype)[0] for _ in range(2))
        for bound in ({}, dict(max_q=700, max_k=700)):
            kw = dict(cu_q=cu, cu_k=cu, sequences=4, **bound)
            o, lse = run(q, k, v, 0.25, causal, **kw)
            for other in (slice(500, 560), slice(1260, 1293)):
                keep = [i for i in range(n) if not other.start <= i < other.stop]
                for change in ("large", "growing", "infinite"):
                    q2 = q.clone()
                    if change == "large":
                        q2[other] *= 1000
                    elif change == "growing":
                        q2[other] *= 4
                    else:
                        q2[other, :, 3] = math.inf
                    o2, lse2 = run(q2, k, v, 0.25, causal, **kw)
                    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[:, keep], lse[:, keep]), change


def guarded(t, value):
    """t [tokens, ...] inside a larger buffer whose other elements are `value`; the view and the buffer."""
    big = torch.full((t.shape[0] + 600, *t.shape[1:]), value, device="cuda", dtype=t.dtype)
    big[300:-300] = t
    return big[300:-300], big


@pytest.mark.parametrize("hq,hk,dim,dtype", [(2, 2, 64, BF), (8, 2, 128, F16)])
@pytest.mark.parametrize("bound", [{}, dict(max_q=300, max_k=300), dict(max_q=40, max_k=70)], ids=str)
@pytest.mark.parametrize("starts,good", [
    ([-5, 120, 1 << 30], [(0, 120), (120, 300)]),                     # taken as 0, 120, 300
    ([0, 120, 300, 90, 90, 2 ** 31 - 1], []),                         # falling, then up past the end, over the others
    ([0, 120, 300, 90, 90], [(0, 120), (120, 300)]),
    ([-2 ** 31, -7, 0, 200, 300, 2 ** 31 - 1], [(0, 200), (200, 300)]),
    ([300, 2 ** 31 - 1, 0], [])])
def test_wrong_starts_leave_the_good_sequences_and_all_else(cuda_lib, starts, good, bound, hq, hk, dim, dtype):
    """Good sequences among wrong starts get their own values; nothing outside the tensors is read (NaN) or written."""
    rng = np.random.default_rng(len(starts))
    (q, _), (k, _), (v, _) = (guarded(place(rng.normal(size=(1, 300, h, dim)), "bshd", dtype)[0], math.nan) for h in (hq, hk, hk))
    o, big_o = guarded(torch.full((300, hq, dim), 9.0, device="cuda", dtype=dtype), 7.0)
    lse_ends = torch.full((hq * 300 + 600,), 7.0, device="cuda")
    lse = lse_ends[300:-300].view(hq, 300).fill_(9.0)
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    d = cba.make_attention_desc(q, k, v, o, causal=True, scale=dim ** -0.5, sequences=len(starts) - 1, **bound)
    ws = torch.full((cba.cba_attention_forward_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    cba.cba_attention_forward(d, q, k, v, cu, cu, o, lse, ws)
    assert cba.cba_get_status(ws) == cba.CBA_OK
    ends = [min(max(s, 0), 300) for s in starts]
    reached = [max(b, a) for a, b in zip(ends, ends[1:])]
    for s, e in good:
        assert sum(a < b and a < e and b > s for a, b in zip(ends, reached)) == 1  # no other sequence writes its rows
        m, n = min(e - s, bound.get("max_q", 300)), min(e - s, bound.get("max_k", 300))
        wo, wl, bo, bl = bars(f8(q[s:s + m]), f8(k[s:s + n]), f8(v[s:s + n]), dim ** -0.5, True, dtype)
        check(o[s:s + m], wo, bo, f"o of {s}")
        check(lse[:, s:s + m], wl, bl, f"lse of {s}")
        assert (o[s + m:e] == 9).all() and (lse[:, s + m:e] == 9).all()
    touched = torch.zeros(300, dtype=torch.bool, device="cuda")
    for a, b in zip(ends, reached):
        touched[a:b] = True
    assert (o[~touched] == 9).all() and (lse[:, ~touched] == 9).all() and torch.isfinite(o.float()).all()
    for ends_of in (big_o[:300], big_o[-300:], lse_ends[:300], lse_ends[-300:]):
        assert (ends_of == 7).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 200])
def test_values_near_the_largest_number(cuda_lib, dim, rows):
    """bf16 values whose sum times 2^8 is just within fp32's range: 1000 of up to 2^109 (2^8 x 1000 x 2^109 < 2^127), under
    logits that come within 2^8 of a new largest one."""
    rng = np.random.default_rng(dim)
    q, k = np.zeros((1, rows, 1, dim)), np.zeros((1, 1000, 1, dim))
    q[..., 0], k[0, 500:, 0, 0] = 1.0, 5.5
    v = 2.0 ** 109 * rng.uniform(0.5, 1, (1, 1000, 1, dim)) * (1 if rows == 1 else rng.choice([-1, 1], (1, 1000, 1, dim)))
    q, k, v = (place(t, "bshd", BF) for t in (q, k, v))
    o, lse = run(q, k, v, 1.0, False)
    compare(q, k, v, o, lse, 1.0, False)
