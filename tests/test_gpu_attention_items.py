"""Attention's backward pass where a block's work items follow one another in unusual orders, or are handed out from loose
bounds, against the 64-bit oracle (the bars are derived in test_gpu_attention)."""
import numpy as np
import pytest
import torch

import activation_backward_gb300 as cba
from .test_gpu_attention import BF, F16, compare, pack, run

pytestmark = pytest.mark.gpu


def check_packed(rng, lens_q, lens_k, hq, hk, dim, dtype, scale, causal, repeat=2, max_q=None, max_k=None):
    parts, args, cu = pack(rng, lens_q, lens_k, hq, hk, dim, dtype, scale, causal)
    kw = dict(cu_q=cu[0], cu_k=cu[1], sequences=len(lens_q), max_q=max_q or max(lens_q), max_k=max_k or max(lens_k))
    outs = [t.clone() for t in run(*args, scale, causal, **kw)]
    at = [0, 0]
    for p, a, b in zip(parts, lens_q, lens_k):
        own = [outs[0][None, at[0]:at[0] + a], outs[1][None, at[1]:at[1] + b], outs[2][None, at[1]:at[1] + b]]
        compare(p, own, scale, causal, dtype)
        at = [at[0] + a, at[1] + b]
    for _ in range(repeat):
        assert all(torch.equal(x, y) for x, y in zip(outs, run(*args, scale, causal, **kw)))
    return outs


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, BF), (96, F16)], ids=str)
def test_query_tiles_without_keys_between_others(cuda_lib, dim, dtype, causal):
    """Sequences whose queries see no key at all among others, and (causal) tiles whose queries come before the first key:
    a block meets tiles with and without work in any order."""
    rng = np.random.default_rng(dim + causal)
    lens_q = [int(x) for x in rng.integers(1, 300, size=90)]
    lens_k = [0 if rng.random() < 0.4 else int(rng.integers(1, 260)) for _ in lens_q]
    check_packed(rng, lens_q, lens_k, 6, 2, dim, dtype, 0.1, causal, repeat=4)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, BF), (128, F16)], ids=str)
def test_items_of_one_step_far_apart(cuda_lib, dim, dtype, causal):
    """Sequences of a tile each beside a long one: an item of one step is over long before its block has walked past the
    tiles that do not exist to the next."""
    rng = np.random.default_rng(dim)
    lens = [int(x) for x in rng.integers(1, 129, size=260)]
    lens[100] = 1500
    check_packed(rng, lens, lens, 4, 4, dim, dtype, 0.1, causal, repeat=3)


def spread(rng, n, longest):
    return [int(x) for x in rng.integers(0, longest, size=n)]


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, BF), (64, F16), (128, F16)], ids=str)
@pytest.mark.parametrize("count,longest", [(60, 420), (33, 130), (300, 40), (5, 700)])
def test_bounds_far_above_the_lengths(cuda_lib, count, longest, dim, dtype, causal):
    """All tokens as the bound of every sequence's length, as when none is given."""
    rng = np.random.default_rng(dim + count)
    lens_q, lens_k = spread(rng, count, longest), spread(rng, count, longest)
    loose = check_packed(rng, lens_q, lens_k, 4, 2, dim, dtype, 0.1, causal, 1, sum(lens_q), sum(lens_k))
    same = np.random.default_rng(dim + count)
    assert (spread(same, count, longest), spread(same, count, longest)) == (lens_q, lens_k)
    tight = check_packed(same, lens_q, lens_k, 4, 2, dim, dtype, 0.1, causal, 0)
    if count > 5:  # (no tile is cut into items)
        assert all(torch.equal(x, y) for x, y in zip(loose, tight))


def test_loose_bounds_and_tiles_cut_into_items(cuda_lib):
    rng = np.random.default_rng(12)
    lens = [0, 1700, 5, 900, 130]
    check_packed(rng, lens, lens, 4, 1, 128, BF, 0.1, True, 2, 1 << 20, 1 << 20)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
def test_tokens_outside_every_sequence_are_left_alone(cuda_lib, dtype, causal):
    """Room before the first sequence and after the last; keys for queries that are not there and the other way round."""
    rng = np.random.default_rng(13)
    lens_q, lens_k = [90, 0, 300, 7, 0, 140] * 4, [130, 60, 0, 200, 0, 129] * 4
    parts, (q, k, v, o, lse, do), cu = pack(rng, lens_q, lens_k, 2, 1, 72, dtype, 0.1, causal)
    pad = [torch.full((200, *t.shape[1:]), float("nan"), device="cuda", dtype=dtype) for t in (q, k, v, o, do)]
    q, k, v, o, do = (torch.cat([p[:150], t, p]) for p, t in zip(pad, (q, k, v, o, do)))
    lse = torch.cat([lse[:, :1].expand(2, 150), lse, lse[:, :1].expand(2, 200)], 1).contiguous()
    outs = run(q, k, v, o, lse, do, 0.1, causal, cu_q=cu[0] + 150, cu_k=cu[1] + 150, sequences=24, max_q=None, max_k=None)
    for t in outs:
        assert torch.all(t[:150] == 9) and torch.all(t[-200:] == 9)
    at = [150, 150]
    for p, a, b in zip(parts, lens_q, lens_k):
        own = [outs[0][None, at[0]:at[0] + a], outs[1][None, at[1]:at[1] + b], outs[2][None, at[1]:at[1] + b]]
        compare(p, own, 0.1, causal, dtype)
        at = [at[0] + a, at[1] + b]


def test_the_torch_call_without_bounds(cuda_lib):
    """1500 short sequences: tiles counted up to the default bound would be half a million a head."""
    from activation_backward_gb300 import transformer as tr
    rng = np.random.default_rng(14)
    lens = spread(rng, 1500, 60)
    _, (q, k, v, o, lse, do), cu = pack(rng, lens, lens, 2, 1, 64, BF, 0.1, True)
    loose = tr.attention_backward(q, k, v, o, lse, do, causal=True, scale=0.1, cu_q=cu[0])
    tight = run(q, k, v, o, lse, do, 0.1, True, cu_q=cu[0], cu_k=cu[0], sequences=1500, max_q=60, max_k=60)
    assert all(torch.equal(x, y) for x, y in zip(loose, tight))


@pytest.mark.parametrize("batch_stride", [0, 1 << 37], ids=["contiguous", "batch strides"])
@pytest.mark.parametrize("dim,dtype", [(64, BF), (72, F16), (128, F16)], ids=str)
def test_packed_batch_strides_are_not_used(cuda_lib, dim, dtype, batch_stride):
    """Strides of 0 (contiguous) or with anything as the batch stride: a packed sequence starts where cu says."""
    rng = np.random.default_rng(15)
    lens_q, lens_k = (40, 0, 150, 9), (60, 30, 140, 200)
    parts, (q, k, v, o, lse, do), cu = pack(rng, lens_q, lens_k, 4, 2, dim, dtype, 0.1, True)
    outs = [torch.full_like(t, 9.0) for t in (q, k, v)]
    d = cba.make_attention_desc(q, k, v, o, do, *outs, causal=True, scale=0.1, sequences=4, max_q=150, max_k=200)
    for name in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
        s = getattr(d, name)
        setattr(d, name, cba.cba_attn_strides_t(batch_stride, s.token, s.head) if batch_stride else cba.cba_attn_strides_t(0, 0, 0))
    ws = torch.empty(cba.cba_attention_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    cba.cba_attention_backward(d, q, k, v, o, lse, do, *cu, *outs, ws)
    assert cba.cba_get_status(ws) == cba.CBA_OK
    at = [0, 0]
    for p, a, b in zip(parts, lens_q, lens_k):
        own = [outs[0][None, at[0]:at[0] + a], outs[1][None, at[1]:at[1] + b], outs[2][None, at[1]:at[1] + b]]
        compare(p, own, 0.1, True, dtype)
        at = [at[0] + a, at[1] + b]


@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
def test_one_packed_query_of_one_head(cuda_lib, dtype):
    """Every axis of q has one index, so that its descriptor has no strides; the query belongs to the third sequence."""
    rng = np.random.default_rng(16)
    check_packed(rng, (0, 0, 1, 0), (30, 7, 50, 0), 1, 1, 64, dtype, 0.1, False)
