"""The power of two by which f16 attention gradients hold dS belongs to one sequence and key/value head, and to its finite
rows: nothing else changes a bit of it (bars and their derivation: test_gpu_attention)."""
import numpy as np
import pytest
import torch

from .test_gpu_attention import BF, F16, bars, check, f8, make, pack, run

pytestmark = pytest.mark.gpu
LENS = (100, 60, 200, 130, 77)
ENDS = np.cumsum((0,) + LENS)


def call(args, cu, causal, max_len=200):
    return [t.clone() for t in run(*args, 0.1, causal, cu_q=cu[0], cu_k=cu[1], sequences=len(cu[0]) - 1, max_q=max_len, max_k=max_len)]


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 6e4])
@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, F16), (128, BF)], ids=str)
def test_another_sequence_changes_no_bit(cuda_lib, dim, dtype, bad, causal):
    """Small gradients beside a sequence of infinities, NaN or the largest numbers."""
    rng = np.random.default_rng(dim)
    parts = [make(rng, 1, n, n, 4, 2, dim, dtype, "bshd", 0.1, causal, 2e-3) for n in LENS]
    args = [torch.cat([p[i][0] for p in parts]) for i in (0, 1, 2, 3)] + [torch.cat([p[4][0] for p in parts], 1).contiguous(),
                                                                          torch.cat([p[5][0] for p in parts])]
    cu = [torch.tensor(ENDS, dtype=torch.int32, device="cuda")] * 2
    clean = call(args, cu, causal)
    for i in (1, 3):
        for t in (args[2], args[3], args[5]):
            t[ENDS[i]:ENDS[i + 1]] = bad
    dirty = call(args, cu, causal)
    for x, y in zip(clean, dirty):
        for i in (0, 2, 4):
            assert torch.equal(x[ENDS[i]:ENDS[i + 1]], y[ENDS[i]:ENDS[i + 1]])


@pytest.mark.parametrize("dim", [64, 128])
def test_tokens_of_no_sequence_change_no_bit(cuda_lib, dim):
    rng = np.random.default_rng(dim)
    _, (q, k, v, o, lse, do), cu = pack(rng, LENS, LENS, 2, 1, dim, F16, 0.1, False)
    do *= 0.02
    clean = call((q, k, v, o, lse, do), cu, False)
    more = [torch.cat([t, torch.full((30, *t.shape[1:]), float("inf"), device="cuda", dtype=F16)]) for t in (q, k, v, o, do)]
    lse = torch.cat([lse, torch.zeros(2, 30, device="cuda")], 1).contiguous()
    dirty = call((*more[:4], lse, more[4]), cu, False)
    for x, y in zip(clean, dirty):
        assert torch.equal(x, y[:len(x)])


@pytest.mark.parametrize("dim", [64, 128])
def test_an_infinite_row_spreads_as_in_the_formulas(cuda_lib, dim):
    """do of one query under the first key/value head: the other queries' dq keep their accuracy, the other head its bits."""
    rng = np.random.default_rng(dim + 1)
    args = make(rng, 2, 150, 170, 4, 2, dim, F16, "bshd", 0.1, False, 2e-3)
    q, k, v, o, lse, do = args
    clean = [t.clone() for t in run(*args, 0.1, False)]
    want, bar = bars(*(f8(a[1]) for a in args), 0.1, False, F16)
    do[1, 40, 1] = float("inf")
    dq, dk, dv = run(*args, 0.1, False)
    for x, y in zip(clean, (dq, dk, dv)):
        assert torch.equal(x[0], y[0])
    assert torch.equal(clean[0][1, :, 2:], dq[1, :, 2:])
    assert torch.equal(clean[1][1, :, 1], dk[1, :, 1]) and torch.equal(clean[2][1, :, 1], dv[1, :, 1])
    rows = np.delete(np.arange(150), 40)
    check(dq[1, rows, :2], want[0][rows, :2], bar[0][rows, :2], "dq")
    assert not torch.isfinite(dq[1, 40, 1].float()).any() and not torch.isfinite(dk[1, :, 0].float()).any()


def test_heads_of_unlike_size(cuda_lib):
    """One key/value head's values and gradients are ten thousand times another's: each keeps its own accuracy."""
    rng = np.random.default_rng(9)
    args = list(make(rng, 1, 140, 160, 4, 2, 64, F16, "bshd", 0.125, False, 1e-3))
    big = make(rng, 1, 140, 160, 4, 2, 64, F16, "bshd", 0.125, False, 300.0)
    for i in (0, 3, 5):
        args[i][:, :, :2] = big[i][:, :, :2]
    for i in (1, 2):
        args[i][:, :, :1] = big[i][:, :, :1]
    args[4][:, :2] = big[4][:, :2]
    outs = run(*args, 0.125, False)
    for j in (0, 1):  # the oracle's bars take the largest rows of the heads that they are given
        a = [f8(t[0]) for t in args]
        h = slice(2 * j, 2 * j + 2)
        want, bar = bars(a[0][:, h], a[1][:, j:j + 1], a[2][:, j:j + 1], a[3][:, h], a[4][h], a[5][:, h], 0.125, False, F16)
        for g, x, y, s, name in zip(outs, want, bar, (h, slice(j, j + 1), slice(j, j + 1)), ("dq", "dk", "dv")):
            check(g[0][:, s], x, y, f"{name} of head {j}")
