"""Rows of attention that see no key: whatever the forward left in their o (and lse, where the mask is the library's), they get
dq = 0 and the other rows the bits that they get beside zeros."""
import numpy as np
import pytest
import torch

from .test_gpu_attention import BF, F16, compare, make, pack, run

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
TYPES = [(64, BF), (128, BF), (64, F16), (128, F16)]


@pytest.mark.parametrize("left_in_o,left_in_lse", [(NAN, -INF), (INF, -INF), (NAN, NAN), (0.0, NAN), (3.0, 0.0)])
@pytest.mark.parametrize("dim,dtype", TYPES, ids=str)
def test_queries_before_the_first_key(cuda_lib, dim, dtype, left_in_o, left_in_lse):
    """Causal, 300 queries and 150 keys: a tile without keys, and 22 rows of one that has some."""
    rng = np.random.default_rng(dim)
    args = make(rng, 2, 300, 150, 4, 2, dim, dtype, "bshd", 0.1, True)
    clean = [t.clone() for t in run(*args, 0.1, True)]
    compare(args, clean, 0.1, True, dtype)
    args[3][:, :150] = left_in_o
    args[4][:, :, :150] = left_in_lse
    dirty = run(*args, 0.1, True)
    assert torch.all(dirty[0][:, :150] == 0)
    assert all(torch.equal(x, y) for x, y in zip(clean, dirty))


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dim,dtype", TYPES, ids=str)
def test_rows_that_the_callers_mask_emptied(cuda_lib, dim, dtype, causal):
    rng = np.random.default_rng(dim + 1)
    args = make(rng, 1, 200, 210, 2, 1, dim, dtype, "bshd", 0.1, causal)
    rows = [0, 7, 131, 199]
    args[3][:, rows] = 0
    args[4][:, :, rows] = -INF
    clean = [t.clone() for t in run(*args, 0.1, causal)]
    compare(args, clean, 0.1, causal, dtype)
    args[3][:, rows] = NAN
    dirty = run(*args, 0.1, causal)
    assert torch.all(dirty[0][:, rows] == 0)
    assert all(torch.equal(x, y) for x, y in zip(clean, dirty))


@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
def test_packed_rows_without_keys(cuda_lib, dtype):
    rng = np.random.default_rng(3)
    lens_q, lens_k = (200, 40, 90), (60, 0, 90)
    _, args, cu = pack(rng, lens_q, lens_k, 4, 2, 72, dtype, 0.1, True)
    kw = dict(cu_q=cu[0], cu_k=cu[1], sequences=3, max_q=200, max_k=90)
    clean = [t.clone() for t in run(*args, 0.1, True, **kw)]
    for rows in (slice(0, 140), slice(200, 240)):
        args[3][rows] = NAN
        args[4][:, rows] = NAN
    dirty = run(*args, 0.1, True, **kw)
    assert torch.all(dirty[0][:140] == 0) and torch.all(dirty[0][200:240] == 0)
    assert all(torch.equal(x, y) for x, y in zip(clean, dirty))
