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
