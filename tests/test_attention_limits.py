"""Which packed attention calls the library accepts (no GPU): the limit is on tiles that can exist, not on what loose bounds of
the sequences' lengths multiply up to."""
import ctypes

import pytest

from activation_backward_gb300 import _binding as B

from .test_transformer_host import at, lib  # noqa: F401


@pytest.mark.parametrize("batch,total", [(4096, 1 << 20), (1 << 16, 1 << 22), (1, 1 << 25), (1 << 20, 1 << 20)])
def test_packed_calls_with_the_default_bounds(lib, batch, total):  # noqa: F811
    """Every length bounded by all tokens, as the torch call does without max_q and max_k."""
    d = at(packed=1, batch=batch, heads_q=32, heads_kv=8, total_q=total, total_k=total, len_q=total, len_k=total)
    need = lib.cba_attention_workspace_bytes(ctypes.byref(d))
    rows = (total + 127) // 128 * 128 + 128 * (batch + 1)
    assert 8 * 32 * rows <= need < 8 * 32 * rows + (1 << 30)


def test_bounds_above_the_tokens_change_nothing(lib):  # noqa: F811
    need = [lib.cba_attention_workspace_bytes(ctypes.byref(at(packed=1, batch=3, total_q=5000, total_k=4000, len_q=a, len_k=b)))
            for a, b in ((5000, 4000), (1 << 20, 1 << 29))]
    assert need[0] == need[1] > 0
