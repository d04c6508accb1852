"""Host-side checks of the transformer-layer operators' entry points (no GPU):
every call below is refused before any CUDA call, so no pointer is read."""
import ctypes

import pytest

import activation_backward_gb300 as cba
from activation_backward_gb300 import _binding as B

FAKE, WS = 1 << 20, 1 << 21  # aligned, never dereferenced
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    from activation_backward_gb300 import build
    build.build()
    return B.load()


# ---- layer norm

def ln(**kw):
    return cba.make_layernorm_desc(**{**dict(rows=4, cols=64), **kw})


LN_BAD = [dict(rows=-1), dict(cols=0), dict(type=3), dict(param_type=-1), dict(accumulate=2), dict(eps=NAN), dict(eps=-1.0),
          dict(ld_x=63), dict(ld_dx=-5)]


def ln_fwd(lib, d, x=FAKE, gamma=FAKE, beta=FAKE, y=FAKE, mean=FAKE, rstd=FAKE):
    return lib.cba_layernorm_forward(ctypes.byref(d), x, gamma, beta, y, mean, rstd, None)


def ln_bwd(lib, d, wsb=1 << 30, **kw):
    a = dict(x=FAKE, dy=FAKE, gamma=FAKE, mean=FAKE, rstd=FAKE, residual=None, dx=FAKE, dgamma=FAKE, dbeta=FAKE, ws=WS)
    a.update(kw)
    return lib.cba_layernorm_backward(ctypes.byref(d), *a.values(), wsb, None)


@pytest.mark.parametrize("bad", LN_BAD, ids=str)
def test_layernorm_rejects_a_bad_descriptor(lib, bad):
    d = ln(**bad)
    assert lib.cba_layernorm_workspace_bytes(ctypes.byref(d)) == 0
    assert ln_fwd(lib, d) == cba.CBA_ERR_ARG and ln_bwd(lib, d) == cba.CBA_ERR_ARG


def test_layernorm_unsupported(lib):
    for d in (ln(type=cba.CBA_F16, param_type=cba.CBA_BF16), ln(type=cba.CBA_F32, param_type=cba.CBA_F16), ln(rows=1 << 31),
              ln(ld_x=1 << 40)):
        assert ln_fwd(lib, d) == cba.CBA_ERR_UNSUPPORTED and ln_bwd(lib, d) == cba.CBA_ERR_UNSUPPORTED
        assert lib.cba_layernorm_workspace_bytes(ctypes.byref(d)) == 0


def test_layernorm_pointers_alignment_workspace(lib):
    d = ln()
    for name in ("x", "y"):
        assert ln_fwd(lib, d, **{name: None}) == cba.CBA_ERR_ARG
    for name in ("x", "dy", "mean", "rstd", "dx"):
        assert ln_bwd(lib, d, **{name: None}) == cba.CBA_ERR_ARG
    for name in ("x", "gamma", "mean"):
        assert ln_fwd(lib, d, **{name: FAKE + 2}) == cba.CBA_ERR_ALIGN
        assert ln_bwd(lib, d, **{name: FAKE + 2}) == cba.CBA_ERR_ALIGN
    need = lib.cba_layernorm_workspace_bytes(ctypes.byref(d))
    assert need >= 2 * 64 * 4 and need % 256 == 0
    assert ln_bwd(lib, d, wsb=need - 1) == cba.CBA_ERR_WORKSPACE
    assert ln_bwd(lib, d, ws=None) == cba.CBA_ERR_WORKSPACE
    assert ln_bwd(lib, d, ws=WS + 16) == cba.CBA_ERR_ALIGN
    assert lib.cba_layernorm_forward(None, *([FAKE] * 6), None) == cba.CBA_ERR_ARG


def test_layernorm_workspace_is_small_beside_the_data(lib):
    for rows, cols in ((1 << 15, 4096), (1 << 20, 256), (64, 1 << 16)):
        d = ln(rows=rows, cols=cols)
        assert lib.cba_layernorm_workspace_bytes(ctypes.byref(d)) < max(rows * cols, 64 * cols * 4)


def test_dtype_code():
    import torch
    assert cba.dtype_code(torch.bfloat16) == cba.CBA_BF16
    with pytest.raises(TypeError):
        cba.dtype_code(torch.int32)
