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


# ---- attention's backward pass

def at(**kw):
    d = B.cba_attention_desc_t()
    base = dict(batch=2, heads_q=4, heads_kv=2, dim=64, len_q=100, len_k=90, packed=0, type=cba.CBA_BF16, total_q=0, total_k=0,
                causal=1, scale=0.125)
    for n, v in {**base, **kw}.items():
        setattr(d, n, v)
    return d


def at_bwd(lib, d, wsb=1 << 40, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, dout=FAKE, cu_q=None, cu_k=None, dq=FAKE, dk=FAKE, dv=FAKE, ws=WS)
    a.update(kw)
    return lib.cba_attention_backward(ctypes.byref(d), *a.values(), wsb, None)


AT_BAD = [dict(batch=0), dict(heads_q=0), dict(heads_kv=3), dict(dim=0), dict(len_q=-1), dict(type=7), dict(causal=2), dict(packed=2),
          dict(scale=NAN), dict(packed=1, total_q=-1), dict(q=cba.cba_attn_strides_t(-8, 64, 64)),
          dict(k=cba.cba_attn_strides_t(0, 128, 64)),  # two batches at the same place
          dict(dv=cba.cba_attn_strides_t(1 << 20, 128, 32))]  # heads that overlap


@pytest.mark.parametrize("bad", AT_BAD, ids=lambda b: "-".join(b))
def test_attention_rejects_a_bad_descriptor(lib, bad):
    d = at(**bad)
    assert lib.cba_attention_workspace_bytes(ctypes.byref(d)) == 0
    assert at_bwd(lib, d) == cba.CBA_ERR_ARG


def test_attention_unsupported(lib):
    for kw in (dict(type=cba.CBA_F32), dict(dim=136), dict(dim=60), dict(len_q=1 << 31 - 1), dict(batch=1 << 24, len_q=1 << 14)):
        assert at_bwd(lib, at(**kw)) == cba.CBA_ERR_UNSUPPORTED, kw
    d = at(o=cba.cba_attn_strides_t(1 << 20, 260, 64))
    assert at_bwd(lib, d) == cba.CBA_ERR_ALIGN and lib.cba_attention_workspace_bytes(ctypes.byref(d)) == 0


def test_attention_pointers_alignment_workspace(lib):
    d = at()
    for name in ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv"):
        assert at_bwd(lib, d, **{name: None}) == cba.CBA_ERR_ARG, name
    for name in ("q", "dout", "dv"):
        assert at_bwd(lib, d, **{name: FAKE + 8}) == cba.CBA_ERR_ALIGN, name
    assert at_bwd(lib, d, cu_q=FAKE) == cba.CBA_ERR_ARG          # dense has no sequence starts
    p = at(packed=1, total_q=50, total_k=60)
    assert at_bwd(lib, p) == cba.CBA_ERR_ARG                     # packed needs them
    assert at_bwd(lib, p, cu_q=FAKE, cu_k=FAKE, wsb=0) == cba.CBA_ERR_WORKSPACE
    need = lib.cba_attention_workspace_bytes(ctypes.byref(d))
    assert need >= 2 * 4 * 128 * 8
    assert at_bwd(lib, d, wsb=need - 1) == cba.CBA_ERR_WORKSPACE
    assert at_bwd(lib, d, ws=WS + 128) == cba.CBA_ERR_ALIGN


def test_attention_descriptor_of_tensors():
    import torch
    qkv = torch.zeros(2, 10, 3, 4, 64, dtype=torch.bfloat16)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    o = torch.zeros(2, 4, 10, 64, dtype=torch.bfloat16).transpose(1, 2)
    d = cba.make_attention_desc(q, k, v, o, o, o, o, o, causal=True)
    assert (d.batch, d.len_q, d.len_k, d.heads_q, d.heads_kv, d.dim, d.packed) == (2, 10, 10, 4, 4, 64, 0)
    assert (d.k.batch, d.k.token, d.k.head) == (10 * 768, 768, 64) and (d.o.batch, d.o.token, d.o.head) == (2560, 64, 640)
    assert abs(d.scale - 0.125) < 1e-7
    p = torch.zeros(30, 4, 64, dtype=torch.float16)
    d = cba.make_attention_desc(p, p, p, p, p, p, p, p, sequences=3, max_q=20)
    assert (d.packed, d.batch, d.total_q, d.len_q, d.len_k) == (1, 3, 30, 20, 30)
    for bad in (dict(q=q.float()), dict(dv=v[:, :5]), dict(o=o[..., :32]), dict(k=k[:1]), dict(q=p), dict(dq=o.transpose(2, 3))):
        a = dict(q=q, k=k, v=v, o=o, dout=o, dq=o, dk=o, dv=o)
        a.update(bad)
        with pytest.raises(ValueError):
            cba.make_attention_desc(**a)


# ---- Newton-Schulz orthogonalisation

def ns(**kw):
    return cba.make_orthogonalize_desc(**{**dict(batch=2, rows=40, cols=70), **kw})


def ns_call(lib, d, G=FAKE, O=FAKE, ws=WS, wsb=1 << 40):
    return lib.cba_orthogonalize(ctypes.byref(d), G, O, ws, wsb, None)


@pytest.mark.parametrize("bad", [dict(batch=0), dict(rows=0), dict(cols=-1), dict(steps=0), dict(in_type=4), dict(out_type=-1),
                                 dict(coefficients=(NAN, 1, 1)), dict(eps=-1.0), dict(scale=float("inf")), dict(ld_in=69),
                                 dict(ld_out=-1), dict(batch_in=2799), dict(batch_out=5)], ids=str)
def test_orthogonalize_rejects_a_bad_descriptor(lib, bad):
    d = ns(**bad)
    assert lib.cba_orthogonalize_workspace_bytes(ctypes.byref(d)) == 0
    assert ns_call(lib, d) == cba.CBA_ERR_ARG


def test_orthogonalize_limits_pointers_workspace(lib):
    for kw in (dict(steps=101), dict(rows=1 << 21, cols=3), dict(batch=1 << 17)):
        assert ns_call(lib, ns(**kw)) == cba.CBA_ERR_UNSUPPORTED
    d = ns()
    assert ns_call(lib, d, G=None) == cba.CBA_ERR_ARG and ns_call(lib, d, O=None) == cba.CBA_ERR_ARG
    assert ns_call(lib, d, G=FAKE + 2) == cba.CBA_ERR_ALIGN and ns_call(lib, d, O=FAKE + 1) == cba.CBA_ERR_ALIGN
    need = lib.cba_orthogonalize_workspace_bytes(ctypes.byref(d))
    assert need > 2 * (2 * 40 * 72 + 2 * 40 * 40) * 2
    assert ns_call(lib, d, wsb=need - 1) == cba.CBA_ERR_WORKSPACE and ns_call(lib, d, ws=None) == cba.CBA_ERR_WORKSPACE
    assert ns_call(lib, d, ws=WS + 64) == cba.CBA_ERR_ALIGN
