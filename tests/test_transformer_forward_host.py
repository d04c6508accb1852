"""Host-side checks of the entry points of attention's forward pass, of query/key norms with rotation and of dropout (no
GPU): every call below is refused before any CUDA call, so no pointer is read."""
import ctypes

import pytest

import activation_backward_gb300 as cba
from activation_backward_gb300 import _binding as B

FAKE, WS = 1 << 20, 1 << 21  # aligned, never dereferenced
NAN = float("nan")
ST = cba.cba_attn_strides_t


@pytest.fixture(scope="module")
def lib():
    from activation_backward_gb300 import build
    build.build()
    return B.load()


def filled(d, base, kw):
    for n, v in {**base, **kw}.items():
        setattr(d, n, v)
    return d


# ---- attention's forward pass

def at(**kw):
    return filled(B.cba_attention_desc_t(), dict(batch=2, heads_q=4, heads_kv=2, dim=64, len_q=100, len_k=90, packed=0,
                                                 type=cba.CBA_BF16, causal=1, scale=0.125), kw)


def at_fwd(lib, d, wsb=1 << 40, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cu_q=None, cu_k=None, o=FAKE, lse=FAKE, ws=WS)
    a.update(kw)
    return lib.cba_attention_forward(ctypes.byref(d), *a.values(), wsb, None)


@pytest.mark.parametrize("bad", [dict(batch=0), dict(heads_q=0), dict(heads_kv=3), dict(dim=0), dict(len_q=-1), dict(type=7),
                                 dict(causal=2), dict(packed=2), dict(scale=NAN), dict(packed=1, total_q=-1), dict(q=ST(-8, 64, 64)),
                                 dict(k=ST(0, 128, 64)), dict(o=ST(1 << 20, 128, 32))], ids=lambda b: "-".join(b))
def test_attention_rejects_a_bad_descriptor(lib, bad):
    d = at(**bad)
    assert lib.cba_attention_forward_workspace_bytes(ctypes.byref(d)) == 0
    assert at_fwd(lib, d) == cba.CBA_ERR_ARG


def test_attention_limits(lib):
    for kw in (dict(type=cba.CBA_F32), dict(dim=136), dict(dim=60), dict(len_q=1 << 31 - 1), dict(batch=1 << 24, len_q=1 << 14),
               dict(batch=(1 << 31) - 1, len_q=1 << 30, heads_q=(1 << 31) - 1, heads_kv=(1 << 31) - 1)):
        assert at_fwd(lib, at(**kw)) == cba.CBA_ERR_UNSUPPORTED, kw
    d = at(o=ST(1 << 20, 260, 64))
    assert at_fwd(lib, d) == cba.CBA_ERR_ALIGN and lib.cba_attention_forward_workspace_bytes(ctypes.byref(d)) == 0


def test_attention_pointers_alignment_workspace(lib):
    d = at()
    for name in ("q", "k", "v", "o"):
        assert at_fwd(lib, d, **{name: None}) == cba.CBA_ERR_ARG, name
        assert at_fwd(lib, d, **{name: FAKE + 8}) == cba.CBA_ERR_ALIGN, name
    assert at_fwd(lib, d, lse=FAKE + 2) == cba.CBA_ERR_ALIGN
    assert at_fwd(lib, d, cu_q=FAKE) == cba.CBA_ERR_ARG          # dense has no sequence starts
    p = at(packed=1, total_q=50, total_k=60)
    assert at_fwd(lib, p) == cba.CBA_ERR_ARG                     # packed needs them
    assert at_fwd(lib, p, cu_q=FAKE, cu_k=FAKE + 1) == cba.CBA_ERR_ALIGN
    assert at_fwd(lib, p, cu_q=FAKE, cu_k=FAKE, wsb=0) == cba.CBA_ERR_WORKSPACE
    for x in (d, p, at(batch=1, len_q=1, len_k=1 << 16)):
        kw = dict(cu_q=FAKE, cu_k=FAKE) if x.packed else {}
        need = lib.cba_attention_forward_workspace_bytes(ctypes.byref(x))
        assert need >= 256 and need % 256 == 0
        assert at_fwd(lib, x, wsb=need - 1, **kw) == cba.CBA_ERR_WORKSPACE and at_fwd(lib, x, ws=None, **kw) == cba.CBA_ERR_WORKSPACE
        assert at_fwd(lib, x, ws=WS + 128, **kw) == cba.CBA_ERR_ALIGN
    assert lib.cba_attention_forward(None, *([FAKE] * 8), 1 << 20, None) == cba.CBA_ERR_ARG


def test_attention_workspace_is_bounded(lib):
    """Sums of cut tiles: a tile of 256 rows for every SM a few times over, whatever the lengths."""
    for kw in (dict(batch=64, len_q=1, len_k=1 << 17), dict(batch=1, len_q=1 << 17, len_k=1 << 17, heads_q=1, heads_kv=1),
               dict(batch=512, len_q=4096, len_k=4096), dict(batch=1, len_q=100, len_k=1 << 29), dict(batch=1 << 16, len_q=1)):
        assert 0 < lib.cba_attention_forward_workspace_bytes(ctypes.byref(at(dim=128, **kw))) < 1 << 28, kw


def test_attention_descriptor_without_gradients():
    import torch
    q, o = torch.zeros(2, 10, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 10, 64, dtype=torch.bfloat16).transpose(1, 2)
    d = cba.make_attention_desc(q, q[:, :, :2], q[:, :, :2], o)
    assert (d.heads_q, d.heads_kv, d.len_q) == (4, 2, 10) and (d.o.batch, d.o.token, d.o.head) == (2560, 64, 640)
    assert (d.k.token, d.dq.token, d.dout.token) == (256, 0, 0)


@pytest.mark.parametrize("kw", [dict(len_q=(1 << 30) + 1), dict(len_k=(1 << 30) + 1), dict(len_q=(1 << 31) - 1),
                                dict(packed=1, total_q=(1 << 30) + 1), dict(packed=1, total_k=1 << 40),
                                dict(q=ST(1 << 38, 256, 64)), dict(type=cba.CBA_F32), dict(dim=136), dict(dim=60),
                                dict(batch=1 << 24, len_q=1 << 14)], ids=str)
def test_attention_past_its_limits_has_no_workspace(lib, kw):
    """Refused by the checks themselves: the workspace query, which needs no driver, refuses the descriptor too."""
    d = at(**kw)
    assert lib.cba_attention_forward_workspace_bytes(ctypes.byref(d)) == 0
    cu = dict(cu_q=FAKE, cu_k=FAKE) if d.packed else {}
    assert at_fwd(lib, d, **cu) == cba.CBA_ERR_UNSUPPORTED


def test_attention_takes_lengths_up_to_its_limit(lib):
    for kw in (dict(len_q=1 << 30), dict(len_k=1 << 30), dict(packed=1, total_q=1 << 30, total_k=1 << 30)):
        assert lib.cba_attention_forward_workspace_bytes(ctypes.byref(at(**kw))) >= 256, kw


# ---- query and key norms with rotation

def qk(**kw):
    return filled(B.cba_qk_norm_rope_desc_t(), dict(batch=2, len=10, heads_q=4, heads_k=2, dim=64, type=cba.CBA_BF16,
                                                    param_type=cba.CBA_F32, norm=1, rot_dim=64, positions=16, eps=1e-6), kw)


def qk_fwd(lib, d, **kw):
    a = dict(q=FAKE, k=FAKE, gamma_q=FAKE, gamma_k=FAKE, table=FAKE, pos=FAKE, yq=FAKE, yk=FAKE)
    a.update(kw)
    return lib.cba_qk_norm_rope_forward(ctypes.byref(d), *a.values(), None)


def qk_bwd(lib, d, wsb=1 << 30, **kw):
    a = dict(q=FAKE, k=FAKE, gamma_q=FAKE, gamma_k=FAKE, table=FAKE, pos=FAKE, dyq=FAKE, dyk=FAKE, dq=FAKE, dk=FAKE, dgamma_q=FAKE,
             dgamma_k=FAKE, ws=WS)
    a.update(kw)
    return lib.cba_qk_norm_rope_backward(ctypes.byref(d), *a.values(), wsb, None)


@pytest.mark.parametrize("bad", [dict(batch=0), dict(len=-1), dict(heads_q=0), dict(heads_k=-1), dict(dim=0), dict(type=3),
                                 dict(param_type=-1), dict(norm=2), dict(interleaved=-1), dict(accumulate=3), dict(rot_dim=-2),
                                 dict(rot_dim=66), dict(rot_dim=7), dict(positions=0), dict(eps=NAN), dict(eps=-1.0),
                                 dict(q=ST(640, -8, 64)), dict(yk=ST(0, 128, 64)), dict(dq=ST(2560, 256, 32))], ids=str)
def test_qk_rejects_a_bad_descriptor(lib, bad):
    d = qk(**bad)
    assert lib.cba_qk_norm_rope_workspace_bytes(ctypes.byref(d)) == 0
    assert qk_fwd(lib, d) == cba.CBA_ERR_ARG and qk_bwd(lib, d) == cba.CBA_ERR_ARG


def test_qk_limits(lib):
    for kw in (dict(dim=60, rot_dim=0), dict(dim=264, rot_dim=0), dict(param_type=cba.CBA_F16), dict(batch=1 << 21, len=1 << 10),
               dict(q=ST(1 << 40, 256, 64))):
        d = qk(**kw)
        assert qk_fwd(lib, d) == cba.CBA_ERR_UNSUPPORTED and qk_bwd(lib, d) == cba.CBA_ERR_UNSUPPORTED, kw
        assert lib.cba_qk_norm_rope_workspace_bytes(ctypes.byref(d)) == 0
    assert qk_fwd(lib, qk(q=ST(2640, 260, 64))) == cba.CBA_ERR_ALIGN
    assert qk_fwd(lib, qk(type=cba.CBA_F32, q=ST(2640, 260, 64)), q=None) == cba.CBA_ERR_ARG  # 1040 bytes: a multiple of 16


@pytest.mark.parametrize("kw", [dict(heads_q=(1 << 31) - 1), dict(heads_k=(1 << 31) - 31), dict(heads_q=(1 << 30) + 1)], ids=str)
def test_qk_heads_past_32_bit_steps(lib, kw):
    """A warp's next head, or the sum of a side's steps, would pass 2^31."""
    d = qk(dim=8, rot_dim=8, **kw)
    assert lib.cba_qk_norm_rope_workspace_bytes(ctypes.byref(d)) == 0
    assert qk_fwd(lib, d) == cba.CBA_ERR_UNSUPPORTED and qk_bwd(lib, d) == cba.CBA_ERR_UNSUPPORTED
    most = qk(dim=256, rot_dim=30, len=3000, heads_q=1 << 30, heads_k=1 << 30)
    assert 0 < lib.cba_qk_norm_rope_workspace_bytes(ctypes.byref(most)) <= 1 << 20


def test_qk_pointers_alignment_workspace(lib):
    d = qk()
    for name in ("q", "k", "yq", "yk", "table"):
        assert qk_fwd(lib, d, **{name: None}) == cba.CBA_ERR_ARG, name
    for name in ("q", "k", "dyq", "dyk", "dq", "dk", "table"):
        assert qk_bwd(lib, d, **{name: None}) == cba.CBA_ERR_ARG, name
    for name in ("q", "gamma_k", "table", "yq"):
        assert qk_fwd(lib, d, **{name: FAKE + 8}) == cba.CBA_ERR_ALIGN, name
    for name in ("dyk", "dq", "gamma_q"):
        assert qk_bwd(lib, d, **{name: FAKE + 8}) == cba.CBA_ERR_ALIGN, name
    assert qk_fwd(lib, d, pos=FAKE + 2) == cba.CBA_ERR_ALIGN and qk_bwd(lib, d, dgamma_q=FAKE + 1) == cba.CBA_ERR_ALIGN
    short = qk(positions=9)
    assert qk_fwd(lib, short, pos=None) == cba.CBA_ERR_ARG and qk_bwd(lib, short, pos=None) == cba.CBA_ERR_ARG
    plain = qk(norm=0)
    assert qk_fwd(lib, plain) == cba.CBA_ERR_ARG                  # gamma belongs to the norm
    assert qk_bwd(lib, plain, gamma_q=None, gamma_k=None) == cba.CBA_ERR_ARG  # and so does dgamma
    need = lib.cba_qk_norm_rope_workspace_bytes(ctypes.byref(d))
    assert need >= 256 and need % 256 == 0
    assert qk_bwd(lib, d, wsb=need - 1) == cba.CBA_ERR_WORKSPACE and qk_bwd(lib, d, ws=None) == cba.CBA_ERR_WORKSPACE
    assert qk_bwd(lib, d, ws=WS + 64) == cba.CBA_ERR_ALIGN
    # refused for the missing query, not for keys that are not there
    assert qk_fwd(lib, qk(heads_k=0), q=None, k=None, yk=None) == cba.CBA_ERR_ARG
    assert lib.cba_qk_norm_rope_forward(None, *([FAKE] * 8), None) == cba.CBA_ERR_ARG


def test_qk_workspace_is_small_beside_the_data(lib):
    for b, n in ((1, 1), (1, 1 << 15), (64, 8192)):
        assert lib.cba_qk_norm_rope_workspace_bytes(ctypes.byref(qk(batch=b, len=n, dim=128))) <= 1 << 20


# ---- dropout

def dr(**kw):
    return cba.make_dropout_desc(**{**dict(rows=4, cols=64), **kw})


def drop(lib, d, x=FAKE, residual=FAKE, step=FAKE, y=FAKE):
    return lib.cba_dropout(ctypes.byref(d), x, residual, step, y, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=0), dict(type=3), dict(p=-0.1), dict(p=1.5), dict(p=NAN), dict(ld_x=63),
                                 dict(ld_residual=-1), dict(ld_y=5)], ids=str)
def test_dropout_rejects_a_bad_descriptor(lib, bad):
    assert drop(lib, dr(**bad)) == cba.CBA_ERR_ARG


def test_dropout_limits_pointers_alignment(lib):
    assert drop(lib, dr(rows=1 << 35)) == cba.CBA_ERR_UNSUPPORTED and drop(lib, dr(ld_y=1 << 40)) == cba.CBA_ERR_UNSUPPORTED
    assert drop(lib, dr(rows=1, cols=(1 << 40) + 1)) == cba.CBA_ERR_UNSUPPORTED
    d = dr()
    assert drop(lib, d, x=None) == cba.CBA_ERR_ARG and drop(lib, d, y=None) == cba.CBA_ERR_ARG
    for name, by in (("x", 2), ("residual", 1), ("y", 2), ("step", 4)):
        assert drop(lib, d, **{name: FAKE + by}) == cba.CBA_ERR_ALIGN, name
    assert drop(lib, dr(rows=0), x=None, y=None) == cba.CBA_OK  # nothing to do
    assert lib.cba_dropout(None, FAKE, FAKE, FAKE, FAKE, None) == cba.CBA_ERR_ARG
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(offset=-5), dict(offset=1 << 64)):
        with pytest.raises(ValueError):
            dr(**kw)
