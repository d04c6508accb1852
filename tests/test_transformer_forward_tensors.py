"""What the torch-tensor calls of attention's forward pass, query/key norms with rotation and dropout read from their
tensors and refuse (no GPU): the library's entry points are replaced by recorders."""
import pytest
import torch

from activation_backward_gb300 import _binding as B
from activation_backward_gb300 import transformer as tr

BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """The arguments of the library calls that were made."""
    seen = []
    for name in ("cba_attention_forward", "cba_qk_norm_rope_forward", "cba_qk_norm_rope_backward", "cba_dropout"):
        monkeypatch.setattr(B, name, lambda *a, _n=name, **kw: seen.append((_n, *a)))
    for name in ("cba_attention_forward_workspace_bytes", "cba_qk_norm_rope_workspace_bytes"):
        monkeypatch.setattr(B, name, lambda d: 256)
    return seen


def refused(calls, match, f, *a, **kw):
    before = len(calls)
    with pytest.raises((ValueError, TypeError), match=match or None):
        f(*a, **kw)
    assert len(calls) == before


# ---- attention

def test_attention_shapes(calls):
    q, kv = torch.zeros(2, 10, 4, 64, dtype=BF), torch.zeros(2, 7, 2, 64, dtype=BF)
    o, lse = tr.attention(q, kv, kv, causal=True)
    assert o.shape == q.shape and o.dtype == BF and lse.shape == (2, 4, 10) and lse.dtype == torch.float32
    d = calls[0][1]
    assert (d.len_q, d.len_k, d.heads_kv, d.causal, d.packed) == (10, 7, 2, 1, 0)
    cu = torch.tensor([0, 4, 10], dtype=torch.int32)
    o, lse = tr.attention(q[0], q[0], q[0], cu_q=cu, max_q=6)
    assert lse.shape == (4, 10)
    d = calls[1][1]
    assert (d.packed, d.batch, d.len_q, d.len_k, d.total_q) == (1, 2, 6, 10, 10) and calls[1][5] is cu and calls[1][6] is cu


def test_attention_refusals(calls):
    q = torch.zeros(2, 10, 4, 64, dtype=BF)
    for name in ("q", "k", "v"):
        for stored in ((2, 10, 1, 64), (1, 1, 4, 64), (1, 10, 4, 64)):
            a = dict(q=q, k=q, v=q)
            a[name] = torch.zeros(stored, dtype=BF).expand(2, 10, 4, 64)
            refused(calls, name, tr.attention, **a)
        a = dict(q=q, k=q, v=q)
        a[name] = q.to("meta")
        refused(calls, "device", tr.attention, **a)
    refused(calls, "sequences", tr.attention, q[0], q[0], q[0])
    cu = torch.tensor([0, 10], dtype=torch.int32)
    refused(calls, "int32", tr.attention, q[0], q[0], q[0], cu_q=cu.long())
    refused(calls, "int32", tr.attention, q[0], q[0], q[0], cu_q=cu, cu_k=torch.tensor([0, 5, 10], dtype=torch.int32))
    refused(calls, "meta", tr.attention, q[0], q[0], q[0], cu_q=cu.to("meta"))
    refused(calls, "", tr.attention, q, q, q, cu_q=cu)
    refused(calls, "v", tr.attention, q, q, q.half())
    refused(calls, "", tr.attention, q, q[:1], q[:1])
    refused(calls, "innermost", tr.attention, q.transpose(2, 3), q.transpose(2, 3), q.transpose(2, 3))


def test_attention_timeout_can_be_asked_for(calls, monkeypatch):
    asked, code = [], [B.CBA_ERR_DEVICE_TIMEOUT]
    monkeypatch.setattr(B, "cba_get_status", lambda ws: asked.append(ws) or code[0])
    q = torch.zeros(1, 4, 1, 64, dtype=BF)
    tr.attention(q, q, q)
    assert not asked
    with pytest.raises(B.CbaError):
        tr.attention(q, q, q, check=True)
    assert asked[0] is calls[1][-1]


# ---- query and key norms with rotation

def qk_args(shape=(2, 6), hq=4, hk=2, dim=16, dtype=BF):
    a = dict(q=torch.zeros(*shape, hq, dim, dtype=dtype), k=torch.zeros(*shape, hk, dim, dtype=dtype))
    a.update(gamma_q=torch.ones(dim), gamma_k=torch.ones(dim), table=torch.zeros(9, dim // 2, 2), pos=torch.zeros(shape, dtype=torch.int32))
    return a


def test_qk_shapes(calls):
    a = qk_args()
    yq, yk = tr.qk_norm_rope(**a)
    assert yq.shape == a["q"].shape and yk.shape == a["k"].shape
    d = calls[0][1]
    assert (d.batch, d.len, d.heads_q, d.heads_k, d.rot_dim, d.positions, d.norm, d.param_type) == (2, 6, 4, 2, 16, 9, 1, B.CBA_F32)
    qkv = torch.zeros(6, 8, 16, dtype=BF)
    tr.qk_norm_rope(qkv[:, :4], qkv[:, 4:6])
    d = calls[1][1]
    assert (d.batch, d.len, d.rot_dim, d.q.token, d.q.head, d.k.token) == (1, 6, 0, 128, 16, 128)
    yq, yk = tr.qk_norm_rope(a["q"], None, table=a["table"], norm=False, interleaved=True)
    d = calls[2][1]
    assert yk is None and (d.heads_k, d.norm, d.interleaved) == (0, 0, 1)


def test_qk_backward_shapes(calls):
    a = qk_args()
    dq, dk, gq, gk = tr.qk_norm_rope_backward(dyq=a["q"].clone(), dyk=a["k"].clone(), **a)
    assert dq.shape == a["q"].shape and dk.shape == a["k"].shape and gq.dtype == gk.dtype == torch.float32 and gq.shape == (16,)
    assert calls[0][1].accumulate == 0
    out = tr.qk_norm_rope_backward(dyq=a["q"], dyk=a["k"], dgamma_q=gq, dgamma_k=gk, **a)
    assert out[2] is gq and out[3] is gk and calls[1][1].accumulate == 1
    assert tr.qk_norm_rope_backward(a["q"], None, a["q"], None)[1::2] == (None, None)
    assert tr.qk_norm_rope_backward(a["q"], a["k"], a["q"], a["k"], norm=False)[2:] == (None, None)


@pytest.mark.parametrize("name,bad", [
    ("gamma_q", lambda t: t[:8]), ("gamma_k", lambda t: torch.ones(32)[::2]), ("gamma_k", lambda t: t.bfloat16()),
    ("table", lambda t: t.double()), ("table", lambda t: t[..., 0]), ("table", lambda t: t.transpose(0, 1)),
    ("pos", lambda t: t.long()), ("pos", lambda t: t[:, :5]), ("pos", lambda t: t.t().contiguous().t()), ("pos", lambda t: t[0]),
    ("k", lambda t: t[:, :5]), ("k", lambda t: t[..., :8]), ("k", lambda t: t.half()), ("k", lambda t: t[:, :, :1].expand(2, 6, 2, 16)),
    ("q", lambda t: t[:1].expand(2, 6, 4, 16)), ("k", lambda t: t.to("meta")), ("table", lambda t: t.to("meta")),
    ("pos", lambda t: t.to("meta")), ("gamma_q", lambda t: t.to("meta"))])
def test_qk_refusals(calls, name, bad):
    a = qk_args()
    a[name] = bad(a[name])
    refused(calls, "", tr.qk_norm_rope, **a)
    refused(calls, "", tr.qk_norm_rope_backward, dyq=torch.zeros(2, 6, 4, 16, dtype=BF), dyk=torch.zeros(2, 6, 2, 16, dtype=BF), **a)


def test_qk_backward_refusals(calls):
    a = qk_args()
    dy = dict(dyq=a["q"], dyk=a["k"])
    g = torch.zeros(16)
    refused(calls, "together", tr.qk_norm_rope_backward, dgamma_q=g, **dy, **a)
    refused(calls, "fp32", tr.qk_norm_rope_backward, dgamma_q=g, dgamma_k=g.bfloat16(), **dy, **a)
    refused(calls, "meta", tr.qk_norm_rope_backward, dgamma_q=g, dgamma_k=g.to("meta"), **dy, **a)
    refused(calls, "dyk", tr.qk_norm_rope_backward, dyq=a["q"], dyk=None, **a)
    refused(calls, "dyq", tr.qk_norm_rope_backward, dyq=a["q"][:, :5], dyk=a["k"], **a)
    refused(calls, "norm", tr.qk_norm_rope_backward, norm=False, **dy, **a)
    refused(calls, "norm", tr.qk_norm_rope, norm=False, **a)


# ---- dropout

def test_dropout_strides(calls):
    x = torch.zeros(4, 5, 3, 8)[:, :, 1]
    y = tr.dropout(x, 0.25, 7, offset=5, residual=torch.zeros(4, 5, 8))
    name, d, rows, res, step, out = calls[0]
    assert (d.rows, d.cols, d.ld_x, d.ld_residual, d.ld_y, d.seed, d.offset, d.p) == (20, 8, 24, 8, 0, 7, 5, 0.25)
    assert out is y and y.is_contiguous() and rows.data_ptr() == x.data_ptr() and step is None


def test_dropout_refusals(calls):
    x = torch.zeros(4, 8)
    refused(calls, "residual", tr.dropout, x, 0.1, 0, residual=x[:3])
    refused(calls, "residual", tr.dropout, x, 0.1, 0, residual=x.half())
    refused(calls, "meta", tr.dropout, x, 0.1, 0, residual=x.to("meta"))
    refused(calls, "expanded", tr.dropout, x[:1].expand(4, 8), 0.1, 0)
    refused(calls, "expanded", tr.dropout, x, 0.1, 0, residual=x[:1].expand(4, 8))
    refused(calls, "int64", tr.dropout, x, 0.1, 0, step=torch.zeros(1, dtype=torch.int32))
    refused(calls, "int64", tr.dropout, x, 0.1, 0, step=torch.zeros(2, dtype=torch.int64))
    refused(calls, "meta", tr.dropout, x, 0.1, 0, step=torch.zeros(1, dtype=torch.int64, device="meta"))
    refused(calls, "seed", tr.dropout, x, 0.1, -1)
    refused(calls, "offset", tr.dropout, x, 0.1, 0, offset=1 << 64)
    refused(calls, "innermost", tr.dropout, torch.zeros(8, 4).t(), 0.1, 0)
