"""What the torch-tensor calls read from their tensors and refuse (no GPU): the library's entry points are replaced by
recorders, so nothing is launched and no pointer is read."""
import pytest
import torch

from activation_backward_gb300 import _binding as B
from activation_backward_gb300 import transformer as tr


@pytest.fixture
def calls(monkeypatch):
    """The arguments of the library calls that were made."""
    seen = []
    for name in ("cba_layernorm_forward", "cba_layernorm_backward", "cba_attention_backward", "cba_orthogonalize"):
        monkeypatch.setattr(B, name, lambda *a, _n=name, **kw: seen.append((_n, *a)))
    for name in ("cba_layernorm_workspace_bytes", "cba_attention_workspace_bytes", "cba_orthogonalize_workspace_bytes"):
        monkeypatch.setattr(B, name, lambda d: 256)
    return seen


# ---- layer norm

def norm_args(*shape):
    rows = torch.zeros(shape).numel() // shape[-1]
    return dict(x=torch.randn(shape), dy=torch.randn(shape), gamma=torch.ones(shape[-1]), mean=torch.zeros(rows), rstd=torch.ones(rows))


@pytest.mark.parametrize("name", ["x", "dy", "residual"])
@pytest.mark.parametrize("stored", [(1, 1, 32), (4, 1, 32), (1, 10, 32)], ids=str)
def test_layer_norm_refuses_rows_that_lie_on_one_another(calls, name, stored):
    """An expanded tensor (the gradient of a sum over positions is one) holds fewer elements than its shape says."""
    a = norm_args(4, 10, 32)
    a[name] = torch.randn(stored).expand(4, 10, 32)
    with pytest.raises(ValueError):
        tr.layer_norm_backward(**a)
    if name == "x":
        with pytest.raises(ValueError):
            tr.layer_norm(a["x"])
    assert not calls


def test_layer_norm_refuses_the_gradient_of_a_sum(calls):
    y, got = torch.randn(6, 8, requires_grad=True), []
    z = y * 1.0
    z.register_hook(got.append)
    z.sum(0).backward(torch.ones(8))
    dy = got[0]
    assert dy.shape == (6, 8) and dy.stride() == (0, 1)
    with pytest.raises(ValueError):
        tr.layer_norm_backward(torch.randn(6, 8), dy, None, torch.zeros(6), torch.ones(6))
    with pytest.raises(ValueError):  # rows that overlap in part
        tr.layer_norm(torch.randn(20).as_strided((6, 8), (2, 1)))
    assert not calls


@pytest.mark.parametrize("t,ld", [(torch.zeros(1, 8).expand(1, 8), 0), (torch.zeros(6, 12)[:, :8], 12), (torch.zeros(6, 8), 8),
                                  (torch.zeros(6, 3)[:, 1:2], 3), (torch.zeros(2, 3, 2, 8)[:, :, 0], 16), (torch.zeros(0, 8), 0)],
                         ids=lambda v: str(tuple(v.shape)) if torch.is_tensor(v) else "")
def test_layer_norm_takes_the_rows_stride(calls, t, ld):
    tr.layer_norm(t)
    (name, d, x, *_), = calls
    assert name == "cba_layernorm_forward" and (d.rows, d.cols) == (t.numel() // t.shape[-1], t.shape[-1])
    assert d.ld_x == ld and x.data_ptr() == t.data_ptr()


@pytest.mark.parametrize("name", ["mean", "rstd"])
@pytest.mark.parametrize("bad", [lambda t: t.bfloat16(), lambda t: t.double(), lambda t: t[:3], lambda t: t[:, None].expand(40, 2),
                                 lambda t: torch.zeros(80)[::2], lambda t: t.new_zeros(1).expand(40)],
                         ids=["bf16", "fp64", "short", "wide", "every second", "expanded"])
def test_layer_norm_backward_refuses_other_statistics(calls, name, bad):
    a = norm_args(4, 10, 32)
    tr.layer_norm_backward(**a)
    assert len(calls) == 1
    a[name] = bad(a[name])
    with pytest.raises(ValueError, match="mean and rstd"):
        tr.layer_norm_backward(**a)
    assert len(calls) == 1


def test_layer_norm_backward_takes_statistics_in_the_shape_of_the_rows(calls):
    a = norm_args(4, 10, 32)
    a["mean"], a["rstd"] = a["mean"].view(4, 10), a["rstd"].view(4, 10, 1)
    tr.layer_norm_backward(**a)
    assert len(calls) == 1


# ---- attention's backward pass

def attn_args(shape=(2, 16, 4, 64), dtype=torch.bfloat16):
    a = {n: torch.randn(shape).to(dtype) for n in ("q", "k", "v", "o", "dout")}
    a["lse"] = torch.zeros(*shape[:-3], shape[-2], shape[-3])
    return a


@pytest.mark.parametrize("name", ["q", "k", "v", "o", "dout"])
@pytest.mark.parametrize("stored", [(1, 1, 1, 64), (2, 1, 1, 64), (1, 16, 1, 64), (1, 1, 4, 64), (1, 16, 4, 64), (2, 1, 4, 64),
                                    (2, 16, 1, 64)], ids=str)
def test_attention_refuses_expanded_tensors(calls, name, stored):
    a = attn_args()
    a[name] = torch.randn(stored).bfloat16().expand(2, 16, 4, 64)
    with pytest.raises(ValueError, match=name):
        tr.attention_backward(**a)
    assert not calls


def test_packed_attention_refuses_expanded_tensors(calls):
    a = attn_args((16, 4, 64))
    cu = torch.tensor([0, 9, 16], dtype=torch.int32)
    tr.attention_backward(**a, cu_q=cu)
    assert len(calls) == 1
    for stored in ((1, 1, 64), (16, 1, 64), (1, 4, 64)):
        a["dout"] = torch.randn(stored).bfloat16().expand(16, 4, 64)
        with pytest.raises(ValueError, match="dout"):
            tr.attention_backward(**a, cu_q=cu)
    assert len(calls) == 1


def test_attention_axes_of_one_index_may_have_any_stride(calls):
    """Of such an axis only index 0 is used: expanding it changes nothing."""
    a = attn_args((1, 16, 1, 64))
    a["dout"] = torch.randn(16, 64).bfloat16().as_strided((1, 16, 1, 64), (0, 64, 0, 1))
    tr.attention_backward(**a)
    d = calls[0][1]
    assert (d.dout.batch, d.dout.token, d.dout.head) == (0, 64, 0) and (d.q.batch, d.q.token, d.q.head) == (0, 64, 0)
    one = attn_args((1, 1, 1, 64))
    tr.attention_backward(**one)
    d = calls[1][1]
    assert (d.q.batch, d.q.token, d.q.head) == (0, 0, 0)


# ---- devices

@pytest.mark.parametrize("name", ["dy", "gamma", "mean", "rstd", "residual", "dgamma", "dbeta"])
def test_layer_norm_backward_refuses_tensors_of_another_device(calls, name):
    a = dict(norm_args(6, 32), residual=torch.zeros(6, 32), dgamma=torch.zeros(32), dbeta=torch.zeros(32))
    tr.layer_norm_backward(**a)
    assert len(calls) == 1
    a[name] = a[name].to("meta")
    with pytest.raises(ValueError, match=f"{name} is on meta"):
        tr.layer_norm_backward(**a)
    assert len(calls) == 1


@pytest.mark.parametrize("name", ["gamma", "beta"])
def test_layer_norm_refuses_tensors_of_another_device(calls, name):
    with pytest.raises(ValueError, match=f"{name} is on meta"):
        tr.layer_norm(torch.zeros(6, 32), **{name: torch.zeros(32, device="meta")})
    assert not calls


@pytest.mark.parametrize("name", ["lse", "cu_q", "cu_k", "o"])
def test_attention_refuses_tensors_of_another_device(calls, name):
    """Sequence starts often live on the host; the kernels read them on the GPU."""
    a = attn_args((16, 4, 64))
    a["cu_q"] = torch.tensor([0, 9, 16], dtype=torch.int32)
    a["cu_k"] = a["cu_q"].clone()
    tr.attention_backward(**a)
    assert len(calls) == 1
    a[name] = a[name].to("meta")
    with pytest.raises(ValueError, match=name):
        tr.attention_backward(**a)
    assert len(calls) == 1


# ---- torch's defaults

@pytest.fixture(params=[torch.bfloat16, torch.float64], ids=str)
def default_type(request):
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield request.param
    torch.set_default_dtype(before)


def test_statistics_and_parameter_gradients_are_fp32_whatever_the_default_type(calls, default_type):
    """The kernels write 4 bytes an element."""
    x = torch.zeros(6, 32, dtype=torch.bfloat16)
    y, mean, rstd = tr.layer_norm(x)
    assert y.dtype == torch.bfloat16 and mean.dtype == rstd.dtype == torch.float32
    dx, dgamma, dbeta = tr.layer_norm_backward(x, x, None, mean, rstd)
    assert dx.dtype == torch.bfloat16 and dgamma.dtype == dbeta.dtype == torch.float32
    assert [c[0] for c in calls] == ["cba_layernorm_forward", "cba_layernorm_backward"]


# ---- device status

@pytest.mark.parametrize("call", [lambda **kw: tr.attention_backward(**attn_args(), **kw),
                                  lambda **kw: tr.orthogonalize(torch.randn(2, 6, 9), **kw)], ids=["attention", "orthogonalize"])
def test_a_timeout_can_be_asked_for(calls, monkeypatch, call):
    """The workspace with the status word is the call's own: `check` reads it before it is gone."""
    asked, code = [], [B.CBA_ERR_DEVICE_TIMEOUT]
    monkeypatch.setattr(B, "cba_get_status", lambda ws: asked.append(ws) or code[0])
    call()
    assert len(calls) == 1 and not asked  # without it the call stays asynchronous
    with pytest.raises(B.CbaError) as e:
        call(check=True)
    assert e.value.code == B.CBA_ERR_DEVICE_TIMEOUT and asked[0] is calls[1][-1]
    code[0] = B.CBA_OK
    call(check=True)
    assert len(asked) == 2
