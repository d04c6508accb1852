"""The torch-tensor calls on tensors that the kernels must not be given."""
import pytest
import torch

import activation_backward_gb300 as cba
from activation_backward_gb300 import transformer as tr

pytestmark = pytest.mark.gpu


def test_host_tensors_are_refused(cuda_lib):
    x, g = torch.randn(6, 64), torch.randn(64)
    q, lse = torch.randn(1, 8, 2, 64).bfloat16(), torch.zeros(1, 2, 8)
    for call in (lambda: tr.layer_norm(x, g, g), lambda: tr.layer_norm_backward(x, x, g, x[:, 0].contiguous(), x[:, 1].contiguous()),
                 lambda: tr.attention_backward(q, q, q, q, lse, q), lambda: tr.orthogonalize(x)):
        with pytest.raises(cba.CbaError) as e:
            call()
        # (a host workspace may also fail its alignment first)
        assert e.value.code in (cba.CBA_ERR_CUDA, cba.CBA_ERR_ALIGN)
    torch.cuda.synchronize()
    y, mean, _ = tr.layer_norm(x.cuda())  # a refused call leaves nothing behind
    assert torch.allclose(mean.cpu(), x.mean(1), atol=1e-5) and torch.isfinite(y).all()


def test_check_reports_a_device_timeout(cuda_lib, monkeypatch):
    """The status word as a bounded wait that ran out leaves it (the library's self-test makes one, of a millisecond)."""
    q, lse = torch.randn(1, 8, 2, 64, device="cuda").bfloat16(), torch.zeros(1, 2, 8, device="cuda")
    G = torch.randn(40, 60, device="cuda")
    calls = (lambda **kw: tr.attention_backward(q, q, q, q, lse, q, **kw), lambda **kw: tr.orthogonalize(G, **kw))
    for call in calls:
        assert all(torch.equal(a, b) for a, b in zip(call(), call(check=True)))
    for name in ("cba_attention_backward", "cba_orthogonalize"):
        plain = getattr(tr.B, name)
        monkeypatch.setattr(tr.B, name, lambda *a, _f=plain: (_f(*a), cba.cba_selftest_bounded_wait(a[-1], timeout_us=1000)))
    for call in calls:
        call()
        with pytest.raises(cba.CbaError) as e:
            call(check=True)
        assert e.value.code == cba.CBA_ERR_DEVICE_TIMEOUT
