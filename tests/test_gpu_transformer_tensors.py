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
