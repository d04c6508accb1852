"""Newton-Schulz of matrices whose squares fp32 cannot hold (bars: test_gpu_ortho)."""
import numpy as np
import pytest
import torch

from .test_gpu_ortho import call, check, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("scale", [1e19, 1e25, 1e36])
@pytest.mark.parametrize("shape", [(1, 40, 60), (2, 64, 333), (1, 333, 64), (1, 200, 330), (2, 301, 201), (1, 1, 1)], ids=str)
def test_squares_past_fp32(cuda_lib, shape, scale, dtype):
    G = draw(shape[1], *shape, scale=scale, dtype=dtype)
    check(call(G, torch.empty(G.shape, device="cuda")), G)


@pytest.mark.parametrize("shape", [(1, 40, 60), (1, 200, 330)], ids=str)
def test_one_huge_element(cuda_lib, shape):
    """It is all that is left of the matrix; fp32's sum of squares would call all of it nothing."""
    G = draw(1, *shape, scale=1.0)
    G[0, 3, 5] = 3e37
    out = call(G, torch.empty_like(G))[0]
    want = torch.zeros_like(out)
    x = 1.0
    for _ in range(5):
        x = 3.4445 * x - 4.775 * x ** 3 + 2.0315 * x ** 5
    want[3, 5] = x
    assert torch.allclose(out, want, atol=8e-3)
