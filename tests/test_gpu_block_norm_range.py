"""The norms around a block at the ends of fp32's range, against float64.  Bounds as in test_gpu_block_norm."""
import pytest
import torch

from test_gpu_block_norm import BF16, F32, Case

pytestmark = pytest.mark.gpu
WIDTHS = [1, 5, 200, 2500, 9000, 20000]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("eps", [1e30, 3e36, 1e38, 3.4e38])
def test_large_eps(K, eps):
    # beside squares that leave fp32 as a sum, or with eps, or not at all: eps has its part in each
    for stream in (F32, BF16):
        c = Case(5, K, stream, F32, gate=None, scale=1.0, eps=eps)
        scales = torch.tensor([1.0, 1e15, 1e18, 5e18, 1e20], device="cuda")[:, None]
        c.h = (c.h.float() * scales).to(stream)
        c.x = (c.x.float() * scales.flip(0)).to(BF16)
        c.check_forward()
        c.check_backward()
