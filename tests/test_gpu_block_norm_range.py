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


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("stream", [F32, BF16])
def test_gradients_of_small_rows(K, stream):
    # a stream of 1e-15 and gradients of 1e-28 with an eps below its squares: their products leave fp32, the sums of the gradient
    # and the norm do not
    c = Case(6, K, stream, F32, gate=1, eps=2.0 ** -126, later=False)
    c.h = (c.h.float() * torch.tensor([1e-15, 1e-17, 1e-12, 1e-18, 1.0, 0.0], device="cuda")[:, None]).to(stream)
    c.dy = (c.dy.float() * torch.tensor([1e-28, 1e-26, 1e-30, 1e-27, 1e-38, 1e-25], device="cuda")[:, None]).to(BF16)
    c.check_backward()
    c.check_backward(need_weights=False)
