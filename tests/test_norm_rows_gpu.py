"""The norms' loops over rows (each block takes several, at every number of
groups a thread) and rows that are constant, whose layer norm is exactly its
bias at every width."""
import pytest
import torch

import test_norm_gpu
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


# widths that are no power of two: one over them is rounded, and that many times a constant is not its sum
@pytest.mark.parametrize("cols", [328, 776, 1000, 1336, 2056, 4104, 515])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
def test_constant_rows(dtype, cols):
    g = torch.Generator(device=DEV).manual_seed(cols)
    value = torch.tensor([1024.0, -1536.0, 7.0, 0.0, 16384.0], device=DEV)  # (sums of `cols` of them are exact)
    x = value[:, None].expand(5, cols).to(dtype).contiguous()
    bias = torch.randn(cols, generator=g, device=DEV).to(dtype)
    weight = torch.randn(cols, generator=g, device=DEV).to(dtype)
    n, h, zero = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(x)
    dopt.dopt_norm("layer", x, n, weight=weight, bias=bias)
    assert torch.equal(n, bias.expand(5, cols))
    dopt.dopt_norm("layer", zero, n, y=x, h=h, post=True, post_weight=weight, post_bias=bias)
    assert torch.equal(h, bias.expand(5, cols))
    # the weights' gradients are sums of zeros
    d = torch.randn(5, cols, generator=g, device=DEV).to(dtype)
    grad = torch.full((2 * cols,), 5.0, device=DEV)
    dopt.dopt_norm_grad("layer", x, d, None, weight=weight, y=x, d_h=d, post=True, post_weight=weight, post_bias=bias, grad=grad,
                        grad_offsets={"weight": 0, "post_weight": cols}, workspace=dopt.norm_workspace(5, cols))
    assert not grad.any()


# more rows than the blocks of a launch take at once: short rows that share a block, one group a thread, two and four
@pytest.mark.parametrize("dtype,size", [(BF16, (9800, 72)), (FP32, (2500, 520)), (FP16, (2600, 1032)), (BF16, (1300, 2056)),
                                        (FP32, (650, 4104)), (BF16, (640, 8200)), (FP16, (2500, 515))], ids=str)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_many_rows(kind, dtype, size):
    test_norm_gpu.test_norm(dtype, kind, size)


@pytest.mark.parametrize("dtype,size", [(FP32, (640, 2048)), (BF16, (640, 2056)), (FP16, (330, 4104)), (BF16, (310, 8200))], ids=str)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_of_many_rows(kind, dtype, size):
    test_norm_gpu.test_norm_grad(dtype, kind, size)
