"""Adding to the grads of a group without rows leaves them as they are, bit for
bit (a zero added would turn -0 into +0 and quieten a NaN)."""
import pytest
import torch

import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("bounds", [(0, 0, 0, 0), (0, 2600, 2600, 5000), (7, 7, 5000, 5000)])
@pytest.mark.parametrize("split", [False, True])
def test_groups_without_rows_are_left_alone(bounds, dtype, split):
    outs, cols, rows, E = 40, 72, 5000, 3
    g = torch.Generator(device=DEV).manual_seed(2)
    c = dopt.checkpoint(rows, cols)
    dopt.dopt_ckpt_save(torch.randn(rows, cols, generator=g, device=DEV).bfloat16(), c)
    dy = torch.randn(rows, outs, generator=g, device=DEV).bfloat16()
    n = outs * cols
    grad = torch.zeros(E * n, dtype=dtype, device=DEV)
    bits = grad.view(torch.int32 if dtype is torch.float32 else torch.int16)
    signalling = {torch.float32: 0x7f800001, torch.bfloat16: 0x7f81, torch.float16: 0x7c01}[dtype]
    bits.fill_(-2 ** 31 if dtype is torch.float32 else -2 ** 15)  # -0
    bits[::7] = signalling
    before = bits.clone()
    dopt.dopt_ckpt_wgrad(c, dy, grad, [k * n for k in range(E)],
                         offsets=torch.tensor(bounds, dtype=torch.int32, device=DEV),
                         row_token=torch.arange(rows, dtype=torch.int32, device=DEV), accumulate=True,
                         workspace=dopt.wgrad_workspace(rows, outs, cols, E) if split else None)
    for k in range(E):
        at = slice(k * n, (k + 1) * n)
        if bounds[k] == bounds[k + 1]:
            assert torch.equal(bits[at], before[at]), f"group {k}"
        else:
            fine = torch.isfinite(grad[at])
            assert int(fine.sum()) == n - len(range(-k * n % 7, n, 7))
            assert float(grad[at][fine].float().abs().max()) > 1
