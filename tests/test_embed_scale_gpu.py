"""The embedding's scale where it is not finite: an id outside the table counts
as nothing all the same."""
import pytest
import torch

import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("cols", [64, 61])
@pytest.mark.parametrize("scale", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_ids_outside(dtype, scale, cols):
    table = torch.randint(1, 5, (9, cols), device=DEV).to(dtype)
    ids = torch.tensor([3, -1, 9, 2 ** 40, 0], device=DEV)
    out = torch.full((5, cols), 7.0, dtype=dtype, device=DEV)
    dopt.dopt_embed(table, ids, out, scale=scale)
    assert not out[1:4].any()
    assert torch.equal(out[[0, 4]].isnan(), torch.full((2, cols), scale != scale, device=DEV))
    assert not bool(torch.isfinite(out[[0, 4]]).any())
    out.fill_(7.0)
    dopt.dopt_embed(table, ids, out, scale=scale, accumulate=True)
    assert bool((out[1:4] == 7).all()) and not bool(torch.isfinite(out[[0, 4]]).any())
