"""The loss and its gradients where the blocks of tokens go through the
vocabulary in more than one group (wide rows: 32 MB of them, or 8 blocks)."""
import pytest
import torch

import test_head_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [(2300, 8192, 600), (4400, 4096, 300)], ids=str)
def test_groups(size):
    test_head_gpu.test_loss(torch.bfloat16, size, "dense")
    test_head_gpu.test_grad(torch.bfloat16, size, "dense")
