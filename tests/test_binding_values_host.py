"""What the optimizer's and the layer operators' bindings keep of numbers is
their value: a learning rate or a place given as a tensor that changes
afterwards counts as what it is at the call."""
import ctypes

import torch

from zero_distributed_optimizer_gb300 import binding as B
from zero_distributed_optimizer_gb300 import layer_ops as L
from test_model_ops_values_host import _Tensor


def test_adam_numbers():
    lr = torch.tensor(0.5)
    for v in (0.5, 0.25, 0.5, 0.125):
        lr.fill_(v)
        assert B.AdamConfig(lr=lr).to_c().lr == v
    config = B.AdamConfig(lr=1e-3, weight_decay=0.0)
    assert config.to_c() is config.to_c()  # one per distinct configuration


def test_weight_gradient_places(monkeypatch):
    seen = []
    monkeypatch.setattr(L, "_call", lambda index, stream, function, *args: seen.append(args))
    keep = L.Checkpoint(_Tensor(torch.uint8, L.ckpt_bytes(4, 8)), 4, 8, torch.bfloat16)
    place = torch.tensor(8)
    for at in (8, 40, 16):
        place.fill_(at)
        L.dopt_ckpt_wgrad(keep, _Tensor(torch.bfloat16, 4, 8), _Tensor(torch.float32, 200), [place])
        starts = next(a for a in seen[-1] if isinstance(a, ctypes.Array))
        assert list(starts) == [at]
