"""What the binding keeps of numbers is their value: a number given as a tensor
that changes afterwards counts as what it is at the call."""
import ctypes

import pytest
import torch

import zero_distributed_optimizer_gb300 as dopt
from zero_distributed_optimizer_gb300 import model_ops as MO


class _Tensor:
    """A stand-in for a CUDA tensor as the binding asks for it (no GPU is used)."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), "cuda:0"

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()


@pytest.fixture
def calls(monkeypatch):
    """The arguments that reach the library, instead of a call."""
    seen = []
    monkeypatch.setattr(MO, "_call", lambda index, stream, function, *args: seen.append(args))
    return seen


def _cfg(args):
    cfg = args[0]._obj
    return cfg.kind, cfg.post, cfg.eps, cfg.scale


def test_norm_numbers(calls):
    x = _Tensor(torch.bfloat16, 4, 8)
    scale, eps = torch.tensor(2.0), torch.tensor(0.5)
    for s, e in ((2.0, 0.5), (3.0, 0.25), (2.0, 0.5)):
        scale.fill_(s)
        eps.fill_(e)
        dopt.dopt_norm("rms", x, x, y=x, scale=scale, eps=eps)
        dopt.dopt_norm_grad("layer", x, x, x, scale=scale, eps=eps, post=True)
        assert _cfg(calls[-2]) == (MO.DOPT_NORM_RMS, 0, e, s)
        assert _cfg(calls[-1]) == (MO.DOPT_NORM_LAYER, 1, e, s)


def test_norm_grad_places(calls):
    x, grad = _Tensor(torch.float32, 4, 8), _Tensor(torch.float32, 100)
    place = torch.tensor(8)
    for at in (8, 40, 16):
        place.fill_(at)
        dopt.dopt_norm_grad("rms", x, x, x, grad=grad, grad_offsets={"weight": place, "gate": 64})
        five = next(a for a in calls[-1] if isinstance(a, ctypes.Array) and a._type_ is ctypes.c_int64)
        assert list(five) == [at, -1, -1, -1, 64]
