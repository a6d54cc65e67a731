"""The experts' layer of the package, which runs the layer operators and the
step together: its gradients against 64-bit autograd of the same layer, and
the loss of a short training run."""
import pytest
import torch

from zero_distributed_optimizer_gb300.moe_layer import MoELayer, teacher_batches

pytestmark = pytest.mark.gpu


def _reference(layer, x, target, rank):
    """Loss and gradients (router, w_in, w_out) in 64 bits, with the layer's own choice of experts."""
    router, w_in, w_out = layer.matrices(rank)
    router = router.double().requires_grad_()
    w_in = torch.stack([w.double() for w in w_in]).requires_grad_()
    w_out = torch.stack([w.double() for w in w_out]).requires_grad_()
    x = x.double()
    top = (x @ router.t()).topk(layer.k, dim=1)
    weights = torch.softmax(top.values, dim=1)
    out = torch.zeros_like(x)
    for j in range(layer.k):
        for e in range(layer.experts):
            t = (top.indices[:, j] == e).nonzero()[:, 0]
            y = torch.nn.functional.gelu(x[t] @ w_in[e].t(), approximate="tanh") @ w_out[e].t()
            out = out.index_add(0, t, weights[t, j, None] * y)
    loss = (out - target.double()).square().mean()
    return loss, torch.autograd.grad(loss, (router, w_in, w_out))


def test_gradients():
    """Within 3 %: a kept value is off by at most half a step, 1/64 of its
    block's largest and so about 1 % of a normal block's root mean square, and
    the bf16 roundings on the way (2^-9 each, rms) add half a percent."""
    layer = MoELayer(width=96, hidden=200, experts=6, k=2, tokens=300, D=2)
    for rank, (x, target) in enumerate(teacher_batches(layer, 5)):
        out, saved = layer.forward(x, rank)
        diff = out.float() - target.float()
        layer.backward((diff * (2.0 / diff.numel())).to(x.dtype), saved, rank)
        loss, (d_router, d_in, d_out) = _reference(layer, x, target, rank)
        assert abs(float(diff.square().mean()) - float(loss.detach())) <= 0.02 * float(loss.detach())
        n = layer.hidden * layer.width
        got = layer.grads[rank].double()
        for e in range(layer.experts):
            for at, want in ((layer.w_in_at[e], d_in[e]), (layer.w_out_at[e], d_out[e])):
                off = (got[at:at + n] - want.reshape(-1)).norm()
                assert off <= 0.03 * want.norm(), f"expert {e}: {float(off / want.norm())}"
        at = layer.router_at
        off = (got[at:at + d_router.numel()] - d_router.reshape(-1)).norm()
        assert off <= 0.03 * d_router.norm(), float(off / d_router.norm())


def test_training_lowers_the_loss():
    layer = MoELayer(width=128, hidden=256, experts=8, k=2, tokens=1024, D=2, lr=4e-3)
    losses = [float(layer.step(teacher_batches(layer, i))) for i in range(30)]
    assert losses[-1] < 0.7 * losses[0], losses
    assert all(torch.equal(layer.params[0], p) for p in layer.params[1:])
