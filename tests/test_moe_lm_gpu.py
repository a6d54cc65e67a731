"""The package's language model of one layer of experts, which runs the
operators of its two ends and of the residual with the layer's and the step:
its loss and gradients against 64-bit autograd of the same model, and a run."""
import pytest
import torch

from zero_distributed_optimizer_gb300 import moe_layer
from zero_distributed_optimizer_gb300.moe_layer import MoELM, token_batches

pytestmark = pytest.mark.gpu


def _reference(model, ids, targets, rank):
    """Loss and gradients (table, the norms' weights, router, w_in, w_out) in 64 bits."""
    router, w_in, w_out = model.matrices(rank)
    leaves = [t.double().requires_grad_() for t in model.ends(rank)] + [
        router.double().requires_grad_(), torch.stack([w.double() for w in w_in]).requires_grad_(),
        torch.stack([w.double() for w in w_out]).requires_grad_()]
    table, norm_in, norm_out, router, w_in, w_out = leaves

    def norm(v, w):
        return v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + 1e-5) * w

    x0 = table[ids]
    n = norm(x0, norm_in)
    # the layer's own choice of experts, from the values it had
    chosen = (model.n_in.double() @ router.detach().t()).topk(model.k, dim=1).indices
    weights = torch.softmax((n @ router.t()).gather(1, chosen), dim=1)
    y = torch.zeros_like(x0)
    for j in range(model.k):
        for e in range(model.experts):
            t = (chosen[:, j] == e).nonzero()[:, 0]
            out = torch.nn.functional.gelu(n[t] @ w_in[e].t(), approximate="tanh") @ w_out[e].t()
            y = y.index_add(0, t, weights[t, j, None] * out)
    logits = norm(x0 + model.scale * y, norm_out) @ table.t()
    loss = torch.nn.functional.cross_entropy(logits, targets, ignore_index=-100)
    return loss, torch.autograd.grad(loss, leaves)


def test_gradients():
    """Within 4 %: the layer's own 3 % (its kept values' 8 bits) and the bf16 roundings of the residual, its norms
    and the gradients on the way (2^-9 each, rms)."""
    model = MoELM(vocab=701, width=96, hidden=200, experts=6, k=2, tokens=300, D=2)
    model.master[model.table_at:model.table_at + 701 * 96] *= 10  # logits of about +-3
    model.params = [model.master.bfloat16() for _ in range(2)]
    for rank, (ids, targets) in enumerate(token_batches(model, 5)):
        model.grads[rank].fill_(float("nan"))  # all of it is written
        got_loss = float(model.loss_and_grads(ids, targets, rank))
        loss, grads = _reference(model, ids, targets, rank)
        assert abs(got_loss - float(loss.detach())) <= 0.02 * float(loss.detach())
        got, n = model.grads[rank].double(), model.hidden * model.width
        places = [[model.table_at], [model.norm_in_at], [model.norm_out_at], [model.router_at], model.w_in_at, model.w_out_at]
        for name, at, want in zip(("table", "norm_in", "norm_out", "router", "w_in", "w_out"), places, grads):
            have = torch.stack([got[a:a + want[0].numel() if len(at) > 1 else a + want.numel()] for a in at]).reshape(want.shape)
            off = float((have - want).norm() / want.norm())
            assert off <= 0.04, (name, off)


def test_a_step_runs(capsys):
    moe_layer.main(["--steps", "2", "--tokens", "256", "--vocab", "1001"])
    assert capsys.readouterr().out.count("loss") == 2
    model = MoELM(vocab=1001, width=64, hidden=96, experts=4, k=2, tokens=200, D=2)
    before = model.params[0].clone()
    model.step(token_batches(model, 1))
    assert all(torch.equal(model.params[0], p) for p in model.params[1:])
    for at, n in ((model.table_at, 1001 * 64), (model.norm_in_at, 64), (model.norm_out_at, 64), (model.router_at, 4 * 64)):
        assert not torch.equal(model.params[0][at:at + n], before[at:at + n])


def test_no_step_on_lost_grads(monkeypatch):
    model = MoELM(vocab=300, width=64, hidden=96, experts=4, k=2, tokens=100, D=2)
    before, seen = model.params[0].clone(), model.head_timeouts
    monkeypatch.setattr(moe_layer.model_ops, "head_timeouts", lambda: seen + 2)
    with pytest.raises(RuntimeError, match="ran out"):
        model.step(token_batches(model, 0))
    assert model.steps == 0 and torch.equal(model.params[0], before)
