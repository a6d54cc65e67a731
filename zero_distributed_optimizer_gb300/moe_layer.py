"""A layer of experts trained with the layer operators and the optimizer step,
alone or in a language model.

    python -m zero_distributed_optimizer_gb300.moe_layer [--steps N] [--vocab V]

Each data-parallel rank routes its tokens to k of E experts (a top-k of a
linear router), sorts them by expert (``dopt_route_sort``,
``dopt_route_dispatch``), runs each expert's two matrices with a GELU between
them and brings the rows back (``dopt_route_combine``).  For the backward pass
it keeps, in 8 bits, the tokens once and the experts' hidden rows before and
after the GELU (``dopt_ckpt_save``); the weight gradients come from there,
straight into the rank's replica of the flat grad buffer
(``dopt_ckpt_wgrad``), and ``dopt_step`` updates the params of all ranks.

The experts' own matrix products are torch's; the layer has no bias.

With ``--vocab`` the layer is the one block of a language model that predicts
the next token (:class:`MoELM`): a table of token vectors (``dopt_embed``), a
norm before the block, one after it with the residual add in the same pass
(``dopt_norm``), and the cross entropy over the vocabulary against the same
table (``dopt_head_loss``).  The table's gradient comes from both ends and adds
up in its place of the flat buffer (``dopt_head_loss_grad``, then
``dopt_embed_grad``).
"""
from __future__ import annotations

import argparse

import torch

from . import binding as B
from . import layer_ops as ops
from . import model_ops


class MoELayer:
    """E experts of two matrices, [hidden, width] and [width, hidden], and a
    router [E, width], in one flat param buffer with D replicas."""

    def __init__(self, width=512, hidden=1408, experts=64, k=8, tokens=4096, D=2, lr=2e-3, seed=0, device="cuda",
                 more_sizes=()):
        self.width, self.hidden, self.experts, self.k, self.tokens, self.D = width, hidden, experts, k, tokens, D
        n = hidden * width
        # router, then w_in and w_out of each expert, then a model's other params
        sizes = [experts * width] + [n] * (2 * experts) + list(more_sizes)
        self.layout = B.dopt_build_range_map(sizes, D, bucket_elems=16 << 20, pad_unit=64).to_device(device)
        N = self.layout.padded_numel
        starts = [start for start, _ in self.layout.param_offsets()]
        experts_end = 1 + 2 * experts
        self.router_at, self.w_in_at, self.w_out_at = starts[0], starts[1:experts_end:2], starts[2:experts_end:2]
        self.more_at = starts[experts_end:]
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = torch.randn(N, generator=g, device=device) * 0.03
        self.exp_avg, self.exp_avg_sq = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.params = [self.master.bfloat16() for _ in range(D)]
        self.grads = [torch.zeros(N, dtype=torch.float32, device=device) for _ in range(D)]
        self.adam = B.AdamConfig(lr=lr, weight_decay=0.0, grad_scale=1.0 / D)
        self.steps, self.timeouts = 0, ops.wgrad_timeouts()
        # what a pass needs, made once
        slots, bf16, i32 = tokens * k, torch.bfloat16, torch.int32

        def rows(cols):
            return torch.zeros(slots, cols, dtype=bf16, device=device)

        self.slot_row = torch.empty(tokens, k, dtype=i32, device=device)
        self.row_token = torch.empty(slots, dtype=i32, device=device)
        self.offsets = torch.empty(experts + 1, dtype=i32, device=device)
        self.route_ws = ops.route_workspace(tokens, k, experts, device)
        self.wgrad_ws = ops.wgrad_workspace(slots, max(width, hidden), max(width, hidden), experts, device)
        self.x_rows, self.y_rows, self.d_y = rows(width), rows(width), rows(width)
        self.h, self.a, self.d_a = rows(hidden), rows(hidden), rows(hidden)
        self.d_weights = torch.empty(tokens, k, device=device)
        self.kept_x = ops.checkpoint(tokens, width, bf16, device)
        self.kept_h = ops.checkpoint(slots, hidden, bf16, device)
        self.kept_a = ops.checkpoint(slots, hidden, bf16, device)

    def matrices(self, rank):
        """(router [E, width], w_in [hidden, width] of each expert, w_out [width, hidden] of each)."""
        p, n = self.params[rank], self.hidden * self.width
        router = p[self.router_at:self.router_at + self.experts * self.width].view(self.experts, self.width)
        return (router, [p[s:s + n].view(self.hidden, self.width) for s in self.w_in_at],
                [p[s:s + n].view(self.width, self.hidden) for s in self.w_out_at])

    def forward(self, x, rank):
        """The layer's output for x [tokens, width] (bf16), and what backward needs."""
        router, w_in, w_out = self.matrices(rank)
        top = (x.float() @ router.float().t()).topk(self.k, dim=1)
        weights = torch.softmax(top.values, dim=1)
        ids = top.indices.contiguous()
        ops.dopt_route_sort(ids, self.experts, self.slot_row, self.row_token, self.offsets, self.route_ws)
        ops.dopt_route_dispatch(x, self.slot_row, self.x_rows)
        ops.dopt_ckpt_save(x, self.kept_x)
        bounds = self.offsets.tolist()
        for e in range(self.experts):
            at = slice(bounds[e], bounds[e + 1])
            torch.matmul(self.x_rows[at], w_in[e].t(), out=self.h[at])
        self.a.copy_(torch.nn.functional.gelu(self.h, approximate="tanh"))
        ops.dopt_ckpt_save(self.h, self.kept_h)
        ops.dopt_ckpt_save(self.a, self.kept_a)
        for e in range(self.experts):
            at = slice(bounds[e], bounds[e + 1])
            torch.matmul(self.a[at], w_out[e].t(), out=self.y_rows[at])
        out = torch.empty_like(x)
        ops.dopt_route_combine(self.y_rows, self.slot_row, weights, out)
        return out, (x, ids, weights, bounds)

    def backward(self, d_out, saved, rank):
        """The params' gradients into the rank's grad replica; the router's
        logits' gradient, for what is before the layer (:meth:`input_grad`)."""
        x, ids, weights, bounds = saved
        _, _, w_out = self.matrices(rank)
        grad = self.grads[rank]
        ops.dopt_route_combine_grad(d_out, self.y_rows, self.slot_row, weights, self.d_y, self.d_weights)
        ops.dopt_ckpt_wgrad(self.kept_a, self.d_y, grad, self.w_out_at, offsets=self.offsets,
                            row_token=None, workspace=self.wgrad_ws)
        for e in range(self.experts):
            at = slice(bounds[e], bounds[e + 1])
            torch.matmul(self.d_y[at], w_out[e], out=self.d_a[at])
        ops.dopt_ckpt_act_grad(self.kept_h, "gelu", self.d_a, self.d_a)
        ops.dopt_ckpt_wgrad(self.kept_x, self.d_a, grad, self.w_in_at, offsets=self.offsets,
                            row_token=self.row_token, workspace=self.wgrad_ws)
        # the router, through the softmax over the chosen logits
        d_top = weights * (self.d_weights - (weights * self.d_weights).sum(dim=1, keepdim=True))
        d_logits = torch.zeros(self.tokens, self.experts, device=x.device).scatter_(1, ids, d_top)
        at = slice(self.router_at, self.router_at + self.experts * self.width)
        grad[at] = (d_logits.t() @ x.float()).reshape(-1)
        return d_logits

    def input_grad(self, d_logits, saved, rank):
        """The gradient of the layer's input, once :meth:`backward` is through."""
        x, _, _, bounds = saved
        router, w_in, _ = self.matrices(rank)
        for e in range(self.experts):
            at = slice(bounds[e], bounds[e + 1])
            torch.matmul(self.d_a[at], w_in[e], out=self.d_y[at])
        d_x = torch.empty_like(x)
        ops.dopt_route_combine(self.d_y, self.slot_row, None, d_x)
        return (d_x.float() + d_logits @ router.float()).to(x.dtype)

    def step(self, batches):
        """One training step on D batches (x, target) of a squared error; the mean loss."""
        losses = []
        for rank, (x, target) in enumerate(batches):
            out, saved = self.forward(x, rank)
            diff = out.float() - target.float()
            losses.append(diff.square().mean())
            self.backward((diff * (2.0 / diff.numel())).to(x.dtype), saved, rank)
        if ops.wgrad_timeouts() != self.timeouts:  # some grads are NaN
            raise RuntimeError("a weight gradient's wait ran out of time: no step is taken")
        self.steps += 1
        B.dopt_step(self.layout, self.adam, self.steps, self.grads, self.master, self.exp_avg, self.exp_avg_sq,
                    self.params)
        return torch.stack(losses).mean()


class MoELM(MoELayer):
    """A language model of one block: token vectors, an RMS norm, the layer of
    experts on a residual, an RMS norm, and logits from the table of token
    vectors again.  The table and the norms' weights lie after the layer's
    params in the flat buffer."""

    def __init__(self, vocab=50257, width=512, hidden=1408, experts=64, k=8, tokens=4096, D=2, lr=2e-3, seed=0,
                 device="cuda"):
        super().__init__(width, hidden, experts, k, tokens, D, lr, seed, device,
                         more_sizes=[vocab * width, width, width])
        self.vocab, self.scale = vocab, 1.0
        self.table_at, self.norm_in_at, self.norm_out_at = self.more_at
        for at in (self.norm_in_at, self.norm_out_at):
            self.master[at:at + width] = 1.0
        self.params = [self.master.bfloat16() for _ in range(D)]
        self.lost, self.head_timeouts = torch.empty(tokens, device=device), model_ops.head_timeouts()
        self.lse = torch.empty(tokens, device=device)
        self.embed_ws = model_ops.embed_workspace(tokens, vocab, width, device)
        self.norm_ws = model_ops.norm_workspace(tokens, width, device)
        aligned = self.table_at % 8 == 0  # in the param replicas
        self.head_ws = model_ops.head_loss_workspace(tokens, width, vocab, aligned, device)
        self.head_grad_ws = model_ops.head_loss_grad_workspace(tokens, width, vocab, torch.float32, 1, aligned, device)
        self.x0, self.n_in, self.residual, self.n_out, self.d_residual, self.d_n, self.d_x0 = (
            torch.empty(tokens, width, dtype=torch.bfloat16, device=device) for _ in range(7))

    def ends(self, rank):
        """(table [vocab, width], the first norm's weight, the last one's)."""
        p = self.params[rank]
        return (p[self.table_at:self.table_at + self.vocab * self.width].view(self.vocab, self.width),
                p[self.norm_in_at:self.norm_in_at + self.width], p[self.norm_out_at:self.norm_out_at + self.width])

    def loss_and_grads(self, ids, targets, rank):
        """The mean loss of the targets in [0, vocab), with all params' gradients
        in the rank's grad replica."""
        table, w_in, w_out = self.ends(rank)
        grad = self.grads[rank]
        model_ops.dopt_embed(table, ids, self.x0)
        model_ops.dopt_norm("rms", self.x0, self.n_in, weight=w_in)
        y, saved = self.forward(self.n_in, rank)
        model_ops.dopt_norm("rms", self.x0, self.n_out, weight=w_out, y=y, h=self.residual, scale=self.scale)
        model_ops.dopt_head_loss(self.n_out, table, targets, self.lost, self.lse, workspace=self.head_ws)
        there = (targets >= 0) & (targets < self.vocab)
        d_loss = there.float() / there.sum().clamp(min=1)
        # backward: the table's gradient from its use as the output matrix first
        model_ops.dopt_head_loss_grad(self.n_out, table, targets, self.lse, d_loss, self.d_n, grad, self.table_at,
                                      workspace=self.head_grad_ws)
        d_y = torch.empty_like(y)
        model_ops.dopt_norm_grad("rms", self.residual, self.d_n, self.d_residual, weight=w_out, y=y, d_y=d_y, scale=self.scale, grad=grad,
                                 grad_offsets={"weight": self.norm_out_at}, workspace=self.norm_ws)
        d_logits = self.backward(d_y, saved, rank)
        d_n_in = self.input_grad(d_logits, saved, rank)
        model_ops.dopt_norm_grad("rms", self.x0, d_n_in, self.d_x0, weight=w_in, d_h=self.d_residual, grad=grad,
                                 grad_offsets={"weight": self.norm_in_at}, workspace=self.norm_ws)
        model_ops.dopt_embed_grad(ids, self.d_x0, grad, self.table_at, self.vocab, accumulate=True, workspace=self.embed_ws)
        return (self.lost * d_loss).sum()

    def step(self, batches):
        """One training step on D batches (ids, targets); the mean loss."""
        losses = [self.loss_and_grads(ids, targets, rank) for rank, (ids, targets) in enumerate(batches)]
        if ops.wgrad_timeouts() != self.timeouts or model_ops.head_timeouts() != self.head_timeouts:
            raise RuntimeError("a wait ran out of time, some grads are NaN: no step is taken")
        self.steps += 1
        B.dopt_step(self.layout, self.adam, self.steps, self.grads, self.master, self.exp_avg, self.exp_avg_sq,
                    self.params)
        return torch.stack(losses).mean()


def token_batches(model, seed, device="cuda"):
    """Tokens with frequencies of about 1 / rank and their successors under a fixed map, D batches; one
    target in 32 is ignored."""
    g = torch.Generator(device=device).manual_seed(seed)
    out = []
    for _ in range(model.D):
        u = torch.rand(model.tokens, generator=g, device=device)
        ids = (model.vocab ** u).long().clamp(max=model.vocab) - 1
        targets = (ids * 7 + 3) % model.vocab
        targets[torch.rand(model.tokens, generator=g, device=device) < 1 / 32] = -100
        out.append((ids, targets))
    return out


def teacher_batches(layer, seed, device="cuda"):
    """Tokens and targets from a fixed random linear map, D batches."""
    g = torch.Generator(device=device).manual_seed(seed)
    m = torch.randn(layer.width, layer.width, generator=torch.Generator(device=device).manual_seed(99),
                    device=device) / layer.width ** 0.5
    out = []
    for _ in range(layer.D):
        x = torch.randn(layer.tokens, layer.width, generator=g, device=device).bfloat16()
        out.append((x, (x.float() @ m).bfloat16()))
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=0, help="train a language model over so many tokens")
    a = ap.parse_args(argv)
    layer = MoELM(vocab=a.vocab, tokens=a.tokens) if a.vocab else MoELayer(tokens=a.tokens)
    batches = token_batches if a.vocab else teacher_batches
    for i in range(a.steps):
        loss = layer.step(batches(layer, i))
        print(f"step {i + 1}: loss {float(loss):.4f}", flush=True)


if __name__ == "__main__":
    main()
