"""A layer of experts trained with the layer operators and the optimizer step.

    python -m zero_distributed_optimizer_gb300.moe_layer [--steps N]

Each data-parallel rank routes its tokens to k of E experts (a top-k of a
linear router), sorts them by expert (``dopt_route_sort``,
``dopt_route_dispatch``), runs each expert's two matrices with a GELU between
them and brings the rows back (``dopt_route_combine``).  For the backward pass
it keeps, in 8 bits, the tokens once and the experts' hidden rows before and
after the GELU (``dopt_ckpt_save``); the weight gradients come from there,
straight into the rank's replica of the flat grad buffer
(``dopt_ckpt_wgrad``), and ``dopt_step`` updates the params of all ranks.

The experts' own matrix products are torch's; the layer has no bias.
"""
from __future__ import annotations

import argparse

import torch

from . import binding as B
from . import layer_ops as ops


class MoELayer:
    """E experts of two matrices, [hidden, width] and [width, hidden], and a
    router [E, width], in one flat param buffer with D replicas."""

    def __init__(self, width=512, hidden=1408, experts=64, k=8, tokens=4096, D=2, lr=2e-3, seed=0, device="cuda"):
        self.width, self.hidden, self.experts, self.k, self.tokens, self.D = width, hidden, experts, k, tokens, D
        n = hidden * width
        sizes = [experts * width] + [n] * (2 * experts)  # router, then w_in and w_out of each expert
        self.layout = B.dopt_build_range_map(sizes, D, bucket_elems=16 << 20, pad_unit=64).to_device(device)
        N = self.layout.padded_numel
        starts = [start for start, _ in self.layout.param_offsets()]
        self.router_at, self.w_in_at, self.w_out_at = starts[0], starts[1::2], starts[2::2]
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
        """The params' gradients into the rank's grad replica."""
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
    a = ap.parse_args(argv)
    layer = MoELayer(tokens=a.tokens)
    for i in range(a.steps):
        loss = layer.step(teacher_batches(layer, i))
        print(f"step {i + 1}: loss {float(loss):.4f}", flush=True)


if __name__ == "__main__":
    main()
