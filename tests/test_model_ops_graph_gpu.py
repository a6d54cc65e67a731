"""The operators of a model's ends and residual, one after another as a training
step uses them: captured in one CUDA graph and replayed on new inputs, from
several host threads at once, on a stream of their own, and with workspaces that
hold anything.  The same bits as one call after another."""
import threading

import pytest
import torch

import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Chain:
    """Tokens to the loss and back, with tied tables, on buffers of its own."""

    def __init__(self, tokens, vocab, width, kind, dtype, seed):
        self.kind, self.vocab, self.width = kind, vocab, width

        def rows():
            return torch.zeros(tokens, width, dtype=dtype, device=DEV)

        n = vocab * width
        self.at = {"table": 7, "weight": 7 + n, "bias": 9 + n + width, "post_weight": 11 + n + 2 * width,
                   "post_bias": 12 + n + 3 * width, "gate": 13 + n + 4 * width}
        self.params = torch.zeros(16 + n + 5 * width, dtype=dtype, device=DEV)
        self.grad = torch.zeros(16 + n + 5 * width, device=DEV)
        self.ids = torch.zeros(tokens, dtype=torch.int64, device=DEV)
        self.targets = torch.zeros(tokens, dtype=torch.int32, device=DEV)
        self.row_gate, self.d_row_gate = torch.zeros(tokens, device=DEV), torch.zeros(tokens, device=DEV)
        self.y, self.x, self.h, self.n, self.d_n, self.d_h, self.d_y = (rows() for _ in range(7))
        self.loss, self.lse, self.d_loss = (torch.zeros(tokens, device=DEV) for _ in range(3))
        self.ws = [dopt.embed_workspace(tokens, vocab, width), dopt.norm_workspace(tokens, width),
                   dopt.head_loss_workspace(tokens, width, vocab, aligned=False),
                   dopt.head_loss_grad_workspace(tokens, width, vocab, torch.float32, 2, aligned=False)]
        for w in self.ws:
            w.fill_(255)
        self.fill(seed)

    def fill(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.ids.copy_(torch.randint(-2, self.vocab, self.ids.shape, generator=g, device=DEV) ** 2 % self.vocab)
        self.targets.copy_(torch.randint(-5, self.vocab, self.targets.shape, generator=g, device=DEV))
        for t in (self.params, self.y, self.row_gate):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV) * 0.5)
        self.d_loss.copy_(torch.rand(self.d_loss.shape, generator=g, device=DEV))

    def run(self, stream=None):
        s = dict(stream=stream)
        n = self.vocab * self.width
        table = self.params[7:7 + n].view(self.vocab, self.width)
        p = {k: self.params[a:a + self.width] for k, a in self.at.items() if k != "table"}
        if self.kind == "rms":
            p["bias"] = p["post_bias"] = None
        bias = p.pop("bias")
        common = dict(y=self.y, post=True, scale=0.5, row_gate=self.row_gate, **p, **s)
        dopt.dopt_embed(table, self.ids, self.x, scale=2.0, **s)
        dopt.dopt_norm(self.kind, self.x, self.n, h=self.h, bias=bias, **common)
        dopt.dopt_head_loss(self.n, table, self.targets, self.loss, self.lse, workspace=self.ws[2], **s)
        dopt.dopt_head_loss_grad(self.n, table, self.targets, self.lse, self.d_loss, self.d_n, self.grad, 7,
                                 workspace=self.ws[3], **s)
        at = {k: a for k, a in self.at.items() if k != "table" and (self.kind == "layer" or "bias" not in k)}
        dopt.dopt_norm_grad(self.kind, self.h, self.d_n, self.d_h, d_y=self.d_y, d_row_gate=self.d_row_gate,
                            grad=self.grad, grad_offsets=at, workspace=self.ws[1], **common)
        dopt.dopt_embed_grad(self.ids, self.d_h, self.grad, 7, self.vocab, scale=2.0, accumulate=True,
                             workspace=self.ws[0], **s)

    def results(self):
        return [t.clone() for t in (self.x, self.h, self.n, self.loss, self.lse, self.d_n, self.d_h, self.d_y,
                                    self.d_row_gate, self.grad)]


SIZES = [(300, 900, 96, "rms", torch.bfloat16), (1000, 5000, 264, "layer", torch.float16),
         (70, 333, 61, "layer", torch.bfloat16), (2500, 700, 136, "rms", torch.bfloat16)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_graph(size):
    chain = Chain(*size, seed=1)
    chain.run()  # the first call looks up what it needs
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain.run()
    for seed in (2, 3):
        chain.fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        want = Chain(*size, seed=seed)
        want.run()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(chain.results(), want.results())):
            assert torch.isfinite(b).all(), i
            assert torch.equal(a, b), i


def test_threads():
    chains = [Chain(*s, seed=k) for k, s in enumerate(SIZES)]
    want = [Chain(*s, seed=k) for k, s in enumerate(SIZES)]
    for c in want:
        c.run()
    torch.cuda.synchronize()
    failed = []

    def work(c):
        stream = torch.cuda.Stream()
        try:
            for _ in range(20):
                c.run(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in chains]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for c, w in zip(chains, want):
        assert all(torch.equal(a, b) for a, b in zip(c.results(), w.results()))
    assert dopt.head_timeouts() == 0


def test_two_graphs_share_workspaces():
    """Graphs of two batch sizes with the larger one's workspaces, replayed in turn."""
    small, large = (200, 900, 96, "rms", torch.bfloat16), (700, 900, 96, "rms", torch.bfloat16)
    chains = [Chain(*small, seed=1), Chain(*large, seed=2)]
    want = [Chain(*small, seed=1), Chain(*large, seed=2)]
    for c in want:
        c.run()
    chains[0].ws = chains[1].ws
    for c in chains:
        c.run()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in chains]
    for g, c in zip(graphs, chains):
        with torch.cuda.graph(g):
            c.run()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for i, (c, w) in enumerate(zip(chains, want)):
        got, right = c.results(), w.results()
        for j, (a, b) in enumerate(zip(got, right)):
            if i == 0 and j in (5, 6, 7, 8, 9):  # another number of pieces: rounding only
                assert float((a.float() - b.float()).norm()) <= 1e-2 * float(b.float().norm()), j
            else:
                assert torch.equal(a, b), (i, j)
