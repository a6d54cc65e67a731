"""The chain of a model's operators, captured and replayed, on ids of which some
are outside the table, another number of them each time: what an earlier replay
left in the workspace past the sorted tokens counts as nothing."""
import pytest
import torch

from test_model_ops_graph_gpu import SIZES, Chain

pytestmark = pytest.mark.gpu


class Outside(Chain):
    def fill(self, seed):
        super().fill(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        u = torch.rand(self.ids.shape, generator=g, device="cuda")
        share = (0.5, 0.1, 0.9)[seed % 3]
        self.ids[u < share] = -1
        self.ids[u < share / 2] = self.vocab + 5
        self.ids[u < share / 4] = 2 ** 40
        inside = int(((self.ids >= 0) & (self.ids < self.vocab)).sum())
        assert 0 < inside < len(self.ids)
        self.inside = inside


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_replays(size):
    chain = Outside(*size, seed=1)
    chain.run()  # the first call looks up what it needs
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain.run()
    seen = set()
    for seed in (1, 2, 3, 5):
        chain.fill(seed)
        seen.add(chain.inside)
        graph.replay()
        torch.cuda.synchronize()
        want = Outside(*size, seed=seed)
        want.run()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(chain.results(), want.results())):
            assert torch.isfinite(b).all(), i
            assert torch.equal(a, b), i
    assert len(seen) > 2


def test_two_graphs_share_workspaces():
    """The larger graph's sorted tokens stay in the workspace behind the smaller one's."""
    sizes = [(200, 900, 96, "rms", torch.bfloat16), (700, 900, 96, "rms", torch.bfloat16)]
    chains = [Outside(*s, seed=k) for k, s in enumerate(sizes)]
    chains[0].ws[0] = chains[1].ws[0]  # the embedding gradient's: the same bits whatever its size
    for c in chains:
        c.run()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in chains]
    for g, c in zip(graphs, chains):
        with torch.cuda.graph(g):
            c.run()
    for seed in (2, 3):
        for c in chains:
            c.fill(seed)
        for g in (graphs[1], graphs[0], graphs[1], graphs[0]):
            g.replay()
        torch.cuda.synchronize()
        for c, s in zip(chains, sizes):
            want = Outside(*s, seed=seed)
            want.run()
            torch.cuda.synchronize()
            for i, (a, b) in enumerate(zip(c.results(), want.results())):
                assert torch.equal(a, b), i
