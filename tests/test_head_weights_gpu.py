"""The loss's gradients where the rows' weights (d_loss, d_lse) are far apart or
one of them is infinite: every row of d_x is as accurate as its own weight
allows, with fp16 as with bf16, whatever the other rows' weights are."""
import pytest
import torch

import model_reference as R
import zero_distributed_optimizer_gb300 as dopt
from test_head_gpu import EPS, F, TINY, Case, _check_grad, _grad

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16]


def _spread(c, low, seed=0):
    """Weights from `low` to 1 over the logarithm, times a loss scale; the ignored rows keep a penalty."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.exp(torch.rand(c.rows, generator=g, device=DEV) * torch.log(torch.tensor(low)).item())
    w[0], w[-1] = 1.0, low
    c.d_loss = w * 4096
    c.d_lse = c.d_loss * (torch.rand(c.rows, generator=g, device=DEV) - 0.25)


def _check_rows(c, lse, d_x, d_lse, rows):
    """d_x of these rows against the formula: the bounds of the gradients' tests, with fp16's least step counted
    by the row's own weight."""
    want_x, _, d = R.head_grad(c.x, c.w, c.targets, lse, c.d_loss, d_lse)
    half = EPS[c.dtype]
    there = ((c.targets >= 0) & (c.targets < c.vocab)).cpu()
    dl = R.f64(c.d_loss) * there
    by = (dl + (0 if d_lse is None else R.f64(d_lse))).abs()[:, None]
    p = torch.exp(R.f64(c.x) @ R.f64(c.w).t() - R.f64(lse)[:, None])
    e32 = by * p * (c.logit_error() + 100 * F) + d.abs() * 4 * F
    # fp16's least step is 2^-24 of numbers scaled so that a row's largest weight is 2^13
    tiny = torch.maximum(by, dl.abs()[:, None]) * 2.0 ** -36 if c.dtype is torch.float16 else 2.0 ** -140
    e16 = e32 + (d.abs() + e32) * half + tiny
    w = R.f64(c.w).abs()
    size = e16 @ w + (d.abs() @ w) * (2 * ((c.vocab + 15) // 16) + 2) * 2.0 ** -23
    err = (R.f64(d_x) - want_x).abs()
    bound = (size + (want_x.abs() + size) * half + TINY[c.dtype]) * 1.01
    bad = (err[rows] > bound[rows]).any(dim=1)
    assert not bool(bad.any()), (int(bad.sum()), float((err / bound)[rows].max()))


def _case(rows, width, vocab, dtype, size=1.0):
    c = Case(rows, width, vocab, dtype, size=size)
    if rows > 40:
        c.targets[10:30] = -1  # rows of which the penalty alone remains
    return c


SIZES = [(70, 64, 5003), (300, 136, 2049), (40, 768, 20011)]


@pytest.mark.parametrize("low", [1e-2, 1e-5, 1e-7])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_weights_far_apart(dtype, size, low):
    c = _case(*size, dtype)
    _spread(c, low)
    _, lse = c.loss()
    every = torch.ones(c.rows, dtype=torch.bool)
    for grad_type, d_lse in ((dtype, c.d_lse), (torch.float32, None)):
        d_x, grad = _grad(c, lse, grad_type, d_lse=d_lse)
        _check_rows(c, lse, d_x, d_lse, every)
        _check_grad(c, lse, grad_type, None, grad, d_lse)
        only_x = _grad(c, lse, grad_type, d_lse=d_lse, want_w=False)[0]
        only_w = _grad(c, lse, grad_type, d_lse=d_lse, want_x=False)[1]
        assert torch.equal(only_x, d_x) and torch.equal(only_w, grad)
        in_pieces = _grad(c, lse, grad_type, pieces=3, d_lse=d_lse)
        _check_rows(c, lse, in_pieces[0], d_lse, every)
        if grad_type is dtype:  # (a column's sums do not depend on the pieces)
            assert torch.equal(in_pieces[1], grad)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_a_weight_that_is_not_finite(dtype, value):
    """Such a row's gradients are not finite; the other rows of d_x are as they are without it."""
    c = _case(300, 136, 2049, dtype)
    c.d_loss = torch.full((300,), 1.0 / 16384, device=DEV)  # (a mean: 2^-14, fp16's least normal number)
    c.targets[c.targets == -1] = 7
    _, lse = c.loss()
    want = _grad(c, lse, dtype)[0]
    c.d_loss[123] = value
    d_x = _grad(c, lse, dtype)[0]
    only = _grad(c, lse, dtype, want_w=False)[0]
    others = torch.arange(300, device=DEV) != 123
    assert not bool(torch.isfinite(d_x[123]).any())
    assert torch.equal(d_x[others], want[others]) and torch.equal(only[others], want[others])


def test_dead_rows_beside_far_weights():
    """Rows that count for nothing add nothing, whatever their logits are, where the others' weights are far apart."""
    c = _case(300, 128, 600, torch.float16)
    _spread(c, 1e-6)
    c.targets[10:30] = torch.arange(20, device=DEV)
    _, lse = c.loss()
    want = _grad(c, lse, torch.float32)
    lse[[1, 2, 3]] = float("nan")  # the ignored ones
    d_x, grad = _grad(c, lse, torch.float32)
    assert torch.equal(d_x, want[0]) and torch.equal(grad, want[1]) and not d_x[[1, 2, 3]].any()


@pytest.mark.parametrize("grad_type", [torch.float16, torch.float32], ids=str)
def test_many_rows_far_apart(grad_type):
    c = _case(9001, 72, 300, torch.float16)
    _spread(c, 1e-6)
    _, lse = c.loss()
    d_x, grad = _grad(c, lse, grad_type, d_lse=c.d_lse)
    _check_rows(c, lse, d_x, c.d_lse, torch.ones(c.rows, dtype=torch.bool))
    _check_grad(c, lse, grad_type, None, grad, c.d_lse)


def test_one_graph_for_equal_weights_and_far_ones():
    """Whether the rows' weights are far apart is found at each replay."""
    c = _case(300, 136, 2049, torch.float16)
    _, lse = c.loss()
    weights = []
    for low in (1.0, 1e-6, 0.5, 1e-3):
        _spread(c, low)
        weights.append((c.d_loss.clone(), c.d_lse.clone()))
    want = []
    for c.d_loss, d_lse in weights:
        want.append(_grad(c, lse, torch.float32, d_lse=d_lse))
    d_loss, d_lse = (torch.zeros(c.rows, device=DEV) for _ in range(2))
    d_x, grad = torch.zeros_like(want[0][0]), torch.full_like(want[0][1], 2.0)
    ws = dopt.head_loss_grad_workspace(c.rows, c.width, c.vocab, torch.float32)
    ws.fill_(255)

    def run():
        dopt.dopt_head_loss_grad(c.x, c.w, c.targets, lse, d_loss, d_x, grad, 3, d_lse=d_lse, workspace=ws)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in (0, 1, 2, 3, 1, 0):
        d_loss.copy_(weights[k][0])
        d_lse.copy_(weights[k][1])
        d_x.fill_(7.0)
        graph.replay()
        assert torch.equal(d_x, want[k][0]) and torch.equal(grad, want[k][1]), k
