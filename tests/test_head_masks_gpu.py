"""The loss where part of the vocabulary is masked: a column of ones in x meets
-1e4, -1e10, the type's lowest value or -inf in the output matrix (a padded
vocabulary, banned entries).  Masks at the front, at the end and over whole
stretches of the columns that one thread takes, all of them but one column, all
of them; and logits that are far above the others."""
import math

import pytest
import torch

import model_reference as R
from test_head_gpu import F, Case, _grad

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16

PLACES = {
    "front of each 128": lambda v: v % 128 < 32,
    "first half tile": lambda v: v < 128,
    "second half tile and the end": lambda v: ((v >= 128) & (v < 256)) | (v >= 640),
    "all but one": lambda v: v != 333,
    "nine of ten": lambda v: v * 7919 % 10 != 0,
    "the last column": lambda v: v == v[-1],
    "the last 32 of each 128": lambda v: v % 128 >= 96,
}
VALUES = [(BF16, -1e4), (BF16, -5e9), (BF16, -1e10), (BF16, -1e20), (BF16, float(torch.finfo(BF16).min)), (BF16, -math.inf),
          (FP16, -1e4), (FP16, float(torch.finfo(FP16).min)), (FP16, -math.inf)]


def _case(dtype, value, masked, vocab=769, rows=150, width=136):
    c = Case(rows, width, vocab, dtype)
    c.x[:, 5] = 1.0
    c.w[:, 5] = 0.0
    c.w[masked, 5] = value
    c.masked = masked
    return c


def _bounds(c):
    """(lse's error, each logit's) as in the tests of the loss: where something is left, masked logits add nothing
    to the sum, whatever their own error."""
    e = c.logit_error()
    there = ~c.masked.cpu() if bool((~c.masked).any()) else torch.ones_like(c.masked).cpu()
    return e[:, there].amax(dim=1), e


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("dtype,value", VALUES, ids=str)
def test_masked_logits(dtype, value, place):
    c = _case(dtype, value, PLACES[place](torch.arange(769, device=DEV)))
    c.targets[5:70] = (~c.masked).nonzero()[:, 0][torch.arange(65, device=DEV) % int((~c.masked).sum())]
    loss, lse = c.loss()
    want_loss, want_lse, _ = R.head(c.x, c.w, c.targets)
    e, of_logit = _bounds(c)
    e_lse = e + 64 * F + want_lse.abs() * 3 * F
    assert bool(torch.isfinite(lse).all())
    assert bool(((R.f64(lse) - want_lse).abs() <= e_lse).all()), float((R.f64(lse) - want_lse).abs().max())
    t = c.targets.cpu().long()
    there = (t >= 0) & (t < c.vocab)
    finite = torch.isfinite(want_loss)  # (a target of -inf: its loss is infinite)
    assert torch.equal(R.f64(loss)[~finite], want_loss[~finite])
    e_loss = e_lse + torch.where(there, of_logit.gather(1, torch.where(there, t, 0)[:, None])[:, 0], 0.0) + want_loss.abs() * F
    assert bool(((R.f64(loss) - want_loss).abs()[finite] <= e_loss[finite]).all())
    if not math.isfinite(value):
        return  # (the gradient of x is a product with the infinite entries)
    c.targets[c.masked[c.targets.clamp(0, c.vocab - 1)]] = -100
    lse = R.head(c.x, c.w, c.targets)[1].float().to(DEV)
    d_x, grad = _grad(c, lse, torch.float32)
    assert bool(torch.isfinite(d_x).all()) and bool(torch.isfinite(grad).all())
    masked = grad[3:3 + c.vocab * c.width].view(c.vocab, c.width)[c.masked]
    assert not masked.any()  # exp of less than -9000: zero in 64 bits too


@pytest.mark.parametrize("dtype,value", VALUES, ids=str)
def test_everything_masked(dtype, value):
    c = _case(dtype, value, torch.ones(500, dtype=torch.bool, device=DEV), vocab=500)
    loss, lse = c.loss()
    want_loss, want_lse, _ = R.head(c.x, c.w, c.targets)
    if math.isinf(value):
        assert bool((lse == -math.inf).all())
    else:
        e = _bounds(c)[0] + 64 * F + want_lse.abs() * 3 * F
        assert bool(((R.f64(lse) - want_lse).abs() <= e).all())
        assert bool(((R.f64(loss) - want_loss).abs() <= 2 * e + want_loss.abs() * F).all())
    assert not loss[1:4].any()  # the ignored targets


@pytest.mark.parametrize("value", [5e9, 1e20, 3.3e38, math.inf])
def test_logits_far_above_the_others(value):
    """One logit of a row is all of its sum: lse is that logit, and its loss nothing."""
    c = _case(BF16, value, torch.arange(600, device=DEV) == 417, vocab=600)
    c.targets[20:40] = 417
    loss, lse = c.loss()
    top = float(c.w[417, 5])
    e = abs(top) * (2 * 9 + 2 + 4) * 2.0 ** -23  # of the logit's 136 products, and lse's rounding
    if math.isinf(value):
        assert bool((lse == math.inf).all())
    else:
        assert bool(((R.f64(lse) - top).abs() <= e).all())
        assert bool((R.f64(loss)[20:40].abs() <= 2 * e).all())


def test_nan_logits_among_masked_ones():
    """A NaN reaches its row's sum from wherever it is, among -inf too."""
    c = _case(BF16, -math.inf, torch.arange(769, device=DEV) % 128 < 32)
    want = c.loss()[1]
    for column in (0, 31, 100, 768):
        w = c.w.clone()
        c.w[column, 9] = float("nan")
        assert bool(torch.isnan(c.loss()[1]).all())
        c.w.copy_(w)
    assert torch.equal(c.loss()[1], want) and bool(torch.isfinite(want).all())
