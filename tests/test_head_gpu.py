"""The loss of the output matrix's logits and its gradients against 64-bit
forms: both types, every grad type, sizes around the tiles' and steps' ends,
strides, ignored targets, one row, pieces of the vocabulary, a penalty on the
logits' scale, accumulation, and products that are exact."""
import pytest
import torch

import model_reference as R
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"
F = 2.0 ** -24
EPS = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def _layout(t, layout):
    rows, cols = t.shape
    if layout == "strided":
        v = torch.full((rows, cols + 24), float("nan"), dtype=t.dtype, device=DEV)[:, 8:8 + cols]
    elif layout == "shifted":
        v = torch.full((rows * cols + 1,), float("nan"), dtype=t.dtype, device=DEV)[1:].view(rows, cols)
    else:
        return t
    v.copy_(t)
    return v


class Case:
    def __init__(self, rows, width, vocab, dtype, layout="dense", seed=0, size=2.0):
        g = torch.Generator(device=DEV).manual_seed(seed + rows * 3 + width * 5 + vocab)
        self.rows, self.width, self.vocab, self.dtype = rows, width, vocab, dtype
        self.aligned = layout != "shifted" and width % 8 == 0
        self.x = _layout(torch.randn(rows, width, generator=g, device=DEV).to(dtype), layout)
        self.w = _layout((torch.randn(vocab, width, generator=g, device=DEV) * size / width ** 0.5).to(dtype), layout)
        self.targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
        if rows > 4:  # ignored ones: before, just past and far past the vocabulary
            self.targets[1], self.targets[2], self.targets[3] = -100, vocab, vocab + 2 ** 33
        if layout == "strided":
            self.targets[self.targets > vocab] = vocab
            self.targets = self.targets.int()
        weight = torch.rand(rows, generator=g, device=DEV) + 0.5
        self.d_loss = weight / rows
        self.d_lse = (torch.rand(rows, generator=g, device=DEV) - 0.25) / rows
        self.layout = layout

    def loss(self, workspace=None):
        loss, lse = (torch.full((self.rows,), 5.0, device=DEV) for _ in range(2))
        ws = dopt.head_loss_workspace(self.rows, self.width, self.vocab, self.aligned) if workspace is None else workspace
        ws.fill_(255)
        dopt.dopt_head_loss(self.x, self.w, self.targets, loss, lse, workspace=ws)
        return loss, lse

    def logit_error(self):
        """Of each logit: the tensor cores add 16 products at a time and cut off (2^-23 of the sum's size each
        time, taken twice: once for the products of a step, once for their addition); at most |x|.|w| in size."""
        return (R.f64(self.x).abs() @ R.f64(self.w).abs().t()) * (2 * ((self.width + 15) // 16) + 2) * 2.0 ** -23


SIZES = [  # rows, width, vocab
    (1, 1, 1), (3, 8, 5), (5, 64, 256), (31, 72, 100), (130, 128, 257), (256, 200, 1000), (257, 264, 777),
    (300, 515, 1030), (70, 768, 5003), (600, 65, 2049), (24, 2048, 700),
]


@pytest.mark.parametrize("layout", ["dense", "strided", "shifted"])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_loss(dtype, size, layout):
    c = Case(*size, dtype, layout)
    loss, lse = c.loss()
    want_loss, want_lse, logits = R.head(c.x, c.w, c.targets)
    e = c.logit_error()
    # lse moves by no more than the largest logit's error; the sum's own: exponentials (2 roundings and the
    # argument's, of up to 2^5 in size), 32 + 8 additions in a row; then the logarithm and the rounding
    own = 64 * F + want_lse.abs() * 3 * F
    e_lse = e.amax(dim=1) + own
    assert bool(((R.f64(lse) - want_lse).abs() <= e_lse).all()), float((R.f64(lse) - want_lse).abs().max())
    there = ((c.targets >= 0) & (c.targets < c.vocab)).cpu()
    at = torch.where(there, c.targets.cpu().long(), 0)
    e_loss = e_lse + e.gather(1, at[:, None])[:, 0] + want_loss.abs() * F
    assert bool(((R.f64(loss) - want_loss).abs() <= e_loss).all())
    assert not loss.cpu()[~there].any()
    again = c.loss()
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


def test_loss_of_large_logits():
    """Logits of thousands: exp alone would overflow, and one logit is all of the sum."""
    c = Case(200, 128, 900, torch.bfloat16, size=400.0)
    loss, lse = c.loss()
    want_loss, want_lse, _ = R.head(c.x, c.w, c.targets)
    e = c.logit_error().amax(dim=1) + want_lse.abs() * 3 * F + 64 * F
    assert bool(((R.f64(lse) - want_lse).abs() <= e).all())
    assert bool(((R.f64(loss) - want_loss).abs() <= 2 * e + want_loss.abs() * F).all())


def test_loss_exact_logits():
    """Whole-number logits are exact: loss and lse are then off by the sum's and the logarithm's own roundings."""
    g = torch.Generator(device=DEV).manual_seed(3)
    rows, width, vocab = 513, 96, 1500
    c = Case(rows, width, vocab, torch.float16)
    c.x.copy_(torch.randint(-2, 3, (rows, width), generator=g, device=DEV))
    c.w.copy_(torch.randint(-1, 2, (vocab, width), generator=g, device=DEV))
    loss, lse = c.loss()
    want_loss, want_lse, _ = R.head(c.x, c.w, c.targets)
    assert float((R.f64(lse) - want_lse).abs().max()) <= 64 * F + float(want_lse.abs().max()) * 3 * F
    assert float((R.f64(loss) - want_loss).abs().max()) <= 64 * F + float(want_lse.abs().max()) * 4 * F


def test_bad_rows_stay_in_their_rows():
    c = Case(300, 128, 600, torch.bfloat16)
    want = c.loss()
    c.x[7, 3], c.x[290, 0] = float("nan"), float("inf")
    loss, lse = c.loss()
    good = [r for r in range(300) if r not in (7, 290)]
    assert torch.equal(loss[good], want[0][good]) and torch.equal(lse[good], want[1][good])
    assert not bool(torch.isfinite(lse[[7, 290]]).any())


def _grad(c, lse, grad_type, pieces=1, first=3, d_lse=None, old=None, want_x=True, want_w=True):
    ws = dopt.head_loss_grad_workspace(c.rows, c.width, c.vocab, grad_type, pieces, c.aligned)
    ws.fill_(255)
    d_x = _layout(torch.full((c.rows, c.width), 7.0, dtype=c.dtype, device=DEV), c.layout) if want_x else None
    grad = None
    if want_w:
        grad = torch.full((first + c.vocab * c.width + 5,), 2.0, dtype=grad_type, device=DEV)
        if old is not None:
            grad[first:first + old.numel()] = old.reshape(-1)
    dopt.dopt_head_loss_grad(c.x, c.w, c.targets, lse, c.d_loss, d_x, grad, first, d_lse=d_lse, accumulate=old is not None,
                             workspace=ws)
    return d_x, grad


def _check_grad(c, lse, grad_type, d_x, grad, d_lse, first=3, old=None):
    want_x, want_w, d = R.head_grad(c.x, c.w, c.targets, lse, c.d_loss, d_lse)
    n = c.vocab * c.width
    half = EPS[c.dtype]
    # d in fp32: the logit's error and the exponential's (its argument is at most some 40, rounded twice), then the
    # coefficient's; d of 16 bits is rounded once more, of two parts twice (their product of half steps)
    there = ((c.targets >= 0) & (c.targets < c.vocab)).cpu()
    by = (R.f64(c.d_loss) * there + (0 if d_lse is None else R.f64(d_lse))).abs()[:, None]
    p = torch.exp(R.f64(c.x) @ R.f64(c.w).t() - R.f64(lse)[:, None])
    e32 = by * p * (c.logit_error() + 100 * F) + d.abs() * 4 * F
    tiny = float(by.max()) * 2.0 ** -36 if c.dtype is torch.float16 else 2.0 ** -140  # fp16's least step, scaled
    e16 = e32 + (d.abs() + e32) * half + tiny
    e_w = e32 + (d.abs() + e32) * half * half + tiny if grad_type is torch.float32 else e16
    x, w = R.f64(c.x).abs(), R.f64(c.w).abs()

    def cut(k):  # the tensor cores' sums of k products, relative to their size
        return (2 * ((k + 15) // 16) + 2) * 2.0 ** -23

    if d_x is not None:
        size = e16 @ w + (d.abs() @ w) * cut(c.vocab)
        err = (R.f64(d_x) - want_x).abs()
        assert bool((err <= (size + (want_x.abs() + size) * half + TINY[c.dtype]) * 1.01).all()), float(err.max())
    if grad is not None:
        got = R.f64(grad)
        assert bool((got[:first] == 2).all()) and bool((got[first + n:] == 2).all())
        k = min(c.rows, 1024) if grad_type is torch.float32 else c.rows
        size = e_w.t() @ x + (d.abs().t() @ x) * (cut(k) + 64 * F)
        if old is not None:
            want_w = want_w + R.f64(old)
            size = size + want_w.abs() * F
        err = (got[first:first + n].view(c.vocab, c.width) - want_w).abs()
        bound = (size + (want_w.abs() + size) * EPS[grad_type] + TINY[grad_type]) * 1.01
        assert bool((err <= bound).all()), (float(err.max()), float((err - bound).max()))


@pytest.mark.parametrize("layout", ["dense", "strided", "shifted"])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_grad(dtype, size, layout):
    c = Case(*size, dtype, layout)
    _, lse = c.loss()
    for grad_type, d_lse in ((dtype, None), (torch.float32, c.d_lse)):
        d_x, grad = _grad(c, lse, grad_type, d_lse=d_lse)
        _check_grad(c, lse, grad_type, d_x, grad, d_lse)
        # either alone, and again
        only_x, only_w = _grad(c, lse, grad_type, d_lse=d_lse, want_w=False)[0], _grad(c, lse, grad_type, d_lse=d_lse, want_x=False)[1]
        assert torch.equal(only_x, d_x) and torch.equal(only_w, grad)


@pytest.mark.parametrize("pieces", [2, 3, 100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_grad_in_pieces(dtype, pieces):
    c = Case(300, 264, 2100, dtype)
    _, lse = c.loss()
    one = _grad(c, lse, dtype)
    for grad_type in (dtype, torch.float32):
        d_x, grad = _grad(c, lse, grad_type, pieces, d_lse=c.d_lse)
        _check_grad(c, lse, grad_type, d_x, grad, c.d_lse)
    d_x, grad = _grad(c, lse, dtype, pieces)
    assert torch.equal(grad, one[1])  # a column's sums do not depend on the pieces
    _check_grad(c, lse, dtype, d_x, grad, None)


@pytest.mark.parametrize("grad_type", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_grad_accumulates(grad_type):
    c = Case(400, 136, 900, torch.bfloat16)
    _, lse = c.loss()
    old = torch.randn(c.vocab, c.width, device=DEV).to(grad_type)
    d_x, grad = _grad(c, lse, grad_type, old=old)
    _check_grad(c, lse, grad_type, d_x, grad, None, old=old)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_long_sums(dtype):
    """Many rows and many columns: split tiles, several sums a tile; fp32 grads keep an fp32 sum's accuracy."""
    c = Case(9000, 256, 700, dtype)
    _, lse = c.loss()
    d_x, grad = _grad(c, lse, torch.float32)
    _check_grad(c, lse, torch.float32, d_x, grad, None)
    _, want, _ = R.head_grad(c.x, c.w, c.targets, lse, c.d_loss)
    got = R.f64(grad)[3:3 + c.vocab * c.width].view(c.vocab, c.width)
    # 2^-16 (bf16) or 2^-22 for what two parts leave of d, at random; some 4e-7 for the sums; 1e-6 for the logits
    assert float((got - want).norm() / want.norm()) <= 4e-6
    c = Case(200, 136, 9001, dtype)
    _, lse = c.loss()
    d_x, grad = _grad(c, lse, dtype)
    _check_grad(c, lse, dtype, d_x, grad, None)


def test_every_target_ignored():
    c = Case(100, 72, 300, torch.float16)
    c.targets.fill_(-1)
    loss, lse = c.loss()
    assert not loss.any()
    assert float((R.f64(lse) - R.head(c.x, c.w, c.targets)[1]).abs().max()) <= float(c.logit_error().max()) + 100 * F
    d_x, grad = _grad(c, lse, torch.float32)
    assert not d_x.any() and not grad[3:-5].any()
    d_x, grad = _grad(c, lse, torch.float32, d_lse=c.d_lse)  # the penalty remains
    _check_grad(c, lse, torch.float32, d_x, grad, c.d_lse)
    d_x, grad = _grad(c, lse, torch.float32, d_lse=c.d_lse * 1e6)
    c.d_lse = c.d_lse * 1e6
    _check_grad(c, lse, torch.float32, d_x, grad, c.d_lse)


@pytest.mark.parametrize("grad_type", [torch.bfloat16, torch.float32], ids=str)
def test_ignored_rows_that_overflow(grad_type):
    """Rows without a target or a penalty whose logits are infinite or NaN add nothing, whatever their lse."""
    c = Case(300, 128, 600, torch.bfloat16)
    _, lse = c.loss()
    want_x, want_w = _grad(c, lse, grad_type, first=3)
    dead = [1, 2, 3]  # the ignored ones
    c.x[dead] = 3e38 * torch.sign(c.x[dead])
    loss, lse = c.loss()
    assert not loss[dead].any() and not bool(torch.isfinite(lse[dead]).any())
    d_x, grad = _grad(c, lse, grad_type, first=3)
    assert torch.equal(d_x, want_x) and torch.equal(grad, want_w) and not d_x[dead].any()


def test_penalty_far_larger_than_the_loss():
    """fp16: what the loss adds to a row's gradient is small beside the penalty, but stays in range."""
    c = Case(150, 136, 400, torch.float16)
    _, lse = c.loss()
    c.d_lse = c.d_lse * 1e4
    d_x, grad = _grad(c, lse, torch.float32, d_lse=c.d_lse)
    _check_grad(c, lse, torch.float32, d_x, grad, c.d_lse)


def test_no_rows():
    c = Case(0, 64, 300, torch.bfloat16)
    empty = torch.empty(0, device=DEV)
    dopt.dopt_head_loss(c.x, c.w, c.targets, empty, empty, workspace=dopt.head_loss_workspace(0, 64, 300))
    grad = torch.full((300 * 64 + 2,), 3.0, device=DEV)
    dopt.dopt_head_loss_grad(c.x, c.w, c.targets, empty, empty, c.x, grad, 1, accumulate=True)
    assert bool((grad == 3).all())
    dopt.dopt_head_loss_grad(c.x, c.w, c.targets, empty, empty, c.x, grad, 1)
    assert not grad[1:-1].any() and bool((grad[[0, -1]] == 3).all())


def test_grad_against_differences():
    """The weighted loss along a direction of x and of the matrix."""
    c = Case(60, 64, 300, torch.float16)
    loss, lse = c.loss()
    d_x, grad = _grad(c, lse, torch.float32, first=0)
    there = ((c.targets >= 0) & (c.targets < c.vocab)).double()

    def value(x, w):
        logits = x @ w.t()
        t = torch.where(there > 0, c.targets, 0)
        return float(((torch.logsumexp(logits, dim=1) - logits.gather(1, t[:, None])[:, 0]) * there * c.d_loss.double()).sum())

    g = torch.Generator(device=DEV).manual_seed(1)
    x, w = c.x.double(), c.w.double()
    for leaf, got in (("x", d_x.double()), ("w", grad[:c.vocab * c.width].view(c.vocab, c.width).double())):
        r = torch.randn(got.shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-5
        up, down = (value(x + s * r, w) if leaf == "x" else value(x, w + s * r) for s in (h, -h))
        slope = float((got * r).sum())
        # d_x: fp16's rounding of its values; both: the gradients' own error
        bound = float((got.abs() * r.abs()).sum()) * (2 * EPS[torch.float16]) + 1e-6
        assert abs((up - down) / (2 * h) - slope) <= bound, leaf
