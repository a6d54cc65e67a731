"""The norms around a block and their gradients against 64-bit forms and torch's
automatic differentiation of them: both kinds, every type, each gate alone and
together, widths from 1 to the most, strides, in-place residuals, no rows, rows
that hold NaN, accumulation."""
import pytest
import torch

import model_reference as R
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = {t: torch.finfo(t).eps / 2 for t in DTYPES}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
PARAMS = ("weight", "bias", "post_weight", "post_bias", "gate")


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
    def __init__(self, kind, rows, cols, dtype, form, layout="dense", seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed + rows * 7 + cols)
        self.kind, self.rows, self.cols, self.dtype, self.layout = kind, rows, cols, dtype, layout

        def rows_of(size, level=0.0):
            return _layout((torch.randn(rows, cols, generator=g, device=DEV) * size + level).to(dtype), layout)

        def param(size, level):
            p = (torch.randn(cols + 1, generator=g, device=DEV) * size + level).to(dtype)
            return p[1:] if layout == "shifted" else p[:cols]

        self.x, self.h, self.d_n, self.d_h = rows_of(1.5, 0.25), rows_of(1.5, 0.25), rows_of(0.5), rows_of(0.5)
        self.y = rows_of(0.75, 0.125) if form != "pre" else None
        every = dict(weight=param(0.25, 1), bias=param(0.25, 0), post_weight=param(0.25, 1), post_bias=param(0.25, 0),
                     gate=param(0.25, 0.75), row_gate=torch.rand(rows, generator=g, device=DEV) + 0.5)
        wanted = {"pre": ("weight", "bias"), "bare": (), "post": ("weight", "bias", "post_weight", "post_bias"),
                  "postonly": (), "gate": ("weight", "gate"), "rowgate": ("bias", "row_gate"), "all": tuple(every)}[form]
        self.post = form in ("post", "postonly", "all")
        if kind == "rms":
            wanted = [n for n in wanted if "bias" not in n]
        self.given = {n: every[n] if n in wanted else None for n in every}
        self.scale, self.eps = (0.625 if self.y is not None else 1.0), 1e-5

    def options(self, but=()):
        return dict(y=self.y, post=self.post, scale=self.scale, eps=self.eps,
                    **{k: v for k, v in self.given.items() if k not in but})

    def new(self):
        return _layout(torch.full((self.rows, self.cols), 9.0, dtype=self.dtype, device=DEV), self.layout)


def _near(got, want, size, dtype, slack=0.0):
    """|got - want| within half a step of the type and `size` fp32 roundings' worth."""
    err = (R.f64(got) - want).abs()
    bound = size + (want.abs() + size) * EPS[dtype] + TINY[dtype] + slack
    worst = float((err - bound).max()) if err.numel() else 0.0
    assert bool((err <= bound).all()), (worst, float(err.max()))


def _sums(n):
    """Relative error, in fp32 roundings, of a sum of n terms as the kernel adds them: up to 32 in a row in a thread,
    then trees and at most 16 warps, so at most 32 + 5 + 16 roundings of the partial sums."""
    return min(n, 53) * 2.0 ** -24


FORMS = ["pre", "bare", "post", "postonly", "gate", "rowgate", "all"]
# rows, cols: one column, one thread, warps' ends, short rows that share a block, several groups a thread, the most
SIZES = [(3, 1), (70, 7), (33, 64), (9, 257), (130, 515), (40, 768), (17, 2048), (6, 2056), (5, 4099), (3, 8192), (2, 16384)]


def _forward_bounds(c, h64, u64, want_h, want_n):
    """fp32 errors of h and n.  A norm's factor is off by half the relative error of its mean square, and by the
    rounding of the root and the quotient; a mean by its sum's."""
    f = 2.0 ** -24

    def hat_error(v):
        mean = v.mean(dim=1, keepdim=True) if c.kind == "layer" else torch.zeros(len(v), 1, dtype=torch.float64)
        size = v.abs().mean(dim=1, keepdim=True)
        root = torch.sqrt(((v - mean) ** 2).mean(dim=1, keepdim=True) + c.eps)
        off = size * (_sums(c.cols) + f) if c.kind == "layer" else torch.zeros_like(mean)
        # the mean's error, the difference's rounding, and the factor's relative error
        return (off + (v - mean).abs() * f) / root + ((v - mean).abs() / root) * (_sums(c.cols) + 5 * f + 2 * off / root)

    def times(e, v, w, b):
        w = 1.0 if w is None else R.f64(w).abs()
        b = 0.0 if b is None else R.f64(b).abs()
        return e * w + (v.abs() * w + b) * 2 * f

    e_h = torch.zeros_like(h64)
    if c.y is not None:
        y = R.f64(c.y)
        hat = R.hat(y, c.kind, c.eps)
        e = times(hat_error(y), hat, c.given["post_weight"], c.given["post_bias"]) if c.post else torch.zeros_like(y)
        by = torch.full((1, 1), abs(c.scale), dtype=torch.float64)
        by = by if c.given["gate"] is None else by * R.f64(c.given["gate"]).abs()
        by = by if c.given["row_gate"] is None else by * R.f64(c.given["row_gate"])[:, None]
        e_h = e * by + u64.abs() * 3 * f + want_h.abs() * f
    hat = R.hat(h64, c.kind, c.eps)
    mean = h64.mean(dim=1, keepdim=True) if c.kind == "layer" else 0.0
    root = torch.sqrt(((h64 - mean) ** 2).mean(dim=1, keepdim=True) + c.eps)
    # h's own error through the norm: no more than twice its size there and in the factor
    worst = e_h.amax(dim=1, keepdim=True)
    through = (2 * e_h + worst) / root + hat.abs() * 2 * worst / root
    return e_h * 1.01, times(hat_error(h64) + through, hat, c.given["weight"], c.given["bias"]) * 1.01


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_norm(dtype, kind, size):
    for k, form in enumerate(FORMS):
        c = Case(kind, *size, dtype, form, ["dense", "strided", "shifted"][k % 3])
        given = {n: R.f64(v) for n, v in c.given.items()}
        y64 = R.f64(c.y)
        u = torch.zeros(size, dtype=torch.float64) if c.y is None else R.branch(
            kind, y64, c.post, given["post_weight"], given["post_bias"], given["gate"], given["row_gate"], c.scale, c.eps)
        want_h, want_n = R.norm(kind, R.f64(c.x), y=y64, post=c.post, scale=c.scale, eps=c.eps, **given)
        e_h, e_n = _forward_bounds(c, want_h, u, want_h, want_n)
        h, n = c.new() if c.y is not None else None, c.new()
        dopt.dopt_norm(kind, c.x, n, h=h, **c.options())
        _near(n, want_n, e_n, dtype)
        if h is None:
            continue
        _near(h, want_h, e_h, dtype)
        # either output alone, and the residual in place
        n2, x2 = c.new(), _layout(c.x.clone(), c.layout)
        dopt.dopt_norm(kind, c.x, n2, h=None, **c.options())
        assert torch.equal(n2, n)
        dopt.dopt_norm(kind, x2, None, h=x2, **c.options())
        assert torch.equal(x2, h)
        x2.copy_(c.x)
        dopt.dopt_norm(kind, x2, n2.fill_(1), h=x2, **c.options())
        assert torch.equal(x2, h) and torch.equal(n2, n)


def _gradients(c):
    """All gradients in 64 bits, from torch's automatic differentiation of the definition."""
    h = R.f64(c.h).requires_grad_()
    leaf = {n: None if v is None else R.f64(v).requires_grad_() for n, v in c.given.items()}
    y = None if c.y is None else R.f64(c.y).requires_grad_()
    ones = {n: torch.ones(c.cols, dtype=torch.float64).requires_grad_() if v is None and "bias" not in n and n != "row_gate"
            else v for n, v in leaf.items()}
    for n in ("bias", "post_bias"):
        if ones[n] is None:
            ones[n] = torch.zeros(c.cols, dtype=torch.float64).requires_grad_()
    n_out = R.affine(R.hat(h, c.kind, c.eps), ones["weight"], ones["bias"])
    first = torch.autograd.grad(n_out, [h, ones["weight"], ones["bias"]], R.f64(c.d_n))
    d_x = R.f64(c.d_h) + first[0]
    found = dict(d_x=d_x, weight=first[1], bias=first[2])
    if y is not None:
        u = R.branch(c.kind, y, c.post, ones["post_weight"], ones["post_bias"], ones["gate"], ones["row_gate"], c.scale, c.eps)
        names = ["gate"] + (["post_weight", "post_bias"] if c.post else []) + (["row_gate"] if ones["row_gate"] is not None else [])
        got = torch.autograd.grad(u, [y] + [ones[n] for n in names], d_x)
        found.update(d_y=got[0], **dict(zip(names, got[1:])))
    return found


@pytest.mark.parametrize("size", SIZES + [(2500, 72), (700, 1032)], ids=str)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_norm_grad(dtype, kind, size):
    rows, cols = size
    ws = dopt.norm_workspace(rows, cols)
    for k, form in enumerate(FORMS):
        c = Case(kind, rows, cols, dtype, form, ["dense", "strided", "shifted"][k % 3], seed=1)
        want = _gradients(c)
        names = [n for n in PARAMS if n in want and (kind == "layer" or "bias" not in n)]
        at = {n: 5 + i * (cols + 3) for i, n in enumerate(names)}
        # errors relative to the largest of a row: a row's results are sums of its terms, each with a handful of
        # fp32 roundings, over a root that is not small (values spread by 0.5 and more)
        f = 64 * 2.0 ** -24
        one_col = cols == 1 and kind == "layer"  # the norm of one column is 0 whatever it holds: its factor is 1 / sqrt(eps)
        for grad_type in (dtype, torch.float32):
            ws.fill_(255)
            grad = torch.full((5 + 5 * (cols + 3),), 2.0, dtype=grad_type, device=DEV)
            d_x, d_y = c.new(), c.new() if c.y is not None else None
            d_row = torch.full((rows,), 9.0, device=DEV) if c.given["row_gate"] is not None else None
            dopt.dopt_norm_grad(kind, c.h, c.d_n, d_x, d_y=d_y, d_h=c.d_h, d_row_gate=d_row, grad=grad, grad_offsets=at,
                                workspace=ws, **c.options(("bias",)))
            size_x = R.f64(c.d_h).abs() + R.f64(c.d_n).abs().amax(dim=1, keepdim=True) * (400 if one_col else 4 if cols > 8 else 100)
            _near(d_x, want["d_x"], size_x * f, dtype)
            if d_y is not None:
                size_y = size_x.amax(dim=1, keepdim=True) * 4 * ((400 if one_col else 4 if cols > 8 else 100) if c.post else 1)
                _near(d_y, want["d_y"], size_y.expand(rows, cols) * f, dtype)
            hats = 6.0  # the largest of the normed values and of y
            used = torch.zeros(len(grad), dtype=torch.bool)
            for n in names:
                total = (R.f64(c.d_n).abs() if n in ("weight", "bias") else size_x).sum(dim=0) * (1.0 if "bias" in n else hats)
                _near(grad[at[n]:at[n] + cols], want[n], total * f * 2, grad_type)
                used[at[n]:at[n] + cols] = True
            assert bool((grad.cpu()[~used] == 2).all())
            if d_row is not None:
                _near(d_row, want["row_gate"], size_x.sum(dim=1) * 2 * hats * f, torch.float32)
        # the same again, in place and without what is not wanted
        d_x2 = _layout(c.d_h.clone(), c.layout)
        dopt.dopt_norm_grad(kind, c.h, c.d_n, d_x2, d_h=d_x2, workspace=ws, **c.options(("bias",)))
        assert torch.equal(d_x2, d_x)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_one_of_two_gradients(kind):
    """Without d_n the residual's gradient passes; without d_h it counts as zeros."""
    c = Case(kind, 50, 136, torch.float32, "all")
    ws = dopt.norm_workspace(50, 136)
    zero = torch.zeros_like(c.d_h)
    for d_n, d_h in ((None, c.d_h), (c.d_n, None)):
        got, want = (c.new(), c.new()), (c.new(), c.new())
        dopt.dopt_norm_grad(kind, c.h, d_n, got[0], d_y=got[1], d_h=d_h, workspace=ws, **c.options(("bias",)))
        dopt.dopt_norm_grad(kind, c.h, zero if d_n is None else d_n, want[0], d_y=want[1], d_h=zero if d_h is None else d_h,
                            workspace=ws, **c.options(("bias",)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_grads_accumulate(kind, dtype):
    c = Case(kind, 77, 264, dtype, "all")
    ws = dopt.norm_workspace(77, 264)
    names = [n for n in PARAMS if kind == "layer" or "bias" not in n]
    at = {n: i * 264 for i, n in enumerate(names)}
    n_grads = 264 * len(names)

    def run(grad, **more):
        dopt.dopt_norm_grad(kind, c.h, c.d_n, None, d_h=c.d_h, grad=grad, grad_offsets=at, workspace=ws,
                            **c.options(("bias",)), **more)
        return grad

    sums = run(torch.zeros(n_grads, device=DEV))
    old = torch.randn(n_grads, device=DEV).to(dtype)
    assert torch.equal(run(old.clone(), accumulate=True), (old.float() + sums).to(dtype))


def test_no_rows():
    for kind in ("rms", "layer"):
        c = Case(kind, 0, 40, torch.bfloat16, "all")
        at = {"weight": 0, "gate": 50}
        grad = torch.full((100,), 3.0, device=DEV)
        keep = grad.clone()
        dopt.dopt_norm(kind, c.x, c.new(), h=c.new(), **c.options())
        run = dict(grad=grad, grad_offsets=at, workspace=dopt.norm_workspace(0, 40))
        dopt.dopt_norm_grad(kind, c.h, c.d_n, None, d_h=c.d_h, accumulate=True, **run, **c.options(("bias",)))
        assert torch.equal(grad, keep)
        dopt.dopt_norm_grad(kind, c.h, c.d_n, None, d_h=c.d_h, **run, **c.options(("bias",)))
        assert not grad[:40].any() and not grad[50:90].any() and bool((grad[40:50] == 3).all())


def test_bad_rows_stay_in_their_rows():
    for kind in ("rms", "layer"):
        c = Case(kind, 30, 520, torch.float32, "all")
        want_h, want_n = c.new(), c.new()
        dopt.dopt_norm(kind, c.x, want_n, h=want_h, **c.options())
        c.x[4, 100], c.y[9, 519] = float("nan"), float("inf")
        h, n = c.new(), c.new()
        dopt.dopt_norm(kind, c.x, n, h=h, **c.options())
        good = [r for r in range(30) if r not in (4, 9)]
        assert torch.equal(h[good], want_h[good]) and torch.equal(n[good], want_n[good])
        assert bool(torch.isnan(n[[4, 9]]).all()) and int(torch.isnan(h[4]).sum()) == 1


def test_large_and_small_values():
    """Mean squares near fp32's ends; a constant row's layer norm is its bias."""
    x = torch.tensor([1e15, 1e-15], device=DEV)[:, None] * torch.randn(2, 300, device=DEV)
    n = torch.empty_like(x)
    dopt.dopt_norm("rms", x, n, eps=0.0)
    _near(n, R.hat(R.f64(x), "rms", 0.0), torch.full((2, 300), 6 * 64 * 2.0 ** -24, dtype=torch.float64), torch.float32)
    x = torch.full((3, 512), 7.0, device=DEV)
    bias = torch.randn(512, device=DEV)
    n = torch.empty_like(x)
    dopt.dopt_norm("layer", x, n, bias=bias)
    assert torch.equal(n, bias.expand(3, 512))
