"""The token embedding and its gradient against 64-bit forms: every type and
id width, odd sizes and strides, ids outside, empty tables' rows, runs of one
token that reach over many blocks, accumulation, and sums that are exact."""
import pytest
import torch

import model_reference as R
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = {t: torch.finfo(t).eps / 2 for t in DTYPES}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half of the least step


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


def _ids(tokens, vocab, how, g, dtype=torch.int64):
    if how == "one":      # all the same: one run over every block
        ids = torch.full((tokens,), vocab // 2, device=DEV)
    elif how == "few":    # long runs next to each other, their ends anywhere in a chunk
        ids = torch.randint(0, min(vocab, 7), (tokens,), generator=g, device=DEV) * max(1, vocab // 7)
    elif how == "most":   # a padding id, the others spread
        ids = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
        ids[torch.rand(tokens, generator=g, device=DEV) < 0.6] = vocab - 1
    elif how == "none":
        ids = torch.full((tokens,), -1, device=DEV)
    else:                 # a third outside on either side
        ids = torch.randint(-vocab // 4, vocab + vocab // 4, (tokens,), generator=g, device=DEV)
        ids[ids < 0] -= 100
    return ids.to(dtype)


@pytest.mark.parametrize("layout", ["dense", "strided", "shifted"])
@pytest.mark.parametrize("cols", [1, 7, 64, 257, 515, 768])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_embed(dtype, cols, layout):
    tokens, vocab = 131, 97
    g = torch.Generator(device=DEV).manual_seed(cols)
    table = _layout(torch.randn(vocab, cols, generator=g, device=DEV).to(dtype), layout)
    for scale, id_type in ((1.0, torch.int64), (-2.7, torch.int32)):
        ids = _ids(tokens, vocab, "outside", g, id_type)
        out = _layout(torch.full((tokens, cols), 3.0, dtype=dtype, device=DEV), layout)
        dopt.dopt_embed(table, ids, out, scale=scale)
        s = float(torch.tensor(scale))  # (as fp32 has it)
        want = R.embed(table, ids, s)
        # the product in fp32, then its rounding to the type
        bound = want.abs() * (EPS[dtype] + 2.0 ** -24) * 1.01 + TINY[dtype]
        if scale == 1.0:
            assert torch.equal(out.cpu().double(), want)
        assert bool(((R.f64(out) - want).abs() <= bound).all())
        before = out.clone()
        dopt.dopt_embed(table, ids, out, scale=scale, accumulate=True)
        inside = ((ids >= 0) & (ids < vocab)).cpu()
        assert torch.equal(out.cpu()[~inside], before.cpu()[~inside])
        want = R.f64(before) + want
        # product, sum and rounding
        bound = (want.abs() * (EPS[dtype] + 2.0 ** -24) + R.embed(table.abs(), ids, abs(s)) * 2.0 ** -24) * 1.01 + TINY[dtype]
        assert bool(((R.f64(out) - want).abs() <= bound).all())


def test_embed_edges():
    table = torch.randn(5, 40, device=DEV)
    table[2, 3] = float("nan")
    table[3, 0] = float("inf")
    out = torch.full((4, 40), 7.0, device=DEV)
    dopt.dopt_embed(table, torch.empty(0, dtype=torch.int64, device=DEV), out[:0])
    assert bool((out == 7).all())
    ids = torch.tensor([2, -1, 2 ** 40, 3], device=DEV)
    dopt.dopt_embed(table, ids, out)
    assert torch.equal(out[[0, 3]].view(torch.int32), table[[2, 3]].view(torch.int32)) and not out[1:3].any()
    out.fill_(-0.0)
    dopt.dopt_embed(table, ids, out, accumulate=True)
    assert bool(torch.signbit(out[1:3]).all())  # left as they were


def test_embed_far_rows():
    """Rows past 2^32 bytes of a table."""
    vocab, cols = 2 ** 21 + 3, 1032
    table = torch.empty(vocab, cols, dtype=torch.bfloat16, device=DEV)
    ids = torch.tensor([vocab - 1, 2 ** 21 - 5, 0], device=DEV)
    table[ids] = torch.randn(3, cols, device=DEV).bfloat16()
    out = torch.empty(3, cols, dtype=torch.bfloat16, device=DEV)
    dopt.dopt_embed(table, ids.int(), out)
    assert torch.equal(out, table[ids])


SIZES = [  # tokens, vocab, cols, ids
    (1, 1, 1, "one"), (31, 50, 96, "outside"), (1000, 97, 64, "outside"), (5000, 3, 40, "one"), (4097, 2000, 257, "few"),
    (3000, 40000, 72, "most"), (1500, 1024 * 3 + 1, 8, "few"), (257, 12, 515, "one"), (300, 90, 33, "none"), (0, 50, 48, "none"),
]


@pytest.mark.parametrize("layout", ["dense", "strided", "shifted"])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_embed_grad(dtype, size, layout):
    tokens, vocab, cols, how = size
    g = torch.Generator(device=DEV).manual_seed(tokens + cols)
    ids = _ids(tokens, vocab, how, g, torch.int32 if layout == "strided" else torch.int64)
    d_out = _layout(torch.randn(tokens, cols, generator=g, device=DEV).to(dtype), layout)
    d_out[(ids < 0) | (ids >= vocab)] = float("nan")
    ws = dopt.embed_workspace(tokens, vocab, cols)
    ws.fill_(255)
    scale = 0.75
    want, size_, count = R.embed_grad(ids, torch.nan_to_num(d_out), vocab, scale)
    # a sum of n terms in any order: n - 1 roundings of at most the sum of magnitudes each; the scale's product
    fp32 = (size_ * (count.double()[:, None] + 1) * 2.0 ** -24) * 1.01
    for grad_type in DTYPES:
        first = 8 if layout == "dense" else 3
        grad = torch.full((first + vocab * cols + 5,), 2.0, dtype=grad_type, device=DEV)
        dopt.dopt_embed_grad(ids, d_out, grad, first, vocab, scale=scale, workspace=ws)
        got = R.f64(grad)
        assert bool((got[:first] == 2).all()) and bool((got[first + vocab * cols:] == 2).all())
        err = (got[first:first + vocab * cols].view(vocab, cols) - want).abs()
        assert bool((err <= fp32 + (want.abs() + fp32) * EPS[grad_type] + TINY[grad_type]).all())
        assert not got[first:first + vocab * cols].view(vocab, cols)[count == 0].any()
        again = torch.full_like(grad, 2.0)
        dopt.dopt_embed_grad(ids, d_out, again, first, vocab, scale=scale, workspace=ws)
        assert torch.equal(again, grad)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_embed_grad_accumulates(dtype):
    tokens, vocab, cols = 700, 300, 136
    g = torch.Generator(device=DEV).manual_seed(5)
    ids = _ids(tokens, vocab // 2, "few", g)
    d_out = torch.randint(-4, 5, (tokens, cols), generator=g, device=DEV).to(dtype)
    grad = torch.randint(-8, 9, (vocab * cols,), generator=g, device=DEV).to(dtype)
    bits = grad.view(torch.int32 if dtype is torch.float32 else torch.int16)
    untouched = torch.ones(vocab, dtype=torch.bool, device=DEV)
    untouched[ids.unique()] = False
    bits.view(vocab, cols)[untouched] = -2 ** 31 if dtype is torch.float32 else -2 ** 15  # -0
    before = grad.clone()
    dopt.dopt_embed_grad(ids, d_out, grad, 0, vocab, accumulate=True, workspace=dopt.embed_workspace(tokens, vocab, cols))
    sums, _, _ = R.embed_grad(ids, d_out, vocab, 1.0)
    want = (R.f64(before).view(vocab, cols) + sums).to(dtype)  # exact sums, one rounding
    assert torch.equal(grad.cpu().view(vocab, cols), want)
    assert torch.equal(grad.view(bits.dtype).view(vocab, cols)[untouched], before.view(bits.dtype).view(vocab, cols)[untouched])


def test_embed_grad_exact_over_many_chunks():
    """Whole numbers: every order of the sums gives the same bits as 64-bit integers."""
    tokens, vocab, cols = 70001, 33, 264
    g = torch.Generator(device=DEV).manual_seed(9)
    ids = _ids(tokens, vocab, "most", g)
    d_out = torch.randint(-3, 4, (tokens, cols), generator=g, device=DEV).bfloat16()
    grad = torch.zeros(vocab * cols, device=DEV)
    dopt.dopt_embed_grad(ids, d_out, grad, 0, vocab, workspace=dopt.embed_workspace(tokens, vocab, cols))
    want = torch.zeros(vocab, cols, dtype=torch.int64, device=DEV).index_add_(0, ids, d_out.long())
    assert torch.equal(grad.view(vocab, cols).long(), want)


def test_embed_grad_is_the_gradient():
    """Against differences of a scalar of the embedding."""
    tokens, vocab, cols = 90, 20, 24
    g = torch.Generator(device=DEV).manual_seed(3)
    table = torch.randn(vocab, cols, generator=g, device=DEV)
    ids = _ids(tokens, vocab, "outside", g)
    r = torch.randint(-4, 5, (tokens, cols), generator=g, device=DEV).float()
    grad = torch.zeros(vocab * cols, device=DEV)
    dopt.dopt_embed_grad(ids, r, grad, 0, vocab, scale=0.5, workspace=dopt.embed_workspace(tokens, vocab, cols))

    def value(t):
        out = torch.empty(tokens, cols, device=DEV)
        dopt.dopt_embed(t, ids, out, scale=0.5)
        return float((out.double() * r.double()).sum())

    for v, c in ((0, 0), (7, 11), (19, 23)):
        up, down = table.clone(), table.clone()
        up[v, c] += 1.0
        down[v, c] -= 1.0
        diff = (value(up) - value(down)) / float(up[v, c].double() - down[v, c].double())
        # linear in the table: fp32's rounding of the two products of each of the id's tokens is all that differs
        n = int((ids == v).sum())
        assert abs(diff - float(grad[v * cols + c])) <= n * 4 * 4 * 2.0 ** -24 + 1e-6 * abs(diff)
