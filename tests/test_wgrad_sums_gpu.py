"""Long sums of the weight gradient: fp32 grads keep an fp32 sum's accuracy at
any number of rows (a tensor core's sum cuts off low bits every 16 rows, so it
may take only so many), and sums that are taken in several parts are whole.

Bounds.  A sum of c additions of 16 rows' products cuts off less than two
units of 2^-23 at each, one of the products' own sum and one of the running
one; sums of 1024 rows (512 with fp16 factors) have c = 64 (32), and adding
them up rounds by 2^-24 of the running sum each."""
import pytest
import torch

import layer_reference as R
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"
CHUNK = {torch.bfloat16: 1024, torch.float16: 512}
TYPES = [torch.bfloat16, torch.float16]


def _kept(x):
    """A checkpoint of x and its values in 64 bits."""
    c = dopt.checkpoint(*x.shape, x.dtype)
    dopt.dopt_ckpt_save(x, c)
    out = torch.empty(x.shape, device=DEV)
    dopt.dopt_ckpt_load(c, out)  # exact in fp32
    return c, out.double()


def _grads(c, dy, starts, outs, cols, dtype, **more):
    grad = torch.full((starts[-1] + outs * cols,), 3.0, dtype=dtype, device=DEV)
    dopt.dopt_ckpt_wgrad(c, dy, grad, starts, **more)
    return [grad[s:s + outs * cols].view(outs, cols) for s in starts]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [40000, 33333])
def test_fp32_grads_of_one_sign(rows, dtype):
    """Every addition cuts the same way."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = (0.5 + 0.5 * torch.rand(rows, 72, generator=g, device=DEV)).to(dtype)
    dy = (0.5 + 0.5 * torch.rand(rows, 40, generator=g, device=DEV)).to(dtype)
    c, kept = _kept(x)
    want = dy.double().t() @ kept
    chunks = -(-rows // CHUNK[dtype])
    room = (2 * (CHUNK[dtype] // 16) * 2.0 ** -23 + (chunks + 1) * 2.0 ** -24) * want
    for ws in (None, dopt.wgrad_workspace(rows, 40, 72)):
        got, = _grads(c, dy, [0], 40, 72, torch.float32, workspace=ws)
        off = (got.double() - want).abs()
        assert torch.all(off <= room), float((off / want).max())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_fp32_grads_of_both_signs(dtype):
    """Sums that wander: each addition cuts off half a unit of the running sum
    on average, whose size grows as the root of the rows: by the 2-norm, c / 3
    units of 2^-23 of the grads at most, and the roundings of the additions."""
    rows = 50001
    g = torch.Generator(device=DEV).manual_seed(1)
    c, kept = _kept(torch.randn(rows, 264, generator=g, device=DEV).to(dtype))
    dy = (torch.randn(rows, 130, generator=g, device=DEV) * 0.1).to(dtype)
    want = dy.double().t() @ kept
    got, = _grads(c, dy, [0], 130, 264, torch.float32)
    chunks = -(-rows // CHUNK[dtype])
    rel = float((got.double() - want).norm() / want.norm())
    assert rel <= CHUNK[dtype] / 16 / 3 * 2.0 ** -23 + chunks ** 0.5 * 2.0 ** -24, rel


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("outs,cols", [(1100, 1100), (40, 300)])
def test_sums_in_parts_are_whole(outs, cols, dtype):
    """Groups of no row to several parts' rows, more tiles than pairs of SMs and
    fewer: whole numbers, so every order gives the same sums."""
    sizes = [0, 1, 1024, 1025, 3000, 64, 0, 512, 2049]
    bounds = [sum(sizes[:k]) + 5 for k in range(len(sizes) + 1)]
    rows, E = bounds[-1] + 9, len(sizes)
    g = torch.Generator(device=DEV).manual_seed(outs)
    c, kept = _kept(torch.randint(-60, 61, (700, cols), generator=g, device=DEV).to(dtype))
    dy = torch.randint(-8, 9, (rows, outs), generator=g, device=DEV).to(dtype)
    token = torch.randint(0, 700, (rows,), generator=g, device=DEV).int()
    starts = [k * outs * cols for k in range(E)]
    offsets = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    got = _grads(c, dy, starts, outs, cols, torch.float32, offsets=offsets, row_token=token)
    for k in range(E):
        at = slice(bounds[k], bounds[k + 1])
        want = dy[at].double().t() @ kept[token[at].long()]
        assert torch.equal(got[k].double(), want), f"group {k}"


@pytest.mark.parametrize("rows,dtype", [(140001, torch.bfloat16), (20003, torch.float16), (131072, torch.bfloat16)],
                         ids=str)
def test_16_bit_grads_of_many_rows(rows, dtype):
    """Rows past what one sum of 16-bit grads takes: whole numbers below 2^24,
    rounded once."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    c, kept = _kept(torch.randint(-9, 10, (rows, 40), generator=g, device=DEV).to(dtype))
    dy = torch.randint(-3, 4, (rows, 24), generator=g, device=DEV).to(dtype)
    want = (dy.double().t() @ kept).float()
    for ws in (None, dopt.wgrad_workspace(rows, 24, 40)):
        got, = _grads(c, dy, [0], 24, 40, dtype, workspace=ws)
        assert torch.equal(got, want.to(dtype))
    R.close(got, want.double().cpu().numpy(), 0.0, dtype, "grads")
