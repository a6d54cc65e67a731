"""Every way in which a weight gradient divides its work, against exact sums:
more tiles than pairs of SMs, tiles of one and of two blocks of outputs, the
second block short or absent, rows of whole tiles and of split ones, joined,
added to what is there, dy aligned, copied and read element by element.  That a
case gets the plan it is there for is checked on the host, so that another
estimate of the plans' times cannot drop one unseen."""
import numpy as np
import pytest
import torch

import zero_distributed_optimizer_gb300 as dopt
from zero_distributed_optimizer_gb300 import build as libbuild

DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
PAIRS = 76

# rows, outs, cols, groups (1: dense), dy's type, the grads', with room for split sums: blocks, whole, split, parts
CASES = [
    # several tiles a pair, one block of outputs (in one sum, and in several)
    (9000, 1200, 1700, 9, BF16, BF16, False, (1, 315, 0, 1)),
    (9000, 1200, 1700, 9, FP16, FP32, True, (1, 315, 0, 1)),
    # two blocks, the last tile's second one short (1950 = 3 * 512 + 414) or absent (1666 = 3 * 512 + 130)
    (6000, 1950, 1290, 12, BF16, BF16, False, (2, 288, 0, 1)),
    (6000, 1950, 1290, 12, FP16, FP16, True, (2, 288, 0, 1)),
    (6000, 1666, 520, 12, BF16, BF16, True, (2, 144, 0, 1)),
    (6000, 1666, 520, 12, FP16, BF16, False, (2, 144, 0, 1)),
    # whole tiles and a split rest, one block and two
    (5000, 2600, 2000, 1, BF16, FP32, True, (1, 76, 12, 6)),
    (5000, 2600, 2000, 1, FP16, FP16, True, (1, 76, 12, 6)),
    (3000, 5600, 2000, 1, BF16, BF16, True, (2, 76, 12, 4)),
    (4500, 5300, 2000, 1, FP16, FP16, True, (2, 76, 12, 5)),
    # only split tiles, of two blocks
    (8192, 2304, 768, 1, FP16, FP16, True, (2, 0, 15, 5)),
    (6000, 1700, 1300, 1, BF16, BF16, True, (2, 0, 24, 3)),
]


@pytest.mark.parametrize("rows,outs,cols,groups,dtype,grad_dtype,room,plan", CASES, ids=str)
def test_each_case_has_its_plan(rows, outs, cols, groups, dtype, grad_dtype, room, plan):
    libbuild.build()
    got = dopt.wgrad_plan(rows, outs, cols, groups, dtype, grad_dtype, 1 << 40 if room else 0)
    assert got == plan
    if room:  # the workspace that is named has room for it, and for the copy of dy
        tiles = dopt.wgrad_plan(rows, outs, cols, groups, dtype, grad_dtype, 1 << 40)
        need = tiles.split * (tiles.parts if tiles.parts > 1 else 0) * tiles.blocks * 4 * 256 * 256
        assert _named(rows, outs, cols, groups) >= need + (rows * -(-outs // 8) * 16 if outs % 8 else 0)


def _named(rows, outs, cols, groups):
    return dopt.wgrad_workspace(rows, outs, cols, groups, device="cpu").numel()


def test_plans_reach_every_form():
    plans = [c[-1] for c in CASES]
    for blocks in (1, 2):
        mine = [p for p in plans if p[0] == blocks]
        assert any(p[1] > 2 * PAIRS and p[3] == 1 for p in mine)  # a pair's third tile
        assert any(p[1] > 0 and p[3] > 1 for p in mine)           # whole tiles before split ones
    two = [c[1] % 512 for c in CASES if c[-1][0] == 2]
    assert any(0 < r <= 256 for r in two) and any(r > 256 for r in two)


def test_plan_refusals():
    for change in (dict(rows=-1), dict(rows=2 ** 31 - 1), dict(outs=0), dict(cols=0), dict(groups=0), dict(groups=257),
                   dict(dy=FP32), dict(ws=-1)):
        a = dict(rows=10, outs=8, cols=8, groups=1, dy=BF16, grad=FP32, ws=0)
        a.update(change)
        with pytest.raises(dopt.DoptError):
            dopt.wgrad_plan(*a.values())


def _cuts(rows, groups):
    """Uneven groups, some empty, the first and last rows in none."""
    cut = np.sort(np.random.default_rng(rows + groups).integers(3, rows - 2, groups + 1))
    cut[0], cut[-1] = 3, rows - 2
    if groups > 5:
        cut[2] = cut[1]
        cut[5] = cut[4]
    return cut.tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["plain", "shifted"])
@pytest.mark.parametrize("rows,outs,cols,groups,dtype,grad_dtype,room,plan", CASES, ids=str)
def test_exact_sums(rows, outs, cols, groups, dtype, grad_dtype, room, plan, layout):
    """Whole numbers whose sums stay below 2^24 (and below fp16's largest):
    every order of summation gives one result, rounded once to the grads' type."""
    g = torch.Generator(device=DEV).manual_seed(rows + outs)
    x = torch.randint(-9, 10, (rows, cols), generator=g, device=DEV).to(dtype)
    dy = torch.randint(-4, 5, (rows, outs), generator=g, device=DEV).to(dtype)
    c = dopt.checkpoint(rows, cols, dtype)
    dopt.dopt_ckpt_save(x, c)
    more, bounds = {}, [0, rows]
    if groups > 1:
        bounds = _cuts(rows, groups)
        token = torch.randint(0, rows, (rows,), generator=g, device=DEV).int()
        more = dict(offsets=torch.tensor(bounds, dtype=torch.int32, device=DEV), row_token=token)
        dy[:bounds[0]] = float("nan")
        dy[bounds[-1]:] = float("nan")
    n = outs * cols
    want = []
    for a, b in zip(bounds, bounds[1:]):
        xe = x[token[a:b].long()] if groups > 1 else x[a:b]
        assert 36 * (b - a) < 2 ** 24  # magnitudes add up to less: the sums are exact in any order
        want.append((dy[a:b].double().t() @ xe.double()).float())
    if layout == "shifted":
        view = torch.full((rows * outs + 1,), float("nan"), dtype=dtype, device=DEV)[1:].view(rows, outs)
        view.copy_(dy)
        dy = view
    starts = [5 + k * (n + 3) for k in range(groups)]
    ws = None
    if room:
        copy = rows * -(-outs // 8) * 16 if layout == "shifted" else 0
        ws = torch.empty(_named(rows, outs, cols, groups) + copy, dtype=torch.uint8, device=DEV)
    grad = torch.full((5 + groups * (n + 3),), 2.0, dtype=grad_dtype, device=DEV)
    for accumulate in (False, True):
        before = grad.clone()
        dopt.dopt_ckpt_wgrad(c, dy, grad, starts, accumulate=accumulate, workspace=ws, **more)
        rest = torch.ones_like(grad, dtype=torch.bool)
        for k in range(groups):
            at = slice(starts[k], starts[k] + n)
            rest[at] = False
            old = before[at].float().view(outs, cols) if accumulate else 0.0
            assert torch.equal(grad[at].view(outs, cols), (old + want[k]).to(grad_dtype)), f"group {k}, {accumulate}"
        assert torch.all(grad[rest] == 2.0)
    assert dopt.wgrad_timeouts() == 0
