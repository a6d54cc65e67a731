"""The weight gradient's bounded waits, made to run out in the test build (the
first pair of blocks issues no products from some item on): the call returns,
both blocks are counted, what the pair did not write is NaN and nothing else
is, and the next call on the same context and workspace is right."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import torch
import zero_distributed_optimizer_gb300 as dopt
from zero_distributed_optimizer_gb300 import binding as B

assert B.LIB_PATH.endswith("libdopt_checked.so"), B.LIB_PATH
DEV = "cuda"
assert torch.cuda.get_device_properties(0).multi_processor_count == 152  # 76 pairs
g = torch.Generator(device=DEV).manual_seed(3)


def case(rows, outs, cols, bounds):
    x = torch.randint(-60, 61, (rows, cols), generator=g, device=DEV).bfloat16()  # kept exactly
    dy = torch.randint(-8, 9, (rows, outs), generator=g, device=DEV).bfloat16()
    c = dopt.checkpoint(rows, cols)
    dopt.dopt_ckpt_save(x, c)
    E = len(bounds) - 1
    more = dict(offsets=torch.tensor(bounds, dtype=torch.int32, device=DEV),
                row_token=torch.arange(rows, dtype=torch.int32, device=DEV)) if E > 1 else {}
    want = torch.stack([dy[a:b].double().t() @ x[a:b].double() for a, b in zip(bounds, bounds[1:])])
    starts = [k * outs * cols for k in range(E)]

    def call(grad, **options):
        dopt.dopt_ckpt_wgrad(c, dy, grad.view(-1), starts, **more, **options)
        torch.cuda.synchronize()
        return grad
    return want, call


assert dopt.wgrad_timeouts(reset=True) == 0
# 200 tiles of 256 x 256: the first pair has three of them, and loses two
want, call = case(2400, 1280, 1280, [300 * k for k in range(9)])
dopt.wgrad_wait_test(1)
got = call(torch.full(want.shape, 5.0, device=DEV))
dopt.wgrad_wait_test(-1)
assert dopt.wgrad_timeouts() == 2, dopt.wgrad_timeouts()
bad = torch.isnan(got)
assert torch.equal(got[~bad].double(), want[~bad])
tiles = bad.view(8, 5, 256, 5, 256).transpose(2, 3).flatten(3)
assert int(tiles.all(dim=3).sum()) == int(tiles.any(dim=3).sum()) == 2
assert torch.equal(call(torch.full(want.shape, 5.0, device=DEV)).double(), want)
assert dopt.wgrad_timeouts(reset=True) == 2

# one tile whose rows are split over pairs, and a workspace that holds numbers
want, call = case(6000, 200, 250, [0, 6000])
ws = dopt.wgrad_workspace(6000, 200, 250)
assert ws.numel() >= 2 * 4 * 256 * 256
for dtype, accumulate in ((torch.float32, False), (torch.bfloat16, True)):
    ws.view(torch.float32).fill_(1.0)
    dopt.wgrad_wait_test(0)
    got = call(torch.full(want.shape, 5.0, dtype=dtype, device=DEV), workspace=ws, accumulate=accumulate)
    dopt.wgrad_wait_test(-1)
    assert torch.isnan(got).all()
    assert dopt.wgrad_timeouts(reset=True) == 2
    got = call(torch.full(want.shape, 5.0, dtype=dtype, device=DEV), workspace=ws, accumulate=accumulate)
    assert torch.equal(got, (want + 5.0 * accumulate).float().to(dtype))
assert dopt.wgrad_timeouts() == 0
print("WAIT_OK")
"""


def test_waits_run_out_without_fault():
    from zero_distributed_optimizer_gb300 import build

    build.build(checked=True)
    env = dict(os.environ, DOPT_CHECKED="1")
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "WAIT_OK" in r.stdout


def test_the_layer_takes_no_step_on_lost_grads(monkeypatch):
    from zero_distributed_optimizer_gb300 import moe_layer

    layer = moe_layer.MoELayer(width=64, hidden=96, experts=4, k=2, tokens=100, D=2)
    before = [t.clone() for t in layer.params]
    seen = layer.timeouts
    monkeypatch.setattr(moe_layer.ops, "wgrad_timeouts", lambda: seen + 2)
    with pytest.raises(RuntimeError, match="ran out"):
        layer.step(moe_layer.teacher_batches(layer, 0))
    assert layer.steps == 0 and all(torch.equal(a, b) for a, b in zip(before, layer.params))
