"""The loss kernels' bounded waits, made to run out in the test build (the first
pair of blocks of each launch issues no products from some item on): the calls
return, what depends on the pair's work is NaN, nothing else is, and the next
calls on the same context and workspaces are right."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import torch
import zero_distributed_optimizer_gb300 as dopt
from zero_distributed_optimizer_gb300 import binding as B

assert B.LIB_PATH.endswith("libdopt_checked.so"), B.LIB_PATH
DEV = "cuda"
g = torch.Generator(device=DEV).manual_seed(3)
rows, width, vocab = 700, 200, 1500
x = torch.randn(rows, width, generator=g, device=DEV).bfloat16()
w = (torch.randn(vocab, width, generator=g, device=DEV) / 8).bfloat16()
targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
d_loss = torch.full((rows,), 1 / rows, device=DEV)
ws = dopt.head_loss_workspace(rows, width, vocab)
ws_grad = dopt.head_loss_grad_workspace(rows, width, vocab, torch.float32)


def loss():
    out = torch.full((2, rows), 5.0, device=DEV)
    dopt.dopt_head_loss(x, w, targets, out[0], out[1], workspace=ws)
    torch.cuda.synchronize()
    return out


def grad(lse):
    d_x, flat = torch.full_like(x, 5.0), torch.full((vocab * width,), 5.0, device=DEV)
    dopt.dopt_head_loss_grad(x, w, targets, lse, d_loss, d_x, flat, workspace=ws_grad)
    torch.cuda.synchronize()
    return d_x, flat


assert dopt.head_timeouts(reset=True) == 0
want = loss()
want_x, want_w = grad(want[1])
# one item a pair here (18 tiles of logits): the first pair's tile is of tokens 0..255
dopt.head_wait_test(0)
got = loss()
dopt.head_wait_test(-1)
assert dopt.head_timeouts(reset=True) == 2, dopt.head_timeouts()
assert torch.isnan(got[:, :256]).all() and torch.equal(got[:, 256:], want[:, 256:])
dopt.head_wait_test(0)
d_x, d_w = grad(want[1])
dopt.head_wait_test(-1)
assert dopt.head_timeouts(reset=True) == 4  # the logits, then both products
assert torch.isnan(d_x[:256]).all() and torch.isnan(d_w[:256 * width]).all()
again = loss()
assert torch.equal(again, want)
d_x, d_w = grad(want[1])
assert torch.equal(d_x, want_x) and torch.equal(d_w, want_w)
assert dopt.head_timeouts() == 0
print("WAIT_OK")
"""


def test_waits_run_out_without_fault():
    from zero_distributed_optimizer_gb300 import build

    build.build(checked=True)
    env = dict(os.environ, DOPT_CHECKED="1")
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "WAIT_OK" in r.stdout
