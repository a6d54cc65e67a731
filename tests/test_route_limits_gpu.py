"""Sorting by expert where a call's shared memory meets the kernels' limit: the
first call of a process at the sizes around 48 KB, and threads that sort with
different numbers of experts at once."""
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import layer_reference as R
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"

FIRST_CALL = """
import torch, zero_distributed_optimizer_gb300 as dopt
tokens, k, experts = {tokens}, 2, {experts}
g = torch.Generator(device="cuda").manual_seed(experts)
ids = torch.randint(0, experts, (tokens, k), generator=g, device="cuda")
i32 = dict(dtype=torch.int32, device="cuda")
slot_row, row_token = torch.empty(tokens, k, **i32), torch.empty(tokens * k, **i32)
offsets = torch.empty(experts + 1, **i32)
dopt.dopt_route_sort(ids, experts, slot_row, row_token, offsets, dopt.route_workspace(tokens, k, experts))
key, order = torch.sort(ids.reshape(-1), stable=True)
assert torch.equal(row_token, (order // k).int())
assert torch.equal(offsets, torch.searchsorted(key, torch.arange(experts + 1, device="cuda")).int())
"""


@pytest.mark.parametrize("tokens", [500, 9000, 40000])  # one block, a cluster, two launches
@pytest.mark.parametrize("experts", [349, 350, 351])
def test_first_call_of_a_process(tokens, experts):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(tokens=tokens, experts=experts)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-1500:]


def _sorts(ids, experts, times, stream, out):
    tokens, k = ids.shape
    with torch.cuda.stream(stream):
        got = [torch.empty(tokens, k, dtype=torch.int32, device=DEV),
               torch.empty(tokens * k, dtype=torch.int32, device=DEV),
               torch.empty(experts + 1, dtype=torch.int32, device=DEV)]
        ws = dopt.route_workspace(tokens, k, experts)
        try:
            for _ in range(times):
                dopt.dopt_route_sort(ids, experts, *got, ws, stream=stream)
            stream.synchronize()
            out[experts] = got
        except dopt.DoptError as e:
            out[experts] = e


def test_threads_with_different_numbers_of_experts():
    cases = {}
    for experts in (1024, 400, 64, 1000, 351):
        ids = np.random.default_rng(experts).integers(-1, experts + 1, (300, 2))
        cases[experts] = ids, torch.from_numpy(ids).to(DEV)
    torch.cuda.synchronize()
    out = {}
    threads = [threading.Thread(target=_sorts, args=(t, experts, 3000, torch.cuda.Stream(), out))
               for experts, (_, t) in cases.items()]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for experts, (ids, _) in cases.items():
        assert not isinstance(out[experts], Exception), out[experts]
        for a, b in zip(out[experts], R.sort(ids, experts)):
            assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("large,small", [(700000, 600000), (622593, 622592), (1245185, 1245184), (2000000, 40000)])
def test_a_larger_batchs_workspace(large, small):
    ws = dopt.route_workspace(large, 1, 5)
    ids = torch.randint(0, 5, (small, 1), generator=torch.Generator(device=DEV).manual_seed(small), device=DEV)
    slot_row, row_token = (torch.empty(s, dtype=torch.int32, device=DEV) for s in ((small, 1), (small,)))
    offsets = torch.empty(6, dtype=torch.int32, device=DEV)
    dopt.dopt_route_sort(ids, 5, slot_row, row_token, offsets, ws)
    key, order = torch.sort(ids.reshape(-1), stable=True)
    assert torch.equal(row_token, order.int())
    assert torch.equal(offsets, torch.searchsorted(key, torch.arange(6, device=DEV)).int())
