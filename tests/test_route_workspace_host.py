"""A sort's workspace made for the largest batch serves every smaller one."""
import ctypes

import pytest

from zero_distributed_optimizer_gb300 import binding as B
from zero_distributed_optimizer_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.lib()


def _bytes(lib, tokens, k=1, experts=8):
    n = ctypes.c_int64(-1)
    assert lib.dopt_route_workspace(tokens, k, experts, ctypes.byref(n)) == 0
    return n.value


STRETCHES = 304 * 2048  # slots of as many stretches as there can be


@pytest.mark.parametrize("experts", [1, 64, 1024])
def test_size_does_not_fall_as_slots_grow(lib, experts):
    sizes = sorted({s + d for m in (1, 2, 3, 7, 50) for s in (STRETCHES * m,) for d in (-2049, -1, 0, 1, 2, 2048, 2049)}
                   | set(range(0, 2 * STRETCHES, 1777)) | {32768, 32769, 2 ** 31 - 1})
    got = [_bytes(lib, s, 1, experts) for s in sizes]
    assert got == sorted(got)
    assert got[-1] == 304 * (experts + 1) * 4
