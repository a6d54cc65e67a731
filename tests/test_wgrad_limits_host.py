"""Sizes that the weight gradient's 32-bit counts cannot hold are refused on the
host, before any CUDA call (the fake pointers are never dereferenced)."""
import ctypes

import pytest

import zero_distributed_optimizer_gb300 as dopt
from zero_distributed_optimizer_gb300 import binding as B
from zero_distributed_optimizer_gb300 import build as libbuild

P = 0x10000  # 16-byte aligned, never read


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.lib()


# The rows of whole steps of 64 that cover so many, in 32 bits, would be negative.
@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 63])
def test_rows_that_overflow_are_refused(lib, rows):
    n = ctypes.c_int64(-1)
    assert lib.dopt_ckpt_wgrad_workspace(rows, 8, 8, 1, ctypes.byref(n)) == B.DOPT_E_ARG
    starts = (ctypes.c_int64 * 1)(0)
    rc = lib.dopt_ckpt_wgrad(P, B.DOPT_BF16, 10, 8, P, P, B.DOPT_BF16, rows, 8, 8, P, 1, starts, P, B.DOPT_FP32, 64, 0,
                             None, 0, None)
    assert rc == B.DOPT_E_ARG
    assert "dy" in lib.dopt_last_error().decode()


def test_the_most_rows_are_taken(lib):
    n = ctypes.c_int64(-1)
    assert dopt.DOPT_WGRAD_MAX_ROWS == 2 ** 31 - 64
    assert lib.dopt_ckpt_wgrad_workspace(2 ** 31 - 64, 8, 8, 1, ctypes.byref(n)) == 0


def test_product_build_has_no_wait_test(lib):
    if B.LIB_PATH.endswith("libdopt_checked.so"):
        pytest.skip("this process runs the checked build")
    for items in (-1, 0):
        with pytest.raises(dopt.DoptError) as e:
            dopt.wgrad_wait_test(items)
        assert e.value.code == B.DOPT_E_STATE
