"""Refusals of the layer operators that come before any CUDA call (the fake
pointers below are never dereferenced), and the sizes the library reports."""
import ctypes

import pytest
import torch

import zero_distributed_optimizer_gb300 as dopt
from zero_distributed_optimizer_gb300 import binding as B
from zero_distributed_optimizer_gb300 import build as libbuild
from zero_distributed_optimizer_gb300 import layer_ops as LO

P = 0x10000  # 16-byte aligned, never read


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.lib()


def _refused(lib, rc, code, text):
    assert rc == code
    assert text in lib.dopt_last_error().decode()


def test_sizes(lib):
    assert dopt.ckpt_bytes(10, 1) == 10 * 128 * 33 // 32
    assert dopt.ckpt_bytes(3, 5632) == 3 * 5632 * 33 // 32
    assert dopt.ckpt_bytes(0, 7) == 0
    assert dopt.ckpt_bytes(2 ** 31 - 1, dopt.DOPT_MAX_COLS) == (2 ** 31 - 1) * dopt.DOPT_MAX_COLS * 33 // 32
    for rows, cols in ((-1, 4), (2 ** 31, 4), (4, 0), (4, dopt.DOPT_MAX_COLS + 1)):
        with pytest.raises(dopt.DoptError):
            dopt.ckpt_bytes(rows, cols)
    n = ctypes.c_int64(-1)
    assert lib.dopt_route_workspace(4096, 8, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.dopt_route_workspace(4097, 8, 8, ctypes.byref(n)) == 0 and n.value > 0
    _refused(lib, lib.dopt_route_workspace(1, 0, 8, ctypes.byref(n)), B.DOPT_E_ARG, "dopt_route_workspace")
    _refused(lib, lib.dopt_route_workspace(1, 1, 0, ctypes.byref(n)), B.DOPT_E_ARG, "n_experts")
    _refused(lib, lib.dopt_ckpt_wgrad_workspace(-1, 1, 1, 1, ctypes.byref(n)), B.DOPT_E_ARG, "wgrad_workspace")
    assert lib.dopt_ckpt_wgrad_workspace(10, 1, 1, 1, None) == B.DOPT_E_ARG


@pytest.mark.parametrize("change,code,text", [
    (dict(id_bytes=2), B.DOPT_E_ARG, "id_bytes"), (dict(tokens=-1), B.DOPT_E_ARG, "tokens"),
    (dict(k=0), B.DOPT_E_ARG, "k 0"), (dict(k=65), B.DOPT_E_ARG, "k 65"),
    (dict(tokens=2 ** 30), B.DOPT_E_ARG, "2^31"), (dict(experts=1025), B.DOPT_E_ARG, "n_experts"),
    (dict(ids=0), B.DOPT_E_ARG, "expert_ids"), (dict(ids=P + 4), B.DOPT_E_ALIGN, "expert_ids"),
    (dict(slot_row=0), B.DOPT_E_ARG, "slot_row"), (dict(row_token=P + 1), B.DOPT_E_ALIGN, "row_token"),
    (dict(offsets=0), B.DOPT_E_ARG, "offsets"), (dict(ws=0), B.DOPT_E_ARG, "workspace"),
    (dict(ws_bytes=8), B.DOPT_E_ARG, "workspace of 8 bytes")])
def test_sort_refusals(lib, change, code, text):
    a = dict(ids=P, id_bytes=8, tokens=600000, k=2, experts=8, slot_row=P, row_token=P, offsets=P, ws=P,
             ws_bytes=1 << 20)
    a.update(change)
    _refused(lib, lib.dopt_route_sort(*a.values(), None), code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(dtype=5), B.DOPT_E_ARG, "dtype"), (dict(cols=0), B.DOPT_E_ARG, "cols"),
    (dict(cols=dopt.DOPT_MAX_COLS + 1, ld=1 << 30), B.DOPT_E_ARG, "cols"), (dict(ld=99), B.DOPT_E_ARG, "stride"),
    (dict(n_rows=2 ** 31), B.DOPT_E_ARG, "n_rows"), (dict(x=0), B.DOPT_E_ARG, "x is NULL"),
    (dict(x=P + 1), B.DOPT_E_ALIGN, "x is not"), (dict(rows=P + 1), B.DOPT_E_ALIGN, "rows"),
    (dict(slot_row=P + 2), B.DOPT_E_ALIGN, "slot_row"), (dict(k=0), B.DOPT_E_ARG, "k 0")])
def test_row_refusals(lib, change, code, text):
    a = dict(x=P, dtype=B.DOPT_BF16, tokens=4, cols=100, ld=100, slot_row=P, k=2, rows=P, n_rows=8)
    a.update(change)
    _refused(lib, lib.dopt_route_dispatch(*a.values(), None), code, text)
    if "x" in change:
        return
    # rows, dtype, n_rows, slot_row, weights, tokens, k, cols, out, ld
    b = [a["rows"], a["dtype"], a["n_rows"], a["slot_row"], P, a["tokens"], a["k"], a["cols"], P, a["ld"]]
    _refused(lib, lib.dopt_route_combine(*b, None), code, text)
    c = [P, a["ld"], a["rows"], a["dtype"], a["n_rows"], a["slot_row"], P, a["tokens"], a["k"], a["cols"], P, P]
    _refused(lib, lib.dopt_route_combine_grad(*c, None), code, text)


def test_combine_grad_needs_weights(lib):
    a = [P, 8, P, B.DOPT_FP32, 8, P, None, 4, 2, 8, P, P]
    _refused(lib, lib.dopt_route_combine_grad(*a, None), B.DOPT_E_ARG, "weights")
    a[6], a[11] = P, P + 2
    _refused(lib, lib.dopt_route_combine_grad(*a, None), B.DOPT_E_ALIGN, "d_weights")


def test_checkpoint_refusals(lib):
    bf = B.DOPT_BF16
    for args, code, text in (
            ((P, bf, -1, 8, 8, P), B.DOPT_E_ARG, "rows"), ((P, bf, 4, 0, 8, P), B.DOPT_E_ARG, "cols"),
            ((P, bf, 4, 8, 7, P), B.DOPT_E_ARG, "stride"), ((P, 9, 4, 8, 8, P), B.DOPT_E_ARG, "dtype"),
            ((0, bf, 4, 8, 8, P), B.DOPT_E_ARG, "x is NULL"), ((P, bf, 4, 8, 8, 0), B.DOPT_E_ARG, "NULL"),
            ((P, bf, 4, 8, 8, P + 8), B.DOPT_E_ALIGN, "16-byte"), ((P + 1, bf, 4, 8, 8, P), B.DOPT_E_ALIGN, "x")):
        _refused(lib, lib.dopt_ckpt_save(*args, None), code, text)
    for args, code, text in (
            ((P, 4, 8, None, 5, P, bf, 8), B.DOPT_E_ARG, "output rows"), ((P, 4, 8, P + 2, 5, P, bf, 8), B.DOPT_E_ALIGN, "row_index"),
            ((P, 4, 8, P, 5, 0, bf, 8), B.DOPT_E_ARG, "out is NULL"), ((P, 4, 8, P, 5, P, 3, 8), B.DOPT_E_ARG, "dtype")):
        _refused(lib, lib.dopt_ckpt_load(*args, None), code, text)
    for args, code, text in (
            ((P, 4, 8, 3, P, 8, bf, P, 8), B.DOPT_E_ARG, "activation"),
            ((P, 4, 9, dopt.DOPT_ACT_SWIGLU, P, 8, bf, P, 9), B.DOPT_E_ARG, "halves"),
            ((P, 4, 8, 0, P, 7, bf, P, 8), B.DOPT_E_ARG, "d_out"), ((P, 4, 8, 0, P, 8, bf, P, 7), B.DOPT_E_ARG, "d_in"),
            ((P, 4, 8, 0, P, 8, bf, P + 1, 8), B.DOPT_E_ALIGN, "d_in")):
        _refused(lib, lib.dopt_ckpt_act_grad(*args, None), code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(x_rows=-1), B.DOPT_E_ARG, "checkpoint"), (dict(cols=0), B.DOPT_E_ARG, "checkpoint"),
    (dict(outs=0), B.DOPT_E_ARG, "dy"), (dict(dy_ld=23), B.DOPT_E_ARG, "stride"),
    (dict(ckpt_dtype=4), B.DOPT_E_ARG, "dtype"), (dict(grad_dtype=4), B.DOPT_E_ARG, "dtype"),
    (dict(dy_dtype=B.DOPT_FP32), B.DOPT_E_ARG, "bf16 or fp16"),
    (dict(dy_dtype=B.DOPT_FP16), B.DOPT_E_ARG, "fp16 dy"), (dict(flags=2), B.DOPT_E_ARG, "flags"),
    (dict(groups=0), B.DOPT_E_ARG, "n_groups"), (dict(groups=257), B.DOPT_E_ARG, "n_groups"),
    (dict(offsets=None), B.DOPT_E_ARG, "n_groups"), (dict(row_token=None), B.DOPT_E_ARG, "row_token"),
    (dict(ckpt=0), B.DOPT_E_ARG, "NULL"), (dict(dy=0), B.DOPT_E_ARG, "NULL"), (dict(grad=0), B.DOPT_E_ARG, "NULL"),
    (dict(ckpt=P + 4), B.DOPT_E_ALIGN, "16-byte"), (dict(grad=P + 2), B.DOPT_E_ALIGN, "aligned"),
    (dict(starts=(0, 767)), B.DOPT_E_ARG, "overlap"), (dict(starts=(768, 1)), B.DOPT_E_ARG, "overlap"),
    (dict(starts=(-1, 768)), B.DOPT_E_ARG, "leave"), (dict(starts=(0, 1233)), B.DOPT_E_ARG, "leave"),
    (dict(numel=700), B.DOPT_E_ARG, "leave"), (dict(ws_bytes=16), B.DOPT_E_ARG, "workspace"),
    (dict(ws=P + 8, ws_bytes=16), B.DOPT_E_ALIGN, "workspace")])
def test_wgrad_refusals(lib, change, code, text):
    a = dict(ckpt=P, ckpt_dtype=B.DOPT_BF16, x_rows=10, cols=32, row_token=P, dy=P, dy_dtype=B.DOPT_BF16, dy_rows=20,
             outs=24, dy_ld=24, offsets=P, groups=2, starts=(0, 768), grad=P, grad_dtype=B.DOPT_FP32, numel=2000,
             flags=0, ws=None, ws_bytes=0)
    a.update(change)
    a["starts"] = (ctypes.c_int64 * 300)(*a["starts"])
    _refused(lib, lib.dopt_ckpt_wgrad(*a.values(), None), code, text)


def test_binding_refuses_what_pointers_cannot_carry(lib):
    x = torch.zeros(4, 8)
    slot_row = torch.zeros(4, 2, dtype=torch.int32)
    c = LO.Checkpoint(torch.zeros(dopt.ckpt_bytes(4, 8), dtype=torch.uint8), 4, 8, torch.float32)
    for call in (lambda: dopt.dopt_route_sort(torch.zeros(4, 2, dtype=torch.int64), 3, slot_row, slot_row, slot_row, x),
                 lambda: dopt.dopt_route_dispatch(x, slot_row, x), lambda: dopt.dopt_route_combine(x, slot_row, None, x),
                 lambda: dopt.dopt_route_combine_grad(x, x, slot_row, x, x, x), lambda: dopt.dopt_ckpt_save(x, c),
                 lambda: dopt.dopt_ckpt_load(c, x), lambda: dopt.dopt_ckpt_act_grad(c, "silu", x, x),
                 lambda: dopt.dopt_ckpt_wgrad(c, x, x, [0])):
        with pytest.raises(dopt.DoptError, match="CUDA tensors are needed"):
            call()
    with pytest.raises(dopt.DoptError, match="dtype"):
        dopt.checkpoint(4, 8, torch.float64, device="cpu")


def test_package_exports_the_layer_operators():
    for name in dir(LO):
        if name.startswith("DOPT_") or name.startswith("dopt_"):
            assert hasattr(dopt, name), name
    for name in ("Checkpoint", "checkpoint", "ckpt_bytes", "route_workspace", "wgrad_workspace"):
        assert getattr(dopt, name) is getattr(LO, name)
