"""Refusals of the operators of a model's ends and residual that come before any
CUDA call (the fake pointers below are never dereferenced), and the sizes the
library reports."""
import ctypes
import os
import re

import pytest
import torch

import zero_distributed_optimizer_gb300 as dopt
from zero_distributed_optimizer_gb300 import binding as B
from zero_distributed_optimizer_gb300 import build as libbuild
from zero_distributed_optimizer_gb300 import model_ops as MO

P = 0x10000  # 16-byte aligned, never read
BF, FP16, FP32 = B.DOPT_BF16, B.DOPT_FP16, B.DOPT_FP32


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.lib()


def _refused(lib, rc, code, text):
    assert rc == code
    assert text in lib.dopt_last_error().decode()


def test_workspaces_are_enough_for_fewer(lib):
    n = ctypes.c_int64()

    def size(f, *a):
        assert f(*a, ctypes.byref(n)) == 0
        return n.value

    for vocab, cols in ((1, 1), (50257, 768), (700, 4096), (200000, 64)):
        sizes = [size(lib.dopt_embed_workspace, t, vocab, cols) for t in (0, 1, 5, 100, 1000, 3000, 10000, 20000, 60000, 200000)]
        assert sizes == sorted(sizes)
    for cols in (1, 515, 16384):
        sizes = [size(lib.dopt_norm_workspace, t, cols) for t in (0, 1, 7, 8, 9, 100, 1000, 1024, 5000)]
        assert sizes == sorted(sizes)
    for aligned in (0, 1):
        sizes = [size(lib.dopt_head_loss_workspace, t, 768, 50257, aligned) for t in (0, 1, 100, 256, 257, 5000)]
        assert sizes == sorted(sizes)
        # more pieces take less
        sizes = [size(lib.dopt_head_loss_grad_workspace, 4096, 768, 50257, BF, p, aligned) for p in (2, 3, 5, 50, 197, 1000)]
        assert sizes == sorted(sizes, reverse=True)
        assert size(lib.dopt_head_loss_grad_workspace, 4096, 768, 50257, FP32, 1, aligned) > size(
            lib.dopt_head_loss_grad_workspace, 4096, 768, 50257, BF, 1, aligned)


@pytest.mark.parametrize("call,args", [
    ("dopt_embed_workspace", (-1, 5, 8)), ("dopt_embed_workspace", (5, 0, 8)), ("dopt_embed_workspace", (5, 5, 0)),
    ("dopt_embed_workspace", (2 ** 31 - 2 ** 16 + 1, 5, 8)), ("dopt_norm_workspace", (5, 0)), ("dopt_norm_workspace", (5, 16385)),
    ("dopt_norm_workspace", (-1, 5)), ("dopt_head_loss_workspace", (5, 8, 0, 1)),
    ("dopt_head_loss_workspace", (2 ** 24 + 1, 8, 5, 1)), ("dopt_head_loss_workspace", (5, 0, 5, 1)),
    ("dopt_head_loss_grad_workspace", (5, 8, 5, BF, 0, 1)), ("dopt_head_loss_grad_workspace", (5, 8, 5, 7, 1, 1)),
    ("dopt_head_loss_grad_workspace", (5, 8, 2 ** 24 + 1, BF, 1, 1))], ids=str)
def test_workspace_refusals(lib, call, args):
    n = ctypes.c_int64()
    _refused(lib, getattr(lib, call)(*args, ctypes.byref(n)), B.DOPT_E_ARG, call)
    good = {"dopt_embed_workspace": (5, 5, 8), "dopt_norm_workspace": (5, 8), "dopt_head_loss_workspace": (5, 8, 5, 1),
            "dopt_head_loss_grad_workspace": (5, 8, 5, BF, 1, 1)}[call]
    _refused(lib, getattr(lib, call)(*good, None), B.DOPT_E_ARG, "NULL")


@pytest.mark.parametrize("change,code,text", [
    (dict(dtype=7), B.DOPT_E_ARG, "dtype"), (dict(vocab=0), B.DOPT_E_ARG, "vocab"), (dict(cols=0), B.DOPT_E_ARG, "cols"),
    (dict(vocab=2 ** 31), B.DOPT_E_ARG, "vocab"), (dict(ld=31), B.DOPT_E_ARG, "strides"), (dict(ld_out=31), B.DOPT_E_ARG, "strides"),
    (dict(ids=0), B.DOPT_E_ARG, "ids"), (dict(ids=P + 4), B.DOPT_E_ALIGN, "ids"), (dict(id_bytes=2), B.DOPT_E_ARG, "id_bytes"),
    (dict(tokens=-1), B.DOPT_E_ARG, "tokens"), (dict(table=0), B.DOPT_E_ARG, "NULL"), (dict(out=0), B.DOPT_E_ARG, "NULL"),
    (dict(table=P + 1), B.DOPT_E_ALIGN, "table"), (dict(out=P + 1), B.DOPT_E_ALIGN, "out"), (dict(flags=2), B.DOPT_E_ARG, "flags")], ids=str)
def test_embed_refusals(lib, change, code, text):
    a = dict(table=P, dtype=BF, vocab=10, cols=32, ld=32, ids=P, id_bytes=8, tokens=4, scale=1.0, out=P, ld_out=32, flags=0)
    a.update(change)
    _refused(lib, lib.dopt_embed(*a.values(), None), code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(ids=0), B.DOPT_E_ARG, "ids"), (dict(id_bytes=1), B.DOPT_E_ARG, "id_bytes"), (dict(d_out=0), B.DOPT_E_ARG, "NULL"),
    (dict(dtype=3), B.DOPT_E_ARG, "dtype"), (dict(grad_dtype=3), B.DOPT_E_ARG, "dtype"), (dict(ld=31), B.DOPT_E_ARG, "stride"),
    (dict(grad=0), B.DOPT_E_ARG, "NULL"), (dict(offset=-1), B.DOPT_E_ARG, "leave"), (dict(offset=181), B.DOPT_E_ARG, "leave"),
    (dict(numel=319), B.DOPT_E_ARG, "leave"), (dict(flags=4), B.DOPT_E_ARG, "flags"), (dict(ws=0), B.DOPT_E_ARG, "workspace"),
    (dict(ws_bytes=100), B.DOPT_E_ARG, "workspace of 100 bytes"), (dict(ws=P + 8), B.DOPT_E_ALIGN, "workspace"),
    (dict(grad=P + 2), B.DOPT_E_ALIGN, "grad"), (dict(d_out=P + 1), B.DOPT_E_ALIGN, "d_out"),
    (dict(tokens=2 ** 31 - 2 ** 16 + 1), B.DOPT_E_ARG, "tokens")], ids=str)
def test_embed_grad_refusals(lib, change, code, text):
    a = dict(ids=P, id_bytes=4, tokens=4, d_out=P, dtype=BF, cols=32, ld=32, vocab=10, scale=1.0, grad=P, grad_dtype=FP32,
             numel=500, offset=180, flags=0, ws=P, ws_bytes=1 << 20)
    a.update(change)
    _refused(lib, lib.dopt_embed_grad(*a.values(), None), code, text)


def _norm(kind=MO.DOPT_NORM_LAYER, post=1, eps=1e-5, params=(P,) * 6):
    cfg = MO._NormCfg(kind, post, eps, 1.0)
    six = MO._SixPointers(*params)
    return ctypes.byref(cfg), six


NORM_BOTH = [
    (dict(kind=2), B.DOPT_E_ARG, "kind"), (dict(post=2), B.DOPT_E_ARG, "post 2"), (dict(eps=-1.0), B.DOPT_E_ARG, "eps"),
    (dict(eps=float("nan")), B.DOPT_E_ARG, "eps"), (dict(kind=0), B.DOPT_E_ARG, "bias"), (dict(post=0), B.DOPT_E_ARG, "without post"),
    (dict(y=0), B.DOPT_E_ARG, "without y"), (dict(dtype=9), B.DOPT_E_ARG, "dtype"), (dict(cols=0), B.DOPT_E_ARG, "columns"),
    (dict(cols=16385, ld=16385), B.DOPT_E_ARG, "columns"), (dict(rows=-1), B.DOPT_E_ARG, "rows"),
    (dict(ld=31), B.DOPT_E_ARG, "stride"), (dict(params=(P + 1,) + (P,) * 5), B.DOPT_E_ALIGN, "param"),
    (dict(params=(P,) * 5 + (P + 2,)), B.DOPT_E_ALIGN, "row_gate"), (dict(y=P + 1), B.DOPT_E_ALIGN, "y is not")]


@pytest.mark.parametrize("change,code,text", NORM_BOTH + [
    (dict(x=0), B.DOPT_E_ARG, "x is NULL"), (dict(h=0, n=0), B.DOPT_E_ARG, "neither"),
    (dict(x=P + 1), B.DOPT_E_ALIGN, "x is not"), (dict(n=P + 1), B.DOPT_E_ALIGN, "n is not"),
    (dict(y=0, post=0, params=(P, P, 0, 0, 0, 0)), B.DOPT_E_ARG, "h without y")], ids=str)
def test_norm_refusals(lib, change, code, text):
    a = dict(dtype=BF, rows=4, cols=32, ld=32, x=P, y=P, h=P, n=P)
    cfg = {k: v for k, v in change.items() if k in ("kind", "post", "eps", "params")}
    a.update({k: v for k, v in change.items() if k not in cfg})
    ld = a["ld"]
    _refused(lib, lib.dopt_norm(*_norm(**cfg), a["dtype"], a["rows"], a["cols"], a["x"], ld, a["y"], ld, a["h"], ld, a["n"], ld,
                                None), code, text)


@pytest.mark.parametrize("change,code,text", NORM_BOTH + [
    (dict(h=0), B.DOPT_E_ARG, "without h"), (dict(d_n=0, d_h=0), B.DOPT_E_ARG, "neither"),
    (dict(grad=0), B.DOPT_E_ARG, "NULL grad"), (dict(grad_dtype=5), B.DOPT_E_ARG, "dtype"), (dict(flags=2), B.DOPT_E_ARG, "flags"),
    (dict(at=(0, 40, 80, 120, 31)), B.DOPT_E_ARG, "overlap"), (dict(at=(0, 40, 80, 120, 170)), B.DOPT_E_ARG, "leave"),
    (dict(at=(-2, 40, 80, 120, 160)), B.DOPT_E_ARG, "leave"), (dict(d_n=0), B.DOPT_E_ARG, "takes no part"),
    (dict(ws=0), B.DOPT_E_ARG, "workspace"), (dict(ws_bytes=64), B.DOPT_E_ARG, "workspace of 64"),
    (dict(ws=P + 4), B.DOPT_E_ALIGN, "workspace"), (dict(grad=P + 2), B.DOPT_E_ALIGN, "grad"),
    (dict(row=P + 2), B.DOPT_E_ALIGN, "d_row_gate"), (dict(params=(P,) * 5 + (0,)), B.DOPT_E_ARG, "without row_gate"),
    (dict(d_x=P + 1), B.DOPT_E_ALIGN, "d_x"), (dict(d_y=P + 1), B.DOPT_E_ALIGN, "d_y"),
    (dict(kind=0, params=(P, 0, P, 0, P, P), at=(-1, 0, -1, -1, -1)), B.DOPT_E_ARG, "takes no part"),
    (dict(post=0, params=(P, P, 0, 0, P, P), at=(-1, -1, 0, -1, -1)), B.DOPT_E_ARG, "takes no part")], ids=str)
def test_norm_grad_refusals(lib, change, code, text):
    a = dict(dtype=BF, rows=4, cols=32, ld=32, h=P, y=P, d_n=P, d_h=P, d_x=P, d_y=P, row=P, grad=P, grad_dtype=FP32, numel=200,
             at=(0, 40, 80, 120, 160), flags=0, ws=P, ws_bytes=1 << 20)
    cfg = {k: v for k, v in change.items() if k in ("kind", "post", "eps", "params")}
    a.update({k: v for k, v in change.items() if k not in cfg})
    ld = a["ld"]
    rows = [v for k in ("h", "y", "d_n", "d_h", "d_x", "d_y") for v in (a[k], ld)]
    _refused(lib, lib.dopt_norm_grad(*_norm(**cfg), a["dtype"], a["rows"], a["cols"], *rows, a["row"], a["grad"],
                                     a["grad_dtype"], a["numel"], (ctypes.c_int64 * 5)(*a["at"]), a["flags"], a["ws"],
                                     a["ws_bytes"], None), code, text)


HEAD_BOTH = [
    (dict(dtype=FP32), B.DOPT_E_ARG, "bf16 or fp16"), (dict(rows=-1), B.DOPT_E_ARG, "rows"), (dict(vocab=0), B.DOPT_E_ARG, "vocab"),
    (dict(rows=2 ** 24 + 1), B.DOPT_E_ARG, "rows"), (dict(vocab=2 ** 24 + 1), B.DOPT_E_ARG, "vocab"), (dict(width=0), B.DOPT_E_ARG, "width"),
    (dict(ld_x=63), B.DOPT_E_ARG, "strides"), (dict(ld_w=63), B.DOPT_E_ARG, "strides"), (dict(x=0), B.DOPT_E_ARG, "NULL"),
    (dict(weight=0), B.DOPT_E_ARG, "NULL"), (dict(targets=0), B.DOPT_E_ARG, "NULL"), (dict(target_bytes=1), B.DOPT_E_ARG, "target_bytes"),
    (dict(x=P + 1), B.DOPT_E_ALIGN, "x, weight"), (dict(targets=P + 4), B.DOPT_E_ALIGN, "targets"),
    (dict(ws=0), B.DOPT_E_ARG, "workspace"), (dict(ws_bytes=1000), B.DOPT_E_ARG, "workspace of 1000 bytes"),
    (dict(ws=P + 8), B.DOPT_E_ALIGN, "workspace"), (dict(lse=P + 2), B.DOPT_E_ALIGN, "lse"), (dict(lse=0), B.DOPT_E_ARG, "NULL")]
HEAD = dict(x=P, dtype=BF, rows=40, width=64, ld_x=64, weight=P, vocab=300, ld_w=64, targets=P, target_bytes=8)


@pytest.mark.parametrize("change,code,text", HEAD_BOTH + [(dict(loss=0), B.DOPT_E_ARG, "NULL loss"),
                                                          (dict(loss=P + 2), B.DOPT_E_ALIGN, "loss")], ids=str)
def test_head_loss_refusals(lib, change, code, text):
    a = dict(HEAD, loss=P, lse=P, ws=P, ws_bytes=1 << 30)
    a.update(change)
    _refused(lib, lib.dopt_head_loss(*a.values(), None), code, text)


@pytest.mark.parametrize("change,code,text", HEAD_BOTH + [
    (dict(d_loss=0), B.DOPT_E_ARG, "NULL"), (dict(d_lse=P + 2), B.DOPT_E_ALIGN, "d_lse"), (dict(d_x=0, grad=0), B.DOPT_E_ARG, "neither"),
    (dict(ld_d_x=63), B.DOPT_E_ARG, "d_x"), (dict(d_x=P + 1), B.DOPT_E_ALIGN, "d_x"), (dict(grad_dtype=4), B.DOPT_E_ARG, "dtype"),
    (dict(grad=P + 2), B.DOPT_E_ALIGN, "grad"), (dict(offset=-1), B.DOPT_E_ARG, "leave"), (dict(offset=801), B.DOPT_E_ARG, "leave"),
    (dict(flags=2), B.DOPT_E_ARG, "flags")], ids=str)
def test_head_loss_grad_refusals(lib, change, code, text):
    a = dict(HEAD, lse=P, d_loss=P, d_lse=P, d_x=P, ld_d_x=64, grad=P, grad_dtype=FP32, numel=20000, offset=800, flags=0, ws=P,
             ws_bytes=1 << 30)
    a.update(change)
    _refused(lib, lib.dopt_head_loss_grad(*a.values(), None), code, text)


def test_head_wait_test_is_of_the_test_build(lib):
    assert lib.dopt_head_wait_test(0) == B.DOPT_E_STATE
    assert lib.dopt_head_timeouts(0, None) == B.DOPT_E_ARG


def test_binding_refuses_what_pointers_cannot_carry(lib):
    x, v = torch.zeros(4, 8), torch.zeros(4)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: dopt.dopt_embed(x, ids, x), lambda: dopt.dopt_embed_grad(ids, x, v, 0, 2), lambda: dopt.dopt_norm("rms", x, x),
                 lambda: dopt.dopt_norm_grad("rms", x, x, x), lambda: dopt.dopt_head_loss(x, x, ids, v, v),
                 lambda: dopt.dopt_head_loss_grad(x, x, ids, v, v, x, v)):
        with pytest.raises(dopt.DoptError, match="CUDA tensors are needed"):
            call()
    with pytest.raises(dopt.DoptError, match="unknown norm"):
        MO._norm_cfg("batch", 0, 1e-5, 1.0)
    with pytest.raises(dopt.DoptError, match="no such params: scale"):
        MO._norm_offsets((("weight", 0), ("scale", 8)))
    with pytest.raises(dopt.DoptError, match="dtype"):
        dopt.head_loss_grad_workspace(4, 8, 8, torch.int32, device="cpu")


def test_package_exports_the_model_operators():
    for name in dir(MO):
        if name.startswith("DOPT_") or name.startswith("dopt_"):
            assert hasattr(dopt, name), name
    for name in ("embed_workspace", "norm_workspace", "head_loss_workspace", "head_loss_grad_workspace", "head_timeouts"):
        assert getattr(dopt, name) is getattr(MO, name)
        assert name in dir(dopt)


def _source(name):
    with open(os.path.join(libbuild.CSRC, name)) as f:
        return re.sub(r'(\\n\\t)?"\s*\n?\s*"', "", f.read())


def test_the_pairs_barriers_are_ordered_at_the_clusters_scope():
    """Both CTAs of a pair arrive on the leader's barriers: every wait acquires and every arrival on another CTA's
    barrier releases at that scope (read on the CPU: a weaker one would be a race, which no run has to show)."""
    text = _source("head.cu")
    waits = re.findall(r"mbarrier\.(?:try|test)_wait[\w.:]*", text)
    arrivals = re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text)
    assert waits and all(".acquire.cluster." in w for w in waits), waits
    assert arrivals and all(".release.cluster." in a for a in arrivals), arrivals
