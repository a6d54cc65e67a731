"""Python binding of the layer operators in include/dopt.h: tokens sorted by
expert and back (``dopt_route_*``) and activations kept in 8 bits for the
backward pass (``dopt_ckpt_*``).

As in :mod:`.binding`, every function checks what raw pointers cannot carry
(device, dtype, shape, strides), passes pointers and sizes to libdopt.so, and
is asynchronous on `stream` (default: torch's current stream).  Outputs and
workspaces are the caller's.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from .binding import (DOPT_BF16, DOPT_E_ARG, DOPT_FP16, DOPT_FP32, DoptError, _check, _on,
                      _stream_handle, lib)

DOPT_MAX_EXPERTS = 1024
DOPT_MAX_TOPK = 64
DOPT_MAX_GROUPS = 256
DOPT_MAX_COLS = 4194304
DOPT_CKPT_BLOCK = 32
DOPT_CKPT_PITCH = 128
DOPT_ACT_SILU = 0
DOPT_ACT_GELU = 1
DOPT_ACT_SWIGLU = 2
DOPT_WGRAD_ACCUMULATE = 1
DOPT_WGRAD_MAX_ROWS = 2147483584

# torch's query of a device's current stream, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

_CODES = {torch.bfloat16: DOPT_BF16, torch.float32: DOPT_FP32, torch.float16: DOPT_FP16}
_ACTS = {"silu": DOPT_ACT_SILU, "gelu": DOPT_ACT_GELU, "swiglu": DOPT_ACT_SWIGLU}


def _bad(message: str):
    return DoptError(DOPT_E_ARG, message)


def _dtype_code(dtype, name: str) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise _bad(f"{name} has dtype {dtype}, expected bf16, fp16 or fp32")
    return code


def _cuda_index(t, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise _bad(f"{name} is on {t.device}: CUDA tensors are needed (no CPU path exists)")
    return index


def _dense(t, name: str, dtype, shape, index: int) -> int:
    """The address of a contiguous tensor of this type, shape and device."""
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != index
            or not t.is_contiguous()):
        raise _bad(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, "
                   f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t, name: str, dtype, shape, index: int):
    """(address, row stride) of a 2-D tensor whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        raise _bad(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{index}, "
                   f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    s0, s1 = t.stride()
    if (s1 != 1 and shape[1] > 1) or (s0 < shape[1] and shape[0] > 1):
        raise _bad(f"{name} must have contiguous rows, got strides {(s0, s1)}")
    return t.data_ptr(), s0 if shape[0] > 1 else shape[1]


def _call(index: int, stream, function, *args):
    """function(*args, stream handle) with the tensors' device current."""
    if index != torch.cuda.current_device():
        with _on(torch.device("cuda", index)):
            return _check(function(*args, _stream_handle(stream)))
    if stream is None and _raw_stream is not None:
        rc = function(*args, _raw_stream(index))
    else:
        rc = function(*args, _stream_handle(stream))
    if rc:
        _check(rc)


# ---------------------------------------------------------------------------
# Tokens sorted by expert and back
# ---------------------------------------------------------------------------

def route_workspace(tokens: int, k: int, n_experts: int, device=None):
    """A workspace for :func:`dopt_route_sort` of these sizes and of any fewer
    tokens (a uint8 tensor)."""
    n = ctypes.c_int64()
    _check(lib().dopt_route_workspace(int(tokens), int(k), int(n_experts), ctypes.byref(n)))
    return torch.empty(max(n.value, 16), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def dopt_route_sort(expert_ids, n_experts: int, slot_row, row_token, offsets, workspace,
                    stream=None) -> None:
    """Sort a router's choices by expert (stable).

    expert_ids: [tokens, k] int32 or int64, contiguous; ids outside
    [0, n_experts) are dropped.  Written, all int32: slot_row [tokens, k] (the
    slot's row, -1 if dropped), row_token [tokens * k] (the row's token, -1
    past the last row), offsets [n_experts + 1] (each expert's first row, then
    the number of rows).  workspace: from :func:`route_workspace`.
    """
    index = _cuda_index(expert_ids, "expert_ids")
    if expert_ids.dim() != 2 or not expert_ids.is_contiguous():
        raise _bad("expert_ids must be a contiguous [tokens, k] tensor")
    tokens, k = expert_ids.shape
    wide = expert_ids.dtype is torch.int64
    if not wide and expert_ids.dtype is not torch.int32:
        raise _bad(f"expert_ids has dtype {expert_ids.dtype}, expected int32 or int64")
    if workspace.get_device() != index or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise _bad(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    i32 = torch.int32
    _call(index, stream, lib().dopt_route_sort, expert_ids.data_ptr(), 8 if wide else 4, tokens, k,
          n_experts, _dense(slot_row, "slot_row", i32, (tokens, k), index),
          _dense(row_token, "row_token", i32, (tokens * k,), index),
          _dense(offsets, "offsets", i32, (n_experts + 1,), index),
          workspace.data_ptr(), workspace.numel())


def _check_slot_row(slot_row, index: int):
    if slot_row.dim() != 2:
        raise _bad("slot_row must be [tokens, k]")
    tokens, k = slot_row.shape
    return _dense(slot_row, "slot_row", torch.int32, (tokens, k), index), tokens, k


def dopt_route_dispatch(x, slot_row, rows, stream=None) -> None:
    """rows[slot_row[t, j]] = x[t]: each token's row to its slots' rows.

    x: [tokens, cols] with contiguous rows; rows: [n_rows, cols], contiguous,
    of x's type; rows that no slot names are not written.
    """
    index = _cuda_index(x, "x")
    sr, tokens, k = _check_slot_row(slot_row, index)
    if rows.dim() != 2:
        raise _bad("rows must be [n_rows, cols]")
    n_rows, cols = rows.shape
    xp, ld = _rows(x, "x", rows.dtype, (tokens, cols), index)
    _call(index, stream, lib().dopt_route_dispatch, xp, _dtype_code(x.dtype, "x"), tokens, cols, ld, sr, k,
          _dense(rows, "rows", x.dtype, (n_rows, cols), index), n_rows)


def dopt_route_combine(rows, slot_row, weights, out, stream=None) -> None:
    """out[t] = sum over j of weights[t, j] * rows[slot_row[t, j]] (fp32 sums).

    rows: [n_rows, cols], contiguous; weights: fp32 [tokens, k], or None for
    ones (the gradient of :func:`dopt_route_dispatch`); out: [tokens, cols]
    with contiguous rows, of the rows' type.
    """
    index = _cuda_index(rows, "rows")
    sr, tokens, k = _check_slot_row(slot_row, index)
    if rows.dim() != 2:
        raise _bad("rows must be [n_rows, cols]")
    n_rows, cols = rows.shape
    op, ld = _rows(out, "out", rows.dtype, (tokens, cols), index)
    wp = None if weights is None else _dense(weights, "weights", torch.float32, (tokens, k), index)
    _call(index, stream, lib().dopt_route_combine, _dense(rows, "rows", rows.dtype, (n_rows, cols), index),
          _dtype_code(rows.dtype, "rows"), n_rows, sr, wp, tokens, k, cols, op, ld)


def dopt_route_combine_grad(d_out, rows, slot_row, weights, d_rows, d_weights, stream=None) -> None:
    """Gradients of :func:`dopt_route_combine` with weights: d_rows[r] =
    weights[t, j] * d_out[t] and d_weights[t, j] = <d_out[t], rows[r]>, with
    r = slot_row[t, j] (d_weights is 0 where it is dropped)."""
    index = _cuda_index(rows, "rows")
    sr, tokens, k = _check_slot_row(slot_row, index)
    if rows.dim() != 2:
        raise _bad("rows must be [n_rows, cols]")
    n_rows, cols = rows.shape
    dt, f32 = rows.dtype, torch.float32
    dp, ld = _rows(d_out, "d_out", dt, (tokens, cols), index)
    _call(index, stream, lib().dopt_route_combine_grad, dp, ld, _dense(rows, "rows", dt, (n_rows, cols), index),
          _dtype_code(dt, "rows"), n_rows, sr, _dense(weights, "weights", f32, (tokens, k), index),
          tokens, k, cols, _dense(d_rows, "d_rows", dt, (n_rows, cols), index),
          _dense(d_weights, "d_weights", f32, (tokens, k), index))


# ---------------------------------------------------------------------------
# Activations kept in 8 bits
# ---------------------------------------------------------------------------

class Checkpoint(NamedTuple):
    """An activation kept in 8 bits: `data` (uint8, dopt_ckpt_bytes long, CUDA)
    holds rows x cols values that were of type `dtype`; dopt.h states the format."""

    data: torch.Tensor
    rows: int
    cols: int
    dtype: torch.dtype


def ckpt_bytes(rows: int, cols: int) -> int:
    """Bytes of a checkpoint of rows x cols values."""
    n = ctypes.c_int64()
    _check(lib().dopt_ckpt_bytes(int(rows), int(cols), ctypes.byref(n)))
    return n.value


def checkpoint(rows: int, cols: int, dtype=torch.bfloat16, device=None) -> Checkpoint:
    """A new, unwritten checkpoint for rows x cols values of `dtype`."""
    _dtype_code(dtype, "checkpoint")
    return Checkpoint(torch.empty(ckpt_bytes(rows, cols), dtype=torch.uint8,
                                  device="cuda" if device is None else device),
                      int(rows), int(cols), dtype)


def _check_ckpt(ckpt: Checkpoint):
    """(address, device index) of a checkpoint's buffer."""
    data = ckpt.data
    index = _cuda_index(data, "checkpoint")
    pitch = -(-ckpt.cols // DOPT_CKPT_PITCH) * DOPT_CKPT_PITCH
    need = ckpt.rows * (pitch + pitch // DOPT_CKPT_BLOCK)
    if data.dtype is not torch.uint8 or not data.is_contiguous() or data.numel() < need:
        raise _bad(f"a checkpoint of {ckpt.rows} x {ckpt.cols} values needs a contiguous uint8 tensor "
                   f"of {need} bytes")
    return data.data_ptr(), index


def dopt_ckpt_save(x, ckpt: Checkpoint, stream=None) -> None:
    """Keep x ([rows, cols], contiguous rows, of the checkpoint's type) in `ckpt`."""
    cp, index = _check_ckpt(ckpt)
    xp, ld = _rows(x, "x", ckpt.dtype, (ckpt.rows, ckpt.cols), index)
    _call(index, stream, lib().dopt_ckpt_save, xp, _dtype_code(x.dtype, "x"), ckpt.rows, ckpt.cols, ld, cp)


def dopt_ckpt_load(ckpt: Checkpoint, out, row_index=None, stream=None) -> None:
    """Read `ckpt` back into out ([rows, cols], contiguous rows, any of the
    three types).  row_index: int32 [n], out is then [n, cols] and gets row
    row_index[i] (zeros where there is no such row)."""
    cp, index = _check_ckpt(ckpt)
    n = ckpt.rows
    ip = None
    if row_index is not None:
        n = row_index.numel()
        ip = _dense(row_index, "row_index", torch.int32, (n,), index)
    op, ld = _rows(out, "out", out.dtype, (n, ckpt.cols), index)
    _call(index, stream, lib().dopt_ckpt_load, cp, ckpt.rows, ckpt.cols, ip, n, op,
          _dtype_code(out.dtype, "out"), ld)


def dopt_ckpt_act_grad(ckpt: Checkpoint, act: str, d_out, d_in, stream=None) -> None:
    """d_in = d_out * act'(h) from the kept input h: act "silu", "gelu" (tanh
    form) or "swiglu" (h = [gate, up] halves; d_out has half the columns).
    For silu and gelu d_in may be d_out."""
    cp, index = _check_ckpt(ckpt)
    code = _ACTS.get(act)
    if code is None:
        raise _bad(f"unknown activation {act!r}: one of {', '.join(_ACTS)}")
    width = ckpt.cols // 2 if code == DOPT_ACT_SWIGLU else ckpt.cols
    dp, ld = _rows(d_out, "d_out", d_out.dtype, (ckpt.rows, width), index)
    ip, ld_in = _rows(d_in, "d_in", d_out.dtype, (ckpt.rows, ckpt.cols), index)
    _call(index, stream, lib().dopt_ckpt_act_grad, cp, ckpt.rows, ckpt.cols, code, dp, ld,
          _dtype_code(d_out.dtype, "d_out"), ip, ld_in)


@functools.lru_cache(maxsize=256)
def _starts(grad_offsets: tuple):
    """The C array of these offsets (kept by value: the library only reads it)."""
    return (ctypes.c_int64 * max(len(grad_offsets), 1))(*grad_offsets)


def wgrad_workspace(dy_rows: int, outs: int, cols: int, n_groups: int = 1, device=None):
    """A workspace for :func:`dopt_ckpt_wgrad` of these sizes and a contiguous dy
    (a uint8 tensor).  A view of dy whose rows are not 16-byte aligned though
    outs is a multiple of 8 is read element by element, three times slower,
    unless the workspace has 2 * dy_rows * outs bytes more."""
    n = ctypes.c_int64()
    _check(lib().dopt_ckpt_wgrad_workspace(int(dy_rows), int(outs), int(cols), int(n_groups),
                                           ctypes.byref(n)))
    return torch.empty(max(n.value, 16), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def dopt_ckpt_wgrad(ckpt: Checkpoint, dy, grad, grad_offsets, offsets=None, row_token=None,
                    accumulate: bool = False, workspace=None, stream=None) -> None:
    """Weight gradients dW[o, c] = sum over rows r of dy[r, o] * x[r, c] from
    the kept input x, written into the flat grad buffer.

    dy: [dy_rows, outs] with contiguous rows, bf16 (or fp16 with a checkpoint
    of fp16 values); grad: a 1-D contiguous bf16, fp16 or fp32 tensor, e.g. a
    grad replica of :func:`dopt_step`; grad_offsets: one start per group
    (``layout.param_offsets()[i][0]``).  offsets: int32 [groups + 1], each
    group's first row of dy and the end (None: one group of all rows).
    row_token: int32 [dy_rows], the row of x that goes with each row of dy
    (None: the same row).  accumulate: add to the grads that are there.
    workspace: from :func:`wgrad_workspace`, optional.
    """
    cp, index = _check_ckpt(ckpt)
    if dy.dim() != 2 or grad.dim() != 1:
        raise _bad("dy must be [rows, outs] and grad one-dimensional")
    dy_rows, outs = dy.shape
    dp, ld = _rows(dy, "dy", dy.dtype, (dy_rows, outs), index)
    n_groups = len(grad_offsets)
    numel = grad.numel()
    gp = _dense(grad, "grad", grad.dtype, (numel,), index)
    op = None if offsets is None else _dense(offsets, "offsets", torch.int32, (n_groups + 1,), index)
    rp = None if row_token is None else _dense(row_token, "row_token", torch.int32, (dy_rows,), index)
    wp, wn = None, 0
    if workspace is not None:
        if workspace.get_device() != index or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
            raise _bad(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
        wp, wn = workspace.data_ptr(), workspace.numel()
    starts = _starts(tuple(grad_offsets))
    _call(index, stream, lib().dopt_ckpt_wgrad, cp, _dtype_code(ckpt.dtype, "checkpoint"), ckpt.rows, ckpt.cols,
          rp, dp, _dtype_code(dy.dtype, "dy"), dy_rows, outs, ld, op, n_groups, starts, gp,
          _dtype_code(grad.dtype, "grad"), numel, DOPT_WGRAD_ACCUMULATE if accumulate else 0, wp, wn)


class WgradPlan(NamedTuple):
    """How a weight gradient divides its work (dopt_ckpt_wgrad_plan in dopt.h)."""

    blocks: int  # of 256 outputs, in a tile
    whole: int   # tiles
    split: int   # tiles whose rows are split
    parts: int   # into so many


def wgrad_plan(dy_rows: int, outs: int, cols: int, n_groups: int, dy_dtype, grad_dtype,
               workspace_bytes: int) -> WgradPlan:
    """The plan of such a :func:`dopt_ckpt_wgrad` on a device of 152 SMs."""
    p = (ctypes.c_int64 * 4)()
    _check(lib().dopt_ckpt_wgrad_plan(int(dy_rows), int(outs), int(cols), int(n_groups), _dtype_code(dy_dtype, "dy"),
                                      _dtype_code(grad_dtype, "grad"), int(workspace_bytes), p))
    return WgradPlan(*p)


def wgrad_timeouts(reset: bool = False) -> int:
    """Blocks of :func:`dopt_ckpt_wgrad` on the current device whose waits ran
    out of time (0 unless a copy or product failed to complete; the grads they
    did not write are then NaN); reset clears it."""
    c = ctypes.c_uint32(0)
    _check(lib().dopt_wgrad_timeouts(1 if reset else 0, ctypes.byref(c)))
    return c.value


def wgrad_wait_test(items: int) -> None:
    """Test build only (dopt_wgrad_wait_test in dopt.h): the first pair of blocks
    of later weight gradients stops after `items` of its items, so that its
    waits run out; -1 restores normal work.  Raises DoptError with DOPT_E_STATE
    in the product build."""
    _check(lib().dopt_wgrad_wait_test(int(items)))
