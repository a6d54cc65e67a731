"""Python binding of the operators of a language model's two ends and of its
residual stream in include/dopt.h: the token embedding (``dopt_embed*``), the
norms around a block (``dopt_norm*``) and the loss of the output matrix's logits
(``dopt_head_loss*``).

As in :mod:`.layer_ops`, every function checks what raw pointers cannot carry
(device, dtype, shape, strides), passes pointers and sizes to libdopt.so, and is
asynchronous on `stream` (default: torch's current stream).  Outputs and
workspaces are the caller's; params' gradients go to offsets of a flat grad
buffer.
"""
from __future__ import annotations

import ctypes
import functools
from operator import index as index_of

import torch

from .binding import _check, lib
from .layer_ops import _bad, _call, _cuda_index, _dense, _dtype_code, _rows

DOPT_EMBED_ACCUMULATE = 1
DOPT_EMBED_MAX_TOKENS = 2147418112
DOPT_NORM_RMS = 0
DOPT_NORM_LAYER = 1
DOPT_NORM_MAX_COLS = 16384
DOPT_NORM_ACCUMULATE = 1
DOPT_HEAD_MAX_ROWS = 16777216
DOPT_HEAD_MAX_VOCAB = 16777216
DOPT_HEAD_ACCUMULATE = 1

_KINDS = {"rms": DOPT_NORM_RMS, "layer": DOPT_NORM_LAYER}
_NORM_PARAMS = ("weight", "bias", "post_weight", "post_bias", "gate")


def _bytes(n: int, device):
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda" if device is None else device)


def _workspace(workspace, index: int):
    """(address, bytes) of a workspace."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != index or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise _bad(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    return workspace.data_ptr(), workspace.numel()


def _numbers(t, name: str, index: int):
    """(address, bytes of an element, count) of contiguous one-dimensional int32 or int64 numbers."""
    if t.dim() != 1 or not t.is_contiguous() or t.get_device() != index:
        raise _bad(f"{name} must be a contiguous one-dimensional tensor on cuda:{index}, got "
                   f"{tuple(t.shape)} on {t.device}")
    wide = t.dtype is torch.int64
    if not wide and t.dtype is not torch.int32:
        raise _bad(f"{name} has dtype {t.dtype}, expected int32 or int64")
    return t.data_ptr(), 8 if wide else 4, t.shape[0]


def _flat(grad, index: int):
    """(address, type code, elements) of a flat grad buffer."""
    if grad.dim() != 1:
        raise _bad("grad must be one-dimensional")
    n = grad.numel()
    return _dense(grad, "grad", grad.dtype, (n,), index), _dtype_code(grad.dtype, "grad"), n


# ---------------------------------------------------------------------------
# Token embedding
# ---------------------------------------------------------------------------

def dopt_embed(table, ids, out, scale: float = 1.0, accumulate: bool = False, stream=None) -> None:
    """out[t] = scale * table[ids[t]]; zeros where ids[t] is outside the table.

    table: [vocab, cols] with contiguous rows; ids: [tokens] int32 or int64;
    out: [tokens, cols] with contiguous rows, of the table's type.  accumulate:
    add to out instead (an id outside then leaves its row as it is).
    """
    index = _cuda_index(table, "table")
    if table.dim() != 2:
        raise _bad("table must be [vocab, cols]")
    vocab, cols = table.shape
    ip, wide, tokens = _numbers(ids, "ids", index)
    tp, ld = _rows(table, "table", table.dtype, (vocab, cols), index)
    op, ld_out = _rows(out, "out", table.dtype, (tokens, cols), index)
    _call(index, stream, lib().dopt_embed, tp, _dtype_code(table.dtype, "table"), vocab, cols, ld, ip, wide, tokens,
          scale, op, ld_out, DOPT_EMBED_ACCUMULATE if accumulate else 0)


def embed_workspace(tokens: int, vocab: int, cols: int, device=None):
    """A workspace for :func:`dopt_embed_grad` of these sizes and of any fewer
    tokens (a uint8 tensor)."""
    n = ctypes.c_int64()
    _check(lib().dopt_embed_workspace(int(tokens), int(vocab), int(cols), ctypes.byref(n)))
    return _bytes(n.value, device)


def dopt_embed_grad(ids, d_out, grad, grad_offset: int, vocab: int, scale: float = 1.0, accumulate: bool = False,
                    workspace=None, stream=None) -> None:
    """The table's gradient, scale times the sum of d_out's rows of each id,
    into grad[grad_offset:grad_offset + vocab * cols].

    ids: [tokens] int32 or int64 (those outside [0, vocab) are left out);
    d_out: [tokens, cols] with contiguous rows; grad: a 1-D contiguous bf16,
    fp16 or fp32 tensor, e.g. a grad replica of :func:`dopt_step`.  accumulate:
    add to the grads that are there.  workspace: from :func:`embed_workspace`.
    """
    index = _cuda_index(d_out, "d_out")
    if d_out.dim() != 2:
        raise _bad("d_out must be [tokens, cols]")
    ip, wide, tokens = _numbers(ids, "ids", index)
    cols = d_out.shape[1]
    dp, ld = _rows(d_out, "d_out", d_out.dtype, (tokens, cols), index)
    gp, code, numel = _flat(grad, index)
    wp, wn = _workspace(workspace, index)
    _call(index, stream, lib().dopt_embed_grad, ip, wide, tokens, dp, _dtype_code(d_out.dtype, "d_out"), cols, ld,
          vocab, scale, gp, code, numel, grad_offset, DOPT_EMBED_ACCUMULATE if accumulate else 0, wp, wn)


# ---------------------------------------------------------------------------
# Norms around a block
# ---------------------------------------------------------------------------

class _NormCfg(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("post", ctypes.c_int32), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float)]


_SixPointers = ctypes.c_void_p * 6  # dopt_norm_params
_FiveOffsets = ctypes.c_int64 * 5


@functools.lru_cache(maxsize=256)
def _norm_cfg(kind, post, eps, scale):
    """The configuration of these values (kept by value, of plain numbers: a tensor
    is the same key whatever it holds; the library only reads it)."""
    code = _KINDS.get(kind)
    if code is None:
        raise _bad(f"unknown norm {kind!r}: one of {', '.join(_KINDS)}")
    return _NormCfg(code, post, eps, scale)


@functools.lru_cache(maxsize=256)
def _norm_offsets(offsets):
    """The places of the params' gradients, -1 for none, from (name, place) pairs."""
    at = dict(offsets)
    found = [at.pop(name, -1) for name in _NORM_PARAMS]
    if at:
        raise _bad(f"no such params: {', '.join(map(str, at))} (of {', '.join(_NORM_PARAMS)})")
    return _FiveOffsets(*found)


def _norm_params(params, row_gate, dtype, shape, index):
    cols, at = shape[1:], []
    for p in params:
        if p is None:
            at.append(None)
        elif p.dtype is dtype and p.shape == cols and p.get_device() == index and p.is_contiguous():
            at.append(p.data_ptr())
        else:
            _dense(p, _NORM_PARAMS[len(at)], dtype, cols, index)  # raises
    at.append(None if row_gate is None else _dense(row_gate, "row_gate", torch.float32, shape[:1], index))
    return _SixPointers(*at)


def _matrices(named, dtype, shape, index):
    """(address, row stride) of each of the matrices, one after another."""
    cols, found = shape[1], []
    for name, t in named:
        if t is None:
            found += (None, cols)
        elif t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
            found += (t.data_ptr(), cols)
        else:
            found += _rows(t, name, dtype, shape, index)
    return found


def _matrix(t, name, dtype, shape, index):
    if t is None:
        return None, shape[1]
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
        return t.data_ptr(), shape[1]
    return _rows(t, name, dtype, shape, index)


def dopt_norm(kind: str, x, n, weight=None, bias=None, y=None, h=None, post: bool = False, post_weight=None,
              post_bias=None, gate=None, row_gate=None, scale: float = 1.0, eps: float = 1e-5, stream=None) -> None:
    """h = x + scale * row_gate * gate * u and n = norm(h), with u the block's
    output y, or with `post` its norm.

    kind: "rms" or "layer".  x, y, h, n: [rows, cols] with contiguous rows, of
    one type; h or n may be None (not wanted), h may be x.  Without y: n =
    norm(x), and h is None.  weight, bias, post_weight, post_bias, gate: [cols] of that type,
    row_gate: fp32 [rows]; None counts as ones (biases: zeros).
    """
    index = _cuda_index(x, "x")
    if x.dim() != 2:
        raise _bad("x must be [rows, cols]")
    dt, shape = x.dtype, x.shape
    _call(index, stream, lib().dopt_norm, ctypes.byref(_norm_cfg(kind, 1 if post else 0, float(eps), float(scale))),
          _norm_params((weight, bias, post_weight, post_bias, gate), row_gate, dt, shape, index), _dtype_code(dt, "x"),
          *shape, *_matrices((("x", x), ("y", y), ("h", h), ("n", n)), dt, shape, index))


def norm_workspace(rows: int, cols: int, device=None):
    """A workspace for :func:`dopt_norm_grad` of these sizes and of any fewer
    rows (a uint8 tensor)."""
    n = ctypes.c_int64()
    _check(lib().dopt_norm_workspace(int(rows), int(cols), ctypes.byref(n)))
    return _bytes(n.value, device)


def dopt_norm_grad(kind: str, h, d_n, d_x, weight=None, y=None, d_y=None, d_h=None, post: bool = False,
                   post_weight=None, post_bias=None, gate=None, row_gate=None, scale: float = 1.0, eps: float = 1e-5,
                   d_row_gate=None, grad=None, grad_offsets=None, accumulate: bool = False, workspace=None,
                   stream=None) -> None:
    """The gradients of :func:`dopt_norm` from h (as it was written; x where
    there was no y), y, and the gradients d_n of n and d_h of h (either may be
    None).

    d_x (may be d_h) and d_y: [rows, cols], or None; d_row_gate: fp32 [rows] or
    None.  grad: a flat grad buffer; grad_offsets: where in it the gradients of
    the params go, a dict of "weight", "bias", "post_weight", "post_bias" and
    "gate" (those that are wanted).  accumulate: add to the grads that are
    there.  workspace: from :func:`norm_workspace`.
    """
    index = _cuda_index(h, "h")
    if h.dim() != 2:
        raise _bad("h must be [rows, cols]")
    dt, shape = h.dtype, h.shape
    at = _norm_offsets(tuple((n, index_of(a)) for n, a in grad_offsets.items()) if grad_offsets else ())
    gp, code, numel = (None, 0, 0) if grad is None else _flat(grad, index)
    wp, wn = _workspace(workspace, index)
    rp = None if d_row_gate is None else _dense(d_row_gate, "d_row_gate", torch.float32, shape[:1], index)
    _call(index, stream, lib().dopt_norm_grad, ctypes.byref(_norm_cfg(kind, 1 if post else 0, float(eps), float(scale))),
          _norm_params((weight, None, post_weight, post_bias, gate), row_gate, dt, shape, index), _dtype_code(dt, "h"),
          *shape, *_matrices((("h", h), ("y", y), ("d_n", d_n), ("d_h", d_h), ("d_x", d_x), ("d_y", d_y)), dt, shape, index),
          rp, gp, code, numel, at,
          DOPT_NORM_ACCUMULATE if accumulate else 0, wp, wn)


# ---------------------------------------------------------------------------
# Loss of the output matrix's logits
# ---------------------------------------------------------------------------

def head_loss_workspace(rows: int, width: int, vocab: int, aligned: bool = True, device=None):
    """A workspace for :func:`dopt_head_loss` of these sizes and of any fewer
    rows (a uint8 tensor).  aligned: the rows of x and weight are 16-byte
    aligned (a width that is not a multiple of 8 counts as False)."""
    n = ctypes.c_int64()
    _check(lib().dopt_head_loss_workspace(int(rows), int(width), int(vocab), 1 if aligned else 0, ctypes.byref(n)))
    return _bytes(n.value, device)


def head_loss_grad_workspace(rows: int, width: int, vocab: int, grad_dtype=torch.bfloat16, pieces: int = 1,
                             aligned: bool = True, device=None):
    """A workspace for :func:`dopt_head_loss_grad` with the vocabulary in
    `pieces` pieces: 1 is the fastest, more take less memory (about 2 * rows *
    vocab / pieces bytes, twice that for fp32 grads)."""
    n = ctypes.c_int64()
    _check(lib().dopt_head_loss_grad_workspace(int(rows), int(width), int(vocab), _dtype_code(grad_dtype, "grad"),
                                               int(pieces), 1 if aligned else 0, ctypes.byref(n)))
    return _bytes(n.value, device)


def _head(x, weight, targets):
    """(device index, the arguments that both directions begin with)."""
    index = _cuda_index(x, "x")
    if x.dim() != 2 or weight.dim() != 2:
        raise _bad("x must be [rows, width] and weight [vocab, width]")
    rows, width = x.shape
    vocab = weight.shape[0]
    xp, ld_x = _rows(x, "x", x.dtype, (rows, width), index)
    wp, ld_w = _rows(weight, "weight", x.dtype, (vocab, width), index)
    tp, wide, n = _numbers(targets, "targets", index)
    if n != rows:
        raise _bad(f"targets must have {rows} elements, got {n}")
    return index, (xp, _dtype_code(x.dtype, "x"), rows, width, ld_x, wp, vocab, ld_w, tp, wide)


def dopt_head_loss(x, weight, targets, loss, lse, workspace=None, stream=None) -> None:
    """lse[t] = log(sum over v of exp(x[t] . weight[v])) and loss[t] = lse[t] -
    x[t] . weight[targets[t]], 0 where the target is outside [0, vocab).  Logits
    masked by values far below the others, down to -inf, add nothing.

    x: [rows, width], weight: [vocab, width], bf16 or fp16 with contiguous rows;
    targets: int32 or int64 [rows]; loss, lse: fp32 [rows].  workspace: from
    :func:`head_loss_workspace`.
    """
    index, args = _head(x, weight, targets)
    rows, f32 = args[2], torch.float32
    wp, wn = _workspace(workspace, index)
    _call(index, stream, lib().dopt_head_loss, *args, _dense(loss, "loss", f32, (rows,), index),
          _dense(lse, "lse", f32, (rows,), index), wp, wn)


def dopt_head_loss_grad(x, weight, targets, lse, d_loss, d_x, grad, grad_offset: int = 0, d_lse=None,
                        accumulate: bool = False, workspace=None, stream=None) -> None:
    """The gradients of :func:`dopt_head_loss` from its lse and the gradients of
    its outputs, d_loss and d_lse (fp32 [rows]; d_lse may be None).

    d_x: [rows, width] of x's type with contiguous rows, or None; grad: a flat
    grad buffer that takes the matrix's gradient at grad_offset, or None.
    accumulate: add to the grads that are there.  workspace: from
    :func:`head_loss_grad_workspace`.  With fp16, where rows' weights (d_loss,
    d_lse) are more than 16 times apart and grad is wanted too, d_x takes a pass
    of its own over the vocabulary.
    """
    index, args = _head(x, weight, targets)
    rows, width, f32 = args[2], args[3], torch.float32
    gp, code, numel = (None, 0, 0) if grad is None else _flat(grad, index)
    wp, wn = _workspace(workspace, index)
    _call(index, stream, lib().dopt_head_loss_grad, *args, _dense(lse, "lse", f32, (rows,), index),
          _dense(d_loss, "d_loss", f32, (rows,), index),
          None if d_lse is None else _dense(d_lse, "d_lse", f32, (rows,), index),
          *_matrix(d_x, "d_x", x.dtype, (rows, width), index), gp, code, numel, grad_offset,
          DOPT_HEAD_ACCUMULATE if accumulate else 0, wp, wn)


def head_timeouts(reset: bool = False) -> int:
    """Blocks of :func:`dopt_head_loss` and its gradient on the current device
    whose waits ran out of time (0 unless a copy or product failed to complete;
    what they did not write is then NaN); reset clears it."""
    c = ctypes.c_uint32(0)
    _check(lib().dopt_head_timeouts(1 if reset else 0, ctypes.byref(c)))
    return c.value


def head_wait_test(items: int) -> None:
    """Test build only (dopt_head_wait_test in dopt.h): the first pair of blocks
    of later launches stops after `items` of its items, so that its waits run
    out; -1 restores normal work.  Raises DoptError with DOPT_E_STATE in the
    product build."""
    _check(lib().dopt_head_wait_test(int(items)))
