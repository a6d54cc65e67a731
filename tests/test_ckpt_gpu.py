"""Activations kept in 8 bits against the format's definition in 64 bits
(equal, not near), and an activation function's backward pass from them."""
import numpy as np
import pytest
import torch

import layer_reference as R
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _values(rows, cols, dtype, kind, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g)
    if kind == "wide":  # magnitudes over the type's whole range, its least values among them
        e = torch.randint(-24, 16, (rows, cols), generator=g) if dtype == torch.float16 else \
            torch.randint(-149, 128, (rows, cols), generator=g)
        x = torch.ldexp(1 + torch.rand(rows, cols, generator=g, dtype=torch.float64), e) * x.sign()
        x = x.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max)
    elif kind == "halves":  # exact ties, the largest values next to a power of two
        x = torch.randint(-255, 256, (rows, cols), generator=g) / 2.0
    elif kind == "zeros":
        x = torch.where(torch.rand(rows, cols, generator=g) < 0.98, 0.0, x)
    return x.to(dtype).to(DEV)


def _strided(x, layout):
    rows, cols = x.shape
    if layout == "strided":
        full = torch.full((rows, cols + 40), 9.0, dtype=x.dtype, device=DEV)
        v = full[:, 16:16 + cols]
    elif layout == "shifted":
        v = torch.full((rows * cols + 1,), 9.0, dtype=x.dtype, device=DEV)[1:].view(rows, cols)
    else:
        return x
    v.copy_(x)
    return v


def _save(x, dtype=None):
    c = dopt.checkpoint(x.shape[0], x.shape[1], x.dtype)
    c.data.fill_(77)
    dopt.dopt_ckpt_save(x, c)
    return c


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("kind", ["normal", "wide", "halves", "zeros"])
@pytest.mark.parametrize("rows,cols,layout", [
    (1, 1, "plain"), (3, 31, "plain"), (2, 32, "plain"), (5, 33, "shifted"), (9, 100, "strided"),
    (17, 512, "plain"), (4, 517, "plain"), (70, 129, "shifted"), (33, 1028, "strided")])
def test_format_and_values(rows, cols, layout, kind, dtype):
    x = _values(rows, cols, dtype, kind)
    half = dtype == torch.float16
    c = _save(_strided(x, layout))
    pitch = -(-cols // 128) * 128
    assert c.data.numel() == rows * pitch * 33 // 32
    codes = c.data[:rows * pitch].view(torch.int8).view(rows, pitch).cpu().numpy()
    exps = c.data[rows * pitch:].view(rows, pitch // 32).cpu().numpy()
    want_codes, want_exps = R.keep(R.f64(x), half)
    assert np.array_equal(exps[:, :want_exps.shape[1]], want_exps)
    assert np.array_equal(codes[:, :want_codes.shape[1]], want_codes)
    assert not codes[:, cols:].any() and np.all(exps != 255)
    want = R.kept_values(R.f64(x), half)
    for out_dtype in (torch.float32, torch.bfloat16) + ((torch.float16,) if half else ()):
        out = _strided(torch.zeros(rows, cols, dtype=out_dtype, device=DEV), layout)
        dopt.dopt_ckpt_load(c, out)
        assert np.array_equal(R.f64(out), want)  # exact in these types
    if layout != "plain":  # nothing beside the rows is written
        base = out._base if out._base is not None else out
        assert int((base.float() == 9).sum()) >= base.numel() - out.numel()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_blocks_with_inf_or_nan(dtype):
    x = _values(6, 200, dtype, "normal")
    x[0, 0], x[1, 63], x[2, 199], x[3, 100] = float("nan"), float("inf"), -float("inf"), float("nan")
    out = torch.zeros_like(x)
    dopt.dopt_ckpt_load(_save(x), out)
    want = R.kept_values(R.f64(x), dtype == torch.float16)
    assert np.isnan(want).sum() == 32 + 32 + 8 + 32
    assert np.array_equal(R.f64(out), want, equal_nan=True)


def test_load_by_row_index():
    x = _values(40, 300, torch.bfloat16, "normal")
    c = _save(x)
    index = torch.tensor([39, 0, 0, -1, 40, 2 ** 31 - 1, 7], dtype=torch.int32, device=DEV)
    out = torch.full((7, 300), 5.0, device=DEV)
    dopt.dopt_ckpt_load(c, out, row_index=index)
    kept = R.kept_values(R.f64(x))
    assert np.array_equal(R.f64(out), np.stack([kept[39], kept[0], kept[0]] + 3 * [0 * kept[0]] + [kept[7]]))
    dopt.dopt_ckpt_load(c, out[:0], row_index=index[:0])
    half = torch.zeros(40, 300, dtype=torch.float16, device=DEV)  # bf16 values rounded to fp16
    dopt.dopt_ckpt_load(c, half)
    R.close(half, kept, 0.0, torch.float16, "fp16 of bf16")


def test_no_rows():
    c = dopt.checkpoint(0, 64)
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    dopt.dopt_ckpt_save(x, c)
    dopt.dopt_ckpt_load(c, x)
    dopt.dopt_ckpt_act_grad(c, "silu", x, x)


def test_checkpoint_past_32_bit_offsets():
    rows, cols = (1 << 20) + 3, 4096  # 4.3 G codes
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-3:] = _values(3, cols, torch.bfloat16, "normal")
    c = _save(x)
    index = torch.tensor([rows - 1, rows - 3, 5], dtype=torch.int32, device=DEV)
    out = torch.zeros(3, cols, device=DEV)
    dopt.dopt_ckpt_load(c, out, row_index=index)
    kept = R.kept_values(R.f64(x[-3:]))
    assert np.array_equal(R.f64(out), np.stack([kept[2], kept[0], 0 * kept[0]]))
    d = torch.ones(rows, cols, dtype=torch.bfloat16, device=DEV)
    dopt.dopt_ckpt_act_grad(c, "silu", d, d)  # in place
    want, bound = R.act_grad("silu", kept, np.ones_like(kept))
    R.close(d[-3:], want, bound, torch.bfloat16, "silu")
    assert torch.all(d[:-3] == 0.5)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("rows,width,layout", [
    (1, 1, "plain"), (3, 32, "plain"), (7, 33, "plain"), (5, 48, "plain"), (20, 500, "shifted"),
    (9, 96, "strided"), (65, 1024, "plain"), (6, 1031, "plain")])
def test_act_grad(rows, width, layout, act, dtype):
    cols = 2 * width if act == "swiglu" else width
    h = _values(rows, cols, dtype, "normal", 1) * 3
    d = _values(rows, width, dtype, "normal", 2)
    h = h.clamp(-9, 9)
    c = _save(h)
    d_in = _strided(torch.zeros(rows, cols, dtype=dtype, device=DEV), layout)
    dopt.dopt_ckpt_act_grad(c, act, _strided(d, layout), d_in)
    want, bound = R.act_grad(act, R.kept_values(R.f64(h), dtype == torch.float16), R.f64(d))
    R.close(d_in, want, bound, dtype, act)
    if act != "swiglu":
        dopt.dopt_ckpt_act_grad(c, act, d, d)  # in place
        assert torch.equal(d, d_in)


@pytest.mark.parametrize("rows,cols,dtype", [
    (1701, 4101, torch.bfloat16), (1701, 2051, torch.float32), (1531, 4112, torch.float16)], ids=str)
def test_blocks_of_several_rows_in_turn(rows, cols, dtype):
    """Enough rows for a thread block to take several groups of them, the last
    ones short of a whole group: every row, kept, read back (by index too, from
    the last row on) and through the activation gradients."""
    half = dtype == torch.float16
    x = _values(rows, cols, dtype, "normal", 3).clamp(-9, 9)
    c, out = _save(x), torch.zeros_like(x)
    kept = R.kept_values(R.f64(x), half)
    dopt.dopt_ckpt_load(c, out)
    assert np.array_equal(R.f64(out), kept)
    index = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device=DEV)
    dopt.dopt_ckpt_load(c, out, row_index=index)
    assert np.array_equal(R.f64(out), kept[::-1])
    for act in ("gelu",) if cols % 2 else ("gelu", "swiglu"):
        d = _values(rows, cols // 2 if act == "swiglu" else cols, dtype, "normal", 4)
        dopt.dopt_ckpt_act_grad(c, act, d, out)
        want, bound = R.act_grad(act, kept, R.f64(d))
        R.close(out, want, bound, dtype, act)


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
def test_act_grad_against_differences(act):
    """Central differences of the function itself at the kept values, in 64
    bits: their own error is eps^2 / 6 times the third derivative (below 4 for
    these functions, times |u| for the gated one) and 2^-50 / eps."""
    h = _values(4, 64, torch.float32, "normal", 5) * 2
    d = _values(4, 32 if act == "swiglu" else 64, torch.float32, "normal", 6)
    d_in = torch.zeros_like(h)
    dopt.dopt_ckpt_act_grad(_save(h), act, d, d_in)
    kept, dn, eps = R.kept_values(R.f64(h)), R.f64(d), 1e-4
    _, bound = R.act_grad(act, kept, dn)
    want = np.zeros_like(kept)
    for j in range(kept.shape[1]):
        up, down = kept.copy(), kept.copy()
        up[:, j] += eps
        down[:, j] -= eps
        want[:, j] = (dn * (R.act(act, up) - R.act(act, down)) / (2 * eps)).sum(axis=1)
    scale = (1 + np.abs(kept).max()) * np.abs(dn).max()
    R.close(d_in, want, bound + scale * (4 * eps ** 2 + 2.0 ** -46 / eps), torch.float32, act)


def test_act_grad_at_the_ends():
    """Far out the slopes are 0 and 1 (and swiglu's silu(g) is 0 and g), NaN
    stays NaN and an Inf gradient stays Inf."""
    big = torch.tensor([[3e38, -3e38, 1e5, -1e5, 200.0, -200.0, 90.0, -90.0]], device=DEV)
    h = torch.zeros(1, 8 * 32, device=DEV)
    h[:, ::32] = big  # one value a block, so that each is kept to 1 part in 64
    ones = torch.ones_like(h)
    for act in ("silu", "gelu"):
        d_in = torch.zeros_like(h)
        dopt.dopt_ckpt_act_grad(_save(h), act, ones, d_in)
        assert torch.allclose(d_in[:, ::32], (big > 0).float(), rtol=0, atol=1e-30)
        assert torch.allclose(d_in[:, 1::32], torch.tensor(0.5, device=DEV), rtol=0, atol=1e-6)
    gated = torch.cat([h, ones], dim=1)
    d_in = torch.zeros_like(gated)
    dopt.dopt_ckpt_act_grad(_save(gated), "swiglu", ones, d_in)
    kept = torch.from_numpy(R.kept_values(R.f64(h))).to(DEV)
    assert torch.allclose(d_in[:, :256:32].double(), (big > 0).double(), rtol=0, atol=1e-30)
    assert torch.allclose(d_in[:, 256::32].double(), kept[:, ::32].clamp(min=0), rtol=1e-6, atol=1e-30)
    h[0, 3], ones[0, 40] = float("nan"), float("inf")
    dopt.dopt_ckpt_act_grad(_save(h), "silu", ones, d_in[:, :256])
    assert torch.all(torch.isnan(d_in[0, :32])) and torch.isinf(d_in[0, 40])


def test_another_stream():
    x = _values(500, 640, torch.bfloat16, "normal")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = dopt.checkpoint(500, 640)
        out = torch.empty_like(x)
    dopt.dopt_ckpt_save(x, c, stream=side)
    dopt.dopt_ckpt_load(c, out, stream=side)
    side.synchronize()
    assert np.array_equal(R.f64(out), R.kept_values(R.f64(x)))
