"""Weight gradients from a kept input into a flat grad buffer, against 64-bit
products: dense and per expert, odd sizes and strides, empty groups, rows of
other groups that hold NaN, accumulation, every grad type, and exactly where
the sums are exact."""
import numpy as np
import pytest
import torch

import layer_reference as R
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _layout(t, layout):
    rows, cols = t.shape
    if layout == "strided":
        v = torch.full((rows, cols + 24), float("nan"), dtype=t.dtype, device=DEV)[:, 8:8 + cols]
    elif layout == "shifted":
        v = torch.full((rows * cols + 1,), float("nan"), dtype=t.dtype, device=DEV)[1:].view(rows, cols)
    else:
        return t
    v.copy_(t)
    return v


def _case(rows, outs, cols, groups, x_rows, dtype, seed=0, integers=False):
    """A checkpoint, dy, and for groups > 0 offsets that leave the first and
    last rows (NaN in dy) to no group, one group empty, and row tokens."""
    g = torch.Generator(device=DEV).manual_seed(seed + rows * 3 + outs + cols)
    if integers:  # kept exactly (the largest of a block is below 128), products and sums exact in fp32
        x = torch.randint(-60, 61, (x_rows, cols), generator=g, device=DEV).to(dtype)
        dy = torch.randint(-8, 9, (rows, outs), generator=g, device=DEV).to(dtype)
    else:
        x = torch.randn(x_rows, cols, generator=g, device=DEV).to(dtype)
        dy = (torch.randn(rows, outs, generator=g, device=DEV) * 0.1).to(dtype)
    c = dopt.checkpoint(x_rows, cols, dtype)
    dopt.dopt_ckpt_save(x, c)
    offsets = row_token = None
    if groups:
        cut = np.sort(np.random.default_rng(seed + rows).integers(2, rows - 1, groups + 1))
        if groups > 2:
            cut[2] = cut[1]
        offsets = torch.tensor(cut, dtype=torch.int32, device=DEV)
        dy[:cut[0]] = float("nan")
        dy[cut[-1]:] = float("nan")
        row_token = torch.randint(0, x_rows, (rows,), generator=g, device=DEV).int()
        row_token[cut[0]] = -1           # rows of no token count as zeros
        row_token[cut[-1] - 1] = x_rows
    return c, R.kept_values(R.f64(x), dtype == torch.float16), dy, offsets, row_token


def _want(kept, dy, offsets, row_token, groups):
    dn = np.nan_to_num(R.f64(dy))
    return R.wgrad(kept, dn, None if offsets is None else offsets.cpu().numpy(),
                   None if row_token is None else row_token.cpu().numpy(), max(groups, 1))


CASES = [  # rows, outs, cols, groups (0: dense), rows of x, layout of dy
    (1, 1, 1, 0, 1, "plain"), (2, 5, 3, 0, 9, "plain"), (64, 64, 64, 0, 64, "plain"),
    (65, 130, 33, 0, 65, "plain"), (300, 200, 264, 0, 300, "strided"), (129, 257, 129, 0, 129, "shifted"),
    (1000, 128, 256, 0, 1000, "plain"), (777, 264, 520, 0, 800, "plain"),
    (40, 72, 40, 3, 25, "plain"), (500, 136, 300, 5, 130, "plain"), (700, 99, 257, 4, 350, "shifted"),
    (2048, 256, 384, 8, 512, "plain"), (900, 512, 128, 64, 300, "plain")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("grad_dtype", ["same", torch.float32], ids=str)
@pytest.mark.parametrize("rows,outs,cols,groups,x_rows,layout", CASES)
def test_wgrad(rows, outs, cols, groups, x_rows, layout, grad_dtype, dtype):
    grad_dtype = dtype if grad_dtype == "same" else grad_dtype
    c, kept, dy, offsets, row_token = _case(rows, outs, cols, groups, x_rows, dtype)
    want = _want(kept, dy, offsets, row_token, groups)
    n, E = outs * cols, max(groups, 1)
    starts = [3 + g * (n + 5) for g in range(E)]
    starts = starts[::-1]  # in falling order: groups may sit anywhere
    ws = dopt.wgrad_workspace(rows, outs, cols, E)
    for workspace in (None, ws):
        grad = torch.full((3 + E * (n + 5),), 2.5, dtype=grad_dtype, device=DEV)
        dopt.dopt_ckpt_wgrad(c, _layout(dy, layout), grad, starts, offsets=offsets, row_token=row_token,
                             workspace=workspace)
        seen = torch.ones_like(grad, dtype=torch.bool)
        for g, (w, mag, m) in enumerate(want):
            at = slice(starts[g], starts[g] + n)
            seen[at] = False
            # at most one rounding (or truncation) of a partial sum a product
            R.close(grad[at].view(outs, cols), w, (m + 8) * 2 * R.F32 * mag, grad_dtype, f"group {g}")
        assert torch.all(grad[seen] == 2.5)  # nothing between the params
        # accumulation onto what is there
        before = grad.clone()
        dopt.dopt_ckpt_wgrad(c, _layout(dy, layout), grad, starts, offsets=offsets, row_token=row_token,
                             accumulate=True, workspace=workspace)
        for g, (w, mag, m) in enumerate(want):
            at = slice(starts[g], starts[g] + n)
            old = R.f64(before[at]).reshape(outs, cols)
            R.close(grad[at].view(outs, cols), old + w, (m + 9) * 2 * R.F32 * (mag + np.abs(old)), grad_dtype,
                    f"group {g} accumulated")
        assert torch.all(grad[seen] == 2.5)


@pytest.mark.parametrize("rows,outs,cols,groups,x_rows", [
    (31, 40, 70, 0, 31), (512, 256, 256, 0, 512), (1100, 300, 520, 0, 1100), (3000, 129, 130, 7, 900),
    (4096, 512, 384, 16, 1024), (5000, 640, 768, 0, 5000), (2500, 264, 1288, 3, 700)])
def test_exact_sums(rows, outs, cols, groups, x_rows):
    """Whole numbers whose sums stay below 2^24: every order of summation gives
    the same fp32 result, so the kernel's has to be equal."""
    c, kept, dy, offsets, row_token = _case(rows, outs, cols, groups, x_rows, torch.bfloat16, integers=True)
    want = _want(kept, dy, offsets, row_token, groups)
    n, E = outs * cols, max(groups, 1)
    starts = [8 + g * n for g in range(E)]
    for workspace in (None, dopt.wgrad_workspace(rows, outs, cols, E)):
        grad = torch.full((8 + E * n,), -1.0, device=DEV)
        dopt.dopt_ckpt_wgrad(c, dy, grad, starts, offsets=offsets, row_token=row_token, workspace=workspace)
        for g, (w, mag, _) in enumerate(want):
            assert mag.max(initial=0) < 2 ** 24
            assert np.array_equal(R.f64(grad[starts[g]:starts[g] + n]).reshape(outs, cols), w), f"group {g}"


def test_groups_without_rows():
    """No rows at all: zeros, or what was there."""
    c = dopt.checkpoint(4, 40)
    dopt.dopt_ckpt_save(torch.ones(4, 40, dtype=torch.bfloat16, device=DEV), c)
    dy = torch.full((6, 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    offsets = torch.tensor([3, 3, 3], dtype=torch.int32, device=DEV)
    token = torch.zeros(6, dtype=torch.int32, device=DEV)
    grad = torch.full((2000,), 7.0, device=DEV)
    dopt.dopt_ckpt_wgrad(c, dy, grad, [0, 1000], offsets=offsets, row_token=token, accumulate=True)
    assert torch.all(grad == 7)
    dopt.dopt_ckpt_wgrad(c, dy, grad, [0, 1000], offsets=offsets, row_token=token)
    assert torch.all(grad[:960] == 0) and torch.all(grad[1000:1960] == 0) and torch.all(grad[960:1000] == 7)
    dopt.dopt_ckpt_wgrad(c, dy[:0], grad, [1000])
    assert torch.all(grad[1000:1960] == 0)


def test_offsets_out_of_range_are_held():
    c, kept, dy, _, _ = _case(50, 16, 24, 0, 50, torch.bfloat16)
    offsets = torch.tensor([-5, 20, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    token = torch.arange(50, dtype=torch.int32, device=DEV)
    grad = torch.zeros(2 * 384, device=DEV)
    dopt.dopt_ckpt_wgrad(c, dy, grad, [0, 384], offsets=offsets, row_token=token)
    for g, (lo, hi) in enumerate(((0, 20), (20, 50))):
        dn, xn = R.f64(dy)[lo:hi], kept[lo:hi]
        R.close(grad[384 * g:384 * (g + 1)].view(16, 24), dn.T @ xn, 2 * 40 * R.F32 * (np.abs(dn).T @ np.abs(xn)),
                torch.float32, f"group {g}")


def test_nonfinite_values_reach_only_their_grads():
    """NaN in x, Inf in dy: the grads they are summed into and no others."""
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(300, 320, generator=g, device=DEV).bfloat16()
    dy = torch.randn(300, 264, generator=g, device=DEV).bfloat16()
    x[299, 70] = float("nan")    # its block: columns 64..95
    dy[150, 9] = float("inf")    # output 9
    c = dopt.checkpoint(300, 320)
    dopt.dopt_ckpt_save(x, c)
    grad = torch.zeros(264 * 320, device=DEV)
    dopt.dopt_ckpt_wgrad(c, dy, grad, [0])
    bad = ~torch.isfinite(grad.view(264, 320))
    want = torch.zeros_like(bad)
    want[:, 64:96] = True
    want[9, :] = True
    assert torch.equal(bad, want)


def test_against_differences():
    """y = x W^T is linear in W: the change of sum(y * dy) over a unit step of
    a weight, in 64 bits on the kept values, is that weight's gradient."""
    c, kept, dy, _, _ = _case(60, 20, 36, 0, 60, torch.bfloat16, seed=9)
    grad = torch.zeros(720, device=DEV)
    dopt.dopt_ckpt_wgrad(c, dy, grad, [0])
    dn, w = R.f64(dy), np.random.default_rng(0).normal(size=(20, 36))
    mag = np.abs(dn).T @ np.abs(kept)
    base = ((kept @ w.T) * dn).sum()
    for o, i in ((0, 0), (7, 35), (19, 11)):
        w2 = w.copy()
        w2[o, i] += 1
        got = float(grad[o * 36 + i])
        assert abs(((kept @ w2.T) * dn).sum() - base - got) <= 2 * 70 * R.F32 * mag[o, i] + 1e-9


def test_repeats_and_another_stream():
    """The same bits at every call, on the current stream and on another."""
    c, _, dy, offsets, row_token = _case(3000, 264, 392, 6, 900, torch.bfloat16)
    starts = [g * 264 * 392 for g in range(6)]
    ws = dopt.wgrad_workspace(3000, 264, 392, 6)
    grads = []
    side = torch.cuda.Stream()
    for k in range(4):
        grad = torch.zeros(6 * 264 * 392, device=DEV)
        if k < 2:
            dopt.dopt_ckpt_wgrad(c, dy, grad, starts, offsets=offsets, row_token=row_token, workspace=ws)
        else:
            side.wait_stream(torch.cuda.current_stream())
            dopt.dopt_ckpt_wgrad(c, dy, grad, starts, offsets=offsets, row_token=row_token, workspace=ws,
                                 stream=side)
            side.synchronize()
        grads.append(grad)
    torch.cuda.synchronize()
    assert all(torch.equal(grads[0], x) for x in grads[1:])


def test_no_wait_ran_out():
    assert dopt.wgrad_timeouts() == 0
