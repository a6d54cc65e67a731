"""Tokens sorted by expert and back, and the gradients, against plain 64-bit
forms: sizes from one token to several sorting tiles, dropped slots, odd
widths, strided and unaligned rows, NaN in places that do not count, other
streams, rows past 32-bit offsets."""
import numpy as np
import pytest
import torch

import layer_reference as R
import zero_distributed_optimizer_gb300 as dopt

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _sort(ids, experts):
    tokens, k = ids.shape
    out = [torch.full((tokens, k), -7, dtype=torch.int32, device=DEV),
           torch.full((tokens * k,), -7, dtype=torch.int32, device=DEV),
           torch.full((experts + 1,), -7, dtype=torch.int32, device=DEV)]
    dopt.dopt_route_sort(ids, experts, *out, dopt.route_workspace(tokens, k, experts))
    return out


@pytest.mark.parametrize("tokens,k,experts,wide", [
    (0, 1, 3, True), (1, 1, 1, True), (1, 8, 64, False), (5, 3, 2, True), (31, 2, 1024, True),
    (512, 8, 64, True), (513, 8, 64, False), (4096, 1, 5, True), (4097, 1, 1024, False),
    (3001, 7, 40, True), (20000, 4, 1023, True), (1000, 64, 8, False)])
@pytest.mark.parametrize("kind", ["spread", "dropped", "one"])
def test_sort(tokens, k, experts, wide, kind):
    rng = np.random.default_rng(tokens * 31 + k)
    if kind == "spread":
        ids = rng.integers(0, experts, (tokens, k))
    elif kind == "dropped":  # ids below and above the range, far beyond 32 bits where they can be
        ids = rng.integers(-2, experts + 3, (tokens, k))
        if wide:
            ids[rng.random((tokens, k)) < 0.1] = 2 ** 32
    else:
        ids = np.full((tokens, k), experts - 1)
    t = torch.from_numpy(ids.astype(np.int64 if wide else np.int32)).to(DEV)
    want = R.sort(ids, experts)
    for a, b in zip(_sort(t, experts), want):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("tokens,k,experts", [
    (4096, 8, 1024), (16384, 2, 300), (16385, 2, 300), (524288, 2, 64), (400000, 3, 1024), (262145, 4, 7),
    (700000, 2, 5), (1300000, 3, 900)])
def test_sort_many_slots(tokens, k, experts):
    """One block of the sort, its cluster, and tiles in two launches, against a stable sort."""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    ids = torch.randint(-1, experts + 1, (tokens, k), generator=g, device=DEV)
    slot_row, row_token, offsets = _sort(ids, experts)
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    key, order = torch.sort(key, stable=True)
    n = int((key < experts).sum())
    assert torch.equal(row_token[:n], (order[:n] // k).int()) and torch.all(row_token[n:] == -1)
    want = torch.full((tokens * k,), -1, dtype=torch.int32, device=DEV)
    want[order[:n]] = torch.arange(n, dtype=torch.int32, device=DEV)
    assert torch.equal(slot_row.view(-1), want)
    assert torch.equal(offsets, torch.searchsorted(key, torch.arange(experts + 1, device=DEV)).int())


def _rows(n, cols, dtype, layout, g):
    """A [n, cols] tensor: contiguous, with a longer row stride, or starting
    one element into its storage."""
    x = torch.randn(n, cols, generator=g, device=DEV)
    if layout == "strided":
        full = torch.zeros(n, cols + 24, dtype=dtype, device=DEV)
        view = full[:, 8:8 + cols]
    elif layout == "shifted":
        view = torch.zeros(n * cols + 1, dtype=dtype, device=DEV)[1:].view(n, cols)
    else:
        view = torch.empty(n, cols, dtype=dtype, device=DEV)
    view.copy_(x)
    return view


def _route(tokens, k, experts, local, g):
    ids = torch.rand(tokens, experts, generator=g, device=DEV).argsort(dim=1)[:, :k].contiguous()
    slot_row, row_token, offsets = _sort(ids, local)
    weights = torch.softmax(torch.randn(tokens, k, generator=g, device=DEV), dim=1).contiguous()
    return slot_row, row_token, int(offsets[-1]), weights


CASES = [  # tokens, k, experts, local, cols, layout
    (1, 1, 1, 1, 1, "plain"), (1, 8, 64, 64, 512, "plain"), (3, 2, 4, 1, 7, "plain"),
    (33, 2, 8, 3, 515, "plain"), (65, 6, 8, 8, 130, "shifted"), (40, 33, 64, 50, 96, "plain"),
    (129, 4, 16, 8, 1028, "strided"), (257, 8, 32, 16, 64, "strided"), (17, 3, 4, 4, 2500, "plain")]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("tokens,k,experts,local,cols,layout", CASES)
def test_dispatch_combine_and_gradients(tokens, k, experts, local, cols, layout, dtype):
    g = torch.Generator(device=DEV).manual_seed(tokens + cols)
    slot_row, row_token, n, weights = _route(tokens, k, experts, local, g)
    sr = slot_row.cpu().numpy()
    x = _rows(tokens, cols, dtype, layout, g)
    rows = torch.full((tokens * k, cols), 3.0, dtype=dtype, device=DEV)
    dopt.dopt_route_dispatch(x, slot_row, rows)
    assert torch.equal(rows[:n], x[row_token[:n].long()])
    assert torch.all(rows[n:] == 3.0)  # rows without a slot are not written

    y = _rows(tokens * k, cols, dtype, "shifted" if layout == "shifted" else "plain", g)
    y[n:] = float("nan")           # not a slot's row
    w = weights.clone()
    w[slot_row < 0] = float("nan")  # a dropped slot's weight
    out = _rows(tokens, cols, dtype, layout, g)
    for wt, wn in ((w, R.f64(weights)), (None, None)):
        dopt.dopt_route_combine(y, slot_row, wt, out)
        want, mag = R.combine(R.f64(y), sr, wn, n)
        R.close(out, want, (k + 1) * R.F32 * mag, dtype, "combine")

    d = _rows(tokens, cols, dtype, layout, g)
    d_rows = torch.full_like(rows, 5.0)
    d_w = torch.full_like(weights, 5.0)
    dopt.dopt_route_combine_grad(d, y, slot_row, w, d_rows, d_w)
    dn, yn, wn = R.f64(d), R.f64(y), R.f64(weights)
    want_w, mag_w, want_r = np.zeros((tokens, k)), np.zeros((tokens, k)), np.full((tokens * k, cols), 5.0)
    for t in range(tokens):
        for j in range(k):
            if sr[t, j] >= 0:
                want_r[sr[t, j]] = wn[t, j] * dn[t]
                want_w[t, j] = dn[t] @ yn[sr[t, j]]
                mag_w[t, j] = np.abs(dn[t]) @ np.abs(yn[sr[t, j]])
    R.close(d_rows, want_r, R.F32 * np.abs(want_r), dtype, "d_rows")
    R.close(d_w, want_w, (cols + 5) * R.F32 * mag_w, torch.float32, "d_weights")


def test_gradients_against_differences():
    """The combine is linear in a weight and in a row: the change of
    sum(out * r) over a step of 1 is the gradient, up to the fp32 roundings of
    the two sums (bounded by their magnitudes)."""
    g = torch.Generator(device=DEV).manual_seed(3)
    tokens, k, cols = 9, 3, 40
    slot_row, _, n, w = _route(tokens, k, 4, 3, g)
    y = torch.randn(tokens * k, cols, generator=g, device=DEV)
    r = torch.randn(tokens, cols, generator=g, device=DEV)
    d_rows, d_w = torch.zeros_like(y), torch.zeros_like(w)
    dopt.dopt_route_combine_grad(r, y, slot_row, w, d_rows, d_w)

    def loss(y, w):
        out = torch.empty(tokens, cols, device=DEV)
        dopt.dopt_route_combine(y, slot_row, w, out)
        return float((out.double() * r.double()).sum())

    room = 16 * R.F32 * float((w.abs().sum() + 1) * y.abs().max() * r.abs().sum())
    base = loss(y, w)
    for t in range(tokens):
        for j in range(k):
            w2 = w.clone()
            w2[t, j] += 1
            assert abs(loss(y, w2) - base - float(d_w[t, j])) <= room
    for row in range(n):
        y2 = y.clone()
        y2[row, row % cols] += 1
        assert abs(loss(y2, w) - base - float(d_rows[row, row % cols])) <= room
    # dispatch and the unweighted combine are each other's transpose
    x = torch.randn(tokens, cols, generator=g, device=DEV)
    rows, back = torch.zeros_like(y), torch.zeros_like(x)
    dopt.dopt_route_dispatch(x, slot_row, rows)
    dopt.dopt_route_combine(y, slot_row, None, back)
    left, right = float((rows.double() * y.double())[:n].sum()), float((x.double() * back.double()).sum())
    assert abs(left - right) <= (k + 2) * R.F32 * float((rows * y)[:n].abs().sum()) + 1e-12


def test_no_token_and_no_row():
    for tokens, n_rows in ((0, 4), (4, 0)):
        slot_row = torch.full((tokens, 2), -1, dtype=torch.int32, device=DEV)
        rows = torch.ones(n_rows, 8, device=DEV)
        x = torch.ones(tokens, 8, device=DEV)
        w, d_w = torch.ones(tokens, 2, device=DEV), torch.ones(tokens, 2, device=DEV)
        dopt.dopt_route_dispatch(x, slot_row, rows)
        dopt.dopt_route_combine(rows, slot_row, w, x)
        dopt.dopt_route_combine_grad(x, rows, slot_row, w, torch.ones_like(rows), d_w)
        assert torch.all(rows == 1) and torch.all(x == 0) and torch.all(d_w == 0)


def test_rows_out_of_range_are_skipped():
    slot_row = torch.tensor([[0, 5], [2 ** 31 - 1, 1], [-9, -1]], dtype=torch.int32, device=DEV)
    x = torch.arange(24, device=DEV, dtype=torch.float32).view(3, 8)
    rows = torch.zeros(2, 8, device=DEV)
    dopt.dopt_route_dispatch(x, slot_row, rows)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[1], x[1])
    out = torch.empty(3, 8, device=DEV)
    dopt.dopt_route_combine(rows, slot_row, torch.full((3, 2), 2.0, device=DEV), out)
    assert torch.equal(out, torch.stack([2 * x[0], 2 * x[1], 0 * x[2]]))


def test_another_stream_and_repeats():
    """On a side stream that waits for nothing but its own inputs, and twice:
    the same bits."""
    g = torch.Generator(device=DEV).manual_seed(8)
    tokens, k, cols = 3000, 4, 256
    ids = torch.randint(0, 16, (tokens, k), generator=g, device=DEV)
    x = torch.randn(tokens, cols, generator=g, device=DEV).bfloat16()
    w = torch.rand(tokens, k, generator=g, device=DEV)
    first = None
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            slot_row = torch.empty(tokens, k, dtype=torch.int32, device=DEV)
            row_token = torch.empty(tokens * k, dtype=torch.int32, device=DEV)
            offsets = torch.empty(17, dtype=torch.int32, device=DEV)
            ws = dopt.route_workspace(tokens, k, 16)
            rows = torch.empty(tokens * k, cols, dtype=x.dtype, device=DEV)
            out, d_rows, d_w = torch.empty_like(x), torch.empty_like(rows), torch.empty_like(w)
        dopt.dopt_route_sort(ids, 16, slot_row, row_token, offsets, ws, stream=side)
        dopt.dopt_route_dispatch(x, slot_row, rows, stream=side)
        dopt.dopt_route_combine(rows, slot_row, w, out, stream=side)
        dopt.dopt_route_combine_grad(x, rows, slot_row, w, d_rows, d_w, stream=side)
        side.synchronize()
        got = [slot_row, row_token, offsets, rows, out, d_rows, d_w]
        if first is None:
            first = [t.clone() for t in got]
            R.close(out, R.f64(x) * R.f64(w).sum(axis=1, keepdims=True),
                    (k + 1) * R.F32 * np.abs(R.f64(x)) * R.f64(w).sum(axis=1, keepdims=True), x.dtype, "combine")
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_rows_past_32_bit_offsets():
    n, cols = (1 << 20) + 5, 4096  # 4.3 G elements, 8.6 GB
    rows = torch.zeros(n, cols, dtype=torch.bfloat16, device=DEV)
    slot_row = torch.tensor([[n - 1, 0], [n - 2, 1]], dtype=torch.int32, device=DEV)
    x = torch.randn(2, cols, device=DEV).bfloat16()
    dopt.dopt_route_dispatch(x, slot_row, rows)
    assert torch.equal(rows[n - 1], x[0]) and torch.equal(rows[n - 2], x[1])
    out = torch.empty_like(x)
    dopt.dopt_route_combine(rows, slot_row, torch.tensor([[0.0, 2.0], [2.0, 0.0]], device=DEV), out)
    assert torch.equal(out, 2 * x)
    d_w = torch.empty(2, 2, device=DEV)
    dopt.dopt_route_combine_grad(x, rows, slot_row, torch.ones(2, 2, device=DEV), rows, d_w)
    norm = R.f64(x)
    R.close(d_w, np.repeat((norm * norm).sum(axis=1)[:, None], 2, axis=1),
            (cols + 5) * R.F32 * (norm * norm).sum(axis=1)[:, None], torch.float32, "d_weights")
