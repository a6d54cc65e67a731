"""Plain 64-bit forms of the layer operators (numpy), written from their
definitions, and the bounds their fp32 kernels have to keep."""
import numpy as np
import torch

F32 = 2.0 ** -24  # half a unit in the last place, relative
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
BLOCK, PITCH = 32, 128


def f64(t):
    return t.detach().cpu().double().numpy()


def sort(ids, experts):
    """(slot_row, row_token, offsets) of [tokens, k] ids."""
    tokens, k = ids.shape
    slot_row = np.full((tokens, k), -1, np.int32)
    row_token = np.full(tokens * k, -1, np.int32)
    offsets, row = [0], 0
    flat = ids.reshape(-1)
    for e in range(experts):
        for s in np.flatnonzero(flat == e):
            slot_row[s // k, s % k] = row
            row_token[row] = s // k
            row += 1
        offsets.append(row)
    return slot_row, row_token, np.array(offsets, np.int32)


def combine(rows, slot_row, weights, n_rows):
    """(sum, sum of magnitudes) over each token's kept slots."""
    tokens, k = slot_row.shape
    out = np.zeros((tokens, rows.shape[1]))
    mag = np.zeros_like(out)
    for t in range(tokens):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < n_rows:
                term = rows[r] * (1.0 if weights is None else weights[t, j])
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def keep(x, from_fp16=False):
    """(codes, exponent bytes) of a checkpoint of x, from the format's text."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    codes = np.zeros((rows, blocks * BLOCK), np.int64)
    exps = np.zeros((rows, blocks), np.int64)
    least = -24 if from_fp16 else -126
    for r in range(rows):
        for b in range(blocks):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.all(np.isfinite(v)):
                exps[r, b] = 255
                continue
            top = np.abs(v).max()
            k = least if top == 0 else max(least, int(np.frexp(top)[1]) - 1 - 6)
            exps[r, b] = k + 127
            q = np.rint(v / 2.0 ** k)  # nearest even; the quotient is exact
            codes[r, b * BLOCK:b * BLOCK + len(v)] = np.clip(q, -127, 127)
    return codes, exps


def kept_values(x, from_fp16=False):
    codes, exps = keep(x, from_fp16)
    step = np.where(exps == 255, np.nan, 2.0 ** (exps - 127.0))
    return (codes * np.repeat(step, BLOCK, axis=1))[:, :x.shape[1]]


def sigmoid(x):
    """With full relative precision on both sides (a form in 1 + tanh loses the lower tail)."""
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


C, A = np.sqrt(2.0 / np.pi), 0.044715


def act(name, h):
    if name == "silu":
        return h * sigmoid(h)
    if name == "gelu":
        return h * sigmoid(2 * C * (h + A * h ** 3))
    g, u = np.split(h, 2, axis=1)
    return g * sigmoid(g) * u


def _slope(t, x, g):
    """p + g p m with p = sigmoid(t), m = 1 - p, and the bound of its fp32
    evaluation: t carries |t| 2^-21 of rounding, the exponential 2 + 1.2 |t|
    units of 2^-23 (so p and m move by p m times that), and the sums,
    products and the quotient 16 roundings of each term."""
    p, m = sigmoid(t), sigmoid(-t)
    d = np.abs(t) * 2.0 ** -21 + (2 + 1.2 * np.abs(t)) * 2.0 ** -23
    bound = p * m * d * (1 + 2 * np.abs(g)) + 16 * F32 * (p + np.abs(g) * p * m)
    return p + g * p * m, bound


def act_grad(name, h, d):
    """(gradient, bound of its fp32 evaluation before the last rounding).
    |h| is at most 80 (9 for gelu) here: the flat ends are tested apart."""
    if name == "silu":
        slope, bound = _slope(h, h, h)
        return d * slope, np.abs(d) * bound
    if name == "gelu":
        slope, bound = _slope(2 * C * (h + A * h ** 3), h, 2 * C * h * (1 + 3 * A * h * h))
        return d * slope, np.abs(d) * bound
    g, u = np.split(h, 2, axis=1)
    slope, bound = _slope(g, g, g)
    s = sigmoid(g)
    ds = s * sigmoid(-g) * (np.abs(g) * 2.0 ** -21 + (2 + 1.2 * np.abs(g)) * 2.0 ** -23) + 8 * F32 * s
    return (np.concatenate([d * u * slope, d * g * s], axis=1),
            np.concatenate([np.abs(d * u) * bound, np.abs(d * g) * ds], axis=1))


def wgrad(x, dy, offsets, row_token, groups):
    """Per group (sum, sum of magnitudes, rows)."""
    out = []
    for g in range(groups):
        lo, hi = (0, dy.shape[0]) if offsets is None else (offsets[g], offsets[g + 1])
        token = np.arange(lo, hi) if row_token is None else row_token[lo:hi]
        there = (token >= 0) & (token < x.shape[0])
        xe = np.where(there[:, None], x[np.where(there, token, 0)] if len(x) else 0.0, 0.0).reshape(hi - lo, x.shape[1])
        out.append((dy[lo:hi].T @ xe, np.abs(dy[lo:hi]).T @ np.abs(xe), hi - lo))
    return out


def close(got, want, bound, dtype, what):
    """got (of `dtype`) within `bound` and one rounding to dtype of want; NaN
    and Inf where want has them (an Inf also where want rounds to one)."""
    g = f64(got)
    assert g.shape == want.shape, f"{what}: shape {g.shape}, expected {want.shape}"
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN in other places"
    fine = np.isfinite(want) & np.isfinite(g)
    inf = ~np.isfinite(g) & ~np.isnan(g)
    limit = float(torch.finfo(dtype).max)
    assert np.all(np.abs(want[inf]) >= limit * (1 - UNIT[dtype])), f"{what}: Inf for a finite value"
    off = np.abs(g[fine] - want[fine])
    room = (np.broadcast_to(bound, want.shape)[fine] * (1 + UNIT[dtype]) + UNIT[dtype] * np.abs(want[fine])
            + TINY[dtype])
    worst = int(np.argmax(off - room)) if off.size else 0
    assert np.all(off <= room), f"{what}: off by {off[worst]} where {room[worst]} is allowed"
