"""Workloads for the operators around the optimizer step that a training layer needs: tokens sorted by expert
and back with their gradients, and activations kept in 8 bits with the uses that the backward pass makes of them.

`listed` and `draw` give the cases, `prepare` makes a case's inputs on the GPU, `run` takes one pass through
an operator and `exact` gives its result in 64 bits.  With `own` the passes are calls of the package;
without, they are the operators' formulas in elementary torch operations in fp32.

Terms: a token takes k of E experts; a slot is one (token, choice) pair; experts 0..local-1 live on this rank
and slots that chose another one are dropped.  A checkpoint holds each row's columns in blocks of 32: one
int8 code per value and one exponent byte per block (value = code * 2**(byte - 127), byte 255: NaN).
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 32      # columns that share an exponent
PITCH = 128     # a checkpoint row's codes are padded to a multiple of this


def listed():
    return [
        # sorting and copying for a decoding batch's few tokens: launch latency counts
        dict(name="dispatch_few", op="dispatch", tokens=24, k=8, experts=64, local=64, cols=2048, dtype="bf16"),
        # one microbatch of a layer of 64 small experts, all on this rank
        dict(name="dispatch_train", op="dispatch", tokens=32768, k=8, experts=64, local=64, cols=512, dtype="bf16"),
        # a rank that holds 3 of 8 experts; an odd width, so that no row is aligned
        dict(name="combine_odd_share", op="combine", tokens=1001, k=2, experts=8, local=3, cols=515, dtype="fp16"),
        # the way back of dispatch_train
        dict(name="combine_train", op="combine", tokens=32768, k=8, experts=64, local=64, cols=512, dtype="bf16"),
        # gradients of the way back in fp32, half of the experts elsewhere
        dict(name="combine_grad_share", op="combine_grad", tokens=4096, k=4, experts=32, local=16, cols=1024, dtype="fp32"),
        # gradients of combine_train
        dict(name="combine_grad_train", op="combine_grad", tokens=32768, k=8, experts=64, local=64, cols=512, dtype="bf16"),
        # a small fp32 activation with a short last block, kept and read back
        dict(name="ckpt_odd", op="ckpt", rows=333, cols=1001, dtype="fp32"),
        # a Llama-1.3B MLP activation of 16384 tokens, kept and read back
        dict(name="ckpt_train", op="ckpt", rows=16384, cols=5632, dtype="bf16"),
        # GELU's backward pass on a ragged number of tokens
        dict(name="act_gelu", op="act_grad", act="gelu", rows=1025, cols=2048, dtype="fp16"),
        # the gated activation of a Llama-1.3B MLP, 16384 tokens
        dict(name="act_swiglu_train", op="act_grad", act="swiglu", rows=16384, cols=5632, dtype="bf16"),
        # weight gradient of a Llama-1.3B up projection over 16384 tokens, bf16 grads
        dict(name="wgrad_train", op="wgrad", tokens=16384, k=1, experts=1, outs=5632, cols=2048, dtype="bf16", grad="bf16"),
        # weight gradients of 64 experts of 512 x 1408, fp32 grads, the tokens' activations kept once
        dict(name="wgrad_experts", op="wgrad", tokens=8192, k=8, experts=64, outs=1408, cols=512, dtype="bf16", grad="fp32"),
    ]


def _size(rng, lo, hi, unit=64):
    """A size spread over [lo, hi]'s logarithm; half of them multiples of `unit`."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        n = -(-n // unit) * unit
    return max(lo, min(hi, n))


def draw(rng):
    while True:
        op = rng.choice(["dispatch", "combine", "combine_grad", "ckpt", "act_grad", "wgrad"])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if op in ("dispatch", "combine", "combine_grad"):
            experts = rng.choice([4, 8, 16, 32, 64, 128])
            c = dict(op=op, tokens=_size(rng, 1, 32768), k=rng.choice([1, 2, 3, 4, 6, 8]), experts=experts,
                     local=rng.choice([experts, experts // 2, max(1, experts // 3)]), cols=_size(rng, 64, 2048), dtype=dtype)
            if c["tokens"] < 32:  # a handful of tokens with every expert at hand
                c["local"] = experts
            if c["k"] <= experts and c["tokens"] * c["k"] * c["cols"] * SIZE[dtype] <= 32768 * 8 * 512 * 2:
                return c
        elif op == "ckpt":
            c = dict(op=op, rows=_size(rng, 1, 16384), cols=_size(rng, 32, 11264), dtype=dtype)
            if c["rows"] * c["cols"] * SIZE[dtype] <= 16384 * 5632 * 2:
                return c
        elif op == "act_grad":
            c = dict(op=op, act=rng.choice(["silu", "gelu", "swiglu"]), rows=_size(rng, 1, 16384), cols=_size(rng, 32, 5632), dtype=dtype)
            if c["rows"] * c["cols"] * SIZE[dtype] <= 16384 * 5632 * 2:
                return c
        else:
            experts = rng.choice([1, 1, 4, 8, 16, 64])
            dtype = rng.choice(["bf16", "fp16"])
            c = dict(op=op, tokens=_size(rng, 64, 16384), k=1 if experts == 1 else rng.choice([1, 2, 4]), experts=experts,
                     outs=_size(rng, 64, 5632), cols=_size(rng, 64, 5632), dtype=dtype, grad=rng.choice([dtype, "fp32"]))
            rows = c["tokens"] * c["k"]
            if (rows * c["outs"] * c["cols"] <= 16384 * 5632 * 2048 and rows * c["outs"] <= 16384 * 5632
                    and experts * c["outs"] * c["cols"] <= 64 * 1408 * 512):
                return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _route(g, c):
    """A router's choices (int64 ids by falling weight, as a top-k gives them) with popular and unpopular
    experts, their softmax weights, and what sorting the slots by expert gives."""
    T, k, E, local = c["tokens"], c["k"], c["experts"], c.get("local", c["experts"])
    logits = torch.randn(T, E, generator=g, device=DEVICE) + 0.5 * torch.randn(E, generator=g, device=DEVICE)
    top = logits.topk(k, dim=1)
    ids, weights = top.indices.contiguous(), torch.softmax(top.values, dim=1).contiguous()
    slot_row, row_token, offsets = _sort(ids, local)
    return ids, weights, slot_row, row_token, offsets


def _activations(g, rows, cols, dtype):
    """Normal values whose columns differ in size, a few of them much larger."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    x *= torch.exp(0.5 * torch.randn(cols, generator=g, device=DEVICE))
    x *= torch.where(torch.rand(cols, generator=g, device=DEVICE) < 0.005, 12.0, 1.0)
    return x.to(DTYPES[dtype])


def _inputs(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 11)
    s = dict(c)
    if c["op"] in ("dispatch", "combine", "combine_grad"):
        T, k, C, dt = c["tokens"], c["k"], c["cols"], DTYPES[c["dtype"]]
        ids, weights, slot_row, row_token, offsets = _route(g, c)
        if c["op"] == "dispatch":
            s.update(ids=ids, x=_activations(g, T, C, c["dtype"]))
        else:
            rows = _activations(g, T * k, C, c["dtype"])
            rows[int(offsets[-1]):] = 0
            s.update(rows=rows, weights=weights, slot_row=slot_row)
            if c["op"] == "combine_grad":
                s.update(d_out=(torch.randn(T, C, generator=g, device=DEVICE) * 1e-2).to(dt))
    elif c["op"] == "ckpt":
        s.update(x=_activations(g, c["rows"], c["cols"], c["dtype"]))
    elif c["op"] == "act_grad":
        width = c["cols"] * (2 if c["act"] == "swiglu" else 1)
        s.update(h=_activations(g, c["rows"], width, c["dtype"]),
                 d_out=(torch.randn(c["rows"], c["cols"], generator=g, device=DEVICE) * 1e-2).to(DTYPES[c["dtype"]]))
    else:
        T, k, O = c["tokens"], c["k"], c["outs"]
        if c["experts"] > 1:
            _, _, _, s["row_token"], s["offsets"] = _route(g, c)
        s.update(x=_activations(g, T, c["cols"], c["dtype"]),
                 dy=(torch.randn(T * k, O, generator=g, device=DEVICE) * 1e-2).to(DTYPES[c["dtype"]]))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, dev = s["op"], DEVICE
    if op == "dispatch":
        T, k, C = s["tokens"], s["k"], s["cols"]
        s.update(slot_row=torch.zeros(T, k, dtype=torch.int32, device=dev),
                 row_token=torch.zeros(T * k, dtype=torch.int32, device=dev),
                 offsets=torch.zeros(s["local"] + 1, dtype=torch.int32, device=dev),
                 rows=torch.zeros(T * k, C, dtype=s["x"].dtype, device=dev),
                 # one int32 per (tile of 1024 slots, expert) and one more tile
                 workspace=torch.zeros((-(-T * k // 1024) + 1) * s["local"] * 4 + 4096, dtype=torch.uint8, device=dev))
    elif op == "combine":
        s.update(out=torch.zeros(s["tokens"], s["cols"], dtype=s["rows"].dtype, device=dev))
    elif op == "combine_grad":
        s.update(d_rows=torch.zeros_like(s["rows"]), d_weights=torch.zeros_like(s["weights"]))
    elif op == "ckpt":
        s.update(data=torch.zeros(_bytes(s["rows"], s["cols"]), dtype=torch.uint8, device=dev),
                 out=torch.zeros_like(s["x"]))
    elif op == "act_grad":
        h = s.pop("h")
        s.update(data=_pack(*_quantise(h)), width=h.shape[1], d_in=torch.zeros_like(h))
    else:
        x = s.pop("x")
        E, n = s["experts"], s["outs"] * s["cols"]
        # the matrices of a flat grad buffer, another param of the same size after each
        s.update(data=_pack(*_quantise(x)), first=64, stride=2 * n, grad_offsets=[64 + 2 * n * e for e in range(E)],
                 grad_buffer=torch.zeros(64 + 2 * n * E, dtype=DTYPES[s["grad"]], device=dev),
                 workspace=torch.zeros(256 << 20, dtype=torch.uint8, device=dev))
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import zero_distributed_optimizer_gb300 as dopt

    op = s["op"]
    if op == "dispatch":
        dopt.dopt_route_sort(s["ids"], s["local"], s["slot_row"], s["row_token"], s["offsets"], s["workspace"])
        dopt.dopt_route_dispatch(s["x"], s["slot_row"], s["rows"])
        return dict(rows=s["rows"], slot_row=s["slot_row"], row_token=s["row_token"], offsets=s["offsets"])
    if op == "combine":
        dopt.dopt_route_combine(s["rows"], s["slot_row"], s["weights"], s["out"])
        return s["out"]
    if op == "combine_grad":
        dopt.dopt_route_combine_grad(s["d_out"], s["rows"], s["slot_row"], s["weights"], s["d_rows"], s["d_weights"])
        return dict(d_rows=s["d_rows"], d_weights=s["d_weights"])
    if op == "ckpt":
        kept = dopt.Checkpoint(s["data"], s["rows"], s["cols"], s["x"].dtype)
        dopt.dopt_ckpt_save(s["x"], kept)
        dopt.dopt_ckpt_load(kept, s["out"])
        return s["out"]
    if op == "act_grad":
        kept = dopt.Checkpoint(s["data"], s["rows"], s["width"], s["d_out"].dtype)
        dopt.dopt_ckpt_act_grad(kept, s["act"], s["d_out"], s["d_in"])
        return s["d_in"]
    kept = dopt.Checkpoint(s["data"], s["tokens"], s["cols"], s["dy"].dtype)
    dopt.dopt_ckpt_wgrad(kept, s["dy"], s["grad_buffer"], s["grad_offsets"], offsets=s.get("offsets"),
                         row_token=s.get("row_token"), workspace=s["workspace"])
    return s["grad_buffer"]


def _plain(s):
    op = s["op"]
    if op == "dispatch":
        slot_row, row_token, offsets = _sort(s["ids"], s["local"])
        rows = torch.where(row_token[:, None] >= 0, s["x"][row_token.clamp(min=0).long()], 0)
        return dict(rows=rows, slot_row=slot_row, row_token=row_token, offsets=offsets)
    if op == "combine":
        there = s["slot_row"] >= 0
        y = s["rows"][s["slot_row"].clamp(min=0).long()].float()
        return torch.where(there[..., None], s["weights"][..., None] * y, 0.0).sum(dim=1).to(s["rows"].dtype)
    if op == "combine_grad":
        slot_row, d = s["slot_row"], s["d_out"].float()
        there = slot_row >= 0
        at = slot_row.clamp(min=0).long()
        y = s["rows"][at].float()
        d_weights = torch.where(there, (y * d[:, None, :]).sum(dim=2), 0.0)
        d_rows = torch.zeros_like(s["rows"])
        d_rows[at[there]] = (s["weights"][..., None] * d[:, None, :])[there].to(d_rows.dtype)
        return dict(d_rows=d_rows, d_weights=d_weights)
    if op == "ckpt":
        return _values(*_quantise(s["x"]), s["cols"]).to(s["x"].dtype)
    if op == "act_grad":
        h = _values(*_unpack(s["data"], s["rows"], s["width"]), s["width"])
        d = s["d_out"].float()
        return _act_grad(s["act"], h, d).to(s["d_out"].dtype)
    x = _values(*_unpack(s["data"], s["tokens"], s["cols"]), s["cols"])
    dy, n = s["dy"].float(), s["outs"] * s["cols"]
    if s["experts"] == 1:
        w = (dy.t() @ x)[None]
    else:  # every expert's rows padded to the longest and multiplied in one batched product
        offsets = s["offsets"].long()
        row = offsets[:-1, None] + torch.arange(int((offsets[1:] - offsets[:-1]).max()), device=x.device)
        there = row < offsets[1:, None]
        row = torch.where(there, row, 0)
        token = s["row_token"][row].long()
        w = torch.where(there[..., None], dy[row], 0.0).transpose(1, 2) @ torch.where(there[..., None], x[token], 0.0)
    s["grad_buffer"][s["first"]:].view(s["experts"], s["stride"])[:, :n] = w.reshape(s["experts"], n).to(s["grad_buffer"].dtype)
    return s["grad_buffer"]


def _sort(ids, experts):
    """(row of each slot or -1, token of each row or -1, first row of each expert and the end), in slot order within an expert."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    sorted_key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(sorted_key, torch.arange(experts + 1, device=ids.device))
    row_of = torch.empty_like(order)
    row_of[order] = torch.arange(T * k, device=ids.device)
    slot_row = torch.where(key < experts, row_of, -1).view(T, k)
    row_token = torch.where(sorted_key < experts, order // k, -1)
    return slot_row.int(), row_token.int(), offsets.int()


def _pow2(e):
    """2.0**e in fp32, e a tensor of whole numbers in -126..127."""
    return ((e + 127).int() << 23).view(torch.float32)


def _quantise(x):
    """(codes int8 [rows, blocks, 32], exponent bytes [rows, blocks]) of a 2-D tensor."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    top = v.abs().amax(dim=2)
    fine = torch.isfinite(top)
    e = torch.frexp(torch.where(fine, top, 1.0)).exponent.int() - 7
    e = torch.where(top == 0, -126, e).clamp(min=-24 if x.dtype == torch.float16 else -126)
    codes = torch.round(v * _pow2(-e)[..., None]).clamp(-127, 127)
    return torch.where(fine[..., None], codes, 0.0).to(torch.int8), torch.where(fine, e + 127, 255).to(torch.uint8)


def _values(codes, scales, cols):
    """The fp32 values that codes and exponent bytes stand for, [rows, cols]."""
    step = torch.where(scales == 255, torch.nan, _pow2(scales.int() - 127))
    return (codes.float() * step[..., None]).flatten(1)[:, :cols]


def _pitch(cols):
    return -(-cols // PITCH) * PITCH


def _bytes(rows, cols):
    return rows * (_pitch(cols) + _pitch(cols) // BLOCK)


def _pack(codes, scales):
    """The one buffer that holds a checkpoint: every row's codes (padded with zeros to the pitch), then every row's bytes (padded with 1)."""
    rows, blocks = scales.shape
    pitch = _pitch(blocks * BLOCK)
    data = torch.zeros(rows, pitch, dtype=torch.int8, device=codes.device)
    data[:, :blocks * BLOCK] = codes.view(rows, -1)
    tail = torch.ones(rows, pitch // BLOCK, dtype=torch.uint8, device=codes.device)
    tail[:, :blocks] = scales
    return torch.cat([data.view(torch.uint8).reshape(-1), tail.reshape(-1)])


def _unpack(data, rows, cols):
    pitch = _pitch(cols)
    codes = data[:rows * pitch].view(torch.int8).view(rows, pitch // BLOCK, BLOCK)
    return codes, data[rows * pitch:].view(rows, pitch // BLOCK)


C_GELU, A_GELU = math.sqrt(2.0 / math.pi), 0.044715


def _act_grad(act, h, d):
    if act == "silu":
        s = torch.sigmoid(h)
        return d * (s * (1 + h * (1 - s)))
    if act == "gelu":
        t = torch.tanh(C_GELU * (h + A_GELU * h * h * h))
        return d * (0.5 * (1 + t) + 0.5 * h * (1 - t * t) * C_GELU * (1 + 3 * A_GELU * h * h))
    g, u = h.chunk(2, dim=1)
    s = torch.sigmoid(g)
    return torch.cat([d * u * (s * (1 + g * (1 - s))), d * (g * s)], dim=1)


def work(case):
    c = dict(case)
    op = c["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, C, b = c["tokens"], c["k"], c["cols"], SIZE[c["dtype"]]
        kept = T * k * c["local"] / c["experts"]
        if op == "dispatch":  # ids, tokens; sorted rows, slot and row indexes, expert offsets
            return dict(bytes=T * k * 8 + T * C * b + kept * C * b + T * k * 8 + 4 * c["local"], flops=0)
        if op == "combine":  # rows, weights, slot indexes; tokens
            return dict(bytes=kept * C * b + T * k * 8 + T * C * b, flops=2 * kept * C)
        # rows, the tokens' gradients, weights, slot indexes; the rows' gradients and the weights'
        return dict(bytes=2 * kept * C * b + T * C * b + T * k * 12, flops=3 * kept * C)
    if op == "ckpt":  # values in, codes and exponents out; the same back
        n, b = c["rows"] * c["cols"], SIZE[c["dtype"]]
        return dict(bytes=2 * n * b + 2 * n * (1 + 1 / BLOCK), flops=4 * n)
    if op == "act_grad":  # codes and exponents, the output's gradient; the input's
        n, b = c["rows"] * c["cols"], SIZE[c["dtype"]]
        wide = 2 if c["act"] == "swiglu" else 1
        return dict(bytes=n * wide * (1 + 1 / BLOCK) + n * b + n * wide * b, flops=20 * n)
    rows = c["tokens"] * c["k"]  # the rows' gradients, codes and exponents, row indexes; the weights' gradients
    return dict(bytes=rows * c["outs"] * SIZE[c["dtype"]] + c["tokens"] * c["cols"] * (1 + 1 / BLOCK)
                + (rows * 4 if c["experts"] > 1 else 0) + c["experts"] * c["outs"] * c["cols"] * SIZE[c["grad"]],
                flops=2 * rows * c["outs"] * c["cols"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _held64(x):
    """What a checkpoint of x stands for: whole multiples, at most 127, of a block's step 2**(floor(log2(largest)) - 6)."""
    rows, cols = x.shape
    v = x.double()
    out = torch.empty_like(v)
    least = -24 if x.dtype == torch.float16 else -126
    for c0 in range(0, cols, 4096):
        w = v[:, c0:c0 + 4096]
        short = -w.shape[1] % BLOCK
        w = torch.cat([w, w.new_zeros(rows, short)], dim=1).view(rows, -1, BLOCK)
        top = w.abs().max(dim=2, keepdim=True).values
        _, e = torch.frexp(top)
        step = torch.exp2((e.double() - 7).clamp(min=least))
        q = torch.round(w / step).clamp(-127, 127) * step
        out[:, c0:c0 + 4096] = q.view(rows, -1)[:, :v[:, c0:c0 + 4096].shape[1]]
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = s["op"]
    if op == "dispatch":
        ids, x = s["ids"].cpu().numpy().reshape(-1), s["x"].double()
        T, k, E = s["tokens"], s["k"], s["local"]
        slot_row, row_token = np.full(T * k, -1, np.int32), np.full(T * k, -1, np.int32)
        offsets, n = [0], 0
        for e in range(E):
            slots = np.flatnonzero(ids == e)
            slot_row[slots] = n + np.arange(len(slots))
            row_token[n:n + len(slots)] = slots // k
            n += len(slots)
            offsets.append(n)
        rows = torch.zeros(T * k, s["cols"], dtype=torch.float64, device=DEVICE)
        rows[:n] = x.index_select(0, torch.from_numpy(row_token[:n].astype(np.int64)).to(DEVICE))
        return dict(rows=rows, slot_row=slot_row.reshape(T, k), row_token=row_token, offsets=np.array(offsets, np.int32))
    if op in ("combine", "combine_grad"):
        there = s["slot_row"] >= 0
        token, choice = there.nonzero(as_tuple=True)
        row = s["slot_row"][there].long()
        w = s["weights"].double()[token, choice]
        if op == "combine":
            out = torch.zeros(s["tokens"], s["cols"], dtype=torch.float64, device=DEVICE)
            return out.index_add_(0, token, s["rows"].double()[row] * w[:, None])
        d = s["d_out"].double()[token]
        d_rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=DEVICE)
        d_rows[row] = d * w[:, None]
        d_weights = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEVICE)
        d_weights[token, choice] = torch.einsum("nc,nc->n", d, s["rows"].double()[row])
        return dict(d_rows=d_rows, d_weights=d_weights)
    if op == "ckpt":
        return _held64(s["x"])
    if op == "act_grad":
        h, d = _held64(s["h"]), s["d_out"].double()
        if s["act"] == "gelu":
            u = C_GELU * (h + A_GELU * h ** 3)
            return d * (0.5 + 0.5 * torch.tanh(u) + 0.5 * h / torch.cosh(u) ** 2 * C_GELU * (1 + 3 * A_GELU * h ** 2))
        n = s["cols"]
        g, up = (h, 1.0) if s["act"] == "silu" else (h[:, :n], h[:, n:])
        slope = (1 + torch.exp(-g) * (1 + g)) / (1 + torch.exp(-g)) ** 2
        return d * slope if s["act"] == "silu" else torch.cat([d * up * slope, d * g / (1 + torch.exp(-g))], dim=1)
    x, n = _held64(s["x"]), s["outs"] * s["cols"]
    out = torch.zeros(64 + 2 * n * s["experts"], dtype=torch.float64, device=DEVICE)
    bounds = s["offsets"].tolist() if s["experts"] > 1 else [0, s["tokens"]]
    for e in range(s["experts"]):
        dy = s["dy"][bounds[e]:bounds[e + 1]].double()
        xe = x if s["experts"] == 1 else x[s["row_token"][bounds[e]:bounds[e + 1]].long()]
        out[64 + 2 * n * e:64 + 2 * n * e + n] = torch.mm(dy.t(), xe).reshape(-1)
    return out
