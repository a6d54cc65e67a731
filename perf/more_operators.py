"""Workloads for the operators at the two ends of a language model and on its residual stream: the token
embedding with its gradient, the norms around a block fused with the block's gates and residual scale, and the
cross entropy of the output matrix's logits, which are never kept.  Gradients of params go into a flat buffer.

`listed` and `draw` give the cases, `prepare` makes a case's inputs on the GPU, `run` takes one pass through
an operator and `exact` gives its result in 64 bits.  With `own` the passes are calls of the package;
without, they are the operators' formulas in elementary torch operations in fp32.

Terms: ids and targets outside [0, vocab) count as nothing (padding, an ignored target, another rank's share
of the vocabulary).  A block's branch is scale * row_gate[t] * gate[c] * post(y)[t, c], h the residual with the
branch added, n the next norm of h; gates and the norm after the block (`post`) may be left out.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5
FIRST = 64  # where the params' gradients start in their flat buffer


def listed():
    return [
        # the embeddings of a handful of sequences' next tokens: launch latency counts
        dict(name="embed_few", op="embed", tokens=24, vocab=32000, cols=2048, dtype="bf16", scale=1.0, share=1),
        # one microbatch's tokens through GPT-2 small's table, scaled
        dict(name="embed_train", op="embed", tokens=16384, vocab=50257, cols=768, dtype="bf16", scale=27.7, share=1),
        # one rank's third of a small vocabulary; an odd width, so that no row is aligned
        dict(name="embed_grad_odd", op="embed_grad", tokens=1001, vocab=5003, cols=515, dtype="fp32", grad="fp32", scale=0.5, share=3),
        # the gradient of embed_train's table
        dict(name="embed_grad_train", op="embed_grad", tokens=16384, vocab=50257, cols=768, dtype="bf16", grad="bf16", scale=27.7, share=1),
        # a layer norm after a gated branch, ragged rows
        dict(name="norm_odd", op="norm", kind="layer", rows=1001, cols=515, dtype="fp16", post=False, gate=True, row_gate=True),
        # the norms around a block of a Llama-1.3B layer, 16384 tokens
        dict(name="norm_train", op="norm", kind="rms", rows=16384, cols=2048, dtype="bf16", post=True, gate=True, row_gate=False),
        # gradients of two layer norms with every gate, ragged rows
        dict(name="norm_grad_odd", op="norm_grad", kind="layer", rows=333, cols=1001, dtype="fp32", grad="fp32", post=True, gate=True, row_gate=True),
        # gradients of norm_train
        dict(name="norm_grad_train", op="norm_grad", kind="rms", rows=16384, cols=2048, dtype="bf16", grad="bf16", post=True, gate=True, row_gate=False),
        # the loss of a few tokens: reading the output matrix is all there is
        dict(name="head_loss_few", op="head_loss", rows=24, width=2048, vocab=32000, dtype="bf16"),
        # the loss of one microbatch of GPT-2 small
        dict(name="head_loss_train", op="head_loss", rows=16384, width=768, vocab=50257, dtype="bf16"),
        # odd sizes everywhere, fp32 gradients, a penalty on the logits' scale
        dict(name="head_grad_odd", op="head_grad", rows=1001, width=515, vocab=5003, dtype="fp16", grad="fp32", z=1e-3),
        # the gradients of head_loss_train
        dict(name="head_grad_train", op="head_grad", rows=16384, width=768, vocab=50257, dtype="bf16", grad="bf16", z=0.0),
    ]


def _size(rng, lo, hi, unit=64):
    """A size spread over [lo, hi]'s logarithm; half of them multiples of `unit`."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        n = -(-n // unit) * unit
    return max(lo, min(hi, n))


def draw(rng):
    while True:
        op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "head_loss", "head_grad"])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if op in ("embed", "embed_grad"):
            c = dict(op=op, tokens=_size(rng, 1, 32768), vocab=_size(rng, 128, 131072), cols=_size(rng, 64, 4096), dtype=dtype,
                     scale=rng.choice([1.0, 0.125, 27.7]), share=rng.choice([1, 1, 3]))
            if op == "embed_grad":
                c["grad"] = rng.choice([dtype, "fp32"])
            if c["tokens"] < 32:
                c["share"] = 1
            if (c["tokens"] * c["cols"] * SIZE[dtype] <= 32768 * 2048 * 2
                    and c["vocab"] * c["cols"] * SIZE[c.get("grad", dtype)] <= 131072 * 1024 * 2):
                return c
        elif op in ("norm", "norm_grad"):
            c = dict(op=op, kind=rng.choice(["rms", "layer"]), rows=_size(rng, 1, 32768), cols=_size(rng, 32, 8192), dtype=dtype,
                     post=rng.random() < 0.5, gate=rng.random() < 0.5, row_gate=rng.random() < 0.3)
            if op == "norm_grad":
                c["grad"] = rng.choice([dtype, "fp32"])
            if c["rows"] * c["cols"] * SIZE[dtype] <= 16384 * 2048 * 2:
                return c
        else:
            dtype = rng.choice(["bf16", "fp16"])
            c = dict(op=op, rows=_size(rng, 1, 32768), width=_size(rng, 64, 4096), vocab=_size(rng, 128, 131072), dtype=dtype)
            if op == "head_grad":
                c.update(grad=rng.choice([dtype, "fp32"]), z=rng.choice([0.0, 1e-3]))
            if (c["rows"] * c["vocab"] * c["width"] <= 16384 * 50257 * 768 and c["rows"] * c["vocab"] <= 16384 * 50257
                    and c["vocab"] * c["width"] <= 50257 * 1024):
                return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _tokens(g, n, vocab, nothing=0.0):
    """Ids as text has them, the most frequent first (frequency about 1 / rank); a part of them -100, which counts as nothing."""
    u = torch.rand(n, generator=g, device=DEVICE, dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)
    return torch.where(torch.rand(n, generator=g, device=DEVICE) < nothing, -100, ids) if nothing else ids


def _normal(g, *shape, size=1.0):
    return torch.randn(*shape, generator=g, device=DEVICE) * size


def _stream(g, rows, cols, dtype):
    """Normal values whose columns differ in size, a few of them much larger, as a residual stream has them."""
    x = _normal(g, rows, cols) * torch.exp(0.3 * _normal(g, cols))
    return (x * torch.where(torch.rand(cols, generator=g, device=DEVICE) < 0.005, 10.0, 1.0)).to(DTYPES[dtype])


def _inputs(case, seed):
    s = dict(case)
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 6971 + 29)
    op, dt = s["op"], DTYPES[s["dtype"]]
    if op in ("embed", "embed_grad"):
        T, V, C = s["tokens"], s["vocab"], s["cols"]
        # ids of the whole vocabulary, of which this table holds one part in `share`: the others fall outside
        ids = _tokens(g, T, V * s["share"])
        s["ids"] = torch.where(ids % s["share"] == 0, ids // s["share"], -1 - ids)
        if op == "embed":
            s["table"] = _normal(g, V, C, size=0.05).to(dt)
        else:
            s["d_out"] = _normal(g, T, C, size=1e-2).to(dt)
    elif op in ("norm", "norm_grad"):
        T, C = s["rows"], s["cols"]
        s["y"] = (0.5 * _stream(g, T, C, "fp32") + 0.1).to(dt)
        s["weight"], s["post_weight"] = (1 + _normal(g, C, size=0.1)).to(dt), (1 + _normal(g, C, size=0.1)).to(dt)
        s["bias"], s["post_bias"] = _normal(g, C, size=0.1).to(dt), _normal(g, C, size=0.1).to(dt)
        if s["kind"] == "rms":
            s["bias"] = s["post_bias"] = None
        if not s["post"]:
            s["post_weight"] = s["post_bias"] = None
        s["gate"] = (0.7 + _normal(g, C, size=0.2)).to(dt) if s["gate"] else None
        s["row_gate"] = torch.sigmoid(_normal(g, T)) if s["row_gate"] else None
        s["scale"] = 0.75
        s["x" if op == "norm" else "h"] = _stream(g, T, C, s["dtype"])
        if op == "norm_grad":
            s["d_n"], s["d_h"] = _normal(g, T, C, size=1e-2).to(dt), _normal(g, T, C, size=1e-2).to(dt)
    else:
        T, H, V = s["rows"], s["width"], s["vocab"]
        s["x"] = _normal(g, T, H).to(dt)
        s["weight"] = _normal(g, V, H, size=2.0 / math.sqrt(H)).to(dt)  # logits of about +-2, the target's raised
        s["targets"] = _tokens(g, T, V, nothing=0.05 if T >= 32 else 0.0)
        there = (s["targets"] >= 0)[:, None]
        s["x"] = (s["x"].float() + torch.where(there, s["weight"][s["targets"].clamp(min=0)].float(), 0.0)).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = s["op"]
    if op == "embed":
        s["out"] = torch.zeros(s["tokens"], s["cols"], dtype=s["table"].dtype, device=DEVICE)
    elif op == "embed_grad":
        n, T = s["vocab"] * s["cols"], s["tokens"]
        s["grad_buffer"] = torch.zeros(FIRST + n + 64, dtype=DTYPES[s["grad"]], device=DEVICE)
        # the sorted tokens, a few words a row of the table, and fp32 sums of parts of long runs
        s["workspace"] = _workspace(64 * T + 16 * s["vocab"] + T * s["cols"] + (1 << 20))
    elif op == "norm":
        s.update(h=torch.zeros_like(s["x"]), n=torch.zeros_like(s["x"]))
    elif op == "norm_grad":
        C, h = s["cols"], s["h"]
        s.update(d_x=torch.zeros_like(h), d_y=torch.zeros_like(h), d_row_gate=torch.zeros(s["rows"], device=DEVICE),
                 # five params' gradients, another param of the same size after each
                 grad_buffer=torch.zeros(FIRST + 10 * C, dtype=DTYPES[s["grad"]], device=DEVICE),
                 workspace=_workspace(1024 * 4 * C * 4 + (1 << 20)))
    else:
        T, H, V = s["rows"], s["width"], s["vocab"]
        s["lse"] = torch.zeros(T, device=DEVICE)
        aligned = 2 * (T + V) * (H + 64)  # copies with aligned rows, where rows are not
        if op == "head_loss":
            s["loss"] = torch.zeros(T, device=DEVICE)
            s["workspace"] = _workspace(aligned + 8 * (T + 256) * (V // 128 + 2) + (1 << 20))
        else:
            s["lse"] = torch.logsumexp(s["x"].float() @ s["weight"].float().t(), dim=1)
            there = s["targets"] >= 0
            # a mean over the targets that count, scaled where fp16 gradients would be too small
            weight = torch.where(there, 4096.0 if s["dtype"] == "fp16" else 1.0, 0.0) / there.sum().clamp(min=1)
            s["d_loss"] = weight
            s["d_lse"] = 2 * s["z"] * s["lse"] * weight if s["z"] else None
            planes = 2 if s["grad"] == "fp32" else 1
            s.update(d_x=torch.zeros_like(s["x"]), grad_buffer=torch.zeros(FIRST + V * H + 64, dtype=DTYPES[s["grad"]], device=DEVICE),
                     workspace=_workspace(aligned + 2 * planes * (T + 256) * (V + 256) + (512 << 20)))
    return s


def _workspace(n):
    return torch.empty(n, dtype=torch.uint8, device=DEVICE)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import zero_distributed_optimizer_gb300 as dopt

    op = s["op"]
    if op == "embed":
        dopt.dopt_embed(s["table"], s["ids"], s["out"], scale=s["scale"])
        return s["out"]
    if op == "embed_grad":
        dopt.dopt_embed_grad(s["ids"], s["d_out"], s["grad_buffer"], FIRST, s["vocab"], scale=s["scale"], workspace=s["workspace"])
        return s["grad_buffer"]
    if op == "norm":
        dopt.dopt_norm(s["kind"], s["x"], s["n"], weight=s["weight"], bias=s["bias"], y=s["y"], h=s["h"],
                       post=s["post"], post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"],
                       row_gate=s["row_gate"], scale=s["scale"], eps=EPS)
        return dict(h=s["h"], n=s["n"])
    if op == "norm_grad":
        C = s["cols"]
        at = {name: FIRST + 2 * C * i for i, name in enumerate(PARAMS) if s[name] is not None}
        gated = s["row_gate"] is not None
        dopt.dopt_norm_grad(s["kind"], s["h"], s["d_n"], s["d_x"], weight=s["weight"], y=s["y"], d_y=s["d_y"], d_h=s["d_h"],
                            post=s["post"], post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"],
                            row_gate=s["row_gate"], scale=s["scale"], eps=EPS, d_row_gate=s["d_row_gate"] if gated else None,
                            grad=s["grad_buffer"], grad_offsets=at, workspace=s["workspace"])
        return dict(d_x=s["d_x"], d_y=s["d_y"], grad=s["grad_buffer"], d_row_gate=s["d_row_gate"])
    if op == "head_loss":
        dopt.dopt_head_loss(s["x"], s["weight"], s["targets"], s["loss"], s["lse"], workspace=s["workspace"])
        return dict(loss=s["loss"], lse=s["lse"])
    dopt.dopt_head_loss_grad(s["x"], s["weight"], s["targets"], s["lse"], s["d_loss"], s["d_x"], s["grad_buffer"], FIRST,
                             d_lse=s["d_lse"], workspace=s["workspace"])
    return dict(d_x=s["d_x"], grad=s["grad_buffer"])


PARAMS = ("weight", "bias", "post_weight", "post_bias", "gate")


def _plain(s):
    op = s["op"]
    if op == "embed":
        there = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
        rows = s["table"][torch.where(there, s["ids"], 0)].float() * s["scale"]
        return torch.where(there[:, None], rows, 0.0).to(s["table"].dtype)
    if op == "embed_grad":
        there = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
        d = torch.zeros(s["vocab"], s["cols"], device=DEVICE)
        d.index_add_(0, torch.where(there, s["ids"], 0), torch.where(there[:, None], s["d_out"].float(), 0.0))
        return _put(s["grad_buffer"], FIRST, d * s["scale"])
    if op == "norm":
        u = _normed(s["y"].float(), s["kind"], s["post_weight"], s["post_bias"]) if s["post"] else s["y"].float()
        h = s["x"].float() + u * _branch(s)
        n = _normed(h, s["kind"], s["weight"], s["bias"])
        return dict(h=h.to(s["x"].dtype), n=n.to(s["x"].dtype))
    if op == "norm_grad":
        h, y, d_n, dt = s["h"].float(), s["y"].float(), s["d_n"].float(), s["h"].dtype
        hat, r = _standard(h, s["kind"])
        d_x = s["d_h"].float() + _back(d_n * s["weight"].float(), hat, r, s["kind"])
        y_hat, y_r = _standard(y, s["kind"]) if s["post"] else (y, None)
        u = y_hat
        if s["post_weight"] is not None:
            u = u * s["post_weight"].float() + (s["post_bias"].float() if s["post_bias"] is not None else 0.0)
        d_u = d_x * _branch(s)
        d_hat = d_u if s["post_weight"] is None else d_u * s["post_weight"].float()
        d_y = _back(d_hat, y_hat, y_r, s["kind"]) if s["post"] else d_hat
        gate = 1.0 if s["gate"] is None else s["gate"].float()
        row = s["scale"] if s["row_gate"] is None else s["scale"] * s["row_gate"][:, None]
        wide = {"weight": d_n * hat, "bias": d_n, "post_weight": d_u * y_hat, "post_bias": d_u, "gate": d_x * u * row}
        _put_params(s, {name: wide[name].sum(dim=0) for name in PARAMS if s[name] is not None})
        if s["row_gate"] is not None:
            s["d_row_gate"].copy_((d_x * u * gate).sum(dim=1) * s["scale"])
        return dict(d_x=d_x.to(dt), d_y=d_y.to(dt), grad=s["grad_buffer"], d_row_gate=s["d_row_gate"])
    x, w = s["x"].float(), s["weight"].float()
    there = (s["targets"] >= 0) & (s["targets"] < s["vocab"])
    target = torch.where(there, s["targets"], 0)[:, None]
    logits = x @ w.t()
    if op == "head_loss":
        top = logits.amax(dim=1, keepdim=True)
        lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(dim=1))
        return dict(loss=torch.where(there, lse - logits.gather(1, target)[:, 0], 0.0), lse=lse)
    at_target = torch.where(there, s["d_loss"], 0.0)
    d = torch.exp(logits - s["lse"][:, None]) * (at_target + (0.0 if s["d_lse"] is None else s["d_lse"]))[:, None]
    d.scatter_add_(1, target, -at_target[:, None])
    return dict(d_x=(d @ w).to(s["x"].dtype), grad=_put(s["grad_buffer"], FIRST, d.t() @ x))


def _put(buffer, at, values):
    buffer[at:at + values.numel()] = values.reshape(-1).to(buffer.dtype)
    return buffer


def _put_params(s, found):
    return [_put(s["grad_buffer"], FIRST + 2 * s["cols"] * i, found[name]) for i, name in enumerate(PARAMS) if name in found]


def _branch(s):
    """What the branch is multiplied by, [rows or 1, cols or 1]."""
    by = torch.full((1, 1), s["scale"], device=DEVICE)
    by = by if s["gate"] is None else by * s["gate"].float()[None]
    return by if s["row_gate"] is None else by * s["row_gate"][:, None]


def _standard(v, kind):
    """(rows of mean square 1, and for a layer norm of mean 0; the factors that made them so)."""
    v = v if kind == "rms" else v - v.mean(dim=1, keepdim=True)
    r = torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)
    return v * r, r


def _normed(v, kind, weight, bias):
    v = _standard(v, kind)[0]
    v = v if weight is None else v * weight.float()
    return v if bias is None else v + bias.float()


def _back(d, hat, r, kind):
    """The gradient of _standard's input from its output's."""
    d = d - hat * (d * hat).mean(dim=1, keepdim=True)
    return r * (d if kind == "rms" else d - d.mean(dim=1, keepdim=True))


def work(case):
    c = dict(case)
    op, b = c["op"], SIZE[c["dtype"]]
    if op in ("embed", "embed_grad"):
        T, V, C = c["tokens"], c["vocab"], c["cols"]
        kept = T / c["share"]
        if op == "embed":  # ids, the rows that are there; tokens
            return dict(bytes=8 * T + min(kept, V) * C * b + T * C * b, flops=T * C)
        return dict(bytes=8 * T + kept * C * b + V * C * SIZE[c["grad"]], flops=kept * C + V * C)
    if op in ("norm", "norm_grad"):
        n, gated = c["rows"] * c["cols"], 4 * c["rows"] if c["row_gate"] else 0
        if op == "norm":  # x, y; h, n
            return dict(bytes=4 * n * b + gated + 5 * c["cols"] * b, flops=16 * n)
        # h, y, the gradients of n and h; of x, y and the params
        return dict(bytes=6 * n * b + 2 * gated + 5 * c["cols"] * (b + SIZE[c["grad"]]), flops=30 * n)
    T, H, V = c["rows"], c["width"], c["vocab"]
    if op == "head_loss":  # tokens, the matrix, targets; loss and lse
        return dict(bytes=(T + V) * H * b + 16 * T, flops=2 * T * V * H)
    # tokens, the matrix, targets, three numbers a row; gradients.  Logits are computed again: three products
    return dict(bytes=(2 * T + V) * H * b + 20 * T + V * H * SIZE[c["grad"]], flops=6 * T * V * H)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f64 = torch.float64
    if op == "embed":
        out = torch.zeros(s["tokens"], s["cols"], dtype=f64, device=DEVICE)
        t = ((s["ids"] >= 0) & (s["ids"] < s["vocab"])).nonzero()[:, 0]
        out[t] = s["table"].index_select(0, s["ids"][t]).double() * s["scale"]
        return out
    if op == "embed_grad":
        out = torch.zeros(s["grad_buffer"].numel(), dtype=f64, device=DEVICE)
        rows = out[FIRST:FIRST + s["vocab"] * s["cols"]].view(s["vocab"], s["cols"])
        t = ((s["ids"] >= 0) & (s["ids"] < s["vocab"])).nonzero()[:, 0]
        rows.index_add_(0, s["ids"][t], s["d_out"][t].double(), alpha=s["scale"])
        return out
    if op in ("norm", "norm_grad"):
        return _exact_norm(s, op)
    T, H, V = s["rows"], s["width"], s["vocab"]
    w = s["weight"].double()
    loss, lse, d_x = (torch.zeros(n, dtype=f64, device=DEVICE) for n in (T, T, (T, H)))
    grad = torch.zeros(s["grad_buffer"].numel() if op == "head_grad" else 0, dtype=f64, device=DEVICE)
    d_w = grad[FIRST:FIRST + V * H].view(V, H) if op == "head_grad" else None
    for t0 in range(0, T, 4096):
        at = slice(t0, t0 + 4096)
        x, target = s["x"][at].double(), s["targets"][at]
        logits = torch.mm(x, w.t())
        row = (target >= 0).nonzero()[:, 0]
        if op == "head_loss":
            lse[at] = torch.logsumexp(logits, dim=1)
            loss[at][row] = lse[at][row] - logits[row, target[row]]
            continue
        d = (logits - s["lse"][at].double()[:, None]).exp_()
        both = torch.zeros(len(target), dtype=f64, device=DEVICE)
        both[row] = s["d_loss"][at].double()[row]
        if s["d_lse"] is not None:
            both += s["d_lse"][at].double()
        d *= both[:, None]
        d[row, target[row]] -= s["d_loss"][at].double()[row]
        d_x[at] = torch.mm(d, w)
        d_w += torch.mm(d.t(), x)
    return dict(loss=loss, lse=lse) if op == "head_loss" else dict(d_x=d_x, grad=grad)


def _exact_norm(s, op):
    """From torch's automatic differentiation of the forward formula, in 64 bits."""
    given = {k: s[k].double().requires_grad_() for k in PARAMS + ("y", "row_gate") if s[k] is not None}

    def norm(v, weight, bias):
        if s["kind"] == "layer":
            v = v - torch.sum(v, dim=1, keepdim=True) / s["cols"]
        v = v / torch.sqrt(torch.sum(v ** 2, dim=1, keepdim=True) / s["cols"] + EPS)
        v = v if weight is None else weight * v
        return v if bias is None else v + bias

    u = given["y"]
    if s["post"]:
        u = norm(u, given.get("post_weight"), given.get("post_bias"))
    if "gate" in given:
        u = u * given["gate"]
    if "row_gate" in given:
        u = u * given["row_gate"][:, None]
    u = s["scale"] * u
    if op == "norm":
        h = s["x"].double() + u
        return dict(h=h.detach(), n=norm(h, given["weight"], given.get("bias")).detach())
    h = s["h"].double().requires_grad_()  # the residual as it was kept
    wanted = [k for k in PARAMS if k in given]
    first = torch.autograd.grad(norm(h, given["weight"], given.get("bias")), [h] + [given[k] for k in ("weight", "bias") if k in given],
                                s["d_n"].double())
    d_x = s["d_h"].double() + first[0]
    found = dict(zip([k for k in ("weight", "bias") if k in given], first[1:]))
    rest = [k for k in ("post_weight", "post_bias", "gate", "y", "row_gate") if k in given]
    found.update(zip(rest, torch.autograd.grad(u, [given[k] for k in rest], d_x)))
    grad = torch.zeros(s["grad_buffer"].numel(), dtype=torch.float64, device=DEVICE)
    for i, name in enumerate(PARAMS):
        if name in wanted:
            grad[FIRST + 2 * s["cols"] * i:FIRST + 2 * s["cols"] * i + s["cols"]] = found[name]
    return dict(d_x=d_x, d_y=found["y"], grad=grad, d_row_gate=found.get("row_gate", torch.zeros(s["rows"], dtype=torch.float64, device=DEVICE)))
