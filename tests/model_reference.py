"""Plain 64-bit forms of the operators of a language model's ends and residual
stream (torch on the CPU), written from their definitions."""
import torch


def f64(t):
    return None if t is None else t.detach().cpu().double()


def embed(table, ids, scale):
    """scale * table[ids], zeros for ids outside."""
    table, ids = f64(table), ids.cpu().long()
    out = torch.zeros(len(ids), table.shape[1], dtype=torch.float64)
    for t, i in enumerate(ids.tolist()):
        if 0 <= i < len(table):
            out[t] = scale * table[i]
    return out


def embed_grad(ids, d_out, vocab, scale):
    """(the table's gradient, the sums of magnitudes that it is made of, tokens of each row)."""
    d = f64(d_out)
    grad = torch.zeros(vocab, d.shape[1], dtype=torch.float64)
    size, count = torch.zeros_like(grad), torch.zeros(vocab, dtype=torch.int64)
    for t, i in enumerate(ids.cpu().tolist()):
        if 0 <= i < vocab:
            grad[i] += scale * d[t]
            size[i] += abs(scale) * d[t].abs()
            count[i] += 1
    return grad, size, count


def hat(v, kind, eps):
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    return v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)


def affine(v, weight, bias):
    v = v if weight is None else v * weight
    return v if bias is None else v + bias


def branch(kind, y, post, post_weight, post_bias, gate, row_gate, scale, eps):
    """What a block adds to the residual; all arguments in 64 bits."""
    u = affine(hat(y, kind, eps), post_weight, post_bias) if post else y
    u = u if gate is None else u * gate
    return scale * (u if row_gate is None else u * row_gate[:, None])


def norm(kind, x, weight=None, bias=None, y=None, post=False, post_weight=None, post_bias=None, gate=None,
         row_gate=None, scale=1.0, eps=1e-5):
    """(h, n)."""
    h = x if y is None else x + branch(kind, y, post, post_weight, post_bias, gate, row_gate, scale, eps)
    return h, affine(hat(h, kind, eps), weight, bias)


def head(x, weight, targets):
    """(loss, lse, logits) of every row; the loss is 0 where the target is outside."""
    logits = f64(x) @ f64(weight).t()
    lse = torch.logsumexp(logits, dim=1)
    t = targets.cpu().long()
    there = (t >= 0) & (t < logits.shape[1])
    at = logits.gather(1, torch.where(there, t, 0)[:, None])[:, 0]
    return torch.where(there, lse - at, torch.zeros_like(lse)), lse, logits


def head_grad(x, weight, targets, lse, d_loss, d_lse=None):
    """(d_x, d_weight, d_logits) from the given lse."""
    x, w = f64(x), f64(weight)
    t = targets.cpu().long()
    there = ((t >= 0) & (t < len(w))).double()
    dl = f64(d_loss) * there
    d = torch.exp(x @ w.t() - f64(lse)[:, None]) * (dl + (0.0 if d_lse is None else f64(d_lse)))[:, None]
    rows = torch.arange(len(t))
    d[rows, torch.where(there > 0, t, torch.zeros_like(t))] -= dl
    return d @ w, d.t() @ x, d
