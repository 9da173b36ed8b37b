"""The embedding, the head's loss and clipping in float64 (torch, CPU), each with a bound on
what fp32 arithmetic in the kernels' order may be off by.  U = 2^-24 is half a step of fp32.

Sums of n terms s_i in fp32 in any order are off by at most (n - 1) U sum|s_i| to first order;
CHAIN(n) below is that n, with a few more for the products and scalings around the sum."""
from __future__ import annotations

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}   # half the least step


def rounded(value, bound, dtype):
    """The bound after one rounding to dtype."""
    return bound + HALF[dtype] * (value.abs() + bound) + TINY[dtype]


def embedding(ids, weight, scale, dtype):
    """(y, bound): one fp32 product, one rounding."""
    V = weight.shape[0]
    inside = (ids >= 0) & (ids < V)
    y = torch.zeros(len(ids), weight.shape[1], dtype=torch.float64)
    y[inside] = scale * weight.double()[ids[inside].long()]
    return y, rounded(y, U * y.abs(), dtype)


def embedding_backward(ids, dy, vocab, scale, dtype, before=None):
    """(dweight, bound): a sum of as many terms as the token occurs, scaled; `before` added."""
    inside = (ids >= 0) & (ids < vocab)
    at, d = ids[inside].long(), dy.double()[inside]
    zero = torch.zeros(vocab, dy.shape[1], dtype=torch.float64)
    dw = scale * zero.index_add(0, at, d)
    size = abs(scale) * zero.index_add(0, at, d.abs())
    n = torch.bincount(at, minlength=vocab).double()[:, None]
    bound = (n + 2) * U * size
    if before is not None:
        dw = dw + before.double()
        bound = bound + U * dw.abs()
        return dw, torch.where(n > 0, rounded(dw, bound, dtype), 0.0)
    return dw, torch.where(n > 0, rounded(dw, bound, dtype), 0.0)


def head(x, weight, targets, logit_scale, dloss=None, dlse=None):
    """{name: (value, bound)} of loss and lse, and of dx and dweight where dloss is given.

    Logits: D products and their sum; products are exact for 2-byte types, and sums of six partial
    products in fp32, which leave out three, of less than 2^-22, 2^-22 and 2^-30: 8 U of the
    product's size in all.  The scaling to log2 units and the exponential (2 U of the argument's
    size each, 4 U relative); the sum over the vocabulary is a sum of V positive terms in runs of
    at most 64 a lane and a tree or a walk over the runs: fewer than 96 + V / 64 additions deep.
    dl is rounded once to the operands' type; its products are summed over V (dx) or M (dweight)."""
    t = x.dtype
    x, w = x.double(), weight.double()
    (M, D), V = x.shape, w.shape[0]
    inside = (targets >= 0) & (targets < V)
    at = targets.clamp(0, V - 1).long()[:, None]
    logits = logit_scale * (x @ w.t())
    off = (D + 12) * U * abs(logit_scale) * (x.abs() @ w.abs().t()) + 4 * U * logits.abs()
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - lse[:, None])
    # a logit's error moves lse by p times it
    off_lse = (p * off).sum(1) + (96 + V / 64 + 8) * U + 6 * U * (lse.abs() + logits.abs().max(1).values)
    loss = torch.where(inside, lse - logits.gather(1, at)[:, 0], 0.0)
    off_loss = torch.where(inside, off_lse + off.gather(1, at)[:, 0] + 2 * U * loss.abs(), 0.0)
    out = dict(loss=(loss, off_loss), lse=(lse, off_lse))
    if dloss is None:
        return out
    own = torch.where(inside, dloss.double(), 0.0)[:, None]
    both = own if dlse is None else own + torch.where(inside, dlse.double(), 0.0)[:, None]
    hot = torch.zeros_like(p).scatter_(1, at, 1.0) * inside[:, None]
    dl = both * p - own * hot
    # the exponent's error makes a relative one of p; then the subtraction, then one rounding.
    # What is held is dl times a scale that brings the largest |dloss| + |dlse| to 2^13
    # or just below.
    rel = off + off_lse[:, None] + 8 * U * (1 + logits.abs() + lse.abs()[:, None])
    # v_exp_f32 gives 0 where its result is below the normal numbers: 2^-126 off in p
    e = both.abs() * (p * rel + 2.0 ** -126) + 4 * U * (both.abs() * p + own.abs() * hot)
    top = (own.abs() + (both - own).abs()).max() if M else 0.0
    e = e + HALF[t] * (dl.abs() + e) + TINY[t] * top / 2.0 ** 12
    x = torch.where(inside[:, None], x, 0.0)
    dx, dw = logit_scale * (dl @ w), logit_scale * (dl.t() @ x)
    size_x, size_w = abs(logit_scale) * (dl.abs() @ w.abs()), abs(logit_scale) * (dl.abs().t() @ x.abs())
    off_x = abs(logit_scale) * (e @ w.abs()) + (V + 28) * U * size_x
    off_w = abs(logit_scale) * (e.t() @ x.abs()) + (M + 12) * U * size_w
    return dict(out, dx=(dx, rounded(dx, off_x, t)), dweight=(dw, rounded(dw, off_w, t)))


def clip(grads, max_norm, scale, dtypes):
    """(norm, bound), [(out, bound)]: squares and sums in fp64, so the norm is off by its rounding
    and the factor by one more; each value by a product and its rounding."""
    square = sum(float((g.double() ** 2).sum()) for g in grads)
    norm = scale * square ** 0.5
    if not norm < float("inf"):
        return (norm, 0.0), [(g.double(), torch.zeros_like(g, dtype=torch.float64)) for g in grads]
    factor = scale * (max_norm / norm if norm > max_norm else 1.0)
    outs = []
    for g, t in zip(grads, dtypes):
        v = g.double() * factor
        outs.append((v, rounded(v, 3 * U * v.abs(), t)))
    return (norm, 2 * U * norm), outs
