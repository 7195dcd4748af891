"""Plain 64-bit forms of the AdamW lane's layers, with bounds on how far an
fp32 evaluation that rounds its outputs once may be from them.

u = 2^-24 is half a step of fp32; half(t) is half a step of an output type
(bf16 2^-8).  A sum of n terms t_i whose additions form a tree of depth h is
off by at most h u sum |t_i| to first order; the bounds below carry an extra
1 % for the second order.
"""
import torch

U = 2.0 ** -24
SECOND = 1.01


def half(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, bound):
    """Every element of got within bound of want (and finite where want is)."""
    got = got.double()
    assert got.shape == want.shape, (got.shape, want.shape)
    assert torch.isfinite(got).all()
    excess = (got - want).abs() - bound * SECOND
    worst = excess.max().item() if excess.numel() else -1.0
    assert worst <= 0, (worst, (got - want).abs().max().item())


# ---- embedding -----------------------------------------------------------------


def embedding(tokens, table, scale):
    return table.double()[tokens] * scale


def embedding_bound(want, out_dtype):
    # one fp32 product, one rounding of the result
    return want.abs() * (U + half(out_dtype))


def embedding_grad(tokens, grad, vocab, scale, padding):
    """(gradient, bound of its error without the final rounding)."""
    t, g = tokens.reshape(-1), grad.reshape(-1, grad.shape[-1]).double()
    keep = (t >= 0) & (t < vocab)
    if padding is not None:
        keep &= t != padding
    t, g = t[keep].long(), g[keep]
    d = torch.zeros(vocab, g.shape[-1], dtype=torch.float64, device=g.device).index_add_(0, t, g)
    a = torch.zeros_like(d).index_add_(0, t, g.abs())
    n = torch.bincount(t, minlength=vocab).double()[:, None]
    # no tree over n terms is deeper than n - 1; the scale's product is one more
    return d * scale, a * abs(scale) * n * U


# ---- LayerNorm -----------------------------------------------------------------


def sum_depth(dim):
    """Additions between an element and the row's sum: up to 32 in a thread, 5
    in a warp, 16 over warps; wider rows: dim / 1024 in a thread, 5, 32."""
    return 53 if dim <= 16384 else dim / 1024 + 40


def norm(x, w, b, eps):
    x = x.double()
    mu = x.mean(-1, keepdim=True)
    var = (x - mu).square().mean(-1, keepdim=True)
    r = (var + eps).rsqrt()
    y = (x - mu) * r
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mu[..., 0], r[..., 0]


def norm_bounds(x, w, b, eps, out_dtype):
    """(bound of y, of mean, of rstd)."""
    x = x.double()
    h = sum_depth(x.shape[-1])
    mu = x.mean(-1, keepdim=True)
    xc = x - mu
    var = xc.square().mean(-1, keepdim=True)
    r = (var + eps).rsqrt()
    # the sum, its scaling by the rounded 1 / dim
    dmu = (h + 2) * U * x.abs().mean(-1, keepdim=True)
    # about a mean off by dmu the squares gain dmu^2 and their sum is off by
    # the differences' rounding (2 u), the tree and the scaling
    dvar = (h + 5) * U * (var + dmu ** 2) + dmu ** 2 + 2 * dmu * U * xc.abs().mean(-1, keepdim=True)
    # var + eps, the square root and the reciprocal: one rounding each
    dr = r * (0.5 * dvar * r * r + 3 * U)
    aw = 1.0 if w is None else w.double().abs()
    ab = 0.0 if b is None else b.double().abs()
    y = (xc * r).abs() * aw + ab
    dy = aw * (r * (dmu + U * (xc.abs() + dmu)) + (xc.abs() + dmu) * (dr + U * r)) + 2 * U * y
    return dy + half(out_dtype) * (y + dy), dmu[..., 0], dr[..., 0]


def norm_grad(dy, x, mean, rstd, w):
    """((dx, dw, db), (bounds)) from the statistics given, before rounding to the output types."""
    dy, x = dy.double(), x.double()
    dim = x.shape[-1]
    h = sum_depth(dim)
    mu, r = mean.double()[..., None], rstd.double()[..., None]
    xh = (x - mu) * r
    q = dy * w.double() if w is not None else dy
    mq, mqx = q.mean(-1, keepdim=True), (q * xh).mean(-1, keepdim=True)
    dx = r * (q - mq - xh * mqx)
    # xh carries 2 u, q one; the two means their trees and scaling; then two
    # differences, one product inside and one outside
    emq = (h + 3) * U * q.abs().mean(-1, keepdim=True)
    emqx = (h + 6) * U * (q * xh).abs().mean(-1, keepdim=True)
    edx = r * (emq + xh.abs() * emqx + 6 * U * (q.abs() + mq.abs() + (xh * mqx).abs()))
    d2 = dy.reshape(-1, dim)
    x2 = xh.reshape(-1, dim)
    rows = d2.shape[0]
    # rows in one CTA's registers, its row groups, the partial rows of a warp, the warps
    depth = rows / 148 + 2 + 4 + 148 * 4 / 8 + 1 + 8
    dw, db = (d2 * x2).sum(0), d2.sum(0)
    return (dx, dw, db), (edx, (depth + 3) * U * (d2 * x2).abs().sum(0), depth * U * d2.abs().sum(0))


# ---- output head ---------------------------------------------------------------


def head(hidden, weight, targets, ignore):
    """(loss, lse, softmax, valid) per token; invalid tokens 0."""
    t = targets.reshape(-1)
    valid = (t != ignore) & (t >= 0) & (t < weight.shape[0])
    h = torch.where(valid[:, None], hidden.reshape(-1, hidden.shape[-1]).double(), 0.0)
    logits = h @ weight.double().T
    lse = torch.logsumexp(logits, 1)
    at = torch.where(valid, t, 0).long()
    loss = lse - logits.gather(1, at[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return torch.where(valid, loss, zero), torch.where(valid, lse, zero), torch.softmax(logits, 1), valid, h, at


def head_bounds(h, weight, lse, valid):
    """(bound of loss, of lse, of one logit): the tensor cores' fp32 sums are
    taken as truncating (2^-23 a term), the worst case over any order."""
    dim, vocab = weight.shape[1], weight.shape[0]
    size = (h.abs() @ weight.double().abs().T).max(1).values
    el = dim * 2.0 ** -23 * size
    # differences to the maximum, their scaling, the exponential (2^-22), and
    # the sums: 128 columns, the pairs of a group, 32 groups, rescalings
    terms = 2.0 ** -21 + (128 + vocab / 4096 + 40) * 2 * U + 2 * U * 2 * size
    elsed = el + terms + 4 * U * (lse.abs() + size)
    return elsed + el + 2 * U * (lse.abs() + size), elsed, el


def head_grad(h, weight, p, valid, at, dloss, elogit, else_):
    """((dhidden, dweight), (bounds before the output rounding))."""
    w = weight.double()
    vocab, n = w.shape[0], h.shape[0]
    dl = torch.where(valid, dloss.double(), 0.0)[:, None]
    onehot = torch.zeros_like(p)
    onehot[torch.arange(n, device=p.device), at] = 1.0
    g = dl * (p - onehot)
    # p is off by the logit's and the log sum's errors and the exponential's;
    # the difference, the product, and one rounding to bf16
    ep = dl.abs() * p * (torch.expm1((elogit + else_)[:, None]) + 2.0 ** -20)
    eg = (ep + 2 * U * g.abs()) + half(torch.bfloat16) * (g.abs() + ep)
    dh, dw = g @ w, g.T @ h
    edh = eg @ w.abs() + vocab * 2.0 ** -23 * (g.abs() @ w.abs())
    edw = eg.T @ h.abs() + n * 2.0 ** -23 * (g.abs().T @ h.abs())
    return (dh, dw), (edh, edw)
