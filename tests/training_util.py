"""Plain 64-bit definitions of the training operators, and how far a
computation that sums in fp32 may be from them.

u is fp32's unit roundoff; a sum of terms t_i in fp32, whatever its order, is
within depth * u * sum |t_i| of the exact one, depth being the longest chain of
additions a term passes through.  U[dtype] is the roundoff of the output type,
and TINY[dtype] half its smallest step (f16's subnormals).
"""

import torch

u = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-37}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def check(got, want, tol):
    """|got - want| <= tol elementwise (an infinite or NaN want wants the same)."""
    got, want = got.double().cpu(), want.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(want)
    assert got.shape == want.shape
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    off = (got - want).abs()[fine] - tol[fine]
    assert off.numel() == 0 or bool((off <= 0).all()), (
        f"{int((off > 0).sum())} of {off.numel()} off, worst over its bound by {float(off.max()):.3e} "
        f"(bound there {float(tol[fine][off.argmax()]):.3e})")


def out_tol(err, want, dtype):
    """Bound of an fp32 result within err of ``want``, rounded to ``dtype``."""
    return err + U[dtype] * (want.abs() + err) + TINY[dtype]


# -- embedding -------------------------------------------------------------------

def table_grad(ids, grad, vocab, scale, padding=None, before=None):
    """(gradient, sum of the terms' absolute values, number of tokens of each row)."""
    ids, g = ids.reshape(-1).long(), grad.double().reshape(-1, grad.shape[-1]) * scale
    keep = (ids >= 0) & (ids < vocab)
    if padding is not None:
        keep &= ids != padding
    ids, g = ids[keep], g[keep]
    dw = torch.zeros((vocab, g.shape[1]), dtype=torch.float64, device=g.device) if before is None else before.double()
    mag = dw.abs()
    dw = dw.index_add(0, ids, g)
    mag = mag.index_add(0, ids, g.abs())
    count = torch.bincount(ids, minlength=vocab)
    return dw, mag, count


def table_grad_tol(dw, mag, count, dtype):
    # every token is added once, the scale and a value that was there before once each
    return out_tol((count[:, None] + 3) * u * mag, dw, dtype)


# -- layer norm ------------------------------------------------------------------

def norm_depth(dim):
    """Additions in a chain of a row's sum: a thread's share of the row (at most
    64 elements, or 1/256 of a long row), 5 shuffles and the warps."""
    return max(64, dim // 256) + 5 + 32


def norm_forward(x, weight, bias, eps):
    x = x.double()
    mean = x.mean(-1)
    d = x - mean[..., None]
    var = (d * d).mean(-1)
    rstd = (var + eps).rsqrt()
    xh = d * rstd[..., None]
    w = torch.ones_like(x[..., :1]) if weight is None else weight.double()
    y = xh * w + (0.0 if bias is None else bias.double())
    depth = norm_depth(x.shape[-1])
    mean_err = (depth + 2) * u * x.abs().mean(-1)
    # the deviations carry the mean's error, which adds its square to the variance
    var_err = (depth + 4) * u * var + mean_err ** 2 + 2 * mean_err * (u * d.abs().mean(-1))
    rstd_rel = 0.5 * var_err / (var + eps) * 1.01 + 4 * u
    y_err = w.abs() * ((mean_err[..., None] + u * d.abs()) * rstd[..., None] * 1.01 + xh.abs() * (rstd_rel[..., None] + 3 * u))
    y_err = y_err + 2 * u * y.abs()
    return (y, mean, rstd), (y_err, mean_err + u * mean.abs(), rstd * rstd_rel)


def norm_backward(grad, x, mean, rstd, weight, before=None):
    """``mean`` and ``rstd`` are inputs, taken as they are."""
    dim = x.shape[-1]
    g, x = grad.double().reshape(-1, dim), x.double().reshape(-1, dim)
    mean, rstd = mean.double().reshape(-1, 1), rstd.double().reshape(-1, 1)
    rows = x.shape[0]
    d = x - mean
    xh = d * rstd
    w = torch.ones(dim, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    a = g * w
    m0, m1 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    dx = rstd * (a - m0 - xh * m1)
    dw, db = (g * xh).sum(0), g.sum(0)
    depth = norm_depth(dim)
    e0 = (depth + 3) * u * a.abs().mean(1, keepdim=True)
    e1 = (depth + 6) * u * (a * xh).abs().mean(1, keepdim=True)
    dx_err = rstd * (e0 + xh.abs() * e1 + 4 * u * (a.abs() + m0.abs() + 2 * (xh * m1).abs())) * 1.01
    # columns: a thread's rows (1/128 of them at most, past the first), the groups of a CTA, the partial rows
    cdepth = rows / 128 + 96
    dw_err = (cdepth + 4) * u * (g * xh).abs().sum(0)
    db_err = (cdepth + 2) * u * g.abs().sum(0)
    if before is not None:
        dw, db = dw + before[0].double(), db + before[1].double()
        dw_err, db_err = dw_err + 2 * u * dw.abs(), db_err + 2 * u * db.abs()
    return (dx.reshape(grad.shape), dw, db), (dx_err.reshape(grad.shape), dw_err, db_err)


# -- distillation ------------------------------------------------------------------

def distill(logits, teacher, index, temperature, weights=None, grad_scale=1.0):
    """((losses, dlogits), (their errors' bounds)) of (rows, vocab) logits."""
    t = float(temperature)
    z = logits.double() / t
    rows, vocab = z.shape
    w = torch.ones(rows, dtype=torch.float64, device=z.device) if weights is None else weights.double()
    index = index.long()
    valid = (index >= 0) & (index < vocab)
    y = torch.where(valid, teacher.double() / t, -torch.inf)
    live = (y != -torch.inf).any(1) & (w != 0)
    top = z.max(1, keepdim=True).values
    arg = z - torch.where(torch.isfinite(top), top, 0.0)
    e = arg.exp()
    total = e.sum(1, keepdim=True)
    q = e / total
    yarg = y - y.max(1, keepdim=True).values
    pe = yarg.exp()
    p = pe / pe.sum(1, keepdim=True)
    at = torch.where(valid, index, 0)
    logq = arg.gather(1, at) - total.log()
    logp = yarg - pe.sum(1, keepdim=True).log()
    some = valid & (p != 0)
    part = torch.where(some, p * (torch.where(some, logp, 0.0) - logq), 0.0)
    losses = torch.where(live, w * t * t * part.sum(1), 0.0)
    target = torch.zeros_like(z).scatter_add_(1, at, torch.where(valid, p, 0.0))
    f = (w * t * grad_scale)[:, None]
    dz = torch.where(live[:, None], f * (q - target), 0.0)
    # exponentials: the argument is rounded a few times relative to its size, then exp2 and the sums
    size = torch.nan_to_num(torch.where(torch.isfinite(arg), arg.abs(), 0.0))
    depth = 64 + vocab / 256
    qrel = u * (4 * size + 4 * (torch.nan_to_num(q) * size).sum(1, keepdim=True) + depth + 24)
    psize = torch.where(torch.isfinite(yarg), yarg.abs(), 0.0)
    prel = u * (4 * psize + 4 * (torch.nan_to_num(p) * psize).sum(1, keepdim=True) + 64 + 24)
    pmax = torch.zeros_like(z).scatter_add_(1, at, torch.where(valid, torch.nan_to_num(p * prel), 0.0))
    dz_err = f.abs() * (torch.nan_to_num(q) * qrel + pmax + 4 * u * (torch.nan_to_num(q) + target) + 1e-37) * 1.01
    dz_err = torch.where(live[:, None], torch.nan_to_num(dz_err, posinf=0.0), 0.0)
    lq = torch.where(some & torch.isfinite(logq), logq.abs(), 0.0)
    lp = torch.where(some, torch.nan_to_num(logp).abs(), 0.0)
    term = torch.where(some, p * (prel * (lp + lq + 1) + 4 * u * (lp + lq + 1) + qrel.gather(1, at) + u * depth), 0.0)
    loss_err = w.abs() * t * t * (torch.nan_to_num(term).sum(1) + 80 * u * torch.nan_to_num(part.abs(), posinf=0.0).sum(1)) * 1.01
    return (losses, dz), (torch.where(live, loss_err, 0.0) + 1e-37, dz_err)
