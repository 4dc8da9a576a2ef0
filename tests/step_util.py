"""64-bit definitions of the operators that keep a step's memory small, and how
far fp32 sums may be from them (training_util has the roundoffs and `check`)."""

import torch

from training_util import TINY, U, check, out_tol, u  # noqa: F401

BLOCK = 128
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
MOST = {E4: 448.0, E5: 57344.0}
BITS = {E4: 3, E5: 2}   # of a significand, behind the leading one
LOW = {E4: -6, E5: -14}  # exponent below which the values are equally spaced


def check_out(got, want, err, dtype):
    """An fp32 result within err of ``want``, rounded to ``dtype``: f16 rounds what is 65520 (the middle of its largest
    value and the next one that it would have) or more to infinity."""
    want, err = want.double(), err.double()
    if dtype == torch.float16:
        over, may = want.abs() - err >= 65520.0, want.abs() + err >= 65520.0
        assert torch.equal(got[over].double(), torch.sign(want[over]) * torch.inf)
        got, want, err = got[~may], want[~may], err[~may]
    check(got, want, out_tol(err, want, dtype))


# -- 8 bits ----------------------------------------------------------------------

def blocks(x):
    n = -(-x.shape[-1] // BLOCK)
    return torch.nn.functional.pad(x, (0, n * BLOCK - x.shape[-1])).unflatten(-1, (n, BLOCK))


def spread(scales, dim):
    """A block's scale at each of its elements."""
    return scales.repeat_interleave(BLOCK, -1)[..., :dim]


def scale_of(top, fmt):
    """The least power of two 2^e, e >= -126, with top <= MOST 2^e, in 64 bits; 1 for 0."""
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0).double() / MOST[fmt]))
    s = torch.exp2(e)
    s = torch.where(top > s * MOST[fmt], 2 * s, s)
    return torch.where(top > 0, s.clamp(min=2.0 ** -126), 1.0)


def step_of(v, fmt):
    """Distance of the format's values around v (scaled)."""
    binade = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** LOW[fmt])))
    return torch.exp2(binade - BITS[fmt])


def eight(x, fmt):
    """(values without scale, scales) of x (..., dim) in 8 bits."""
    x = x.double()
    finite = torch.isfinite(x)
    scales = scale_of(blocks(torch.where(finite, x, 0.0)).abs().amax(-1), fmt)
    v = torch.where(finite, x, 0.0) / spread(scales, x.shape[-1])
    step = step_of(v, fmt)
    v = torch.round(v / step) * step
    if fmt == E5:
        v = torch.where(torch.isinf(x), x, v)
    else:
        v = torch.where(torch.isinf(x), torch.nan, v)
    return torch.where(torch.isnan(x), torch.nan, v), scales


def check_eight(codes, scales, x, fmt):
    """Codes and scales of x itself: the very values."""
    want, want_scales = eight(x, fmt)
    assert codes.dtype == fmt and torch.equal(scales.double(), want_scales)
    got = codes.float().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0, posinf=1e9, neginf=-1e9),
                       torch.nan_to_num(want, nan=0.0, posinf=1e9, neginf=-1e9))


def check_eight_near(codes, scales, y, err, fmt):
    """Codes and scales of something within err of y: half a step of the format and err from it, the scale that of some
    value within err."""
    top = blocks(y.abs()).amax(-1)
    e = blocks(err).amax(-1)
    s = scales.double()
    assert bool(((s == scale_of((top - e).clamp(min=0), fmt)) | (s == scale_of(top + e, fmt))).all())
    s = spread(s, y.shape[-1])
    half = 0.5 * step_of((y.abs() + err) / s, fmt) * s
    check(codes.float().double() * s, y, half + err)


# -- root-mean-square norm ---------------------------------------------------------

def norm_depth(dim):
    """Additions in a chain of a row's sum: a thread's 16 elements (or 1/512 of a long row), the warp's 5 and the
    warps' 5."""
    return max(16, -(-dim // 512) + 4) + 10


def rms_forward(s, weight, eps):
    """(y, rstd), (their errors in fp32) of the sum s as it is kept."""
    s = s.double()
    mean = (s * s).mean(-1)
    rstd = (mean + eps).rsqrt()
    w = torch.ones_like(s) if weight is None else weight.double().expand_as(s)
    y = s * rstd[..., None] * w
    # all terms are positive; rsqrt is within 2 ulp, the division by dim and eps one rounding each
    rel = 0.5 * (norm_depth(s.shape[-1]) + 3) * u * 1.01 + 4 * u
    return (y, rstd), ((rel + 3 * u) * y.abs(), rel * rstd)


def rms_backward(grad, s, rstd, weight, add=None, before=None):
    """(dx, dw), (their errors) with s the values that were kept."""
    g, s, r = grad.double(), s.double(), rstd.double()[..., None]
    w = torch.ones_like(s) if weight is None else weight.double().expand_as(s)
    xh, a = s * r, g * w
    m = (a * xh).mean(-1, keepdim=True)
    own = r * (a - xh * m)
    dx = own if add is None else own + add.double()
    m_err = (norm_depth(s.shape[-1]) + 4) * u * (a * xh).abs().mean(-1, keepdim=True)
    dx_err = r * (4 * u * a.abs() + xh.abs() * (m_err + 4 * u * m.abs())) + 2 * u * own.abs() + u * dx.abs()
    t = (g * xh).flatten(0, -2)
    dw, mag = t.sum(0), t.abs().sum(0)
    # a thread's rows (at most 32, or one in 304), the groups of a CTA, the partial rows in 16 runs, those
    depth = 32 + t.shape[0] // 300 + 15 + 20 + 16
    if before is not None:
        dw, mag = dw + before.double(), mag + before.double().abs()
    return (dx, dw), (dx_err, (depth + 4) * u * mag)


# -- products ------------------------------------------------------------------------

def product(a, b, scale=1.0, before=None):
    """(a^T b * scale [+ before], its error where products are exact and sums fp32, whatever their order)."""
    a, b = a.double(), b.double()
    d, mag = a.t() @ b * scale, a.abs().t() @ b.abs() * abs(scale)
    if before is not None:
        d, mag = d + before.double(), mag + before.double().abs()
    return d, (a.shape[0] + 4) * u * mag


# -- cross entropy of a linear layer ---------------------------------------------------

def live_tokens(targets, weights, vocab):
    t = targets.reshape(-1).long()
    w = torch.ones(t.shape, dtype=torch.float64, device=t.device) if weights is None else weights.reshape(-1).double()
    return t, w, (t >= 0) & (t < vocab) & (w != 0)


def _logits(h, weight):
    """(z, the error of each in fp32: exact products, sums in any order)."""
    h, weight = h.double(), weight.double()
    return h @ weight.t(), (h.shape[1] + 4) * u * (h.abs() @ weight.abs().t())


def loss_forward(hidden, weight, targets, weights):
    """(losses, lse), (their errors); rows that do not count are 0 with an error of 0."""
    v = weight.shape[0]
    t, w, live = live_tokens(targets, weights, v)
    h = hidden.reshape(-1, hidden.shape[-1])[live]
    z, ez = _logits(h, weight)
    lse = torch.logsumexp(z, 1)
    at = t[live][:, None]
    zt, et = z.gather(1, at)[:, 0], ez.gather(1, at)[:, 0]
    # the logits' errors, weighted by the probabilities; an exponential is within 4 u and |x| u of its argument x (|x| e^x < 0.4,
    # so 90 u in all at most); a chain of 46 additions in 128 columns, then of the columns' pieces
    p = torch.exp(z - lse[:, None])
    el = (p * ez).sum(1) * 1.01 + (150 + v / 128 / 32 + 40) * u + 3 * u * lse.abs()
    out = [torch.zeros(t.shape, dtype=torch.float64, device=t.device) for _ in range(4)]
    out[0][live] = w[live] * (lse - zt)
    out[1][live] = lse
    out[2][live] = w[live].abs() * (el + et + 3 * u * (lse.abs() + zt.abs()))
    out[3][live] = el
    return tuple(x.view(targets.shape) for x in out[:2]), tuple(x.view(targets.shape) for x in out[2:])


def loss_backward(hidden, weight, targets, lse, weights, scale=1.0, before=None):
    """(dhidden, dweight), (their errors) for the lse that is given."""
    v, d, dtype = weight.shape[0], weight.shape[1], hidden.dtype
    t, w, live = live_tokens(targets, weights, v)
    h = hidden.reshape(-1, d)[live]
    z, ez = _logits(h, weight)
    x = z - lse.reshape(-1).double()[live][:, None]
    q = torch.exp(x)
    # q's error: its argument's (the logit's and the difference's), the exponential's; then the difference from 1
    eq = q * (torch.expm1(ez + 2 * u * (z.abs() + x.abs()) + 4 * u))
    q.scatter_add_(1, t[live][:, None], torch.full_like(q[:, :1], -1.0))
    eq += u * q.abs()
    wl = w[live]
    size = torch.exp2(torch.floor(torch.log2(wl.abs())))[:, None]  # a weight's power of two
    # one rounding to the operands' type, of f16 2^14 times the value
    low = 2.0 ** -39 if dtype == torch.float16 else 0.0
    eg = (eq + (U[dtype] + 2 * u) * (q.abs() + eq)) * wl.abs()[:, None] + low * size
    g = q * wl[:, None]
    dh = torch.zeros((t.shape[0], d), dtype=torch.float64, device=h.device)
    eh, wd, hd = torch.zeros_like(dh), weight.double(), h.double()
    dh[live] = g @ wd * scale
    mag = (g.abs() + eg) @ wd.abs()
    eh[live] = (eg @ wd.abs() + (v + 40) * u * mag) * abs(scale)
    dw, mag = g.t() @ hd * scale, (g.abs() + eg).t() @ hd.abs()
    ew = (eg.t() @ hd.abs() + (h.shape[0] + 40) * u * mag) * abs(scale)
    if dtype == torch.float16 and h.shape[0]:
        # a row of h times its weight's power of two relative to the largest may meet f16's smallest step
        ew = ew + (((g.abs() + eg) / size).sum(0) * 2.0 ** -25 * float(size.max()) * abs(scale))[:, None]
    if before is not None:
        dw, ew = dw + before.double(), ew + u * (dw.abs() + before.double().abs())
    return (dh.view(hidden.shape), dw), (eh.view(hidden.shape), ew)
