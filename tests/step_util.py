"""64-bit definitions of the operators that keep a step's memory small, and how
far fp32 sums may be from them (training_util has the roundoffs and `check`)."""

import torch

from training_util import TINY, U, check, out_tol, u  # noqa: F401

BLOCK = 128
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
MOST = {E4: 448.0, E5: 57344.0}
BITS = {E4: 3, E5: 2}   # of a significand, behind the leading one
LOW = {E4: -6, E5: -14}  # exponent below which the values are equally spaced


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
