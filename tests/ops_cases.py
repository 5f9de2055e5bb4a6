"""Shared by the tests of the norms, the embedding and the distillation loss:
definitions in 64 bits (CPU) and the roundings that a result may be off by.

U is half a step of fp32 relative to the value; half(t) that of type t.  A sum
whose terms each pass at most k fp32 additions is within k U sum|terms| of the
exact one (to first order), which the bounds below count."""
import math

import torch

U = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]
CODE = {t: k for k, t in enumerate(TYPES)}   # lopt_dtype
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def half(t):
    return torch.finfo(t).eps / 2


def close(got, want, tol, what):
    """|got - want| <= tol element by element (want, tol in 64 bits), equal where not finite."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaNs differ"
    inf = ~fine & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    off = (got - want).abs()[fine]
    bound = (torch.zeros_like(want) + tol)[fine]
    if off.numel():
        worst = (off / bound.clamp(min=1e-300)).max().item()
        assert bool((off <= bound).all()), f"{what}: {worst:.3g} times the bound, off by {off.max().item():.3g}"


def rounding(want, t):
    """One rounding to t, and fp16's and fp32's smallest steps (t's subnormal values; the units flush fp32's)."""
    return half(t) * want.abs() + TINY[t]


# ---- norms

def depth(cols):
    """Additions that a term of a row's sum passes: at most 16 in a thread (longer rows: cols / 1024), 6 over a wave,
    16 over a block."""
    return 16 + 6 + 16 + cols // 1024


def norm_forward(x, w, b, eps, rms):
    x = x.double()
    mean = torch.zeros(x.shape[0], 1, dtype=torch.float64) if rms else x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    xh = (x - mean) * rstd
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if b is None else b.double()
    return xh * w + b, mean[:, 0], rstd[:, 0], xh, w, b


def norm_forward_tols(y, mean, rstd, xh, w, b, t, x):
    """xh: the sums' roundings (each within depth U of the mean size of its terms, |xh| about 1) and a dozen of its own."""
    k = (2 * depth(x.shape[1]) + 12) * U
    ty = rounding(y, t) + k * ((xh.abs() + 1) * w.abs() + b.abs())
    # the first sum's own error, of the size of x, is taken out by the second one: U of the mean, and of the spread
    tm = 2 * U * mean.abs() + k / rstd + TINY[torch.float32]
    return ty, tm, k * rstd


def norm_backward(dy, x, w, mean, rstd, rms):
    """With the statistics as given."""
    dy, x = dy.double(), x.double()
    mean = torch.zeros(x.shape[0], 1, dtype=torch.float64) if rms else mean.double()[:, None]
    rstd = rstd.double()[:, None]
    xh = (x - mean) * rstd
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()
    a = dy * w
    c1 = (a * xh).mean(1, keepdim=True)
    c2 = torch.zeros_like(c1) if rms else a.mean(1, keepdim=True)
    dx = rstd * (a - xh * c1 - c2)
    k = (2 * depth(x.shape[1]) + 12) * U
    size = rstd * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True) + (0 if rms else a.abs().mean(1, keepdim=True)))
    return dx, (dy * xh).sum(0), dy.sum(0), k * size, (dy * xh).abs().sum(0), dy.abs().sum(0)


def row_depth(rows):
    """Additions that a term of a column's sum passes: the rows of one thread (at least 4 blocks' worth of rows share
    them), 8 groups, 4 waves, blocks / 32 and 32; below 200 for the sizes here, and one product."""
    return min(rows, 16 + rows // 512) + 8 + 4 + 32 + 32 + 4


# ---- distillation

def teacher(ids, u, tau, cols):
    there = (ids >= 0) & (ids < cols) & ~(u == -math.inf)
    v = torch.where(there, u.double() / tau, -math.inf)
    some = there.any(1, keepdim=True)
    p = torch.where(some, v, 0.0).softmax(1) * there
    return there, some[:, 0], p, torch.where(there, v, 0.0)


def distill(z, ids, u, tau, lse=None):
    """(loss, lse, q - p over the vocabulary, and what the bounds need)."""
    cols = z.shape[1]
    there, some, p, v = teacher(ids, u, tau, cols)
    zt = z.double() / tau
    exact = torch.logsumexp(zt, 1)
    at = zt.gather(1, ids.clamp(0, cols - 1).long())
    logp = torch.where(p > 0, p.log(), 0.0)
    terms = torch.where(p > 0, p * (logp - at + exact[:, None]), 0.0)
    loss = torch.where(some, tau * tau * terms.sum(1), 0.0)
    q = torch.exp(zt - (exact if lse is None else lse.double())[:, None])
    dense = torch.zeros_like(q).scatter_add_(1, ids.clamp(0, cols - 1).long(), p)
    finite = torch.where(torch.isfinite(zt), zt, 0.0).abs().max(1).values + torch.where(torch.isfinite(exact), exact.abs(), 0.0)
    size = 1 + finite + v.abs().max(1).values           # largest exponents of the row
    terms_size = torch.where(torch.isfinite(terms), terms, 0.0).abs().sum(1)
    return loss, exact, torch.where(some[:, None], q - dense, 0.0), q, dense, size, terms_size
