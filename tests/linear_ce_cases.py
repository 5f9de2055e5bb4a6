"""The cross entropy of a linear layer in 64 bits, for the tests, with the roundings that a result may be off by.  Computed
where its tensors are (the larger cases on the GPU, in float64 products of two dimensions)."""
import torch

from ops_cases import U, half


def product_depth(k, t):
    """Additions in a row that a term of a product over k passes: one for each matrix instruction (of 16 k; of 2 in fp32),
    a dozen within it, and those of splits and pieces."""
    return (k // 2 if t == torch.float32 else k // 16) + 40


def forward(x, w, targets):
    """(loss, lse, logits, their bounds' parts)"""
    t = x.dtype
    x, w = x.double(), w.double()
    z = x @ w.t()
    ez = product_depth(x.shape[1], t) * U * (x.abs() @ w.abs().t())
    lse = torch.logsumexp(z, 1)
    there = (targets >= 0) & (targets < w.shape[0])
    at = torch.where(there, targets, 0).long()[:, None]
    loss = torch.where(there, lse - z.gather(1, at)[:, 0], 0.0)
    # each tile's sum: 64 in a thread, a few across; the tiles': a quarter of them and a few; an exponential is off by 2 U
    count = (120 + w.shape[0] // 1024) * U
    top = z.max(1).values.abs()
    e = ez.max(1).values
    tl = e + count + U * (lse.abs() + 3 * top)
    return loss, lse, z, ez, torch.where(there, e + tl + 2 * U * loss.abs(), 0.0), tl, there


def backward(g, x, w, targets):
    """(dx, dw, their bounds before the last rounding)"""
    t = x.dtype
    loss, lse, z, ez, _, tl, there = forward(x, w, targets)
    xd, wd, g = x.double(), w.double(), torch.where(there, g.double(), 0.0)[:, None]
    p = torch.exp(z - lse[:, None])
    onehot = torch.zeros_like(p).scatter_(1, torch.where(there, targets, 0).long()[:, None], 1.0)
    G = g * (p - onehot)
    # p from logits and lse off by ez and tl, and lse kept in fp32; G's own rounding; fp16's least step, 2^-35 of the largest g
    eG = g.abs() * p * (2 * (ez + tl[:, None]) + (8 + 3 * lse.abs()[:, None]) * U) + (half(t) + 2 * U) * G.abs()
    if t == torch.float16:
        eG = eG + 2.0 ** -35 * g.abs().max()
    xz = torch.where(there[:, None], xd, 0.0)   # a row to ignore is not read
    G, eG = torch.where(there[:, None], G, 0.0), torch.where(there[:, None], eG, 0.0)
    dx, dw = G @ wd, G.t() @ xz
    tx = eG @ wd.abs() + product_depth(w.shape[0], t) * U * (G.abs() @ wd.abs())
    tw = eG.t() @ xz.abs() + product_depth(x.shape[0], t) * U * (G.abs().t() @ xz.abs())
    return dx, dw, tx, tw
