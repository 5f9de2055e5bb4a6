"""The residual update with its norms in 64 bits on the CPU, for the tests, with the roundings that a result may be off by."""
import torch

from ops_cases import TINY, U, depth, norm_backward, norm_forward, norm_forward_tols, rounding


def vec(v, cols, fill):
    return torch.full((cols,), fill, dtype=torch.float64) if v is None else v.double()


def update(x, y, gate, w1, b1, eps, o):
    """(h, its bound before the last rounding, mean and rstd of y with their bounds)"""
    cols = x.shape[1]
    u, tu, stats = y.double(), 0.0, None
    if o["post"]:
        want = norm_forward(y, w1, b1, eps, o["rms"])
        ty, tm, tr = norm_forward_tols(*want, torch.float32, y)
        u, tu, stats = want[0], ty, (want[1], tm, want[2], tr)
    g = torch.ones(cols, dtype=torch.float64) if gate is None else gate.double()
    branch = o["beta"] * g * u
    h = o["alpha"] * x.double() + branch
    tol = abs(o["beta"]) * g.abs() * tu + 4 * U * ((o["alpha"] * x.double()).abs() + branch.abs())
    return h, tol, stats


def sums_depth(rows):
    """Additions that a term of a column's sum passes: the rows of one thread, 8 groups, 4 waves, 64 and 32 of the join."""
    return min(rows, 16 + rows // 512) + 8 + 4 + 64 + 32 + 8


def backward(dh, dz, y, h, stats, gate, w1, b1, w2, o):
    """{name: (gradient, bound before the last rounding)} with the statistics as given."""
    rows, cols = y.shape
    rms, k = o["rms"], sums_depth(y.shape[0]) * U
    D = torch.zeros(rows, cols, dtype=torch.float64) if dh is None else dh.double()
    tD = U * D.abs()
    out = {}
    if o["pre"]:
        z = torch.zeros(rows, cols, dtype=torch.float64) if dz is None else dz
        d, dw, db, tol, dwa, dba = norm_backward(z, h, w2, stats[2], stats[3], rms)
        tD = tol + U * (D.abs() + d.abs())
        D = D + d
        out["weight"] = (dw, k * dwa)
        if not rms:
            out["bias"] = (db, k * dba)
    out["x"] = (o["alpha"] * D, abs(o["alpha"]) * tD + U * (o["alpha"] * D).abs())
    E, tE = o["beta"] * D, abs(o["beta"]) * tD + U * (o["beta"] * D).abs()
    yd = y.double()
    if o["post"]:
        mean = torch.zeros(rows, 1, dtype=torch.float64) if rms else stats[0].double()[:, None]
        yh = (yd - mean) * stats[1].double()[:, None]
        W, B = vec(w1, cols, 1.0), vec(b1, cols, 0.0)
        u, tu = yh * W + B, 4 * U * ((yh * W).abs() + B.abs())
    else:
        u, tu = yd, torch.zeros_like(yd)
    du, tdu = E, tE
    if gate is not None:
        dg, tg = E * u, tE * u.abs() + E.abs() * tu + U * (E * u).abs()
        out["gate"] = (dg, tg) if gate.dim() == 2 else (dg.sum(0), tg.sum(0) + k * dg.abs().sum(0))
        g = gate.double()
        du, tdu = E * g, tE * g.abs() + U * (E * g).abs()
    if not o["post"]:
        out["y"] = (du, tdu)
        return out
    dy, dw, db, tol, dwa, dba = norm_backward(du, y, w1, None if rms else stats[0], stats[1], rms)
    ta, r = tdu * W.abs(), stats[1].double()[:, None]
    out["y"] = (dy, tol + r * (ta + yh.abs() * (ta * yh.abs()).mean(1, keepdim=True) + (0 if rms else ta.mean(1, keepdim=True))))
    out["post_weight"] = (dw, (tdu * yh.abs()).sum(0) + k * dwa)
    if not rms:
        out["post_bias"] = (db, tdu.sum(0) + k * dba)
    return out


def bound(want, tol, t):
    return rounding(want, t) + tol


__all__ = ["TINY", "U", "backward", "bound", "depth", "update"]
