"""64-bit references of the block-seam tests, with the error each output may
have, counted from the roundings it goes through (U: half a step of binary32).
A row's sums lose at most 64 half steps of the mean of what they add: a thread
adds up to 16 elements, then 10 levels of a tree."""

from __future__ import annotations

import torch

from tests._operators import U, layernorm_ref


def param(p, none):
    return none if p is None else p.double()


def norm_ref(a, kind, gamma, beta, eps):
    """y, rstd and mean of a's rows in binary64 and their errors; a is exact."""
    a = a.double()
    if kind == "layer":
        (y, dy), (mean, dmean), (rstd, drstd) = layernorm_ref(a, gamma, beta, eps)
        return (y, dy), (rstd, drstd), (mean, dmean)
    ms = (a * a).mean(1)
    rstd = 1.0 / torch.sqrt(ms + eps)
    # a square's rounding, the sum's, the mean's, eps's; then root and quotient
    drstd = rstd * (64 + 4) * U
    h = a * rstd[:, None]
    g, b = param(gamma, 1.0), param(beta, 0.0)
    y = h * g + b
    dy = abs(h * g) * (64 + 4 + 4) * U + 2 * U * abs(y)
    return (y, dy), (rstd, drstd), (0 * rstd, 0 * rstd)


def gate_ref(gate, kind):
    if kind == "none":
        return 1.0
    return gate.double() if kind == "column" else torch.sigmoid(gate.double())


# exp within 2 half steps of a step's size, 1 + t, the quotient, a product: 8 half steps
GATE = 8 * U


def sum_ref(x, n, dn, gate, scale):
    """The residual sum before its rounding, and its error."""
    s = scale * x.double() + gate * n
    return s, abs(gate) * dn + (GATE + 2 * U) * abs(gate * n) + 2 * U * abs(s)


def backward_ref(dy, dsum, total, block, gate, kind, gate_kind, post, scale, gamma0, beta0, gamma,
                 stats, serial):
    """Every gradient in binary64 with its error; `serial`: the longest chain of
    additions of a column's sum."""
    layer = kind == "layer"
    col = lambda i: stats[i].double()[:, None]
    d1, total = dy.double(), total.double()
    h1 = (total - col(3) if layer else total) * col(1)
    one = torch.ones_like(h1)
    out = {}

    def through(g, dg, h, r):
        """N' of g (with error dg), and its error."""
        e1 = 64 * U * abs(g).mean(1, keepdim=True) + dg.mean(1, keepdim=True)
        e2 = 64 * U * abs(g * h).mean(1, keepdim=True) + (dg * abs(h)).mean(1, keepdim=True)
        c1 = g.mean(1, keepdim=True) if layer else 0 * e1
        c2 = (g * h).mean(1, keepdim=True)
        v = r * (g - c1 - h * c2)
        dv = r * (dg + (e1 if layer else 0) + abs(h) * e2
                  + 8 * U * (abs(g) + abs(c1) + abs(h * c2))) + 2 * U * abs(v)
        return v, dv

    g = d1 * param(gamma, 1.0)
    D, dD = through(g, U * abs(g), h1, col(1))
    if dsum is not None:
        D = D + dsum.double()
        dD = dD + 2 * U * (abs(D) + abs(dsum.double()))
    out["dx"] = (scale * D, abs(scale) * dD + 2 * U * abs(scale * D))

    def column(v, dv):
        return v.sum(0), dv.sum(0) + serial * U * abs(v).sum(0)

    out["dgamma"] = column(d1 * h1, 4 * U * abs(d1 * h1))
    out["dbeta"] = column(d1, 0 * d1)
    if block is None:
        return out
    b = block.double()
    h0 = (b - col(2) if layer else b) * col(0) if post else b
    r0 = col(0) if post else one[:, :1]
    gp, bp = (param(gamma0, 1.0), param(beta0, 0.0)) if post else (1.0, 0.0)
    n = h0 * gp + bp
    dn = 4 * U * (abs(h0 * gp) + abs(bp))
    gain = gate_ref(gate, gate_kind) * one
    wide = gate_kind == "sigmoid"
    E, dE = (D * gain, gain * dD + GATE * abs(D * gain)) if wide else (D, dD)
    if wide:
        slope = gain * torch.sigmoid(-gate.double())
        dz = D * n * slope
        out["dgate"] = (dz, dD * abs(n * slope) + abs(D * slope) * dn + 2 * GATE * abs(dz))
    A1, eA1 = column(E * h0, dE * abs(h0) + 4 * U * abs(E * h0))
    A0, eA0 = column(E, dE)
    cg = param(gate, 1.0) if gate_kind == "column" else torch.ones_like(A0)
    if post:
        out["dgamma_post"] = (cg * A1, abs(cg) * eA1 + 2 * U * abs(cg * A1))
        out["dbeta_post"] = (cg * A0, abs(cg) * eA0 + 2 * U * abs(cg * A0))
    if gate_kind == "column":
        v = gp * A1 + bp * A0
        gp, bp = gp * torch.ones_like(A0), bp * torch.ones_like(A0)
        out["dgate"] = (v, abs(gp) * eA1 + abs(bp) * eA0 + 3 * U * (abs(gp * A1) + abs(bp * A0)))
    f = cg * gp
    G, dG = E * f, abs(f) * dE + 3 * U * abs(E * f)
    out["dblock"] = through(G, dG, h0, r0) if post else (G, dG)
    return out
