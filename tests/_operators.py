"""Inputs and 64-bit references of the layer-norm and Muon tests, with the
error each output may have, counted from the roundings it goes through."""

from __future__ import annotations

import torch

HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}


def half_step(t, size):
    """Half a step of type t at values of this size; under the smallest normal
    value (6.1e-5 in binary16) the steps shrink no further."""
    return torch.clamp(HALF[t] * size, min=torch.finfo(t).smallest_normal * HALF[t])


U = 2.0 ** -24  # half a step of binary32


def randn(*shape, dtype=torch.float32, pad=0, seed=0, scale=1.0):
    """A tensor whose last-but-one stride is padded by `pad` elements."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn(*shape[:-1], shape[-1] + pad, device="cuda", generator=g) * scale
    return a.to(dtype)[..., :shape[-1]]


def within(name, got, ref, tol):
    got, bad = got.double(), None
    off = (got - ref).abs()
    ok = (off <= tol) | (torch.isnan(got) & torch.isnan(ref)) | (got == ref)
    if not bool(ok.all()):
        i = int(torch.where(ok.reshape(-1), -1.0, off.reshape(-1)).argmax())
        bad = (i, float(got.reshape(-1)[i]), float(ref.reshape(-1)[i]),
               float((tol + 0 * ref).reshape(-1)[i]))
    assert bad is None, f"{name}: element {bad[0]}: {bad[1]!r} for {bad[2]!r} +- {bad[3]:.3e}"


def layernorm_ref(x, gamma, beta, eps):
    """y, mean, rstd in binary64, and the error that each may have besides its
    own rounding: the row's sums lose at most 64 half steps (a thread adds up
    to 32 elements, then 10 levels of a tree) of the mean of what they add."""
    s = x.double()
    mean = s.mean(1)
    c = s - mean[:, None]
    var = (c * c).mean(1)
    rstd = 1.0 / torch.sqrt(var + eps)
    g = 1.0 if gamma is None else gamma.double()
    b = 0.0 if beta is None else beta.double()
    h = c * rstd[:, None]
    y = h * g + b
    # mean: two sweeps, so the error is of the mean's own rounding and of the
    # second sweep's sum of deviations
    dmean = 64 * U * c.abs().mean(1) + 2 * U * s.abs().amax(1)
    drstd = rstd * (64 * U + rstd ** 2 * dmean ** 2 + rstd * 4 * U * s.abs().amax(1))
    dh = (dmean[:, None] + 2 * U * s.abs().amax(1)[:, None]) * rstd[:, None] \
        + (drstd / rstd)[:, None] * h.abs()
    dy = dh * abs(g) + 4 * U * (h * g).abs() + 2 * U * abs(y)
    return (y, dy), (mean, dmean), (rstd, drstd)


def layernorm_bwd_ref(dy, x, gamma, mean, rstd, dsum, serial):
    """dx, dgamma, dbeta in binary64 and their errors; `serial`: the longest
    chain of additions of a column's sum."""
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    n = x.shape[1]
    h = (x - mean) * rstd
    dh = 2 * U * h.abs() + U * (x.abs() + mean.abs()) * rstd * 0  # x, mean are exact in binary32
    g = dy if gamma is None else dy * gamma.double()
    c1 = g.sum(1, keepdim=True) / n
    c2 = (g * h).sum(1, keepdim=True) / n
    dx = rstd * (g - c1 - h * c2)
    if dsum is not None:
        dx = dx + dsum.double()
    e1 = 64 * U * g.abs().mean(1, keepdim=True)
    e2 = 64 * U * (g * h).abs().mean(1, keepdim=True)
    ddx = rstd * (e1 + h.abs() * e2 + 8 * U * (g.abs() + c1.abs() + (h * c2).abs())) \
        + 2 * U * dx.abs()
    if dsum is not None:
        ddx = ddx + 2 * U * dsum.double().abs()
    dgamma, dbeta = (dy * h).sum(0), dy.sum(0)
    egamma = (serial + 4) * U * (dy * h).abs().sum(0) + (dy.abs() * dh).sum(0)
    ebeta = (serial + 4) * U * dy.abs().sum(0)
    return (dx, ddx), (dgamma, egamma), (dbeta, ebeta)


COEFFS = (3.4445, -4.7750, 2.0315)


def ortho_ref(g, coeffs, eps, rounding=None):
    """Newton-Schulz of one matrix in binary64; `rounding` (the storage
    type's, if any) is applied to X, A and aI + bA + cAA between products."""
    keep = (lambda v: v) if rounding is None else rounding
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T.contiguous()
    x = keep(x / (torch.linalg.norm(x) + eps))
    for a, b, c in coeffs:
        gram = keep(x @ x.T.contiguous())
        poly = b * gram + c * (gram @ gram)
        poly.diagonal().add_(a)
        x = keep(keep(poly) @ x)
    return x.T.contiguous() if tall else x


def binary16(v):
    return (v * 2048.0).half().double() / 2048.0


def ortho_check(name, got, g, coeffs, eps):
    """The 2-norm error against binary64 is at most twice that of the same
    iteration with binary16 storage emulated in binary64, plus half a bf16
    step (the output's own rounding)."""
    ref = ortho_ref(g, coeffs, eps)
    model = ortho_ref(g, coeffs, eps, binary16)
    norm = float(torch.linalg.norm(ref))
    off = float(torch.linalg.norm(got.double() - ref))
    mod = float(torch.linalg.norm(model - ref))
    assert off <= 2 * mod + HALF[torch.bfloat16] * norm, (
        f"{name}: off by {off / norm:.3e}, the storage model by {mod / norm:.3e}")
