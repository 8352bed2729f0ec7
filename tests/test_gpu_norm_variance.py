"""Layer norm of rows whose variance is below what binary32 resolves beside their
mean: constant rows far from zero give beta, and finite statistics."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _check(values, cols, eps, dtype=F32):
    rows = len(values)
    x = torch.tensor(values, device="cuda", dtype=F32).to(dtype)[:, None].repeat(1, cols)
    beta = R.randn(cols, dtype=dtype, seed=3)
    y = torch.empty_like(x)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=dtype, eps=eps)
    ln.forward(x, y, beta=beta)
    assert torch.isfinite(ln.rstd).all() and torch.isfinite(ln.mean).all() and torch.isfinite(y).all()
    # eps in binary32, its root and quotient
    most = float(torch.tensor(eps, dtype=F32)) ** -0.5
    assert float(ln.rstd.max()) <= most * (1 + 4 * R.U)
    size = x.double().abs().amax(1, keepdim=True)
    # A sum of the row is off by at most 64 half steps (32 elements a thread, 10
    # levels) of its size, and so is that of the deviations from such a mean, which
    # are that error: their square, with its own roundings, is what is left.
    off = (66 * R.U) ** 2 * size * most + 2 * R.U * beta.double().abs()
    R.within("y", y, beta.double().expand(rows, cols), off + R.half_step(dtype, beta.double().abs() + off))
    # the mean: corrected once, then rounded
    R.within("mean", ln.mean, x[:, 0].double(), 2 * R.U * size[:, 0])


@pytest.mark.parametrize("cols,eps,value", [
    (1000, 1e-12, 13304.465), (1000, 1e-6, 1.37e7), (1000, 1e-5, 1.85e9), (1601, 1e-5, 64653680.0),
    (2000, 1e-5, 58262704.0)])
def test_one_constant_row(cols, eps, value):
    _check([value], cols, eps)


# one wave a row, several, sixteen columns a thread, sweeps; rows one and two at a
# time
@pytest.mark.parametrize("rows", [300, 2050])
@pytest.mark.parametrize("cols", [3, 100, 1000, 1601, 2000, 5120, 8200, 16385, 16400])
def test_constant_rows(rows, cols):
    g = torch.Generator().manual_seed(cols)
    values = (10.0 ** (3 + 7 * torch.rand(rows, generator=g))).tolist()
    for eps in (1e-5, 1e-12):
        _check(values, cols, eps)
    _check(values[:64], cols, 1e-5, BF)
