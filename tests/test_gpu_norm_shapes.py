"""Layer norm over many rows, where a workgroup goes on from rows to rows, two
at a time, and several row groups share a workgroup: forward and backward, even
and odd widths, every type, against the formulas in 64 bits."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# one column to more than the registers take; rows one short of and past two
# at a time, more than all workgroups hold at once
SIZES = [(1024, 1), (5001, 7), (9000, 100), (4097, 512), (3001, 520), (2500, 1001), (1025, 2049),
         (1024, 8192), (1100, 8200), (1030, 9001), (1027, 16385)]


@pytest.mark.parametrize("dtype,ptype", [(F32, F32), (BF, BF), (F16, F32)])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_many_rows(rows, cols, dtype, ptype):
    x = R.randn(rows, cols, dtype=dtype, seed=1)
    res = R.randn(rows, cols, dtype=dtype, seed=2)
    gamma = (1.0 + R.randn(cols, seed=3, scale=0.2)).to(ptype)
    beta = R.randn(cols, seed=4, scale=0.3).to(ptype)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=dtype, param_dtype=ptype, eps=1e-5)
    y, s, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    ln.forward(x, y, gamma=gamma, beta=beta, residual=res, sum_out=s)
    assert torch.equal(s, (x.float() + res.float()).to(dtype))
    (ry, ty), (rm, tm), (rr, tr) = R.layernorm_ref(s, gamma, beta, 1e-5)
    R.within("y", y, ry, ty + R.half_step(dtype, ry.abs() + ty))
    R.within("mean", ln.mean, rm, tm + R.U * rm.abs())
    R.within("rstd", ln.rstd, rr, tr + 2 * R.U * rr)
    dy = R.randn(rows, cols, dtype=dtype, seed=5)
    dsum = R.randn(rows, cols, dtype=dtype, seed=6)
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
    ln.backward(dy, s, dx, gamma=gamma, dgamma=dgamma, dbeta=dbeta, dsum=dsum)
    # a column's longest chain: a workgroup's rows (at least 256 workgroups share
    # them), up to 16 row groups, a quarter of the partials of one of 64 groups
    serial = rows // 256 + 2 + 16 + 4 + 64
    (rx, tx), (rg, tg), (rb, tb) = R.layernorm_bwd_ref(dy, s, gamma, ln.mean, ln.rstd, dsum, serial)
    R.within("dx", dx, rx, tx + R.half_step(dtype, rx.abs() + tx))
    R.within("dgamma", dgamma, rg, tg + R.half_step(ptype, rg.abs() + tg))
    R.within("dbeta", dbeta, rb, tb + R.half_step(ptype, rb.abs() + tb))


@pytest.mark.parametrize("rows,cols", [(2049, 72), (1500, 1001), (1024, 8200)])
def test_many_rows_in_place_and_again(rows, cols):
    """In place and a second time: the same bits."""
    x = R.randn(rows, cols, dtype=BF, seed=1)
    dy = R.randn(rows, cols, dtype=BF, seed=2)
    gamma = R.randn(cols, dtype=BF, seed=3)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=BF)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    ln.forward(x, y, gamma=gamma)
    ln.backward(dy, x, dx, gamma=gamma, dgamma=dg, dbeta=db)
    z, dz, eg, eb = x.clone(), dy.clone(), torch.empty_like(gamma), torch.empty_like(gamma)
    ln.workspace.fill_(255)
    ln.backward(dz, x, dz, gamma=gamma, dgamma=eg, dbeta=eb)
    ln.forward(z, z, gamma=gamma)
    assert torch.equal(z, y) and torch.equal(dz, dx)
    assert torch.equal(eg, dg) and torch.equal(eb, db)
