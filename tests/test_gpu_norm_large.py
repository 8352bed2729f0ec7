"""Layer norm's backward pass over rows whose mean times rstd is beyond binary32:
the threads past a row's end have nothing to add to its sums."""

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


# rows that end inside a thread's eight columns, and between threads
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 7), (5, 96), (1030, 100), (4, 128), (3, 1001),
                                       (2, 8200), (3, 8203), (2, 16385)])
def test_constant_rows(rows, cols, dtype):
    """x = mean everywhere: h is 0, dx = rstd (g - mean of g) and dgamma = 0."""
    value = 2.0 ** 121
    x = torch.full((rows, cols), value, device="cuda", dtype=dtype)
    mean = torch.full((rows,), value, device="cuda")
    rstd = torch.full((rows,), 316.0, device="cuda")
    dy = R.randn(rows, cols, dtype=dtype, seed=5)
    gamma = R.randn(cols, dtype=dtype, seed=6)
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=dtype)
    for g in (gamma, None):
        ln.backward(dy, x, dx, gamma=g, dgamma=dgamma, dbeta=dbeta, mean=mean, rstd=rstd)
        (rx, tx), _, (rb, tb) = R.layernorm_bwd_ref(dy, x, g, mean, rstd, None, rows // 256 + 86)
        R.within("dx", dx, rx, tx + R.half_step(dtype, rx.abs() + tx))
        assert not dgamma.any()
        R.within("dbeta", dbeta, rb, tb + R.half_step(dtype, rb.abs() + tb))
