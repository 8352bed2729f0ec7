"""Layer norm of more rows, each too long for registers, than a launch has
workgroups: every row is taken, in place, in both directions."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_more_long_rows_than_workgroups():
    rows, cols = (1 << 22) + 3, 16385
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 160e9:
        pytest.skip("137 GB for the rows")
    buf = torch.zeros(rows, cols, device="cuda", dtype=BF)
    at = torch.tensor([0, 1, 4194302, 4194303, 4194304, rows - 1], device="cuda")
    x = R.randn(len(at), cols, dtype=BF, seed=1)
    small = Z.ZeroLayerNorm(rows=len(at), cols=cols, dtype=BF)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    small.forward(x, y)
    small.backward(y, y, dx)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=BF)
    buf[at] = x
    ln.forward(buf, buf)
    assert torch.equal(buf[at], y)
    ln.backward(buf, buf, buf)
    assert torch.equal(buf[at], dx)
    buf[at] = 0.0
    assert float(buf.amax()) == 0.0 == float(buf.amin())  # the rows of zeros stay
    del buf
    torch.cuda.empty_cache()
