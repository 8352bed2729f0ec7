"""Element gates of a seam on the GPU near the ends of binary32: right to their rounding
while they are normal numbers, zeros below."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R
from tests._seam import GATE
from tests.test_gpu_seam import _gpu_cleanup  # noqa: F401

pytestmark = pytest.mark.gpu
F32 = torch.float32
NORMAL = 2.0 ** -126
ZS = [-20.0, -50.0, -80.0, -86.0, -87.0, -87.3, -87.35, -87.5, -88.0, -95.0, -100.0, -103.9,
      -110.0, -149.0, -151.0, -1e30, 20.0, 50.0, 86.0, 87.3, 87.35, 88.0, 100.0, 151.0, 1e30]


@pytest.mark.parametrize("size", [1.0, 2.0 ** 90])
@pytest.mark.parametrize("cols", [len(ZS), 64 * len(ZS)])
def test_gates_where_they_leave_binary32(size, cols):
    """sum = sigmoid(z) block beside no residual; dz = dsum block slope, dblock = dsum
    sigmoid(z) without gradients of y.  Blocks of 2^90 bring gates of 2^-126 to where a
    subnormal one would show."""
    rows = 3
    z = torch.tensor(ZS, device="cuda").repeat(rows, cols // len(ZS))
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=F32, gate="sigmoid", post=False)
    block, zeros = torch.full_like(z, size), torch.zeros_like(z)
    total, y, dx, db, dz = (torch.empty_like(z) for _ in range(5))
    plan.forward(zeros, block, total, y, gate=z)
    plan.backward(zeros, total, block, dx, db, dsum=torch.ones_like(z), gate=z, dgate=dz)
    gate, other = torch.sigmoid(z.double()), torch.sigmoid(-z.double())
    slope = gate * other
    for name, got, part, by in (("sum", total, gate, size), ("dblock", db, gate, 1.0),
                                ("dz", dz, slope, size)):
        want = torch.where(part >= NORMAL, part, 0.0) * by
        # a gate or slope, and a product's rounding
        R.within(name, got, want, (2 * GATE + 2 * R.U) * want)


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,cols", [(40, 7), (700, 511), (1500, 1601), (300, 5123), (20, 9001)])
def test_y_over_the_gates(rows, cols, kind, dtype):
    """The bits of a new buffer, sum over x or block at once."""
    x, block, z = (R.randn(rows, cols, seed=k).to(dtype) for k in range(3))
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=dtype, kind=kind, gate="sigmoid")
    total, y = torch.empty_like(x), torch.empty_like(x)
    plan.forward(x, block, total, y, gate=z)
    for over in (None, "x", "block"):
        t = {"x": x.clone(), "block": block.clone(), None: torch.empty_like(x)}
        gates = z.clone()
        plan.forward(t["x"], t["block"], t[over], gates, gate=gates)
        assert torch.equal(t[over], total) and torch.equal(gates, y), over
