"""How near the orthogonalised matrix comes to one in 64 bits rounded to bf16,
where the singular values lie close together, so that one rounding's effect on
them is the same everywhere and the polynomial's slope makes it larger.

A bf16 value is off by at most 2^-8 of itself, at the lower end of a binade, and
evenly spread: 2^-8 / sqrt(3) at the root of the mean square.  Over a whole binade
it is 0.7 of that, so that this bound leaves everything before the last rounding
as much again."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R

pytestmark = pytest.mark.gpu
BOUND = 2.0**-8 / 3**0.5


@pytest.fixture(autouse=True)
def _gpu_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _off(g):
    o = torch.empty_like(g, dtype=torch.bfloat16)
    Z.ZeroOrtho(rows=g.shape[0], cols=g.shape[1], dtype=g.dtype)(g, o)
    ref = R.ortho_ref(g, [R.COEFFS] * 5, 1e-7)
    return float((o.double() - ref).norm() / ref.norm())


# in one workgroup, and in strips, both orientations
@pytest.mark.parametrize("rows,cols", [(32, 256), (40, 320), (64, 64), (28, 13824), (32, 13824),
                                       (48, 13824), (13824, 40), (60, 870), (100, 700)])
def test_short(rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(3)
    assert _off(torch.randn(rows, cols, device="cuda", generator=gen)) < BOUND


@pytest.mark.parametrize("rows,cols", [(24, 100), (32, 600), (50, 3000), (128, 500)])
def test_short_equal(rows, cols):
    """All singular values the same."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    q = torch.linalg.qr(torch.randn(cols, rows, device="cuda", generator=gen))[0]
    assert _off(q.T.contiguous()) < BOUND


# products of tiles, cut and not, one step at a time and two
@pytest.mark.parametrize("rows,cols", [(136, 136), (256, 300), (400, 13824), (13824, 430),
                                       (480, 9000), (1000, 1000)])
def test_long(rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(5)
    assert _off(torch.randn(rows, cols, device="cuda", generator=gen)) < BOUND


@pytest.mark.parametrize("rows,cols", [(150, 700), (300, 400), (1024, 1500)])
def test_long_equal(rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(6)
    q = torch.linalg.qr(torch.randn(cols, rows, device="cuda", generator=gen))[0]
    assert _off(q.T.contiguous()) < BOUND


@pytest.mark.parametrize("rows,cols", [(40, 320), (48, 5000), (200, 210), (430, 5000)])
def test_batch(rows, cols):
    """Each matrix has the rests of its own diagonals."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    g = torch.randn(3, rows, cols, device="cuda", generator=gen)
    g[1] = torch.linalg.qr(g[1].T)[0].T
    o = torch.empty_like(g, dtype=torch.bfloat16)
    Z.ZeroOrtho(batch=3, rows=rows, cols=cols, dtype=g.dtype)(g, o)
    for i in range(3):
        ref = R.ortho_ref(g[i], [R.COEFFS] * 5, 1e-7)
        assert float((o[i].double() - ref).norm() / ref.norm()) < BOUND
