"""The Muon update's elementwise passes over more elements than one of their
launches takes: the elements around the seams equal those of a short call."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
N = (1 << 34) + 1003
PARTS = [slice(0, 2048), slice((1 << 34) - 2048, N)]  # the second: both sides of the seam


@pytest.fixture(autouse=True)
def _gpu_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 160e9:
        pytest.skip("137 GB for the ranges")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _range(dtype, seed):
    t = torch.zeros(N, device="cuda", dtype=dtype)
    for i, p in enumerate(PARTS):
        t[p] = R.randn(p.stop - p.start, dtype=dtype, seed=seed + i)
    return t


def _short(t):
    return [t[p].clone() for p in PARTS]


def test_momentum():
    g, m = _range(BF, 1), _range(F32, 5)
    u = torch.full((N,), 3.0, device="cuda", dtype=BF)
    sg, sm = _short(g), _short(m)
    Z.check(Z.zero_shard_muon_momentum(Z.muon_desc(n=N), [g], m, m, u))
    for p, a, b in zip(PARTS, sg, sm):
        out, v = torch.empty_like(b), torch.empty_like(a)
        Z.check(Z.zero_shard_muon_momentum(Z.muon_desc(n=b.numel()), [a], b, out, v))
        assert torch.equal(m[p], out) and torch.equal(u[p], v)
    assert float(u[4096:1 << 33].amax()) == 0.0 == float(u[4096:1 << 33].amin())


def test_apply():
    o, w = _range(BF, 1), _range(F32, 5)
    param = torch.full((N,), 3.0, device="cuda", dtype=BF)
    so, sw = _short(o), _short(w)
    Z.check(Z.zero_shard_muon_apply(Z.muon_desc(n=N, weight_decay=0.1), o, 0.02, 0.2, w, w, param))
    for p, a, b in zip(PARTS, so, sw):
        out, v = torch.empty_like(b), torch.empty_like(a)
        Z.check(Z.zero_shard_muon_apply(Z.muon_desc(n=b.numel(), weight_decay=0.1), a, 0.02, 0.2, b,
                                        out, v))
        assert torch.equal(w[p], out) and torch.equal(param[p], v)
    assert float(param[4096:1 << 33].amax()) == 0.0 == float(param[4096:1 << 33].amin())
