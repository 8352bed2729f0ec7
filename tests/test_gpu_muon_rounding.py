"""The bf16 update of the Muon momentum is the bf16 of its binary32 value: where
that value is half way between two bf16 ones, what binary32 dropped does not
decide."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("n", [3, 1024])
def test_bf16_update_is_rounded_from_binary32(n):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.ones(n, device="cuda", dtype=BF)
    m = torch.full((n,), 2.0 ** -7 + 2.0 ** -29, device="cuda")
    # 1 + 2^-8 + 2^-30 in binary64, 1 + 2^-8 in binary32, half way to bf16's next
    exact = 0.5 * m.double() + 1.0
    assert (exact.float() == 1.0 + 2.0 ** -8).all() and (exact > 1.0 + 2.0 ** -8).all()
    for dtype in (F32, BF):
        out, u = torch.empty_like(m), torch.empty(n, device="cuda", dtype=dtype)
        Z.check(Z.zero_shard_muon_momentum(
            Z.muon_desc(n=n, mu=0.5, nesterov=False, dtype=dtype), [g], m, out, u))
        assert torch.equal(out, exact.float())
        assert torch.equal(u, exact.float().to(dtype))
    assert (u == 1.0).all()
