"""States in 8 bits on the GPU, number for number: every byte and every scale is the one
that the definition in binary32 gives, over gradients of every type and size."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R
from tests.test_gpu_adamw import LR, Case, _gpu_cleanup, reference  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _is_the_definitions(case, before, t, key, coef=1.0):
    for k, (it, old) in enumerate(zip(case.items, before)):
        want = reference(case, k, old, t, coef, key)
        for name in ("m", "v"):
            scale = it[name + "_scale"].cpu().numpy()
            bad = scale.view(np.uint32) != want[name + "_scale"].view(np.uint32)
            assert not bad.any(), (name, k, "scales", int(bad.sum()), int(bad.argmax()))
            bad = it[name].cpu().numpy() != want[name][0]
            assert not bad.any(), (name, k, "numbers", int(bad.sum()), int(bad.argmax()))


@pytest.mark.parametrize("grad", [F32, BF, F16])
def test_stored_numbers(grad):
    case = Case([3_000_001, 70_001, 257, 5], 8, grad)
    opt = Z.ZeroAdamW(case.tensors())
    for t in (1, 2, 7):
        before = case.state()
        opt.step(case.grads(), LR, t, key=77 + t)
        _is_the_definitions(case, before, t, 77 + t)


def test_stored_numbers_of_clipped_gradients():
    case = Case([300_001, 4096], 8, BF)
    opt = Z.ZeroAdamW(case.tensors(), max_norm=0.25)
    sumsq = torch.full((1,), 3.0, device="cuda", dtype=torch.float64)
    before = case.state()
    opt.step(case.grads(), LR, 3, sumsq, key=5)
    _is_the_definitions(case, before, 3, 5, coef=0.25 / (3.0 ** 0.5 + 1e-6))


@pytest.mark.parametrize("spread", [0.0, 12.0])
def test_stored_numbers_of_gradients_of_every_size(spread):
    """Blocks of gradients around 2^-110 to 2^46, from a state of zeros: below and above
    what is stored as zeros, squares that are no normal numbers."""
    blocks = 157 * 8
    size = torch.arange(blocks, device="cuda", dtype=F32).view(-1, 1) / 8 - 110
    sign = torch.sign(R.randn(blocks * 256, seed=2)).view(blocks, 256)
    g = sign * torch.exp2(size + spread * (R.randn(blocks * 256, seed=1).view(blocks, 256)
                                           .clamp(-3, 0)))
    case = Case([blocks * 256], 8, F32, param=None)
    it = case.items[0]
    it["grad"].copy_(g.reshape(-1))
    for k in ("m", "v"):
        it[k].zero_()
        it[k + "_scale"].zero_()
    opt = Z.ZeroAdamW(case.tensors())
    for t in (1, 2):
        before = case.state()
        opt.step(case.grads(), LR, t, key=t)
        _is_the_definitions(case, before, t, t)


@pytest.mark.parametrize("beta2", [0.0, 0.9, 0.999, 0.9999])
def test_roots_from_2_48_on_are_infinities_and_below_2_91_zeros(beta2):
    """Whatever beta2 is: blocks of one gradient each, whose roots are just below and just
    above either border."""
    root = (1.0 - float(np.float32(beta2))) ** 0.5
    size = torch.tensor([0.999 * 2.0 ** 48, 1.001 * 2.0 ** 48, 1.01 * 2.0 ** -91,
                         0.99 * 2.0 ** -91], device="cuda") / root
    case = Case([1024], 8, F32, param=None)
    it = case.items[0]
    it["grad"].copy_(size.repeat_interleave(256))
    for k in ("m", "v"):
        it[k].zero_()
        it[k + "_scale"].zero_()
    Z.ZeroAdamW(case.tensors(), beta2=beta2).step(case.grads(), LR, 1, key=1)
    scale = it["v_scale"].tolist()
    assert abs(scale[0] / (0.999 * 2.0 ** 40) - 1) < 1e-6 and scale[1] == float("inf")
    # its square times 2^32 is the least number, 2^-149
    assert abs(scale[2] * 2.0 ** 98.5 - 1) < 1e-6
    assert scale[3] == 0.0 and (it["v"][768:] == 0).all()
