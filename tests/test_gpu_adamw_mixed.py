"""AdamW on the GPU over lists of tensors whose states are in 32 and in 8 bits: the norm of long
lists, whose waves go on from tensor to tensor, and steps of more tensors than a launch takes,
with their weights and copies."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R
from tests.test_gpu_adamw import LR, Case, _gpu_cleanup, reference  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
TYPES = (BF, F32, F16)


def _norm_of(sizes, shift):
    """gnorm of tensors of these (elements, bits, type), of whole numbers whose sum of
    squares binary64 holds: any element left out or taken twice is seen."""
    tensors, grads, want = [], [], 0
    for k, (n, bits, dtype) in enumerate(sizes):
        gen = torch.Generator(device="cuda").manual_seed(k)
        g = torch.randint(-3, 4, (n + shift,), device="cuda", generator=gen)[shift:]
        # ends, and borders of chunks, waves and workgroups, stand out
        for c in (1, 256, 1024, 2048, 8192, 16384, 65536):
            g[c - 1:: c * 7][:50] = 128
            g[c::c * 5][:50] = -192
        g[-1:] = 240
        want += int((g * g).sum())
        buf = torch.full((n + shift + 9,), 255.0, device="cuda").to(dtype)
        buf[shift:shift + n] = g.to(dtype)
        grads.append(buf[shift:shift + n] if n else None)
        state = Z.adamw_state(n, bits)
        tensors.append(Z.adamw_tensor(torch.empty(n, device="cuda"), state["m"], state["v"],
                                      m_scale=state.get("m_scale"), v_scale=state.get("v_scale"),
                                      grad_dtype=dtype))
    assert want < 2 ** 53
    opt = Z.ZeroAdamW(tensors, max_norm=1.0)
    got = torch.full((1,), -1.0, device="cuda", dtype=F64)
    opt.gnorm(grads, got)
    assert float(got) == want, (float(got), want)


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("big", [(17_000_005, 8, BF), (8_500_001, 32, F32), (17_000_005, 8, F16)])
def test_norm_of_a_long_list(big, shift):
    """More than 8192 chunks: a wave has eight, of one tensor or of several, of both lengths."""
    short = [((k * 977) % 9000, (8, 32)[k * k % 3 % 2], TYPES[k % 3]) for k in range(300)]
    _norm_of([*short[:100], big, *short[100:], (4097, 32, BF)], shift)


def test_norm_of_many_short_tensors_beside_one_another():
    """As many chunks of tensors of a chunk or two each, both kinds in every group."""
    sizes = [(40_000 + (k * 977) % 9000, (8, 32)[k % 2], TYPES[k % 3]) for k in range(500)]
    _norm_of(sizes, 0)


def test_norm_at_the_border_of_a_short_list():
    """8191, 8192 and 8193 chunks of a state in 32 bits."""
    for chunks in (8191, 8192, 8193):
        _norm_of([(1024 * (chunks - 2) - 5, 32, BF), (1, 32, F16), (1024, 32, F32)], 0)


def _mixed(sizes, clip):
    cases = [Case([n], bits, grad, param=(BF, F16, None)[k % 3], seed=1000 + 7 * k)
             for k, (n, bits, grad) in enumerate(sizes)]
    opt = Z.ZeroAdamW([c.tensors()[0] for c in cases], max_norm=0.5 if clip else 0.0)
    grads = [c.grads()[0] if c.sizes[0] else None for c in cases]
    coef, sumsq = 1.0, None
    if clip:
        sumsq = torch.zeros(1, device="cuda", dtype=F64)
        opt.gnorm(grads, sumsq)
        want = sum(float((g.double() ** 2).sum()) for g in grads if g is not None)
        # 2^-53 for each of the additions behind a sum, 16 and 10 levels at most
        assert abs(float(sumsq) - want) <= 64 * 2.0 ** -53 * want
        coef = min(1.0, 0.5 / (float(sumsq) ** 0.5 + 1e-6))
        assert coef < 1.0
    for t in (1, 4):
        before = [c.state()[0] for c in cases]
        opt.step(grads, LR, t, sumsq, key=70 + t)
        for k, (c, old) in enumerate(zip(cases, before)):
            it = c.items[0]
            for name, ref in reference(c, k, old, t, coef, key=70 + t).items():
                got = it[name].cpu().numpy()
                if name == "master":
                    # Binary64 to a few of its half steps, then one rounding.  In 8 bits u's
                    # denominator (a product, a sum), its inverse (two half steps) and the
                    # product with m' are within 5 half steps of binary32, the reference's
                    # three roundings within 3: 8 half steps of what the step moves.  That is not
                    # bounded by the rate: an r of 0 beside an m that is not, and gradients
                    # clipped to a hundredth, leave m' / sqrt(v') at 1000 and more.
                    keep = old["master"].double().cpu().numpy() * (1 - LR * c.decay)
                    moved = np.abs(ref - keep) + R.U * np.abs(ref)
                    off = np.abs(got.astype(np.float64) - ref.astype(np.float64))
                    ok = off <= 2 * R.U * np.abs(ref) + (8 * R.U * moved if c.bits == 8 else 0)
                    assert ok.all(), (k, c.sizes, moved[~ok], off[~ok], ref[~ok])
                else:  # states in 32 bits and scales are the definition's, and so are numbers
                    assert np.array_equal(got, ref[0] if isinstance(ref, list) else ref), (k, name)
            if it["param"] is not None:
                assert torch.equal(it["param"], it["master"].to(it["param"].dtype)), k


@pytest.mark.parametrize("clip", [False, True])
def test_a_plan_of_both_kinds(clip):
    _mixed([(5000, 8, BF), (100, 32, F32), (4096, 8, F32), (77, 32, F16), (9000, 8, F16),
            (70_001, 32, BF), (0, 8, BF), (2049, 32, F32)], clip)


@pytest.mark.parametrize("clip", [False, True])
def test_more_tensors_of_both_kinds_than_a_launch_takes(clip):
    """Empty ones among them; a group of states in 32 bits only, and one of both behind it."""
    sizes = [((k * 37) % 2100 if k % 11 else 0, 32 if k < 440 else (8, 32)[k % 2], TYPES[k % 3])
             for k in range(900)]
    _mixed(sizes, clip)
