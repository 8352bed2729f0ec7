"""The example block learns: its loss falls."""

from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_muon_block_learns():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("muon_block",
                                                  os.path.join(ROOT, "examples", "muon_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=30)
    assert all(l == l for l in losses)
    assert losses[-1] < 0.5 * losses[0]
