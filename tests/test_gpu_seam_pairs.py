"""Seams of many rows of 16-bit types on the GPU, which are taken two at a time: wide rows,
those that end inside a thread's eight columns among them, odd numbers of rows, the next
rows loaded ahead from buffers that are written in place."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests.test_gpu_seam import (BF, F16, F32, SCALE, _backward, _check_forward, _gpu_cleanup,  # noqa: F401
                                 _inputs, _rows)

pytestmark = pytest.mark.gpu
EPS = 1e-5

# one pass over the rows and several, an odd row at the end, the widest rows of two at a
# time, one column more and less than a thread's
SIZES = [(1030, 4099), (1100, 6143), (1025, 4097), (1027, 6137), (1030, 5120), (1024, 6144),
         (2051, 5128), (1025, 72), (3333, 1024)]
TYPES = [(BF, BF), (BF, F32), (F16, F16), (F16, F32)]
WAYS = [("rms", "none"), ("rms", "column"), ("layer", "none"), ("layer", "column")]


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward_of_pairs(rows, cols, dtype, ptype):
    for i, (kind, gate) in enumerate(WAYS):
        pad, affine, post = (0, 8, 3, 0)[i], i != 1, i != 2
        p = _inputs(rows, cols, dtype, ptype, gate, pad, affine)
        if not post:
            p["gamma_post"] = p["beta_post"] = None
        plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=dtype, param_dtype=ptype, kind=kind,
                               gate=gate, post=post, eps=EPS, residual_scale=SCALE)
        total, y = _rows(rows, cols, dtype, pad, 5), _rows(rows, cols, dtype, 0, 6)
        plan.forward(p["x"], p["block"], total, y,
                     **{k: v for k, v in p.items() if k not in ("x", "block")})
        _check_forward(plan, p, kind, gate, post, total, y, float(torch.tensor(SCALE)))


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward_of_pairs(rows, cols, dtype, ptype):
    for i, (kind, gate) in enumerate(WAYS):
        _backward(rows, cols, dtype, ptype, kind, gate, (0, 8, 3, 0)[i], i != 1, i != 2,
                  dsum=i != 3)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("cols", [96, 515, 1000, 4099, 5120, 6143])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_pairs_in_place(kind, cols, dtype):
    """The bits of new buffers: sum over x or block, y over the other; dx and dblock over
    what they are the gradients from."""
    rows, gate = 2501, "column"
    p = _inputs(rows, cols, dtype, F32, gate, 0)
    args = {k: v for k, v in p.items() if k not in ("x", "block")}
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=dtype, param_dtype=F32, kind=kind,
                           gate=gate, residual_scale=SCALE)
    total, y = torch.empty_like(p["x"]), torch.empty_like(p["x"])
    plan.forward(p["x"], p["block"], total, y, **args)
    for swap in (False, True):
        x, b = p["x"].clone(), p["block"].clone()
        s2, y2 = (b, x) if swap else (x, b)
        plan.forward(x, b, s2, y2, **args)
        assert torch.equal(s2, total) and torch.equal(y2, y)
    dy, ds = _rows(rows, cols, dtype, 0, 30), _rows(rows, cols, dtype, 0, 31)
    dx, db = torch.empty_like(dy), torch.empty_like(dy)
    pars = {k: p[k] for k in ("gate", "gamma_post", "beta_post", "gamma")}
    grads = {"d" + k: torch.empty(cols, device="cuda") for k in (*pars, "beta")}
    plan.backward(dy, total, p["block"], dx, db, dsum=ds, **pars, **grads)
    want = {k: v.clone() for k, v in grads.items()}
    for use in (("dy", "block"), ("dsum", "sum"), ("sum", "dy"), ("block", "dsum")):
        t = {"dy": dy.clone(), "dsum": ds.clone(), "sum": total.clone(),
             "block": p["block"].clone()}
        plan.backward(t["dy"], t["sum"], t["block"], t[use[0]], t[use[1]], dsum=t["dsum"], **pars,
                      **grads)
        assert torch.equal(t[use[0]], dx) and torch.equal(t[use[1]], db), use
        assert all(torch.equal(grads[k], want[k]) for k in want), use
