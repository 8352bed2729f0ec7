"""The block-seam calls on the CPU: struct layout, refusals before any device
is touched, empty sizes.  No kernel is launched here."""

from __future__ import annotations

import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests.test_owner_refusals import on_device

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an aligned stand-in address: never dereferenced by the checks
BF = torch.bfloat16


def layout_matches(cls, consts: dict):
    """Offsets and constants of the header, against the binding's."""
    fields = [f for f, _ in cls._fields_]
    prog = ["#include <stddef.h>", "#include <stdio.h>", '#include "zero_shard.h"',
            "int main(void) {", f'printf("size %zu\\n", sizeof({cls.__name__}));']
    prog += [f'printf("{f} %zu\\n", offsetof({cls.__name__}, {f}));' for f in fields]
    prog += [f'printf("{c} %d\\n", (int){c});' for c in consts] + ["return 0; }"]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(src, "w").write("\n".join(prog))
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), src, "-o", exe],
                       check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    got = dict(line.split() for line in out.strip().splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f
    for c, v in consts.items():
        assert int(got[c]) == v, c


def test_struct_layout_matches_header():
    layout_matches(Z.zs_blocknorm_desc, {c: getattr(Z, c) for c in (
        "ZS_NORM_LAYER", "ZS_NORM_RMS", "ZS_GATE_NONE", "ZS_GATE_COLUMN", "ZS_GATE_SIGMOID",
        "ZS_BLOCKNORM_MAX_COLS")})


def _desc(**kw):
    base = dict(rows=4, cols=64, dtype=Z.ZS_BF16, param_dtype=Z.ZS_BF16, kind=Z.ZS_NORM_RMS,
                post=1, gate=Z.ZS_GATE_COLUMN, eps=1e-5, residual_scale=1.0)
    base.update(kw)
    return Z.zs_blocknorm_desc(**base)


def _fwd(d, x=P, block=P, gate=P, gamma_post=P, beta_post=P, gamma=P, beta=P, total=2 * P,
         y=3 * P, stats=P):
    return Z._lib.zero_shard_blocknorm(ctypes.byref(d), x, block, gate, gamma_post, beta_post,
                                       gamma, beta, total, y, stats)


def _bwd(d, dy=P, dsum=None, total=P, block=P, gate=P, gamma_post=P, beta_post=P, gamma=P,
         stats=P, dx=2 * P, dblock=3 * P, dgate=P, dgamma_post=P, dbeta_post=P, dgamma=P, dbeta=P,
         ws=P, size=1 << 40):
    return Z._lib.zero_shard_blocknorm_bwd(
        ctypes.byref(d), dy, dsum, total, block, gate, gamma_post, beta_post, gamma, stats, dx,
        dblock, dgate, dgamma_post, dbeta_post, dgamma, dbeta, ws, size)


BAD = [dict(rows=-1), dict(cols=0), dict(cols=Z.ZS_BLOCKNORM_MAX_COLS + 1), dict(dtype=3),
       dict(dtype=-1), dict(param_dtype=Z.ZS_F16), dict(dtype=Z.ZS_F32), dict(kind=2),
       dict(kind=-1), dict(post=2), dict(post=-1), dict(gate=3), dict(gate=-1), dict(eps=-1e-5),
       dict(eps=float("nan")), dict(eps=float("inf")), dict(residual_scale=float("nan")),
       dict(residual_scale=float("-inf"))]
BAD += [{"ld_" + n: ld} for n in ("x", "block", "gate", "sum", "y", "dy", "dsum", "dx", "dblock",
                                  "dgate") for ld in (63, -1)]


@pytest.mark.parametrize("kw", BAD)
def test_refuses_bad_descriptors(kw):
    d = _desc(**kw)
    assert _fwd(d) == Z.ZS_EINVAL
    assert _bwd(d) == Z.ZS_EINVAL
    assert Z.zero_shard_blocknorm_workspace(d) == -1


@pytest.mark.parametrize("kw,desc,code", [
    (dict(x=None), {}, Z.ZS_EINVAL), (dict(y=None), {}, Z.ZS_EINVAL),
    (dict(block=None), {}, Z.ZS_EINVAL), (dict(total=None), {}, Z.ZS_EINVAL),
    (dict(total=3 * P), {}, Z.ZS_EINVAL),  # y would overwrite the sum
    (dict(gate=None), {}, Z.ZS_EINVAL), (dict(), dict(gate=Z.ZS_GATE_NONE), Z.ZS_EINVAL),
    (dict(), dict(post=0), Z.ZS_EINVAL),  # a gain of a norm that is not there
    (dict(beta_post=None), dict(post=0), Z.ZS_EINVAL),
    # no block, but a gate, a first norm or a scale for it
    (dict(block=None, total=None), {}, Z.ZS_EINVAL),
    (dict(block=None, total=None, gate=None, gamma_post=None, beta_post=None),
     dict(gate=0, post=0, residual_scale=2.0), Z.ZS_EINVAL),
    (dict(block=None, total=None, gate=None), dict(gate=0), Z.ZS_EINVAL),
    (dict(x=P + 1), {}, Z.ZS_EALIGN), (dict(block=P + 1), {}, Z.ZS_EALIGN),
    (dict(gate=P + 1), {}, Z.ZS_EALIGN), (dict(gate=P + 2), dict(param_dtype=0), Z.ZS_EALIGN),
    (dict(gamma=P + 1), {}, Z.ZS_EALIGN), (dict(beta=P + 1), {}, Z.ZS_EALIGN),
    (dict(gamma_post=P + 1), {}, Z.ZS_EALIGN), (dict(beta_post=P + 1), {}, Z.ZS_EALIGN),
    (dict(total=P + 1), {}, Z.ZS_EALIGN), (dict(y=P + 1), {}, Z.ZS_EALIGN),
    (dict(stats=P + 2), {}, Z.ZS_EALIGN),
])
def test_forward_refuses_bad_pointers(kw, desc, code):
    assert _fwd(_desc(**desc), **kw) == code


@pytest.mark.parametrize("kw,desc,code", [
    (dict(dy=None), {}, Z.ZS_EINVAL), (dict(total=None), {}, Z.ZS_EINVAL),
    (dict(stats=None), {}, Z.ZS_EINVAL), (dict(dx=None), {}, Z.ZS_EINVAL),
    (dict(block=None), {}, Z.ZS_EINVAL), (dict(dblock=None), {}, Z.ZS_EINVAL),
    (dict(dx=3 * P), {}, Z.ZS_EINVAL), (dict(gate=None), {}, Z.ZS_EINVAL),
    (dict(gate=None), dict(gate=Z.ZS_GATE_NONE), Z.ZS_EINVAL),  # a gradient of no gate
    (dict(gamma_post=None, beta_post=None), dict(post=0), Z.ZS_EINVAL),
    (dict(ws=None), {}, Z.ZS_EINVAL), (dict(size=0), {}, Z.ZS_EINVAL),
    (dict(block=None, dblock=None), {}, Z.ZS_EINVAL),
    (dict(ws=P + 8), {}, Z.ZS_EALIGN), (dict(dy=P + 1), {}, Z.ZS_EALIGN),
    (dict(dsum=P + 1), {}, Z.ZS_EALIGN), (dict(dx=P + 1), {}, Z.ZS_EALIGN),
    (dict(dblock=P + 1), {}, Z.ZS_EALIGN), (dict(dgate=P + 1), {}, Z.ZS_EALIGN),
    (dict(dgamma=P + 1), {}, Z.ZS_EALIGN), (dict(dbeta=P + 1), {}, Z.ZS_EALIGN),
    (dict(dgamma_post=P + 1), {}, Z.ZS_EALIGN), (dict(dbeta_post=P + 1), {}, Z.ZS_EALIGN),
    (dict(stats=P + 2), {}, Z.ZS_EALIGN),
])
def test_backward_refuses_bad_pointers(kw, desc, code):
    assert _bwd(_desc(**desc), **kw) == code


def test_workspace_bound_is_exact():
    d = _desc(rows=1000, cols=777)
    need = Z.zero_shard_blocknorm_workspace(d)
    assert need > 0 and need % (4 * 777 * 4) == 0
    assert _bwd(d, size=need - 1) == Z.ZS_EINVAL
    assert Z.zero_shard_blocknorm_workspace(_desc(rows=0)) == 0


def test_no_rows_is_nothing():
    d = _desc(rows=0)
    none = dict.fromkeys(("x", "block", "gate", "total", "y", "stats"))
    assert _fwd(d, **none) == Z.ZS_OK
    none = dict.fromkeys(("dy", "total", "block", "gate", "stats", "dx", "dblock", "dgate",
                          "dgamma_post", "dbeta_post", "dgamma", "dbeta", "ws"))
    assert _bwd(d, **none, size=0) == Z.ZS_OK


def test_valid_calls_reach_the_device_check():
    """Here there is none; on a GPU machine these pointers must not be used."""
    if torch.cuda.is_available():
        pytest.skip("stand-in pointers")
    assert _fwd(_desc()) == Z.ZS_EDEVICE
    assert _bwd(_desc()) == Z.ZS_EDEVICE
    plain = dict(block=None, gate=None, gamma_post=None, beta_post=None)
    d = _desc(gate=0, post=0)
    assert _fwd(d, total=None, **plain) == Z.ZS_EDEVICE
    assert _bwd(d, dblock=None, dgate=None, dgamma_post=None, dbeta_post=None,
                **plain) == Z.ZS_EDEVICE


def _owner(gate="column", rows=4, cols=64):
    o = object.__new__(Z.ZeroBlockNorm)
    o.shape, o.dtype, o.param_dtype, o.gate = (rows, cols), BF, BF, gate
    o.desc = _desc(rows=rows, cols=cols)
    o.stats = on_device(torch.zeros(2, rows))
    return o


@pytest.mark.parametrize("name", ["x", "block", "sum_out", "y", "gate"])
def test_owner_refuses_rows_that_share_memory(name):
    o = _owner("sigmoid")
    t = {n: on_device(torch.zeros(4, 64, dtype=BF)) for n in ("x", "block", "sum_out", "y", "gate")}
    t[name] = on_device(torch.zeros(64, dtype=BF).expand(4, 64))
    with pytest.raises(Z.ZeroShardError):
        o.forward(t["x"], t["block"], t["sum_out"], t["y"], gate=t["gate"])


@pytest.mark.parametrize("bad", [dict(gate=(4, 64)), dict(gamma=(63,)), dict(beta=(65,)),
                                 dict(gamma_post=(4, 64)), dict(beta_post=(1,))])
def test_owner_refuses_parameters_of_other_shapes(bad):
    o, row = _owner(), on_device(torch.zeros(4, 64, dtype=BF))
    p = {n: on_device(torch.zeros(shape, dtype=BF)) for n, shape in bad.items()}
    with pytest.raises(Z.ZeroShardError):
        o.forward(row, row, row, row, **p)


def test_owner_refuses_other_types_and_stats():
    o, row = _owner(), on_device(torch.zeros(4, 64, dtype=BF))
    with pytest.raises(Z.ZeroShardError):
        o.forward(on_device(torch.zeros(4, 64)), row, row, row)
    with pytest.raises(Z.ZeroShardError):
        o.backward(row, row, row, row, row, stats=on_device(torch.zeros(4, 4)))
    for kw in (dict(kind="batch"), dict(gate="tanh")):
        with pytest.raises(Z.ZeroShardError):
            Z.blocknorm_desc(rows=4, cols=64, **kw)
