"""The layer-norm and Muon calls on the CPU: struct layouts match the header,
bad arguments are refused before any device is touched, empty sizes queue
nothing, and valid calls get as far as the device check.  No kernel is
launched here."""

from __future__ import annotations

import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an aligned stand-in address: never dereferenced by the checks


@pytest.mark.parametrize("name", ["zs_layernorm_desc", "zs_muon_desc", "zs_ortho_desc"])
def test_struct_layout_matches_header(name):
    cls = getattr(Z, name)
    fields = [f for f, _ in cls._fields_]
    prog = ["#include <stddef.h>", "#include <stdio.h>", '#include "zero_shard.h"',
            "int main(void) {", f'printf("size %zu\\n", sizeof({name}));']
    prog += [f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f in fields]
    prog += ['printf("consts %d\\n", ZS_F32 + 10 * ZS_BF16 + 100 * ZS_F16 + '
             '1000 * ZS_ORTHO_MAX_STEPS);', "return 0; }"]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(src, "w").write("\n".join(prog))
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), src, "-o", exe],
                       check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    got = dict(line.split() for line in out.strip().splitlines())
    assert int(got.pop("size")) == ctypes.sizeof(cls)
    assert int(got.pop("consts")) == (Z.ZS_F32 + 10 * Z.ZS_BF16 + 100 * Z.ZS_F16
                                      + 1000 * Z.ZS_ORTHO_MAX_STEPS)
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f


def _norm_desc(**kw):
    base = dict(rows=4, cols=64, dtype=Z.ZS_BF16, param_dtype=Z.ZS_BF16, eps=1e-5)
    base.update(kw)
    return Z.zs_layernorm_desc(**base)


NORM_BAD = [dict(rows=-1), dict(cols=0), dict(cols=(1 << 31) + 1), dict(dtype=3), dict(dtype=-1),
            dict(param_dtype=Z.ZS_F16), dict(dtype=Z.ZS_F32), dict(eps=-1e-5),
            dict(eps=float("nan")), dict(eps=float("inf")), dict(ld_x=63), dict(ld_residual=-1),
            dict(ld_sum=1), dict(ld_y=63), dict(ld_dy=63), dict(ld_dsum=63), dict(ld_dx=63)]


def _fwd(d, x=P, residual=None, gamma=P, beta=P, total=None, y=2 * P, mean=P, rstd=P):
    return Z._lib.zero_shard_layernorm(ctypes.byref(d), x, residual, gamma, beta, total, y, mean,
                                       rstd)


def _bwd(d, dy=P, x=P, gamma=P, mean=P, rstd=P, dsum=None, dx=2 * P, dgamma=P, dbeta=P, ws=P,
         size=1 << 40):
    return Z._lib.zero_shard_layernorm_bwd(ctypes.byref(d), dy, x, gamma, mean, rstd, dsum, dx,
                                           dgamma, dbeta, ws, size)


@pytest.mark.parametrize("kw", NORM_BAD)
def test_layernorm_refuses_bad_descriptors(kw):
    d = _norm_desc(**kw)
    assert _fwd(d) == Z.ZS_EINVAL
    assert _bwd(d) == Z.ZS_EINVAL
    assert Z.zero_shard_layernorm_workspace(d) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), Z.ZS_EINVAL), (dict(y=None), Z.ZS_EINVAL),
    (dict(residual=P), Z.ZS_EINVAL), (dict(total=P), Z.ZS_EINVAL),
    (dict(residual=P, total=3 * P, y=3 * P), Z.ZS_EINVAL),  # y would overwrite the sum
    (dict(x=P + 1), Z.ZS_EALIGN), (dict(y=P + 1), Z.ZS_EALIGN),
    (dict(gamma=P + 1), Z.ZS_EALIGN), (dict(beta=P + 1), Z.ZS_EALIGN),
    (dict(mean=P + 2), Z.ZS_EALIGN), (dict(rstd=P + 2), Z.ZS_EALIGN),
    (dict(residual=P + 1, total=3 * P), Z.ZS_EALIGN),
])
def test_layernorm_refuses_bad_pointers(kw, code):
    assert _fwd(_norm_desc(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), Z.ZS_EINVAL), (dict(x=None), Z.ZS_EINVAL), (dict(dx=None), Z.ZS_EINVAL),
    (dict(mean=None), Z.ZS_EINVAL), (dict(rstd=None), Z.ZS_EINVAL),
    (dict(ws=None), Z.ZS_EINVAL), (dict(size=0), Z.ZS_EINVAL),
    (dict(ws=P + 8), Z.ZS_EALIGN), (dict(dy=P + 1), Z.ZS_EALIGN), (dict(dx=P + 1), Z.ZS_EALIGN),
    (dict(dsum=P + 1), Z.ZS_EALIGN), (dict(dgamma=P + 1), Z.ZS_EALIGN),
    (dict(dbeta=P + 1), Z.ZS_EALIGN), (dict(mean=P + 2), Z.ZS_EALIGN),
])
def test_layernorm_bwd_refuses_bad_pointers(kw, code):
    assert _bwd(_norm_desc(), **kw) == code


def test_layernorm_workspace_bound_is_exact():
    d = _norm_desc(rows=1000, cols=777)
    need = Z.zero_shard_layernorm_workspace(d)
    assert need > 0 and need % (2 * 777 * 4) == 0
    assert _bwd(d, size=need - 1) == Z.ZS_EINVAL
    assert Z.zero_shard_layernorm_workspace(_norm_desc(rows=0)) == 0


def test_layernorm_of_no_rows_is_nothing():
    d = _norm_desc(rows=0)
    assert _fwd(d, x=None, y=None, mean=None, rstd=None, gamma=None, beta=None) == Z.ZS_OK
    assert _bwd(d, dy=None, x=None, dx=None, mean=None, rstd=None, dgamma=None, dbeta=None,
                ws=None, size=0) == Z.ZS_OK


def _muon(**kw):
    base = dict(n=100, n_d=2, nesterov=1, dtype=Z.ZS_BF16, mu=0.95, weight_decay=0.1)
    base.update(kw)
    return Z.zs_muon_desc(**base)


def _table(*p):
    return (ctypes.c_void_p * len(p))(*p)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=1 << 62), dict(n_d=0), dict(n_d=65), dict(nesterov=2), dict(dtype=Z.ZS_F16),
    dict(mu=1.0), dict(mu=-0.1), dict(mu=float("nan")), dict(weight_decay=-1.0),
    dict(weight_decay=float("inf"))])
def test_muon_refuses_bad_descriptors(kw):
    d = ctypes.byref(_muon(**kw))
    assert Z._lib.zero_shard_muon_momentum(d, _table(*[P] * 65), P, P, P) == Z.ZS_EINVAL
    assert Z._lib.zero_shard_muon_apply(d, P, 0.1, 1.0, P, P, P) == Z.ZS_EINVAL


def test_muon_refuses_bad_arguments():
    d = ctypes.byref(_muon())
    mom, app = Z._lib.zero_shard_muon_momentum, Z._lib.zero_shard_muon_apply
    assert mom(None, _table(P, P), P, P, P) == Z.ZS_EINVAL
    assert mom(d, None, P, P, P) == Z.ZS_EINVAL
    assert mom(d, _table(P, None), P, P, P) == Z.ZS_EINVAL
    for i in range(3):
        args = [P, P, P]
        args[i] = None
        assert mom(d, _table(P, P), *args) == Z.ZS_EINVAL
        args[i] = P + 8
        assert mom(d, _table(P, P), *args) == Z.ZS_EALIGN
    assert mom(d, _table(P, P + 2), P, P, P) == Z.ZS_EALIGN
    for lr, scale in ((-1.0, 1.0), (float("nan"), 1.0), (0.1, float("inf")),
                      (0.1, float("nan"))):
        assert app(d, P, lr, scale, P, P, P) == Z.ZS_EINVAL
    for i in range(4):
        args = [P, P, P, P]
        args[i] = None
        assert app(d, args[0], 0.1, 1.0, *args[1:]) == Z.ZS_EINVAL
        args[i] = P + 8
        assert app(d, args[0], 0.1, 1.0, *args[1:]) == Z.ZS_EALIGN
    empty = ctypes.byref(_muon(n=0))
    assert mom(empty, None, None, None, None) == Z.ZS_OK
    assert app(empty, None, 0.1, 1.0, None, None, None) == Z.ZS_OK


def _ortho(**kw):
    base = dict(batch=2, rows=33, cols=70, dtype=Z.ZS_F32, steps=5, eps=1e-7)
    base.update(kw)
    d = Z.zs_ortho_desc(**{k: v for k, v in base.items() if k != "coeffs"})
    if "coeffs" in base:
        d._keep = (ctypes.c_float * len(base["coeffs"]))(*base["coeffs"])
        d.coeffs = ctypes.cast(d._keep, ctypes.POINTER(ctypes.c_float))
    return d


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(batch=65536), dict(rows=(1 << 20) + 1),
    dict(cols=(1 << 20) + 1), dict(dtype=3), dict(steps=0), dict(steps=Z.ZS_ORTHO_MAX_STEPS + 1),
    dict(eps=-1.0), dict(eps=float("nan")), dict(ld_in=69), dict(ld_out=69), dict(stride_in=-1),
    dict(stride_out=-1), dict(steps=1, coeffs=[3.0, float("nan"), 2.0])])
def test_ortho_refuses_bad_descriptors(kw):
    d = _ortho(**kw)
    assert Z.zero_shard_ortho_workspace(d) == -1
    assert Z._lib.zero_shard_ortho(ctypes.byref(d), P, 2 * P, 4 * P, 1 << 60) == Z.ZS_EINVAL


def test_ortho_refuses_bad_arguments():
    d = _ortho()
    need = Z.zero_shard_ortho_workspace(d)
    call = Z._lib.zero_shard_ortho
    assert need > 0
    assert call(None, P, P, P, need) == Z.ZS_EINVAL
    assert call(ctypes.byref(d), None, P, P, need) == Z.ZS_EINVAL
    assert call(ctypes.byref(d), P, None, P, need) == Z.ZS_EINVAL
    assert call(ctypes.byref(d), P, P, None, need) == Z.ZS_EINVAL
    assert call(ctypes.byref(d), P, P, P, need - 1) == Z.ZS_EINVAL
    assert call(ctypes.byref(d), P + 2, P, P, need) == Z.ZS_EALIGN
    assert call(ctypes.byref(d), P, P + 1, P, need) == Z.ZS_EALIGN
    assert call(ctypes.byref(d), P, P, P + 16, need) == Z.ZS_EALIGN
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0)):
        e = _ortho(**kw)
        assert Z.zero_shard_ortho_workspace(e) == 0
        assert call(ctypes.byref(e), None, None, None, 0) == Z.ZS_OK


def test_ortho_outputs_of_one_batch_may_not_overlap():
    # a batch stride shorter than a matrix would let its matrices overwrite
    # each other
    assert Z.zero_shard_ortho_workspace(_ortho(stride_out=33 * 70 - 1)) == -1
    assert Z.zero_shard_ortho_workspace(_ortho(stride_out=33 * 70)) > 0
    assert Z.zero_shard_ortho_workspace(_ortho(ld_out=80, stride_out=32 * 80 + 70)) > 0
    assert Z.zero_shard_ortho_workspace(_ortho(ld_out=80, stride_out=32 * 80 + 69)) == -1
    assert Z.zero_shard_ortho_workspace(_ortho(batch=1, stride_out=1)) > 0


def test_python_desc_refuses_odd_dtypes_and_coeffs(monkeypatch):
    monkeypatch.setattr(Z, "_stream", lambda s: 0)
    with pytest.raises(Z.ZeroShardError):
        Z.layernorm_desc(rows=1, cols=1, dtype=torch.float64)
    with pytest.raises(Z.ZeroShardError):
        Z.ortho_desc(rows=1, cols=1, steps=2, coeffs=[(1, 2, 3)])
    with pytest.raises(Z.ZeroShardError):
        Z.ortho_desc(rows=1, cols=1, steps=1, coeffs=(1, 2))
    d = Z.ortho_desc(rows=1, cols=1, steps=2, coeffs=(1, 2, 3))
    assert [d.coeffs[i] for i in range(6)] == [1, 2, 3, 1, 2, 3]


def test_valid_calls_need_the_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    assert _fwd(_norm_desc()) == Z.ZS_EDEVICE
    assert _bwd(_norm_desc()) == Z.ZS_EDEVICE
    m, o = _muon(), _ortho()
    assert Z._lib.zero_shard_muon_momentum(ctypes.byref(m), _table(P, P), P, P, P) == Z.ZS_EDEVICE
    assert Z._lib.zero_shard_muon_apply(ctypes.byref(m), P, 0.1, 1.0, P, P, P) == Z.ZS_EDEVICE
    assert Z._lib.zero_shard_ortho(ctypes.byref(o), P, 2 * P, 4 * P, 1 << 60) == Z.ZS_EDEVICE
