"""The AdamW calls on the CPU: struct layouts, what plans and calls refuse
before any device is touched, empty sizes.  No kernel is launched here."""

from __future__ import annotations

import ctypes
import math

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests.test_owner_refusals import on_device
from tests.test_seam_host import layout_matches

P = 1 << 20  # an aligned stand-in address: never dereferenced by the checks
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("name,consts", [
    ("zs_adamw_desc", ("ZS_ADAMW_BLOCK", "ZS_ADAMW_MAX_TENSORS")),
    ("zs_adamw_tensor", ("ZS_STATE_32", "ZS_STATE_8"))])
def test_struct_layouts_match_header(name, consts):
    layout_matches(getattr(Z, name), {c: getattr(Z, c) for c in consts})


def _desc(**kw):
    return Z.zs_adamw_desc(**{**dict(count=1, beta1=0.9, beta2=0.999, eps=1e-8, bias_correction=1,
                                     max_norm=0.0), **kw})


def _tensor(at=0, state=Z.ZS_STATE_32, **kw):
    """Stand-in arrays 64 KiB apart, 32 of them a tensor."""
    a = [P + (32 * at + k) * 65536 for k in range(12)]
    base = dict(n=1000, master_in=a[0], master_out=a[0], m_in=a[1], m_out=a[1], v_in=a[2],
                v_out=a[2], param_out=a[3], weight_decay=0.1, lr_scale=1.0, state=state,
                grad_dtype=Z.ZS_BF16, param_dtype=Z.ZS_BF16)
    if state == Z.ZS_STATE_8:
        base.update(m_scale_in=a[4], m_scale_out=a[4], v_scale_in=a[5], v_scale_out=a[5])
    base.update(kw)
    return Z.zs_adamw_tensor(**base)


def _plan(tensors, **kw):
    d = _desc(count=len(tensors), **kw)
    array = (Z.zs_adamw_tensor * max(1, len(tensors)))(*tensors)
    size = Z.zero_shard_adamw_plan_bytes(d, array)
    if size < 0:
        return size, d, None
    plan = torch.zeros(size, dtype=torch.uint8)
    return Z.zero_shard_adamw_plan(d, array, plan), d, plan


BAD_DESC = [dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=NAN), dict(beta2=1.0), dict(beta2=-1.0),
            dict(eps=0.0), dict(eps=-1.0), dict(eps=INF), dict(eps=NAN), dict(bias_correction=2),
            dict(max_norm=NAN), dict(max_norm=INF)]


@pytest.mark.parametrize("kw", BAD_DESC)
def test_refuses_bad_descriptors(kw):
    assert _plan([_tensor()], **kw)[0] < 0
    ok, d, plan = _plan([_tensor()])
    assert ok == Z.ZS_OK
    grads = (ctypes.c_void_p * 1)(P)
    bad = _desc(**kw)
    assert Z.zero_shard_adamw(bad, plan, on_device(torch.zeros(1)), grads, 1e-3, 1, 0) == Z.ZS_EINVAL
    assert Z.zero_shard_adamw_consts(bad, 1e-3, 1, 0)[0] == Z.ZS_EINVAL


@pytest.mark.parametrize("count", [-1, Z.ZS_ADAMW_MAX_TENSORS + 1])
def test_refuses_bad_counts(count):
    d = _desc(count=count)
    assert Z.zero_shard_adamw_plan_bytes(d, (Z.zs_adamw_tensor * 1)(_tensor())) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), Z.ZS_EINVAL), (dict(n=Z.ZS_ADAMW_MAX_ELEMENTS + 1), Z.ZS_EINVAL),
    (dict(state=2), Z.ZS_EINVAL), (dict(grad_dtype=3), Z.ZS_EINVAL),
    (dict(param_dtype=Z.ZS_F32), Z.ZS_EINVAL), (dict(weight_decay=-0.1), Z.ZS_EINVAL),
    (dict(weight_decay=NAN), Z.ZS_EINVAL), (dict(lr_scale=-1.0), Z.ZS_EINVAL),
    (dict(lr_scale=INF), Z.ZS_EINVAL), (dict(master_in=None), Z.ZS_EINVAL),
    (dict(master_out=None), Z.ZS_EINVAL), (dict(m_in=None), Z.ZS_EINVAL),
    (dict(m_out=None), Z.ZS_EINVAL), (dict(v_in=None), Z.ZS_EINVAL),
    (dict(v_out=None), Z.ZS_EINVAL), (dict(m_scale_in=P), Z.ZS_EINVAL),
    (dict(v_scale_out=P), Z.ZS_EINVAL), (dict(master_in=P + 2), Z.ZS_EALIGN),
    (dict(m_in=P + 1), Z.ZS_EALIGN), (dict(v_out=P + 2), Z.ZS_EALIGN),
    (dict(param_out=P + 1), Z.ZS_EALIGN)])
def test_plan_refuses_bad_tensors(kw, code):
    rc = _plan([_tensor(**kw)])[0]
    assert rc == code or (rc == -1 and code == Z.ZS_EINVAL)


@pytest.mark.parametrize("kw", [dict(m_scale_in=None), dict(v_scale_in=None),
                                dict(m_scale_out=None), dict(v_scale_out=None)])
def test_plan_refuses_states_in_8_bits_without_scales(kw):
    assert _plan([_tensor(state=Z.ZS_STATE_8, **kw)])[0] == Z.ZS_EINVAL
    assert _plan([_tensor(state=Z.ZS_STATE_8, **{next(iter(kw)): P + 2})])[0] == Z.ZS_EALIGN


def test_plan_refuses_outputs_that_overlap():
    a = _tensor(0)
    assert _plan([a, _tensor(1)])[0] == Z.ZS_OK
    assert _plan([a, a])[0] == Z.ZS_EINVAL  # the same tensor twice
    assert _plan([a, _tensor(1, master_out=a.master_out + 3996)])[0] == Z.ZS_EINVAL
    assert _plan([a, _tensor(1, master_out=a.master_out + 4000)])[0] == Z.ZS_OK
    assert _plan([a, _tensor(1, param_out=a.v_out + 4)])[0] == Z.ZS_EINVAL
    assert _plan([_tensor(0, m_out=a.v_out)])[0] == Z.ZS_EINVAL
    e = _tensor(0, state=Z.ZS_STATE_8)
    assert _plan([e, _tensor(1, state=Z.ZS_STATE_8, v_scale_out=e.m_scale_out + 12)])[0] \
        == Z.ZS_EINVAL
    assert _plan([e, _tensor(1, state=Z.ZS_STATE_8, v_scale_out=e.m_scale_out + 16)])[0] == Z.ZS_OK
    # empty tensors overlap nothing, and need no arrays
    assert _plan([a, _tensor(0, n=0)])[0] == Z.ZS_OK
    assert _plan([Z.zs_adamw_tensor(n=0)])[0] == Z.ZS_OK


def test_plan_bound_is_exact_and_too_many_elements_are_refused():
    d, array = _desc(), (Z.zs_adamw_tensor * 1)(_tensor())
    need = Z.zero_shard_adamw_plan_bytes(d, array)
    assert Z.zero_shard_adamw_plan(d, array, torch.zeros(need - 1, dtype=torch.uint8)) \
        == Z.ZS_EINVAL
    assert Z.zero_shard_adamw_plan(d, array, None) == Z.ZS_EINVAL
    big = (Z.zs_adamw_tensor * 3)(*[_tensor(k, n=Z.ZS_ADAMW_MAX_ELEMENTS) for k in range(3)])
    assert Z.zero_shard_adamw_plan_bytes(_desc(count=1), big) > 0
    assert Z.zero_shard_adamw_plan_bytes(_desc(count=3), big) == -1


def _calls(d, plan, dev, grads, lr=1e-3, t=1, sumsq=None, consts=P):
    at = lambda a: None if a is None else a
    f = Z._lib
    host = None if plan is None else plan.data_ptr()
    return {
        "gnorm": f.zero_shard_adamw_gnorm(ctypes.byref(d), host, at(dev), grads, P),
        "step": f.zero_shard_adamw(ctypes.byref(d), host, at(dev), grads, lr, t, 0, sumsq),
        "dev": f.zero_shard_adamw_dev(ctypes.byref(d), host, at(dev), grads, consts, sumsq)}


def test_calls_refuse():
    if torch.cuda.is_available():
        pytest.skip("stand-in pointers")
    rc, d, plan = _plan([_tensor(0), _tensor(1, n=0), _tensor(2, grad_dtype=Z.ZS_F32)])
    assert rc == Z.ZS_OK
    ok = (ctypes.c_void_p * 3)(P, None, P)
    every = lambda code, *a, **kw: all(v == code for v in _calls(*a, **kw).values())
    assert every(Z.ZS_EDEVICE, d, plan, P, ok)
    assert every(Z.ZS_EINVAL, d, None, P, ok)
    assert every(Z.ZS_EINVAL, d, torch.zeros_like(plan), P, ok)  # no plan
    assert every(Z.ZS_EINVAL, _desc(count=2), plan, P, ok)       # another plan
    assert every(Z.ZS_EINVAL, d, plan, None, ok)
    assert every(Z.ZS_EALIGN, d, plan, P + 16, ok)
    assert every(Z.ZS_EINVAL, d, plan, P, None)
    assert every(Z.ZS_EINVAL, d, plan, P, (ctypes.c_void_p * 3)(P, None, None))
    assert every(Z.ZS_EALIGN, d, plan, P, (ctypes.c_void_p * 3)(P, None, P + 2))
    assert every(Z.ZS_EALIGN, d, plan, P, (ctypes.c_void_p * 3)(P + 1, None, P))
    for kw in (dict(lr=-1.0), dict(lr=NAN), dict(t=0)):
        assert _calls(d, plan, P, ok, **kw)["step"] == Z.ZS_EINVAL
    assert _calls(d, plan, P, ok, consts=None)["dev"] == Z.ZS_EINVAL
    assert _calls(d, plan, P, ok, consts=P + 4)["dev"] == Z.ZS_EALIGN
    # S goes with clipping
    for dd, s, code in ((d, P, Z.ZS_EINVAL), (_desc(count=3, max_norm=1.0), None, Z.ZS_EINVAL),
                        (_desc(count=3, max_norm=1.0), P + 4, Z.ZS_EALIGN),
                        (_desc(count=3, max_norm=1.0), P, Z.ZS_EDEVICE)):
        got = _calls(dd, plan, P, ok, sumsq=s)
        assert got["step"] == code and got["dev"] == code


def test_no_tensors_and_empty_ones_are_nothing():
    for tensors in ([], [_tensor(n=0)]):
        rc, d, plan = _plan(tensors)
        assert rc == Z.ZS_OK
        grads = (ctypes.c_void_p * 1)(None)
        got = _calls(d, plan, None, grads)
        assert got["step"] == Z.ZS_OK and got["dev"] == Z.ZS_OK


def test_consts():
    rc, got = Z.zero_shard_adamw_consts(_desc(), 0.25, 3, 7 + (1 << 32))
    b1, b2 = (float(torch.tensor(b)) for b in (0.9, 0.999))
    assert rc == Z.ZS_OK and got == [0.25, 1.0 - math.pow(b1, 3), 1.0 - math.pow(b2, 3), 7.0]
    rc, got = Z.zero_shard_adamw_consts(_desc(bias_correction=0), 0.25, 3, 0xFFFFFFFF)
    assert rc == Z.ZS_OK and got == [0.25, 1.0, 1.0, float(0xFFFFFFFF)]
    assert Z.zero_shard_adamw_consts(_desc(), -1.0, 3, 0)[0] == Z.ZS_EINVAL
    assert Z.zero_shard_adamw_consts(_desc(), 1.0, 0, 0)[0] == Z.ZS_EINVAL


def _of(n=600, eight=True, **kw):
    t = {"master": torch.zeros(n), "m": torch.zeros(n, dtype=torch.uint8).view(F8),
         "v": torch.zeros(n, dtype=torch.uint8).view(F8), "m_scale": torch.zeros(3),
         "v_scale": torch.zeros(3), "param_out": torch.zeros(n, dtype=BF)}
    if not eight:
        t.update(m=torch.zeros(n), v=torch.zeros(n))
        t.pop("m_scale"), t.pop("v_scale")
    t.update(kw)
    t = {k: None if v is None else on_device(v) for k, v in t.items()}
    return Z.adamw_tensor(t.pop("master"), t.pop("m"), t.pop("v"), **t)


def test_tensors_of_either_state():
    t = _of()
    assert t.n == 600 and t.state == Z.ZS_STATE_8 and t.master_in == t.master_out
    assert _of(eight=False).state == Z.ZS_STATE_32 and _of(eight=False).m_scale_in is None
    assert _of(m=torch.zeros(600, dtype=torch.uint8), v=torch.zeros(600, dtype=torch.uint8)).state
    assert _of(param_out=None).param_out is None


@pytest.mark.parametrize("eight,kw", [
    (True, dict(m=torch.zeros(600))), (True, dict(v=torch.zeros(600))),
    (True, dict(master=torch.zeros(600, dtype=BF))), (True, dict(master=torch.zeros(601))),
    (True, dict(m_scale=None)), (True, dict(v_scale=torch.zeros(2))),
    (True, dict(m_scale=torch.zeros(3, dtype=BF))), (True, dict(master=torch.zeros(1200)[::2])),
    (True, dict(param_out=torch.zeros(600))), (True, dict(param_out=torch.zeros(599, dtype=BF))),
    (True, dict(master_out=torch.zeros(599))), (True, dict(m_out=torch.zeros(600))),
    (False, dict(m_scale=torch.zeros(3))), (False, dict(m=torch.zeros(600, dtype=BF)))])
def test_tensors_that_do_not_fit_are_refused(eight, kw):
    with pytest.raises(Z.ZeroShardError):
        _of(eight=eight, **kw)


def test_tensors_on_the_cpu_are_refused():
    with pytest.raises(Z.ZeroShardError):
        Z.adamw_tensor(torch.zeros(4), torch.zeros(4), torch.zeros(4))


def test_owner_refuses_gradients_that_do_not_fit():
    o = object.__new__(Z.ZeroAdamW)
    o.tensors = [_of(), Z.zs_adamw_tensor(n=0, grad_dtype=Z.ZS_BF16)]
    g = lambda *a, **kw: on_device(torch.zeros(*a, **{"dtype": BF, **kw}))
    assert len(o._grads([g(600), None])) == 2 and len(o._grads([g(20, 30), None])) == 2
    for bad in ([g(600)], [g(599), None], [g(600, dtype=F32), None], [None, None],
                [g(1200)[::2], None], [torch.zeros(600, dtype=BF), None], [g(600), g(3)],
                (ctypes.c_void_p * 1)(P)):
        with pytest.raises(Z.ZeroShardError):
            o._grads(bad)
