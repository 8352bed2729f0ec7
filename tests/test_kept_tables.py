"""Tables of gradients that a program keeps: what fits is taken, what does not is refused
as a list of the same tensors is, before anything is queued."""

from __future__ import annotations

import ctypes

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests.test_owner_refusals import on_device

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _opt(*sizes, dtype=BF):
    o = object.__new__(Z.ZeroAdamW)
    o.tensors = [Z.zs_adamw_tensor(n=n, grad_dtype=Z.dtype_code(dtype)) for n in sizes]
    return o


def _new(*shape, dtype=BF):
    return on_device(torch.zeros(*shape, dtype=dtype))


def test_tables_that_fit():
    o = _opt(600, 0, 32)
    table = Z.contrib_table([_new(600), None, _new(4, 8)])
    for _ in range(3):
        assert o._grads(table) is table
    assert _opt(600, 0, 32)._grads(table) is table  # another plan of the same sizes
    assert o._grads(table) is table
    rows = Z.contrib_table(_new(2, 40))
    assert _opt(40, 40)._grads(rows) is rows
    assert len(_opt()._grads(Z.contrib_table([]))) == 1


@pytest.mark.parametrize("grads", [
    lambda: [_new(600)], lambda: [_new(600), _new(3), _new(32)], lambda: [_new(600), None],
    lambda: [_new(599), None, _new(32)], lambda: [_new(601), None, _new(32)],
    lambda: [_new(600, dtype=F32), None, _new(32)], lambda: [_new(600, dtype=F16), None, _new(32)],
    lambda: [None, None, _new(32)], lambda: [_new(1200)[::2], None, _new(32)],
    lambda: [_new(1).expand(600), None, _new(32)],
    lambda: [torch.zeros(600, dtype=BF), None, _new(32)],        # on the host
    lambda: [_new(600), None, _new(32), _new(32)]])
def test_tables_that_do_not_fit_are_refused(grads):
    o = _opt(600, 0, 32)
    for _ in range(2):
        with pytest.raises(Z.ZeroShardError, match="grads"):
            o._grads(Z.contrib_table(grads()))
    table = Z.contrib_table(grads())
    for _ in range(2):  # nor the second time
        with pytest.raises(Z.ZeroShardError, match="grads"):
            o._grads(table)


def test_a_table_of_another_plan_is_looked_at_again():
    table = Z.contrib_table([_new(600)])
    assert _opt(600)._grads(table) is table
    for other in (_opt(601), _opt(600, dtype=F32), _opt(600, 600), _opt()):
        with pytest.raises(Z.ZeroShardError, match="grads"):
            other._grads(table)


def test_entries_that_are_not_the_tensors_are_refused():
    o = _opt(600, 600)
    a, b, c = (_new(600) for _ in range(3))
    table = Z.contrib_table([a, b])
    assert o._grads(table) is table
    table[1] = c.data_ptr()
    with pytest.raises(Z.ZeroShardError, match="entries"):
        o._grads(table)
    table[1] = b.data_ptr()
    assert o._grads(table) is table
    table[0] = None
    with pytest.raises(Z.ZeroShardError, match="entries"):
        o._grads(table)
    bare = (ctypes.c_void_p * 2)(a.data_ptr(), b.data_ptr())
    with pytest.raises(Z.ZeroShardError, match="contrib_table"):
        o._grads(bare)


def _muon(n=32, n_d=3):
    muon = object.__new__(Z.ZeroMuon)
    muon.desc = Z.zs_muon_desc(n=n, n_d=n_d)
    return muon


def test_contributions_that_fit():
    muon = _muon()
    table = Z.contrib_table([_new(32), _new(4, 8), _new(40)])
    for _ in range(2):
        assert muon._table(table) is table
    rows = Z.contrib_table(_new(3, 40))
    assert muon._table(rows) is rows
    bare = (ctypes.c_void_p * 3)(*[_new(32).data_ptr() for _ in range(3)])
    assert muon._table(bare) is bare


@pytest.mark.parametrize("bad", [
    lambda: _new(31), lambda: _new(32, dtype=F32), lambda: _new(32, dtype=F16),
    lambda: _new(64)[::2], lambda: torch.zeros(32, dtype=BF), lambda: None])
def test_contributions_that_do_not_fit_are_refused(bad):
    muon = _muon()
    table = Z.contrib_table([_new(32), bad(), _new(32)])
    for _ in range(2):
        with pytest.raises(Z.ZeroShardError, match="contrib"):
            muon._table(table)
    table = Z.contrib_table([_new(32)] * 3)
    assert muon._table(table) is table
    table[0] = 1 << 20
    with pytest.raises(Z.ZeroShardError, match="entries"):
        muon._table(table)


def _desc(count):
    return Z.zs_adamw_desc(count=count, beta1=0.9, beta2=0.999, eps=1e-8, bias_correction=1)


def _tensors(count):
    at = [(1 << 20) + k * 65536 for k in range(3 * count)]  # stand-in addresses
    return (Z.zs_adamw_tensor * max(1, count))(*[
        Z.zs_adamw_tensor(n=1000, master_in=a, master_out=a, m_in=b, m_out=b, v_in=c, v_out=c,
                          lr_scale=1.0, grad_dtype=Z.ZS_BF16, param_dtype=Z.ZS_BF16)
        for a, b, c in zip(at[0::3], at[1::3], at[2::3])])


def test_named_calls_refuse_fewer_tensors_or_gradients_than_counted(monkeypatch):
    """The host arrays are not read past their ends: the library is not called."""
    class Closed:
        def __getattr__(self, name):
            raise AssertionError(name)

    d, two = _desc(3), _tensors(2)
    plan = torch.zeros(Z.zero_shard_adamw_plan_bytes(d, _tensors(3)), dtype=torch.uint8)
    assert Z.zero_shard_adamw_plan(d, _tensors(3), plan) == Z.ZS_OK
    monkeypatch.setattr(Z, "_lib", Closed())
    assert Z.zero_shard_adamw_plan_bytes(d, two) == -1
    assert Z.zero_shard_adamw_plan(d, two, plan) == Z.ZS_EINVAL
    assert Z.zero_shard_adamw_plan(d, _tensors(3), on_device(plan)) == Z.ZS_EINVAL
    dev, s = _new(1), _new(1, dtype=torch.float64)
    three = [_new(1000) for _ in range(3)]
    for p, grads in ((plan, three[:2]), (plan, Z.contrib_table(three[:2])), (plan, []),
                     (on_device(plan), three)):
        assert Z.zero_shard_adamw_gnorm(d, p, dev, grads, s) == Z.ZS_EINVAL
        assert Z.zero_shard_adamw(d, p, dev, grads, 1e-3, 1, 0) == Z.ZS_EINVAL
        assert Z.zero_shard_adamw_dev(d, p, dev, grads, s) == Z.ZS_EINVAL
