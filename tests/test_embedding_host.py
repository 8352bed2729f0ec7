"""The embedding calls on the CPU: struct layout, refusals before any device
is touched, empty sizes.  No kernel is launched here."""

from __future__ import annotations

import ctypes

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests.test_owner_refusals import on_device
from tests.test_seam_host import layout_matches

P = 0x10000  # an aligned stand-in address: never dereferenced by the checks
BF = torch.bfloat16


def test_struct_layout_matches_header():
    layout_matches(Z.zs_embedding_desc, {c: getattr(Z, c) for c in (
        "ZS_EMBEDDING_MAX_TOKENS", "ZS_EMBEDDING_MAX_VOCAB")})


def _desc(**kw):
    base = dict(tokens=2000, vocab=50, cols=64, id_bytes=8, dtype=Z.ZS_BF16,
                table_dtype=Z.ZS_BF16, grad_dtype=Z.ZS_F32, scale=1.0)
    base.update(kw)
    return Z.zs_embedding_desc(**base)


def _fwd(d, ids=P, table=P, y=P):
    return Z._lib.zero_shard_embedding(ctypes.byref(d), ids, table, y)


def _bwd(d, ids=P, dy=P, dtable=P, ws=P, size=1 << 40):
    return Z._lib.zero_shard_embedding_bwd(ctypes.byref(d), ids, dy, dtable, ws, size)


BAD = [dict(tokens=-1), dict(tokens=Z.ZS_EMBEDDING_MAX_TOKENS + 1), dict(vocab=0),
       dict(vocab=Z.ZS_EMBEDDING_MAX_VOCAB + 1), dict(cols=0), dict(cols=(1 << 20) + 1),
       dict(first=(1 << 63) - 49), dict(tokens=1 << 27, cols=128), dict(vocab=1 << 30, cols=129),
       dict(id_bytes=2), dict(id_bytes=0), dict(dtype=3), dict(table_dtype=Z.ZS_F16),
       dict(grad_dtype=Z.ZS_F16), dict(dtype=Z.ZS_F32), dict(accumulate=2), dict(pad_set=-1),
       dict(scale=float("nan")), dict(scale=float("inf"))]
BAD += [{"ld_" + n: ld} for n in ("table", "y", "dy", "dtable") for ld in (63, -1, 1 << 40)]


@pytest.mark.parametrize("kw", BAD)
def test_refuses_bad_descriptors(kw):
    d = _desc(**kw)
    assert _fwd(d) == Z.ZS_EINVAL and _bwd(d) == Z.ZS_EINVAL
    assert Z.zero_shard_embedding_workspace(d) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), Z.ZS_EINVAL), (dict(table=None), Z.ZS_EINVAL), (dict(y=None), Z.ZS_EINVAL),
    (dict(ids=P + 4), Z.ZS_EALIGN), (dict(table=P + 1), Z.ZS_EALIGN), (dict(y=P + 1), Z.ZS_EALIGN)])
def test_forward_refuses_bad_pointers(kw, code):
    assert _fwd(_desc(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), Z.ZS_EINVAL), (dict(dy=None), Z.ZS_EINVAL), (dict(dtable=None), Z.ZS_EINVAL),
    (dict(ws=None), Z.ZS_EINVAL), (dict(size=0), Z.ZS_EINVAL), (dict(ids=P + 4), Z.ZS_EALIGN),
    (dict(dy=P + 1), Z.ZS_EALIGN), (dict(dtable=P + 2), Z.ZS_EALIGN), (dict(ws=P + 128), Z.ZS_EALIGN)])
def test_backward_refuses_bad_pointers(kw, code):
    assert _bwd(_desc(), **kw) == code


def test_workspace_bound_is_exact():
    for tokens, cols in ((1025, 64), (1000, 4096), (2048, 64), (2049, 64), (8192, 64), (8193, 64)):
        d = _desc(tokens=tokens, cols=cols)
        need = Z.zero_shard_embedding_workspace(d)
        assert need > 0
        assert _bwd(d, size=need - 1) == Z.ZS_EINVAL
    for tokens, cols in ((0, 64), (1, 5120), (1024, 64), (600, 5120)):  # nothing is sorted
        d = _desc(tokens=tokens, cols=cols)
        assert Z.zero_shard_embedding_workspace(d) == 0
        if not torch.cuda.is_available():
            assert _bwd(d, ws=None, size=0) == Z.ZS_EDEVICE


def test_products_no_launch_takes_are_refused():
    d = _desc(tokens=1 << 27, cols=1 << 20)
    assert _fwd(d) == Z.ZS_EINVAL and _bwd(d, size=(1 << 63) - 1) == Z.ZS_EINVAL


def test_no_tokens_is_nothing():
    d = _desc(tokens=0)
    assert _fwd(d, ids=None, table=None, y=None) == Z.ZS_OK
    assert _bwd(_desc(tokens=0, accumulate=1), ids=None, dy=None, dtable=None, ws=None,
                size=0) == Z.ZS_OK
    assert _bwd(d, dtable=None) == Z.ZS_EINVAL  # its rows become zeros


def test_valid_calls_reach_the_device_check():
    if torch.cuda.is_available():
        pytest.skip("stand-in pointers")
    assert _fwd(_desc()) == Z.ZS_EDEVICE and _bwd(_desc()) == Z.ZS_EDEVICE
    assert _bwd(_desc(tokens=0), ids=None, dy=None, ws=None, size=0) == Z.ZS_EDEVICE


def _owner(tokens=6, vocab=5, cols=8):
    o = object.__new__(Z.ZeroEmbedding)
    o.rows, o.shape = (vocab, cols), (tokens, cols)
    o.dtype = o.table_dtype = o.grad_dtype = BF
    o.id_dtype, o.desc = torch.int64, _desc(tokens=tokens, vocab=vocab, cols=cols)
    o._workspace, o._workspace_bytes = on_device(torch.zeros(4)), 16
    return o


@pytest.mark.parametrize("bad", [
    dict(ids=torch.zeros(5, dtype=torch.int64)), dict(ids=torch.zeros(6, dtype=torch.int32)),
    dict(ids=torch.zeros(12, dtype=torch.int64)[::2]), dict(ids=torch.zeros(1, dtype=torch.int64).expand(6)),
    dict(table=torch.zeros(4, 8, dtype=BF)), dict(table=torch.zeros(5, 8)),
    dict(table=torch.zeros(8, dtype=BF).expand(5, 8)), dict(table=torch.zeros(8, 5, dtype=BF).T),
    dict(rows=torch.zeros(5, 8, dtype=BF)), dict(rows=torch.zeros(8, dtype=BF).expand(6, 8))])
def test_owner_refuses(bad):
    o = _owner()
    t = dict(ids=torch.zeros(6, dtype=torch.int64), table=torch.zeros(5, 8, dtype=BF),
             rows=torch.zeros(6, 8, dtype=BF))
    t.update(bad)
    t = {k: on_device(v) for k, v in t.items()}
    with pytest.raises(Z.ZeroShardError):
        o.forward(t["ids"], t["table"], t["rows"])
    with pytest.raises(Z.ZeroShardError):
        o.backward(t["ids"], t["rows"], t["table"])


def test_id_types():
    with pytest.raises(Z.ZeroShardError):
        Z.embedding_desc(tokens=1, vocab=1, cols=1, id_dtype=torch.int16)
