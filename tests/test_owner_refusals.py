"""What the owner objects of layer norm and Muon refuse before anything is
queued.  On the CPU stand-ins take the place of device tensors, whose memory the
checks do not touch."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""

    @property
    def is_cuda(self):
        return True


def on_device(t):
    return t.as_subclass(OnDevice)


def _norm(rows, cols, dtype=BF):
    ln = object.__new__(Z.ZeroLayerNorm)
    ln.shape, ln.dtype = (rows, cols), dtype
    return ln


EXPANDED_ROWS = [lambda r, c: torch.zeros(c, dtype=BF).expand(r, c),
                 lambda r, c: torch.zeros((), dtype=BF).expand(r, c),
                 lambda r, c: torch.zeros(r * c, dtype=BF).as_strided((r, c), (c // 2, 1))]


@pytest.mark.parametrize("make", EXPANDED_ROWS)
@pytest.mark.parametrize("rows,cols", [(2, 2), (8, 5120)])
def test_layernorm_refuses_rows_that_share_memory(make, rows, cols):
    with pytest.raises(Z.ZeroShardError):
        _norm(rows, cols)._row(on_device(make(rows, cols)), "dy")


def test_layernorm_refuses_a_single_column_expanded():
    with pytest.raises(Z.ZeroShardError):
        _norm(4, 1)._row(on_device(torch.zeros(1, 1, dtype=BF).expand(4, 1)), "dy")


def test_layernorm_takes_single_rows_and_padded_ones():
    row = _norm(1, 64)._row(on_device(torch.zeros(64, dtype=BF).expand(1, 64)), "x")
    assert row == 0  # one row: whatever its stride
    wide = on_device(torch.zeros(4, 80, dtype=BF)[:, :64])
    assert _norm(4, 64)._row(wide, "x") == 80
    assert _norm(4, 64)._row(on_device(torch.zeros(4, 64, dtype=BF)), "x") == 64
    column = on_device(torch.zeros(4, 7, dtype=BF)[:, 3:4])
    assert _norm(4, 1)._row(column, "x") == 7
    assert _norm(4, 64)._row(None, "x") == 0


@pytest.mark.gpu
def test_layernorm_refuses_expanded_operands():
    """Every operand, before anything is queued."""
    ln = Z.ZeroLayerNorm(rows=4, cols=64, dtype=BF)
    new = lambda: torch.full((4, 64), 3.0, device="cuda", dtype=BF)
    bad = torch.zeros(64, device="cuda", dtype=BF).expand(4, 64)
    out = new()
    for kw in (dict(x=bad), dict(y=bad), dict(residual=bad, sum_out=new()),
               dict(residual=new(), sum_out=bad)):
        with pytest.raises(Z.ZeroShardError):
            ln.forward(**{"x": new(), "y": out, **kw})
    for kw in (dict(dy=bad), dict(x=bad), dict(dx=bad), dict(dsum=bad)):
        with pytest.raises(Z.ZeroShardError):
            ln.backward(**{"dy": new(), "x": new(), "dx": out, **kw})
    torch.cuda.synchronize()
    assert (out == 3.0).all()
    # what autograd hands back for y.sum(0) is such a tensor
    y = new().requires_grad_()
    grad, = torch.autograd.grad(y.sum(0), y, torch.ones(64, device="cuda", dtype=BF))
    assert grad.stride() == (0, 1)
    with pytest.raises(Z.ZeroShardError):
        ln.backward(grad, new(), out)
    ln.forward(new(), out)
    ln.backward(grad.contiguous(), new(), out)


def _ortho(b, r, c):
    orth = object.__new__(Z.ZeroOrtho)
    orth.shape, orth.dtype = (b, r, c), F32
    return orth


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(8, 16).expand(4, 8, 16), lambda: torch.zeros(4, 1, 16).expand(4, 8, 16),
    lambda: torch.zeros(16).expand(4, 8, 16)])
def test_ortho_refuses_matrices_that_share_memory(make):
    with pytest.raises(Z.ZeroShardError):
        _ortho(4, 8, 16)._strides(on_device(make()), F32, "g")


@pytest.mark.parametrize("b,r,c", [(3, 1, 9), (3, 5, 1), (1, 5, 9)])
def test_ortho_refuses_expanded_rows_columns_and_batches(b, r, c):
    t = torch.zeros(1, 1, c).expand(b, r, c)
    with pytest.raises(Z.ZeroShardError):
        _ortho(b, r, c)._strides(on_device(t), F32, "g")
    if b == 1:
        with pytest.raises(Z.ZeroShardError):
            _ortho(b, r, c)._strides(on_device(t[0]), F32, "g")


def test_ortho_takes_what_does_not_share_memory():
    strides = lambda b, r, c, t: _ortho(b, r, c)._strides(on_device(t), F32, "g")
    assert strides(4, 8, 16, torch.zeros(4, 9, 20)[:, :8, :16]) == (20, 180)
    assert strides(4, 8, 16, torch.zeros(8, 4, 16).transpose(0, 1)) == (64, 16)  # between each other
    assert strides(1, 8, 16, torch.zeros(1, 8, 16).expand(1, 8, 16)) == (16, 128)
    assert strides(1, 1, 16, torch.zeros(16).expand(1, 16)) == (16, 16)
    strides(4, 0, 16, torch.zeros(0, 16).expand(4, 0, 16))  # empty: nothing is read


@pytest.mark.gpu
def test_ortho_refuses_expanded_operands():
    orth = Z.ZeroOrtho(batch=4, rows=8, cols=16, dtype=F32)
    g = torch.randn(4, 8, 16, device="cuda")
    o = torch.full((4, 8, 16), 3.0, device="cuda", dtype=BF)
    for bad in (g[0].expand(4, 8, 16), g[:, :1].expand(4, 8, 16)):
        with pytest.raises(Z.ZeroShardError):
            orth(bad, o)
        with pytest.raises(Z.ZeroShardError):
            orth(g, bad.to(BF)[:1].expand(4, 8, 16))
    torch.cuda.synchronize()
    assert (o == 3.0).all()
    between = torch.randn(8, 4, 16, device="cuda").transpose(0, 1)
    orth(between, o)
    again = torch.empty_like(o)
    orth(between.contiguous(), again)
    assert torch.equal(o, again)


def _muon(n, n_d):
    muon = object.__new__(Z.ZeroMuon)
    muon._no_elements, muon.scale = Z.zs_muon_desc(n=0, n_d=1), 1.0
    muon.desc = Z.zs_muon_desc(n=n, n_d=n_d, mu=0.95)
    muon.momentum = muon.update = torch.zeros(n)
    return muon


GOOD = lambda: on_device(torch.zeros(32, dtype=BF))


@pytest.mark.parametrize("contrib", [
    lambda: [GOOD()] * 2, lambda: [GOOD()] * 4, lambda: [], lambda: [GOOD(), None, GOOD()],
    lambda: [GOOD(), GOOD(), on_device(torch.zeros(32))],             # fp32
    lambda: [GOOD(), GOOD(), on_device(torch.zeros(32, dtype=F16))],
    lambda: [GOOD(), on_device(torch.zeros(31, dtype=BF)), GOOD()],   # short
    lambda: [GOOD(), on_device(torch.zeros(64, dtype=BF))[::2], GOOD()],
    lambda: [GOOD(), on_device(torch.zeros(1, dtype=BF)).expand(32), GOOD()],
    lambda: [GOOD(), torch.zeros(32, dtype=BF), GOOD()],              # on the host
    lambda: on_device(torch.zeros(2, 32, dtype=BF)), lambda: on_device(torch.zeros(3, 30, dtype=BF)),
    lambda: on_device(torch.zeros(32, 3, dtype=BF)).T,
    lambda: Z.contrib_table([GOOD()] * 2)])
def test_muon_refuses_wrong_contributions(contrib):
    with pytest.raises(Z.ZeroShardError, match="contrib"):
        _muon(32, 3).step(contrib(), 0.1)


@pytest.mark.parametrize("contrib", [
    lambda: [GOOD()] * 3, lambda: iter([GOOD()] * 3), lambda: tuple([GOOD().view(4, 8)] * 3),
    lambda: on_device(torch.zeros(3, 40, dtype=BF))[:, :32],
    lambda: on_device(torch.zeros(3, 40, dtype=BF)),                  # padded at the rows' ends
    lambda: [GOOD().view(torch.int16), GOOD().view(torch.uint16), GOOD()],
    lambda: Z.contrib_table([GOOD()] * 3)])
def test_muon_takes_contributions(contrib):
    assert len(_muon(32, 3)._table(contrib())) == 3


def test_momentum_refuses_a_short_table():
    d = Z.zs_muon_desc(n=32, n_d=3, nesterov=1, dtype=Z.ZS_BF16, mu=0.95)
    t = [torch.zeros(32, dtype=BF)] * 2
    assert Z.zero_shard_muon_momentum(d, t, None, None, None) == Z.ZS_EINVAL
    assert Z.zero_shard_muon_momentum(d, Z.contrib_table(t), t[0], t[0], t[0]) == Z.ZS_EINVAL
    d.n = 0  # nothing is read
    assert Z.zero_shard_muon_momentum(d, [], None, None, None) == Z.ZS_OK


@pytest.mark.gpu
def test_muon_refuses_state_of_another_type():
    n = 32 * 16
    new = lambda t: torch.zeros(n, device="cuda", dtype=t)
    good = dict(n_d=2, rows=32, cols=16, master=new(F32), momentum=new(F32), param_out=new(BF))
    for kw in (dict(master=new(torch.int32)), dict(momentum=new(torch.int32)),
               dict(param_out=new(F16)), dict(param_out=new(F32)), dict(master=new(BF))):
        with pytest.raises(Z.ZeroShardError):
            Z.ZeroMuon(**{**good, **kw})
    muon = Z.ZeroMuon(**{**good, "param_out": new(torch.int16)})
    rows = [torch.ones(n, device="cuda", dtype=BF) for _ in range(2)]
    for bad in (rows[:1], rows + rows[:1], [rows[0], rows[1].float()], [rows[0], rows[1][:-1]]):
        with pytest.raises(Z.ZeroShardError):
            muon.step(bad, 0.1)
    torch.cuda.synchronize()
    assert not muon.momentum.any() and not muon.master.any()
    muon.step(rows, 0.1)
    muon.step(Z.contrib_table(rows), 0.1)
    muon.step(torch.stack(rows), 0.1)
    assert torch.isfinite(muon.master).all() and muon.master.any()


def test_a_refused_rate_queues_nothing(monkeypatch):
    """The momentum does not move on when the weight update would be refused."""
    called = []
    monkeypatch.setattr(Z, "zero_shard_muon_momentum", lambda *a: called.append(a) or Z.ZS_OK)
    muon = _muon(32, 3)
    for lr in (-1.0, float("nan"), float("inf")):
        with pytest.raises(Z.ZeroShardError):
            muon.step([GOOD()] * 3, lr)
    muon.scale = float("nan")
    with pytest.raises(Z.ZeroShardError):
        muon.step([GOOD()] * 3, 0.1)
    assert not called


@pytest.mark.gpu
def test_muon_refuses_before_the_state_moves():
    n = 32 * 16
    new = lambda t=F32, k=n: torch.zeros(k, device="cuda", dtype=t)
    good = dict(n_d=1, rows=32, cols=16, master=new(), momentum=new(), param_out=new(BF))
    for kw in (dict(master=new(k=n + 1)[1:]), dict(momentum=new(k=n + 1)[1:]),
               dict(param_out=new(BF, n + 4)[4:])):
        with pytest.raises(Z.ZeroShardError):
            Z.ZeroMuon(**{**good, **kw})
    muon = Z.ZeroMuon(**good)
    rows = [torch.ones(n, device="cuda", dtype=BF)]
    for lr in (-1.0, float("nan")):
        with pytest.raises(Z.ZeroShardError):
            muon.step(rows, lr)
    torch.cuda.synchronize()
    assert not muon.momentum.any()
    muon.step(rows, 0.1)
    assert muon.momentum.any()
