"""Layer norm, forward and backward, on the GPU against the formulas in 64
bits: every type, register shape and the long-row path, odd widths, padded
and unaligned rows, a fused residual, absent parameters, infinities and NaN,
buffers used in place, another stream, and a captured graph."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# (rows, cols): every register shape and its edges, one row, one column, odd
# widths, more rows than workgroups, and rows too long for registers
SIZES = [(1, 1), (3, 2), (5, 8), (1, 5120), (7, 511), (6, 512), (5, 1000), (9, 1601), (4, 2048),
         (3, 2056), (2, 4099), (5, 5120), (3, 8192), (2, 8200), (2, 16384), (2, 16385), (3, 20480),
         (2100, 64), (1030, 2064)]
TYPES = [(F32, F32), (BF, BF), (BF, F32), (F16, F16), (F16, F32)]


def _inputs(rows, cols, dtype, ptype, pad, seed=1):
    size = 1.0 + torch.arange(rows, device="cuda", dtype=F32)[:, None] % 7
    x = R.randn(rows, cols, dtype=F32, pad=pad, seed=seed)
    full = torch.empty(rows, cols + pad, device="cuda", dtype=dtype)
    full[:, :cols] = (x * size + 0.5).to(dtype)
    gamma = (1.0 + R.randn(cols, seed=seed + 1, scale=0.2)).to(ptype)
    beta = R.randn(cols, seed=seed + 2, scale=0.3).to(ptype)
    return full[:, :cols], gamma, beta


def _serial(rows):
    """Longest chain of additions behind a column's sum: a partial's rows, the
    four waves of a workgroup, and the partials of one of 16 groups."""
    return rows // 512 + 1 + 4 + 512 // 16 + 16


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, dtype, ptype):
    for pad, residual, affine in ((0, False, True), (8, True, True), (3, True, False)):
        x, gamma, beta = _inputs(rows, cols, dtype, ptype, pad)
        gamma, beta = (gamma, beta) if affine else (None, None)
        ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=dtype, param_dtype=ptype, eps=1e-5)
        y = R.randn(rows, cols, dtype=dtype, pad=pad)
        res = R.randn(rows, cols, dtype=dtype, pad=pad, seed=9) if residual else None
        total = torch.empty(rows, cols, device="cuda", dtype=dtype) if residual else None
        ln.forward(x, y, gamma=gamma, beta=beta, residual=res, sum_out=total)
        s = x
        if residual:
            s = (x.float() + res.float()).to(dtype)
            assert torch.equal(total, s)
        (ry, ty), (rm, tm), (rr, tr) = R.layernorm_ref(s, gamma, beta, 1e-5)
        R.within("y", y, ry, ty + R.half_step(dtype, ry.abs() + ty))
        R.within("mean", ln.mean, rm, tm + R.U * rm.abs())
        R.within("rstd", ln.rstd, rr, tr + 2 * R.U * rr)


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, dtype, ptype):
    for pad, residual, affine in ((0, False, True), (8, True, True), (3, True, False)):
        x, gamma, _ = _inputs(rows, cols, dtype, ptype, pad)
        gamma = gamma if affine else None
        dy = R.randn(rows, cols, dtype=dtype, pad=pad, seed=5)
        dsum = R.randn(rows, cols, dtype=dtype, pad=pad, seed=6) if residual else None
        mean = x.double().mean(1).float()
        rstd = (1.0 / torch.sqrt(x.double().var(1, correction=0) + 1e-5)).float()
        dx = R.randn(rows, cols, dtype=dtype, pad=pad)
        dgamma = torch.empty(cols, device="cuda", dtype=ptype)
        dbeta = torch.empty(cols, device="cuda", dtype=ptype)
        ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=dtype, param_dtype=ptype)
        ln.backward(dy, x, dx, gamma=gamma, dgamma=dgamma, dbeta=dbeta, dsum=dsum, mean=mean,
                    rstd=rstd)
        (rx, tx), (rg, tg), (rb, tb) = R.layernorm_bwd_ref(dy, x, gamma, mean, rstd, dsum,
                                                           _serial(rows))
        R.within("dx", dx, rx, tx + R.half_step(dtype, rx.abs() + tx))
        R.within("dgamma", dgamma, rg, tg + R.half_step(ptype, rg.abs() + tg))
        R.within("dbeta", dbeta, rb, tb + R.half_step(ptype, rb.abs() + tb))


@pytest.mark.parametrize("cols", [96, 1601, 5120, 17000])
def test_backward_is_the_forward_differentiated(cols):
    """dx, dgamma and dbeta against central differences of the formula in 64
    bits along random directions."""
    rows, eps = 6, 1e-5
    x, gamma, beta = _inputs(rows, cols, F32, F32, 0)
    dy = R.randn(rows, cols, seed=5)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=F32, eps=eps)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
    ln.forward(x, y, gamma=gamma, beta=beta)
    ln.backward(dy, x, dx, gamma=gamma, dgamma=dgamma, dbeta=dbeta)

    def loss(x, gamma, beta):
        c = x - x.mean(1, keepdim=True)
        return float(((c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * gamma + beta)
                      * dy.double()).sum())

    at = [x.double(), gamma.double(), beta.double()]
    for k, grad in enumerate((dx, dgamma, dbeta)):
        for seed in range(3):
            v = R.randn(*at[k].shape, seed=20 + seed).double()
            hi, lo = list(at), list(at)
            hi[k], lo[k] = at[k] + 1e-4 * v, at[k] - 1e-4 * v
            want = (loss(*hi) - loss(*lo)) / 2e-4
            got = float((grad.double() * v).sum())
            # binary32 gradients (2^-20 of the sum's size) and the difference's
            # own error, of third order in the step
            size = float(torch.linalg.norm(grad.double()) * torch.linalg.norm(v))
            assert abs(got - want) <= size * (2.0 ** -20 + 1e-6), (k, got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [64, 777, 5120, 16385])
def test_constant_and_far_rows(cols, dtype):
    """A constant row gives beta (variance 0), also far from zero; a row far
    from zero keeps its deviations."""
    x = torch.empty(3, cols, device="cuda", dtype=dtype)
    x[0], x[1] = 1000.0, -3.0
    x[2] = (4096.0 + 32.0 * (torch.arange(cols, device="cuda") % 3)).to(dtype)
    beta = R.randn(cols, dtype=dtype, seed=3)
    y = torch.empty_like(x)
    ln = Z.ZeroLayerNorm(rows=3, cols=cols, dtype=dtype)
    ln.forward(x, y, beta=beta)
    (ry, ty), _, _ = R.layernorm_ref(x, None, beta, 1e-5)
    # deviations of a constant row: the mean's rounding, 2 half steps of 1000,
    # times rstd = 1/sqrt(1e-5)
    R.within("y", y, ry, ty + R.half_step(dtype, ry.abs() + ty))


@pytest.mark.parametrize("cols", [64, 1601, 5120, 16400])
def test_nonfinite_rows_stay_in_their_rows(cols):
    x, gamma, beta = _inputs(5, cols, F32, F32, 0)
    x[1, cols // 2] = float("inf")
    x[3, 0] = float("nan")
    y = torch.empty_like(x)
    ln = Z.ZeroLayerNorm(rows=5, cols=cols, dtype=F32)
    ln.forward(x, y, gamma=gamma, beta=beta)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    assert torch.isfinite(y[[0, 2, 4]]).all()
    assert float(ln.mean[1]) == float("inf") and torch.isnan(ln.mean[3])
    dy = R.randn(5, cols, seed=4)
    dy[2, 1] = float("inf")
    dx = torch.empty_like(x)
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
    mean, rstd = torch.zeros(5, device="cuda"), torch.ones(5, device="cuda")
    x[1], x[3] = 1.0, 2.0
    ln.backward(dy, x, dx, gamma=gamma, dgamma=dgamma, dbeta=dbeta, mean=mean, rstd=rstd)
    assert not torch.isfinite(dx[2]).any()
    assert torch.isfinite(dx[[0, 1, 3, 4]]).all()
    assert float(dbeta[1]) == float("inf") and torch.isfinite(dbeta[2:]).all()
    assert not torch.isfinite(dgamma[1]) and torch.isfinite(dgamma[2:]).all()


@pytest.mark.parametrize("cols", [100, 5120, 17000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(cols, dtype):
    rows = 9
    x, gamma, beta = _inputs(rows, cols, dtype, dtype, 0)
    x = x.contiguous()
    res = R.randn(rows, cols, dtype=dtype, seed=8)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=dtype)
    y, total = torch.empty_like(x), torch.empty_like(x)
    ln.forward(x, y, gamma=gamma, beta=beta, residual=res, sum_out=total)
    y1 = torch.empty_like(x)
    ln.forward(x, y1, gamma=gamma, beta=beta)
    a, b = x.clone(), res.clone()
    y2 = torch.empty_like(x)
    ln.forward(a, y2, gamma=gamma, beta=beta, residual=res, sum_out=a)  # the sum over x
    assert torch.equal(a, total) and torch.equal(y2, y)
    ln.forward(x, y2, gamma=gamma, beta=beta, residual=b, sum_out=b)    # over the residual
    assert torch.equal(b, total) and torch.equal(y2, y)
    a = x.clone()
    ln.forward(a, a, gamma=gamma, beta=beta)                            # y over x
    assert torch.equal(a, y1)
    a, t2 = x.clone(), torch.empty_like(x)
    ln.forward(a, a, gamma=gamma, beta=beta, residual=res, sum_out=t2)  # y over x, a sum besides
    assert torch.equal(a, y) and torch.equal(t2, total)
    dy, dsum = R.randn(rows, cols, dtype=dtype, seed=5), R.randn(rows, cols, dtype=dtype, seed=6)
    outs = []
    for where in ("new", "dy", "dsum", "x"):
        u, w, xx = dy.clone(), dsum.clone(), total.clone()
        dx = {"new": torch.empty_like(x), "dy": u, "dsum": w, "x": xx}[where]
        dg, db = torch.empty_like(gamma), torch.empty_like(beta)
        ln.backward(u, xx, dx, gamma=gamma, dgamma=dg, dbeta=db, dsum=w)
        outs.append((dx.clone(), dg, db))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


def test_no_rows_give_zero_gradients():
    ln = Z.ZeroLayerNorm(rows=0, cols=70, dtype=BF)
    e = torch.empty(0, 70, device="cuda", dtype=BF)
    dg, db = (torch.full((70,), 7.0, device="cuda", dtype=BF) for _ in range(2))
    ln.forward(e, e.clone())
    ln.backward(e, e, e.clone(), dgamma=dg, dbeta=db)
    assert not dg.any() and not db.any()


@pytest.mark.parametrize("cols", [96, 5120, 17000])
def test_gradients_one_at_a_time_and_none(cols):
    rows = 40
    x, gamma, _ = _inputs(rows, cols, BF, BF, 0)
    dy = R.randn(rows, cols, dtype=BF, seed=5)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=BF)
    y, dx0 = torch.empty_like(x), torch.empty_like(x)
    ln.forward(x, y, gamma=gamma)
    dg0, db0 = torch.empty_like(gamma), torch.empty_like(gamma)
    ln.backward(dy, x, dx0, gamma=gamma, dgamma=dg0, dbeta=db0)
    for want_g, want_b in ((1, 0), (0, 1), (0, 0)):
        dx = torch.empty_like(x)
        dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
        ln.backward(dy, x, dx, gamma=gamma, dgamma=dg if want_g else None,
                    dbeta=db if want_b else None)
        assert torch.equal(dx, dx0)
        assert not want_g or torch.equal(dg, dg0)
        assert not want_b or torch.equal(db, db0)


def test_unaligned_buffers():
    """Rows that start between 16-byte boundaries give the aligned result's
    values up to the order of the row sums."""
    rows, cols = 6, 1024
    base = R.randn(rows * cols + 1, dtype=BF, seed=2)
    x = base[1:].view(rows, cols)
    gamma = R.randn(cols + 1, dtype=BF, seed=3)[1:]
    y = torch.empty(rows * cols + 1, device="cuda", dtype=BF)[1:].view(rows, cols)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=BF)
    ln.forward(x, y, gamma=gamma)
    (ry, ty), _, _ = R.layernorm_ref(x, gamma, None, 1e-5)
    R.within("y", y, ry, ty + R.half_step(BF, ry.abs() + ty))


def test_far_offsets():
    """Row offsets past 32 bits (elements and bytes)."""
    rows, cols, ld = 3, 100, (1 << 31) + 7
    x = torch.empty(2 * ld + cols, device="cuda", dtype=BF)
    rowsx = torch.as_strided(x, (rows, cols), (ld, 1))
    vals = R.randn(rows, cols, dtype=BF, seed=1)
    rowsx.copy_(vals)
    y = torch.empty(rows, cols, device="cuda", dtype=BF)
    ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=BF)
    ln.forward(rowsx, y)
    y1 = torch.empty_like(y)
    ln.forward(vals, y1)
    assert torch.equal(y, y1)
    dy = R.randn(rows, cols, dtype=BF, seed=5)
    dx, dx1 = torch.empty_like(dy), torch.empty_like(dy)
    ln.backward(dy, rowsx, dx)
    ln.backward(dy, vals, dx1)
    assert torch.equal(dx, dx1)


def test_another_stream_and_determinism():
    rows, cols = 700, 1601
    side = torch.cuda.Stream()
    x, gamma, beta = _inputs(rows, cols, BF, F32, 0)
    dy = R.randn(rows, cols, dtype=BF, seed=5)
    torch.cuda.synchronize()
    outs = []
    for stream in (None, side, side):
        ln = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=BF, param_dtype=F32, stream=stream)
        y, dx = torch.empty_like(dy), torch.empty_like(dy)
        dg, db = torch.empty_like(gamma), torch.empty_like(beta)
        torch.cuda.synchronize()
        ln.forward(x, y, gamma=gamma, beta=beta)
        ln.backward(dy, x, dx, gamma=gamma, dgamma=dg, dbeta=db)
        torch.cuda.synchronize()
        outs.append((y, dx, dg, db))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


def test_graph_replays_match_eager():
    rows, cols = 300, 768
    side = torch.cuda.Stream()
    x, gamma, beta = _inputs(rows, cols, BF, BF, 0)
    x = x.contiguous()
    dy = R.randn(rows, cols, dtype=BF, seed=5)
    eager = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=BF)
    caught = Z.ZeroLayerNorm(rows=rows, cols=cols, dtype=BF, stream=side)
    new = lambda: [torch.empty_like(x), torch.empty_like(x), torch.empty_like(gamma),
                   torch.empty_like(beta)]
    a, b = new(), new()

    def both(ln, o):
        ln.forward(x, o[0], gamma=gamma, beta=beta)
        ln.backward(dy, x, o[1], gamma=gamma, dgamma=o[2], dbeta=o[3])

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both(caught, b)
    for rep in range(4):
        x.copy_(R.randn(rows, cols, dtype=BF, seed=50 + rep))
        both(eager, a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, b)), rep


def test_owner_refuses_wrong_tensors():
    ln = Z.ZeroLayerNorm(rows=4, cols=32, dtype=BF)
    good = R.randn(4, 32, dtype=BF)
    for bad in (R.randn(4, 31, dtype=BF), R.randn(4, 32), R.randn(32, 4, dtype=BF).T,
                good.cpu()):
        with pytest.raises(Z.ZeroShardError):
            ln.forward(bad, torch.empty_like(good))
        with pytest.raises(Z.ZeroShardError):
            ln.backward(good, bad, torch.empty_like(good))
    with pytest.raises(Z.ZeroShardError):
        ln.forward(good, torch.empty_like(good), gamma=R.randn(32))
    with pytest.raises(Z.ZeroShardError):
        ln.forward(good, torch.empty_like(good), residual=good)
    with pytest.raises(Z.ZeroShardError):
        Z.ZeroLayerNorm(rows=4, cols=0, dtype=BF)
