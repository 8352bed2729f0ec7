"""The Muon update on the GPU: momentum and weight update against the formulas
in 64 bits (one rounding per stored value), the orthogonalisation against 64
bits within the error of its binary16 storage, over types, strides, batches,
odd and tall shapes, zero, tiny, huge and non-finite matrices, other
coefficients, another stream, a captured graph, and the whole step."""

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


def _rows(n_d, n, seed=1):
    return [R.randn((n + 7) // 8 * 8, dtype=BF, seed=seed + k, scale=1e-3)[:n] for k in range(n_d)]


def _momentum_ref(rows, m, mu, nesterov):
    s = torch.zeros(m.numel(), device="cuda", dtype=torch.float64)
    for r in rows:
        s += r.double()
    g = (s / len(rows)).float().double()
    mu = float(torch.tensor(mu, dtype=F32))
    mm = mu * m.double() + g
    return mm, (g + mu * mm if nesterov else mm)


@pytest.mark.parametrize("n", [1, 7, 8, 9, 2048, 2049, 1_000_003])
@pytest.mark.parametrize("n_d", [1, 3, 8, 13, 64])
def test_momentum(n, n_d):
    rows, m = _rows(n_d, n), R.randn(n, seed=99, scale=1e-2)
    for nesterov in (True, False):
        rm, ru = _momentum_ref(rows, m, 0.95, nesterov)
        for dtype in (F32, BF):
            d = Z.muon_desc(n=n, n_d=n_d, mu=0.95, nesterov=nesterov, dtype=dtype)
            out, u = torch.empty_like(m), torch.empty(n, device="cuda", dtype=dtype)
            Z.check(Z.zero_shard_muon_momentum(d, rows, m, out, u))
            assert torch.equal(out, rm.float())           # one rounding of the 64-bit value
            assert torch.equal(u, ru.float().to(dtype))   # bf16: of the binary32 value
            again = m.clone()
            Z.check(Z.zero_shard_muon_momentum(d, rows, again, again, u))
            assert torch.equal(again, out)


@pytest.mark.parametrize("n", [1, 7, 8, 9, 2048, 2049, 1_000_003])
def test_apply(n):
    w, o = R.randn(n, seed=1, scale=0.02), R.randn(n, dtype=BF, seed=2)
    f = lambda v: float(torch.tensor(v, dtype=F32))
    for wd in (0.0, 0.1):
        d = Z.muon_desc(n=n, weight_decay=wd)
        out, p = torch.empty_like(w), torch.empty(n, device="cuda", dtype=BF)
        Z.check(Z.zero_shard_muon_apply(d, o, 0.02, 0.2, w, out, p))
        x = w.double()
        ref = (x - (f(0.02) * f(wd)) * x) - (f(0.02) * f(0.2)) * o.double()
        assert torch.equal(out, ref.float())
        assert torch.equal(p, out.to(BF))
        again = w.clone()
        Z.check(Z.zero_shard_muon_apply(d, o, 0.02, 0.2, again, again, p))
        assert torch.equal(again, out)


def test_elementwise_passes_keep_nonfinite_values_in_place():
    n = 100
    rows, m = _rows(4, n), R.randn(n, seed=9)
    rows[2][7], m[50] = float("inf"), float("nan")
    out, u = torch.empty_like(m), torch.empty(n, device="cuda", dtype=BF)
    Z.check(Z.zero_shard_muon_momentum(Z.muon_desc(n=n, n_d=4), rows, m, out, u))
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[7] = bad[50] = True
    assert torch.equal(~torch.isfinite(out), bad) and torch.equal(~torch.isfinite(u.float()), bad)


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 3), (16, 16), (63, 65), (64, 64), (65, 64), (96, 128),
          (128, 128), (129, 128), (130, 300), (300, 130), (20, 5000), (5000, 20), (513, 257),
          (700, 900), (2100, 2300)]


def _matrix(b, r, c, dtype, pad=0, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = 1e-3 * torch.exp(0.5 * torch.randn(b, r, 1, device="cuda", generator=g))
    return (torch.randn(b, r, c + pad, device="cuda", generator=g) * size).to(dtype)[:, :, :c]


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_ortho(rows, cols, dtype):
    for pad in (0, 5):
        g = _matrix(1, rows, cols, dtype, pad)
        o = torch.full((rows, cols + pad), 7.0, device="cuda", dtype=BF)
        Z.ZeroOrtho(rows=rows, cols=cols, dtype=dtype)(g[0], o[:, :cols])
        R.ortho_check(f"{rows}x{cols}", o[:, :cols], g[0], [R.COEFFS] * 5, 1e-7)
        assert (o[:, cols:] == 7.0).all()  # nothing beside the matrix is written


@pytest.mark.parametrize("batch,rows,cols", [(3, 200, 100), (5, 64, 64), (2, 130, 700),
                                             (300, 20, 30), (40, 257, 300), (12, 1024, 768)])
def test_ortho_batches_equal_single_matrices(batch, rows, cols):
    g = _matrix(batch, rows, cols, F32, pad=3)
    o = torch.zeros(batch, rows + 1, cols, device="cuda", dtype=BF)[:, :rows]
    Z.ZeroOrtho(batch=batch, rows=rows, cols=cols, dtype=F32)(g, o)
    for i in (0, 1, batch - 1):
        R.ortho_check(f"matrix {i}", o[i], g[i], [R.COEFFS] * 5, 1e-7)


@pytest.mark.parametrize("rows,cols", [(1, 9), (50, 40), (300, 200), (200, 1100)])
@pytest.mark.parametrize("steps,coeffs", [
    (1, None), (2, [(3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375)]),
    (12, (1.875, -1.25, 0.375)), (7, (1.5, -0.5, 0.0))])
def test_ortho_steps_and_coefficients(rows, cols, steps, coeffs):
    g = _matrix(1, rows, cols, F32)
    o = torch.empty(rows, cols, device="cuda", dtype=BF)
    Z.ZeroOrtho(rows=rows, cols=cols, dtype=F32, steps=steps, coeffs=coeffs)(g[0], o)
    k = R.COEFFS if coeffs is None else coeffs
    k = k if hasattr(k[0], "__len__") else [k] * steps
    k = [[float(torch.tensor(v, dtype=F32)) for v in t] for t in k]
    R.ortho_check("o", o, g[0], k, 1e-7)


def test_ortho_of_orthogonal_rows():
    """Singular values of one under the coefficients that hold one fixed: the
    rows of a scaled orthogonal matrix come back as unit vectors."""
    m, n = 64, 200
    q = torch.linalg.qr(R.randn(n, m).double().cpu())[0].T.contiguous().cuda()
    o = torch.empty(m, n, device="cuda", dtype=BF)
    # X0 has singular values 1/8; 1.875 s - 1.25 s^3 + 0.375 s^5 brings them to 1
    Z.ZeroOrtho(rows=m, cols=n, dtype=F32, steps=12, coeffs=(1.875, -1.25, 0.375))(
        (5.0 * q).float(), o)
    off = o.double() - q
    # binary16 storage of X and B (2^-11 each, at a fixed point) and bf16 out
    assert float(torch.linalg.norm(off) / torch.linalg.norm(q)) <= 2 ** -8 + 4 * 2 ** -11


@pytest.mark.parametrize("rows,cols", [(40, 70), (200, 150), (700, 900)])
def test_ortho_special_matrices(rows, cols):
    g = _matrix(6, rows, cols, F32)
    g[1] = 0.0
    g[2, 1, 3] = float("nan")
    g[3, rows - 1, cols - 1] = float("inf")
    g[4] = g[0] * 2.0 ** 100        # far from 1: the norm is taken in binary64
    g[5] = g[0] * 2.0 ** -100       # far below eps
    o = torch.empty(6, rows, cols, device="cuda", dtype=BF)
    Z.ZeroOrtho(batch=6, rows=rows, cols=cols, dtype=F32)(g, o)
    R.ortho_check("matrix 0", o[0], g[0], [R.COEFFS] * 5, 1e-7)
    assert not o[1].any() and not o[5].any()
    assert torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
    R.ortho_check("matrix 4", o[4], g[4], [R.COEFFS] * 5, 1e-7)


@pytest.mark.parametrize("rows,cols", [(60, 50), (333, 444)])
def test_ortho_is_free_of_the_scale(rows, cols):
    """With eps = 0 a power of two cancels exactly."""
    g = _matrix(1, rows, cols, F32)[0]
    a, b = (torch.empty(rows, cols, device="cuda", dtype=BF) for _ in range(2))
    orth = Z.ZeroOrtho(rows=rows, cols=cols, dtype=F32, eps=0.0)
    orth(g, a)
    orth(g * 64.0, b)
    assert torch.equal(a, b)


def test_ortho_on_another_stream_repeats_itself():
    side = torch.cuda.Stream()
    for shape in ((1, 90, 100), (2, 300, 500), (1, 1500, 1300)):
        g = _matrix(*shape, BF)
        outs = []
        for stream in (None, side, side):
            orth = Z.ZeroOrtho(batch=shape[0], rows=shape[1], cols=shape[2], stream=stream)
            o = torch.empty(*shape, device="cuda", dtype=BF)
            orth.workspace.fill_(255)  # nothing is read that this call has not written
            torch.cuda.synchronize()
            orth(g, o)
            torch.cuda.synchronize()
            outs.append(o)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[1], outs[2])


def test_ortho_graph_replays_match_eager():
    side = torch.cuda.Stream()
    for shape in ((1, 100, 120), (2, 300, 260)):
        g = _matrix(*shape, F32).contiguous()
        eager = Z.ZeroOrtho(batch=shape[0], rows=shape[1], cols=shape[2], dtype=F32)
        caught = Z.ZeroOrtho(batch=shape[0], rows=shape[1], cols=shape[2], dtype=F32, stream=side)
        a, b = (torch.empty(*shape, device="cuda", dtype=BF) for _ in range(2))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            caught(g, b)
        for rep in range(3):
            g.copy_(_matrix(*shape, F32, seed=70 + rep))
            eager(g, a)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(a, b), (shape, rep)


def test_ortho_owner_refuses_wrong_tensors():
    orth = Z.ZeroOrtho(batch=2, rows=8, cols=16, dtype=F32)
    g, o = R.randn(2, 8, 16), torch.empty(2, 8, 16, device="cuda", dtype=BF)
    for bad in (g[0], g.to(BF), R.randn(2, 16, 8).transpose(1, 2), g.cpu()):
        with pytest.raises(Z.ZeroShardError):
            orth(bad, o)
    with pytest.raises(Z.ZeroShardError):
        orth(g, torch.empty(2, 8, 16, device="cuda"))
    with pytest.raises(Z.ZeroShardError):
        Z.ZeroOrtho(rows=8, cols=16, steps=0)


@pytest.mark.parametrize("batch,rows,cols,n_d", [(1, 40, 56, 4), (3, 128, 64, 2), (1, 300, 520, 8)])
def test_whole_step(batch, rows, cols, n_d):
    """Two steps of ZeroMuon: momentum, orthogonalised update and weights, each
    against 64 bits from the state before it."""
    n = batch * rows * cols
    w, m = R.randn(n, seed=1, scale=0.02), torch.zeros(n, device="cuda")
    p = torch.empty(n, device="cuda", dtype=BF)
    mu = Z.ZeroMuon(n_d=n_d, batch=batch, rows=rows, cols=cols, master=w, momentum=m, param_out=p,
                    weight_decay=0.1, update_dtype=F32)
    f = lambda v: float(torch.tensor(v, dtype=F32))
    for t in range(2):
        contrib = _rows(n_d, n, seed=100 * t)
        rm, ru = _momentum_ref(contrib, m.clone(), 0.95, True)
        before = w.double()
        mu.step(contrib, 0.02)
        assert torch.equal(m, rm.float())
        u = ru.float().view(batch, rows, cols)
        for i in range(batch):
            R.ortho_check(f"step {t} matrix {i}", mu.o[i], u[i], [R.COEFFS] * 5, 1e-7)
        ref = (before - f(0.02) * f(0.1) * before) - f(0.02) * f(mu.scale) * mu.o.double().view(-1)
        assert torch.equal(w, ref.float()) and torch.equal(p, w.to(BF))
