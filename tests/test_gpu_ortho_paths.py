"""The orthogonalisation's ways to spread its work, each against 64 bits: one
workgroup per matrix, strips of columns, every tile shape of the products, tiles
cut along k, two steps at a time; with odd sizes, batches, types, unaligned
rows, ill-conditioned and rank-deficient matrices, coefficients that allow and
forbid pairs, non-finite values, other streams and captured graphs."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
STEPS5 = [R.COEFFS] * 5


@pytest.fixture(autouse=True)
def _gpu_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _matrix(b, r, c, dtype=F32, pad=0, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = 1e-3 * torch.exp(0.5 * torch.randn(b, r, 1, device="cuda", generator=g))
    return (torch.randn(b, r, c + pad, device="cuda", generator=g) * size).to(dtype)[:, :, :c]


def _ortho(g, **kw):
    b, r, c = g.shape
    o = torch.empty(b, r, c, device="cuda", dtype=BF)
    Z.ZeroOrtho(batch=b, rows=r, cols=c, dtype=g.dtype, **kw)(g, o)
    return o


# the last sizes that one workgroup takes, and strips: one row, one strip and
# two, a last strip of one column, every number of row blocks, tall ones
SHORT = [(128, 128), (128, 160), (33, 448), (32, 1056), (1, 1100), (128, 161), (128, 256),
         (128, 257), (65, 1001), (96, 2049), (33, 3000), (1, 20000), (20000, 1), (3001, 64),
         (500, 100), (7000, 127)]


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("rows,cols", SHORT)
def test_short(rows, cols, dtype):
    for pad in (0, 3):
        g = _matrix(1, rows, cols, dtype, pad)
        o = torch.full((1, rows, cols + pad), 7.0, device="cuda", dtype=BF)
        Z.ZeroOrtho(rows=rows, cols=cols, dtype=dtype)(g, o[:, :, :cols])
        R.ortho_check(f"{rows}x{cols}", o[0, :, :cols], g[0], STEPS5, 1e-7)
        assert (o[:, :, cols:] == 7.0).all()  # nothing beside the matrix is written


@pytest.mark.parametrize("batch,rows,cols", [(16, 32, 2000), (3, 100, 1500), (5, 900, 70),
                                             (300, 40, 400)])
def test_short_batches(batch, rows, cols):
    g = _matrix(batch, rows, cols, pad=1)
    o = _ortho(g)
    for i in (0, 1, batch - 1):
        R.ortho_check(f"matrix {i}", o[i], g[i], STEPS5, 1e-7)
        assert torch.equal(o[i], _ortho(g[i:i + 1])[0])


# in the order of the shapes: 64 x 64, 128 x 128, 128 x 256, 192 x 256, 224 x
# 256 and 256 x 256 tiles among their products; the long ones cut the tiles of
# X X^T along k and take two steps at a time
LARGE = [(1, 129, 130), (1, 500, 700), (2, 640, 640), (4, 1024, 1000), (1, 2100, 2900),
         (1, 3000, 3100), (1, 4096, 4096), (1, 5000, 5120), (1, 200, 4000), (1, 512, 4099),
         (1, 700, 5000), (1, 5000, 1300), (2, 1001, 7003), (16, 300, 2000)]


@pytest.mark.parametrize("batch,rows,cols", LARGE)
def test_large(batch, rows, cols):
    g = _matrix(batch, rows, cols, BF if rows % 2 else F32)
    o = _ortho(g)
    for i in (0, batch - 1):
        R.ortho_check(f"matrix {i}", o[i], g[i], STEPS5, 1e-7)


@pytest.mark.parametrize("rows,cols", [(100, 300), (90, 4000), (300, 260), (700, 5000), (4000, 600)])
@pytest.mark.parametrize("kind", ["rank 8", "rank 8 and noise", "decay"])
def test_ill_conditioned(rows, cols, kind):
    m = min(rows, cols)
    if kind == "decay":  # singular values from 1 down to 1e-6
        u = torch.linalg.qr(R.randn(rows, m, seed=1))[0]
        v = torch.linalg.qr(R.randn(cols, m, seed=2))[0]
        g = (u * 10.0 ** (-6.0 * torch.arange(m, device="cuda") / m)) @ v.T.contiguous()
    else:
        g = R.randn(rows, 8, seed=3) @ R.randn(8, cols, seed=4)
        if kind != "rank 8":
            g = g + 1e-3 * R.randn(rows, cols, seed=5)
    o = _ortho(g[None].contiguous())[0]
    assert torch.isfinite(o).all()
    R.ortho_check(kind, o, g, STEPS5, 1e-7)


# the first pair's product is above the limit, the others' below it
FALLING = [(4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037),
           (2.8769, -3.1427, 1.2046), (2.8366, -3.0525, 1.2012)]


@pytest.mark.parametrize("rows,cols", [(60, 50), (120, 1500), (2000, 70), (700, 5000)])
@pytest.mark.parametrize("coeffs", [FALLING, FALLING[:4], FALLING[:1], [(1.5, -0.5, 0.0)] * 7])
def test_coefficients(rows, cols, coeffs):
    g = _matrix(1, rows, cols)
    o = _ortho(g, steps=len(coeffs), coeffs=coeffs)
    k = [[float(torch.tensor(v, dtype=F32)) for v in t] for t in coeffs]
    R.ortho_check("o", o[0], g[0], k, 1e-7)


@pytest.mark.parametrize("rows,cols", [(90, 1200), (1300, 60), (700, 5000)])
def test_special_matrices(rows, cols):
    g = _matrix(6, rows, cols)
    g[1] = 0.0
    g[2, 1, 3] = float("nan")
    g[3, rows - 1, cols - 1] = float("inf")
    g[4] = g[0] * 2.0 ** 100   # far from 1: the norm is taken in binary64
    g[5] = g[0] * 2.0 ** -100  # far below eps
    o = _ortho(g)
    R.ortho_check("matrix 0", o[0], g[0], STEPS5, 1e-7)
    assert not o[1].any() and not o[5].any()
    assert torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
    R.ortho_check("matrix 4", o[4], g[4], STEPS5, 1e-7)


@pytest.mark.parametrize("batch,rows,cols", [(2, 96, 128), (2, 100, 3000), (1, 512, 4096),
                                             (1, 700, 5000)])
def test_streams_and_graphs(batch, rows, cols):
    """The same bits on another stream, over workspaces that hold anything, and
    from every replay of a captured call."""
    side = torch.cuda.Stream()
    g = _matrix(batch, rows, cols).contiguous()
    eager = Z.ZeroOrtho(batch=batch, rows=rows, cols=cols, dtype=F32)
    caught = Z.ZeroOrtho(batch=batch, rows=rows, cols=cols, dtype=F32, stream=side)
    a, b = (torch.empty(batch, rows, cols, device="cuda", dtype=BF) for _ in range(2))
    caught.workspace.fill_(255)
    torch.cuda.synchronize()
    caught(g, b)
    eager(g, a)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        caught(g, b)
    for rep in range(3):
        g.copy_(_matrix(batch, rows, cols, seed=70 + rep))
        eager.workspace.fill_(rep)
        eager(g, a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b), rep


@pytest.mark.parametrize("rows,cols", [(30, 40), (100, 3000), (3000, 100), (300, 500)])
def test_unaligned_buffers(rows, cols):
    """Matrices that start between 16-byte boundaries give the aligned bits."""
    n = rows * cols
    g = R.randn(n + 1, dtype=BF, seed=2)[1:].view(1, rows, cols)
    o = torch.empty(n + 1, device="cuda", dtype=BF)[1:].view(1, rows, cols)
    Z.ZeroOrtho(rows=rows, cols=cols)(g, o)
    assert torch.equal(o, _ortho(g.clone()))
