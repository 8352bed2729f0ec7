"""The embedding and the gradient of its table on the GPU against 64 bits:
types, odd widths, strides, tables split over ranks, padding, rows of every
length up to all tokens, more tokens than a sorted tile, accumulation, streams,
captured graphs, differences."""

from __future__ import annotations

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(autouse=True)
def _gpu_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


TYPES = [(F32, F32), (BF, BF), (BF, F32), (F16, F16), (F16, F32)]
SCALE = 1.7


def _ids(tokens, lo, hi, seed=0, dtype=I64, power=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(tokens, device="cuda", generator=g, dtype=torch.float64) ** power
    return (lo + u * (hi - lo)).floor().to(dtype)


def _plan(ids, vocab, cols, dtype, other, **kw):
    return Z.ZeroEmbedding(tokens=ids.numel(), vocab=vocab, cols=cols, dtype=dtype,
                           table_dtype=other, grad_dtype=other, id_dtype=ids.dtype, scale=SCALE,
                           **kw)


@pytest.mark.parametrize("dtype,other", TYPES)
@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (1, 32000, 5120), (3, 7, 2), (17, 100, 8),
                                               (333, 50, 1601), (1000, 9, 64), (40, 40, 4104),
                                               (5000, 300, 24), (70, 31, 9), (65, 40, 515)])
def test_forward(tokens, vocab, cols, dtype, other):
    for pad, ids_t, first in ((0, I64, 0), (3, I32, 5), (8, I64, -4)):
        ids = _ids(tokens, first - 2, first + vocab + 2, dtype=ids_t)
        table = R.randn(vocab, cols, dtype=other, pad=pad, seed=1)
        y = R.randn(tokens, cols, dtype=dtype, pad=pad, seed=2)
        _plan(ids, vocab, cols, dtype, other, first=first).forward(ids, table, y)
        row = ids.long() - first
        live = (row >= 0) & (row < vocab)
        ref = torch.where(live[:, None], table[row.clamp(0, vocab - 1)].float() * SCALE, 0.0)
        assert torch.equal(y, ref.to(dtype))  # one product, one rounding


def _reference(ids, dy, vocab, first=0, padding=None, old=None):
    """The table's gradient in 64 bits and its error: a row's tokens in runs of
    32 (8 up to 2048 tokens in all), the runs in 4 stretches."""
    row = ids.long().reshape(-1) - first
    live = (row >= 0) & (row < vocab)
    if padding is not None:
        live &= ids.reshape(-1) != padding
    ref = torch.zeros(vocab, dy.shape[1], device="cuda", dtype=torch.float64)
    size, count = ref.clone(), torch.zeros(vocab, device="cuda", dtype=torch.float64)
    ref.index_add_(0, row[live], dy.double()[live])
    size.index_add_(0, row[live], dy.double().abs()[live])
    count.index_add_(0, row[live], torch.ones_like(row[live], dtype=torch.float64))
    run = 8 if ids.numel() <= 2048 else 32
    chain = torch.minimum(count, run + torch.ceil(count / (4 * run)) + 4)[:, None]
    s = float(torch.tensor(SCALE))
    ref, tol = ref * s, size * s * chain * R.U + 2 * R.U * abs(ref) * s
    if old is not None:
        ref, tol = ref + old.double(), tol + 2 * R.U * (abs(ref) + abs(old.double()))
    return ref, tol, count > 0


def _backward(ids, vocab, cols, dtype, other, pad=0, accumulate=False, first=0, padding=None):
    dy = R.randn(ids.numel(), cols, dtype=dtype, pad=pad, seed=3)
    out = R.randn(vocab, cols, dtype=other, pad=pad, seed=4)
    old = out.clone() if accumulate else None
    plan = _plan(ids, vocab, cols, dtype, other, first=first, padding=padding)
    plan.backward(ids, dy, out, accumulate=accumulate)
    ref, tol, used = _reference(ids, dy, vocab, first, padding, old)
    R.within("dtable", out, ref, tol + R.half_step(other, ref.abs() + tol))
    if accumulate:
        assert torch.equal(out[~used], old[~used])
    else:
        assert (out[~used] == 0).all()
    return out


@pytest.mark.parametrize("dtype,other", TYPES)
@pytest.mark.parametrize("tokens,vocab,cols", [
    (1, 1, 1), (1, 1000, 5120), (2, 3, 5), (31, 4, 64), (32, 1, 64), (33, 1, 64), (64, 1, 40),
    (65, 2, 1601), (333, 1009, 1601), (1023, 40, 72), (1024, 3, 520), (1025, 40, 72),
    (600, 50, 5120), (601, 50, 5120), (64, 5000, 37), (1500, 60, 9), (1500, 40, 515),
    (9000, 200, 13), (4096, 7, 256), (1000, 300, 2056), (8191, 5000, 72),
    (8192, 1, 16), (8192, 32000, 136)])
def test_backward(tokens, vocab, cols, dtype, other):
    for pad, ids_t, first, acc in ((0, I64, 0, False), (3, I32, 7, True), (8, I64, -3, False)):
        ids = _ids(tokens, first - 1, first + vocab + 1, dtype=ids_t, power=2.0)
        _backward(ids, vocab, cols, dtype, other, pad, acc, first, padding=first + vocab // 2)


@pytest.mark.parametrize("tokens", [8193, 16384, 20001, 65536, 65537, 150_000, 600_000])
@pytest.mark.parametrize("power", [1.0, 4.0])
def test_more_tokens_than_a_sorted_tile(tokens, power):
    ids = _ids(tokens, 0, 3000, seed=tokens, power=power)
    _backward(ids, 3000, 24, BF, F32, padding=0)


@pytest.mark.parametrize("lengths", [
    [1] * 100, [32] * 8, [33] * 8, [31, 33, 1, 64, 65, 32, 96, 2], [5, 200, 1, 1, 30, 2, 33],
    [8] * 20, [9] * 20, [7, 8, 9, 16, 17, 1], [1000], [31, 1000, 1], [63, 64, 65, 66], [16, 17] * 9, [257 * 32 + 5, 3], [40000, 17, 300]])
def test_rows_of_every_length(lengths):
    """Rows of these many tokens, the tokens shuffled: parts that begin and end at
    every place of a piece."""
    ids = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))
    g = torch.Generator().manual_seed(1)
    ids = ids[torch.randperm(len(ids), generator=g)].cuda()
    for cols in (8, 520):
        _backward(ids, len(lengths) + 2, cols, F32, F32)


@pytest.mark.parametrize("shift", range(0, 34, 3))
def test_long_rows_at_every_offset(shift):
    few = [0] * shift + [1] * 100 + [2] * (70 - shift) + [3] * 3
    for ids in (few, few + [9] * 3000, [0] * (1000 + shift) + few[shift:] * 20):
        ids = torch.sort(torch.tensor(ids, device="cuda")).values
        for cols in (16, 520):
            _backward(ids, 5, cols, F32, F32)


@pytest.mark.parametrize("cols", [24, 1601])
@pytest.mark.parametrize("tokens", [1, 8, 9, 32, 33, 65, 260, 1000, 1024])
def test_few_tokens_sum_as_sorted_ones_do(tokens, cols):
    """Beside tokens of other ranks' rows, so many that all are sorted, the same bits."""
    ids = torch.cat([_ids(tokens, 0, 40, power=3.0), torch.full((1500 - tokens,), -1, device="cuda")])
    dy = R.randn(1500, cols, seed=7) * torch.exp(4 * R.randn(1500, 1, seed=8))
    outs = [torch.empty(40, cols, device="cuda") for _ in range(2)]
    for n, out in zip((tokens, 1500), outs):
        Z.ZeroEmbedding(tokens=n, vocab=40, cols=cols, dtype=F32).backward(ids[:n], dy[:n], out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("shift", [0, 1, 4, 8])
@pytest.mark.parametrize("tokens", [5, 1200])
def test_cleared_stretches_at_every_alignment(tokens, shift):
    """Gradients that begin anywhere and whose rows end anywhere: all of them are written
    and nothing beside them."""
    for vocab, cols in ((3001, 37), (257, 1000), (2, 5121), (70_000, 8), (5000, 1)):
        buf = torch.full((vocab * cols + 32,), 3.0, device="cuda", dtype=BF)
        out = buf[8 + shift:8 + shift + vocab * cols].view(vocab, cols)
        ids = _ids(tokens, 0, vocab, seed=5)
        Z.ZeroEmbedding(tokens=tokens, vocab=vocab, cols=cols).backward(
            ids, torch.ones(tokens, cols, device="cuda", dtype=BF), out)
        want = torch.bincount(ids, minlength=vocab)[:, None].expand(vocab, cols).to(BF)
        assert torch.equal(out, want)
        assert (buf[:8 + shift] == 3).all() and (buf[8 + shift + vocab * cols:] == 3).all()


def test_the_order_of_a_rows_sum():
    """A row's sum is that of its tokens in order, bit for bit: in runs of 8 or,
    among many tokens, of 32."""
    for n, others, run in ((5, 0, 8), (8, 0, 8), (32, 0, 8), (20, 3000, 32), (128, 3000, 32)):
        dy = R.randn(n + others, 16, seed=7) * torch.exp(4 * R.randn(n + others, 1, seed=8))
        ids = torch.full((n + others,), 3, device="cuda")
        ids[n:] = -1
        out = torch.empty(5, 16, device="cuda")
        plan = Z.ZeroEmbedding(tokens=n + others, vocab=5, cols=16, dtype=F32)
        plan.backward(ids, dy, out)
        want = torch.zeros(16, device="cuda")
        for at in range(0, n, run):
            part = torch.zeros(16, device="cuda")
            for t in range(at, min(n, at + run)):
                part = part + dy[t]
            want = want + part
        assert torch.equal(out[3], want), (n, others)


@pytest.mark.parametrize("tokens", [500, 9000])
def test_ranks_parts_add_up(tokens):
    """A table split over four ranks: the outputs add up to the whole's, and
    the gradients are its rows."""
    vocab, cols = 1000, 96
    ids = _ids(tokens, 0, vocab, power=2.0)
    table = R.randn(vocab, cols, dtype=BF, seed=1)
    dy = R.randn(tokens, cols, dtype=BF, seed=2)
    whole = _plan(ids, vocab, cols, BF, BF, padding=17)
    y, dw = torch.empty_like(dy), torch.empty_like(table)
    whole.forward(ids, table, y)
    whole.backward(ids, dy, dw)
    total = torch.zeros(tokens, cols, device="cuda")
    for r in range(4):
        part = _plan(ids, 250, cols, BF, BF, first=250 * r, padding=17)
        yr, dr = torch.empty_like(dy), torch.empty(250, cols, device="cuda", dtype=BF)
        part.forward(ids, table[250 * r:250 * (r + 1)], yr)
        part.backward(ids, dy, dr)
        total += yr.float()
        assert torch.equal(dr, dw[250 * r:250 * (r + 1)])
    assert torch.equal(total.to(BF), y)


def test_far_ids():
    """Ids at the ends of 64 bits, and a table whose first id lies there."""
    lo, hi = -(1 << 63), (1 << 63) - 1
    ids = torch.tensor([lo, lo + 1, -1, 0, 1, hi - 1, hi], device="cuda")
    table = R.randn(3, 40, seed=1)
    for first in (lo, -1, 0, hi - 2):
        y, dw = torch.empty(7, 40, device="cuda"), torch.empty(3, 40, device="cuda")
        plan = Z.ZeroEmbedding(tokens=7, vocab=3, cols=40, dtype=F32, first=first)
        plan.forward(ids, table, y)
        dy = R.randn(7, 40, seed=2)
        plan.backward(ids, dy, dw)
        want, grad = torch.zeros_like(y), torch.zeros_like(dw)
        for t, i in enumerate(ids.tolist()):
            if 0 <= i - first < 3:
                want[t], grad[i - first] = table[i - first], dy[t]
        assert torch.equal(y, want) and torch.equal(dw, grad), first


def test_every_token_is_padding_or_elsewhere():
    ids = torch.tensor([4, 4, 99, -1, 4] * 30, device="cuda")
    dy = R.randn(150, 64, dtype=BF, seed=1)
    plan = Z.ZeroEmbedding(tokens=150, vocab=50, cols=64, padding=4)
    out = torch.full((50, 64), 3.0, device="cuda", dtype=BF)
    plan.backward(ids, dy, out, accumulate=True)
    assert (out == 3.0).all()
    plan.backward(ids, dy, out)
    assert (out == 0).all()


def test_no_tokens():
    plan = Z.ZeroEmbedding(tokens=0, vocab=50, cols=64)
    ids, rows = torch.empty(0, device="cuda", dtype=I64), torch.empty(0, 64, device="cuda", dtype=BF)
    out = torch.full((50, 64), 3.0, device="cuda", dtype=BF)
    plan.forward(ids, out, rows)
    plan.backward(ids, rows, out, accumulate=True)
    assert (out == 3.0).all()
    plan.backward(ids, rows, out)
    assert (out == 0).all()


def test_infinities_and_nan_stay_in_their_rows():
    """A token of no row may hold anything."""
    ids = torch.tensor([0, 1, 2, 3, 1, 9, 0] * 40, device="cuda")
    dy = R.randn(280, 72, seed=1)
    dy[ids == 9] = float("nan")
    dy[1, 5], dy[2, 6] = float("inf"), float("nan")
    out = torch.empty(5, 72, device="cuda")
    Z.ZeroEmbedding(tokens=280, vocab=5, cols=72, dtype=F32).backward(ids, dy, out)
    bad = ~torch.isfinite(out)
    assert bad.sum() == 2 and out[1, 5] == float("inf") and torch.isnan(out[2, 6])


def test_outside_the_outputs_nothing_is_written():
    bufs = [torch.full((n + 2, 40 + 5), 3.0, device="cuda", dtype=BF) for n in (70, 9)]
    y, dw = bufs[0][1:71, :37], bufs[1][1:10, :37]
    ids = _ids(70, 0, 9)
    plan = Z.ZeroEmbedding(tokens=70, vocab=9, cols=37)
    table = R.randn(9, 37, dtype=BF)
    plan.forward(ids, table, y)
    plan.backward(ids, y, dw)
    for b in bufs:
        assert (b[0] == 3.0).all() and (b[-1] == 3.0).all() and (b[:, 37:] == 3.0).all()


def test_gradient_is_the_forward_differentiated():
    """The forward pass is linear: <dy, y(W + V) - y(W)> = <dW, V>."""
    ids = _ids(700, 0, 90, power=3.0)
    plan = Z.ZeroEmbedding(tokens=700, vocab=90, cols=100, dtype=F32, scale=SCALE)
    w, v, dy = (R.randn(*s, seed=i) for i, s in enumerate([(90, 100), (90, 100), (700, 100)]))
    y0, y1, dw = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(w)
    plan.forward(ids, w, y0)
    plan.forward(ids, w + v, y1)
    plan.backward(ids, dy, dw)
    got = float((dw.double() * v.double()).sum())
    want = float((dy.double() * (y1.double() - y0.double())).sum())
    # y0 and y1 are rounded once, w + v once
    size = float((dy.double().abs() * (y0.double().abs() + y1.double().abs())).sum())
    assert abs(got - want) <= 200 * R.U * size


def test_the_same_bits_every_time_and_on_another_stream():
    ids = _ids(20000, 0, 500, power=3.0)
    dy = R.randn(20000, 264, dtype=BF, seed=1)
    torch.cuda.synchronize()
    outs = []
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.current_stream()):
        with torch.cuda.stream(stream):
            plan = Z.ZeroEmbedding(tokens=20000, vocab=500, cols=264)
            out = torch.empty(500, 264, device="cuda", dtype=BF)
            plan.backward(ids, dy, out)
            stream.synchronize()
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("tokens", [300, 9000])
def test_in_a_captured_graph(tokens):
    side = torch.cuda.Stream()
    ids = _ids(tokens, 0, 200)
    dy = R.randn(tokens, 136, dtype=BF, seed=1)
    table = R.randn(200, 136, dtype=BF, seed=2)
    with torch.cuda.stream(side):
        plan = Z.ZeroEmbedding(tokens=tokens, vocab=200, cols=136)
        eager = Z.ZeroEmbedding(tokens=tokens, vocab=200, cols=136)
        y, dw = torch.empty_like(dy), torch.empty_like(table)
        plan.backward(ids, dy, dw)  # the workspace is there before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan.forward(ids, table, y)
        plan.backward(ids, dy, dw)
    for k in range(3):
        with torch.cuda.stream(side):
            ids.copy_(_ids(tokens, -3, 210, seed=10 + k, power=3.0))
            dy.copy_(R.randn(tokens, 136, dtype=BF, seed=20 + k))
            graph.replay()
            want = torch.empty_like(y), torch.empty_like(dw)
            eager.forward(ids, table, want[0])
            eager.backward(ids, dy, want[1])
        side.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dw, want[1])


def test_rows_past_32_bit_offsets():
    """A table, a gradient and dy whose rows lie past 2^32 bytes."""
    ld, cols = (1 << 30) + 8, 64
    buf = torch.zeros(3 * ld + cols, device="cuda", dtype=BF)
    far = buf.as_strided((4, cols), (ld, 1))
    near = R.randn(4, cols, dtype=BF, seed=1)
    far.copy_(near)
    ids = torch.tensor([3, 0, 3, 2], device="cuda")
    plan = Z.ZeroEmbedding(tokens=4, vocab=4, cols=cols)
    y, yf = torch.empty_like(near), torch.empty_like(near)
    plan.forward(ids, near, y)
    plan.forward(ids, far, yf)
    assert torch.equal(y, yf)
    dw, dwf = torch.empty_like(near), torch.empty_like(near)
    plan.backward(ids, near, dw)
    plan.backward(ids, far, dwf)
    assert torch.equal(dw, dwf)
    plan.backward(ids, near, far)
    assert torch.equal(far, dw)
