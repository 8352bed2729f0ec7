"""Embedding, seams and AdamW in one program: the example model runs and its
gradients are the model's; a step of the operators captured in a graph gives what the
eager one does."""

from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("token_model",
                                                  os.path.join(ROOT, "examples", "token_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _plain_gradients(model, ids, targets):
    """The model in binary64 on the CPU, by autograd."""
    leaf = lambda p: p.detach().cpu().double().requires_grad_()
    weights, table = [leaf(w) for w in model.matrices], leaf(model.words)
    gains = [leaf(p) for p in model.gains]
    ids, targets = ids.cpu(), targets.cpu()
    rms = lambda v: v * (v.square().mean(-1, keepdim=True) + model.norm.desc.eps).rsqrt()
    used = table[ids]
    if model.padding is not None:  # its rows take part, without a gradient
        used = torch.where((ids == model.padding)[:, None], used.detach(), used)
    x = used * model.width ** 0.5
    y = rms(x) * gains[0]
    for i in range(len(model.seams)):
        gate, post, gain = gains[1 + 3 * i:4 + 3 * i]
        b = torch.nn.functional.silu(y @ weights[2 * i].T) @ weights[2 * i + 1].T
        x = x + gate * (rms(b) * post)
        y = rms(x) * gain
    logp = (y @ table.T).log_softmax(-1).gather(1, targets[:, None])[:, 0]
    if model.padding is not None:
        logp = logp[targets != model.padding]
    loss = -logp.sum() / max(1, len(logp))
    loss.backward()
    return loss.detach(), [w.grad for w in weights], [table.grad] + [p.grad for p in gains]


@pytest.mark.parametrize("tokens,vocab,width,hidden,padding", [
    (37, 101, 48, 96, None), (64, 19, 129, 64, 3), (1, 50, 64, 32, None)])
def test_gradients_are_the_models(example, tokens, vocab, width, hidden, padding):
    """In binary32, where a sum of k products is off by at most k 2^-24 of its terms'
    magnitudes: k is at most 129 here, the chain has 9 such sums one behind the other
    each way (4 products, 3 norms, the loss, the table's sum) and a norm's own gradient
    magnifies by what it divides by, some ten times.  18 x 129 x 2^-24 x 10 = 1.4e-3 of
    the gradient's norm in the worst case of all signs alike; with signs as they fall
    the root of the count, 18 x 11 x 2^-24 x 10 = 1.2e-4.  Held: 3e-4."""
    model = example.TokenModel(tokens, vocab, width, hidden, dtype=F32, padding=padding)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(vocab, (tokens,), device="cuda", generator=g)
    targets = torch.randint(vocab, (tokens,), device="cuda", generator=g)
    loss, dweights, rest = model.gradients(ids, targets)
    want_loss, want_weights, want_rest = _plain_gradients(model, ids, targets)
    assert abs(float(loss) - float(want_loss)) <= 3e-4 * abs(float(want_loss))
    for got, want in zip(dweights + rest, want_weights + want_rest):
        assert got.shape == want.shape
        off = (got.cpu().double() - want).norm()
        assert off <= 3e-4 * want.norm(), (tuple(want.shape), float(off / want.norm()))


@pytest.mark.parametrize("bits", [8, 32])
def test_steps_move_what_has_a_gradient(example, bits):
    model = example.TokenModel(65, 300, 128, 256, state_bits=bits, padding=7)
    g = torch.Generator(device="cuda").manual_seed(2)
    before = [model.table.clone()] + [p.clone() for p in model.gains]
    for _ in range(3):
        ids = torch.randint(300, (65,), device="cuda", generator=g)
        assert math.isfinite(model.step(ids, ids.roll(-1)))
    for was, now in zip(before, [model.table] + model.gains):
        assert torch.isfinite(now).all() and not torch.equal(was, now)
    assert torch.equal(model.table_bf, model.table.to(BF))
    assert float(model.sumsq) > 0


class _Step:
    """Lookup, seam, a given gradient, and the update of table and gains."""

    def __init__(self, tokens, vocab, width, consts):
        g = torch.Generator(device="cuda").manual_seed(11)
        randn = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.table = randn(vocab, width)
        self.table_bf = self.table.to(BF)
        self.gains = [torch.ones(width, device="cuda") for _ in range(3)]
        self.block, self.dy = randn(tokens, width).to(BF), randn(tokens, width).to(BF)
        new = lambda: torch.empty(tokens, width, device="cuda", dtype=BF)
        self.x, self.s, self.y, self.dx, self.dblock = (new() for _ in range(5))
        self.dtable = torch.empty(vocab, width, device="cuda", dtype=BF)
        self.dgains = [torch.empty_like(p) for p in self.gains]
        self.embed = Z.ZeroEmbedding(tokens=tokens, vocab=vocab, cols=width, scale=2.0)
        self.seam = Z.ZeroBlockNorm(rows=tokens, cols=width, param_dtype=F32, gate="column")
        self.state = Z.adamw_state(vocab * width, 8)
        self.adam = Z.ZeroAdamW(
            [Z.adamw_tensor(self.table, param_out=self.table_bf, weight_decay=0.1, **self.state)]
            + [Z.adamw_tensor(p, grad_dtype=F32, **Z.adamw_state(width)) for p in self.gains],
            max_norm=0.5)
        self.grads = Z.contrib_table([self.dtable] + self.dgains)
        self.sumsq = torch.zeros(1, device="cuda", dtype=F64)
        self.consts = consts

    def queue(self, ids):
        gate, post, gain = self.gains
        self.embed.forward(ids, self.table_bf, self.x)
        self.seam.forward(self.x, self.block, self.s, self.y, gate=gate, gamma_post=post,
                          gamma=gain)
        self.seam.backward(self.dy, self.s, self.block, self.dx, self.dblock, gate=gate,
                           gamma_post=post, gamma=gain, dgate=self.dgains[0],
                           dgamma_post=self.dgains[1], dgamma=self.dgains[2])
        self.embed.backward(ids, self.dx, self.dtable)
        self.adam.gnorm(self.grads, self.sumsq)
        self.adam.step_dev(self.grads, self.consts, self.sumsq)

    def results(self):
        return [self.table, self.table_bf, *self.gains, *self.state.values(), self.y, self.dtable,
                self.sumsq]


@pytest.mark.parametrize("tokens,vocab,width", [(33, 77, 257), (3000, 401, 64)])
def test_captured_steps_are_the_eager_ones(tokens, vocab, width):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        consts = [torch.empty(4, device="cuda", dtype=F64) for _ in range(2)]
        eager, captured = (_Step(tokens, vocab, width, c) for c in consts)
        ids = torch.zeros(tokens, device="cuda", dtype=torch.int64)
        captured.embed.workspace  # before the capture
        graph = torch.cuda.CUDAGraph()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            captured.queue(ids)
        g = torch.Generator(device="cuda").manual_seed(3)
        for t in range(1, 6):
            ids.copy_(torch.randint(vocab, (tokens,), device="cuda", generator=g))
            for c in consts:
                c.copy_(torch.tensor(eager.adam.consts(0.01 / t, t), dtype=F64))
            eager.queue(ids)
            graph.replay()
            stream.synchronize()
            for a, b in zip(eager.results(), captured.results()):
                assert torch.equal(a.view(torch.uint8) if a.element_size() == 1 else a,
                                   b.view(torch.uint8) if b.element_size() == 1 else b), t
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens,vocab,width", [(700, 300, 520), (9000, 500, 72)])
def test_two_programs_at_once(tokens, vocab, width):
    """On two streams, call by call in turn, each what it gives alone."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(9)
    ids = [torch.randint(vocab, (tokens,), device="cuda", generator=g) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)] + [torch.cuda.current_stream()]
    steps = []
    for stream in streams:
        with torch.cuda.stream(stream):
            steps.append(_Step(tokens, vocab, width, torch.empty(4, device="cuda", dtype=F64)))
    consts = [torch.tensor(steps[0].adam.consts(0.01, t + 1), dtype=F64, device="cuda")
              for t in range(4)]
    torch.cuda.synchronize()
    for t in range(4):
        for stream, step in zip(streams[:2], steps):
            with torch.cuda.stream(stream):
                step.consts.copy_(consts[t])
                step.queue(ids[t])
    torch.cuda.synchronize()
    for t in range(4):
        steps[2].consts.copy_(consts[t])
        steps[2].queue(ids[t])
        torch.cuda.synchronize()
    for step in steps[:2]:
        for a, b in zip(step.results(), steps[2].results()):
            assert torch.equal(a.view(torch.uint8) if a.element_size() == 1 else a,
                               b.view(torch.uint8) if b.element_size() == 1 else b)
