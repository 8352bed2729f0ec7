"""A small token model trained with the library's operators: the embedding (its
table also the output's), blocks joined by the fused seams (norm of a block's
output, gate, scaled residual sum, norm before the next block), Muon for the
blocks' matrices and one AdamW call for all that is no matrix: the table with its
state in 8 bits, gains and gates.

    python examples/token_model.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sharded_mixed_precision_zero_amd as Z  # noqa: E402

BF = torch.bfloat16


class TokenModel:
    """Blocks silu(y W1^T) W2^T between seams over (tokens, width) activations of
    ``dtype`` (bf16 or fp32); bf16 matrices, fp32 gains and gates."""

    def __init__(self, tokens: int, vocab: int, width: int, hidden: int, blocks: int = 2,
                 dtype=BF, state_bits: int = 8, max_norm: float = 1.0, padding: int | None = None,
                 seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens, self.width, self.dtype, self.padding = tokens, width, dtype, padding
        self.table = torch.randn(vocab, width, device="cuda", generator=g) * width ** -0.5
        self.table_bf = self.table.to(BF)
        self.words = self.table_bf if dtype is BF else self.table  # what the lookup reads
        self.embed = Z.ZeroEmbedding(tokens=tokens, vocab=vocab, cols=width, dtype=dtype,
                                     scale=width ** 0.5, padding=padding)
        # the norm before the first block, and the seam behind each
        self.norm = Z.ZeroBlockNorm(rows=tokens, cols=width, dtype=dtype, post=False,
                                    param_dtype=torch.float32)
        self.seams = [Z.ZeroBlockNorm(rows=tokens, cols=width, dtype=dtype, gate="column",
                                      param_dtype=torch.float32) for _ in range(blocks)]
        self.matrices, self.muon = [], []
        for rows, cols in ((hidden, width), (width, hidden)) * blocks:
            master = torch.randn(rows * cols, device="cuda", generator=g) * cols ** -0.5
            weight = master.to(BF)
            self.matrices.append(weight.view(rows, cols))
            self.muon.append(Z.ZeroMuon(n_d=1, rows=rows, cols=cols, master=master,
                                        momentum=torch.zeros_like(master), param_out=weight))
        # the first norm's gain; of each seam the gate and the two norms' gains
        one = lambda x: torch.full((width,), x, device="cuda")
        self.gains = [one(1.0)] + [one(x) for _ in range(blocks) for x in (0.5, 1.0, 1.0)]
        self.adam = Z.ZeroAdamW(
            [Z.adamw_tensor(self.table, param_out=self.table_bf, grad_dtype=dtype,
                            **Z.adamw_state(vocab * width, state_bits))]
            + [Z.adamw_tensor(p, grad_dtype=torch.float32, **Z.adamw_state(width))
               for p in self.gains], max_norm=max_norm)
        self.sumsq = torch.zeros(1, device="cuda", dtype=torch.float64)
        self.t = 0

    def _new(self):
        return torch.empty(self.tokens, self.width, device="cuda", dtype=self.dtype)

    def gradients(self, ids, targets):
        """The loss, the gradients of the matrices, and those of the table and
        the gains (in the order of self.matrices and of self.adam's tensors)."""
        dtype = self.dtype
        weights = [w.to(dtype) for w in self.matrices]
        table = self.words
        seams = [self.gains[1 + 3 * i:4 + 3 * i] for i in range(len(self.seams))]

        x, y = self._new(), self._new()
        self.embed.forward(ids, table, x)
        self.norm.forward(x, None, None, y, gamma=self.gains[0])
        total, ys, zs, outs = [x], [y], [], []
        for i, seam in enumerate(self.seams):
            gate, post, gain = seams[i]
            zs.append(ys[-1] @ weights[2 * i].T)
            outs.append(torch.nn.functional.silu(zs[-1]) @ weights[2 * i + 1].T)
            s, y = self._new(), self._new()
            seam.forward(total[-1], outs[-1], s, y, gate=gate, gamma_post=post, gamma=gain)
            total.append(s)
            ys.append(y)

        logits = (ys[-1] @ table.T).float()
        logp = logits.log_softmax(-1)
        use = torch.ones_like(targets, dtype=torch.bool)
        if self.padding is not None:
            use = targets != self.padding
        n = use.sum().clamp(min=1)
        loss = -(logp.gather(1, targets[:, None])[:, 0] * use).sum() / n
        dlogits = logp.exp()
        dlogits[torch.arange(len(targets), device="cuda"), targets] -= 1.0
        dlogits = (dlogits * (use[:, None] / n)).to(dtype)

        dtable = dlogits.T.contiguous() @ ys[-1]
        dy, dtotal = dlogits @ table, None
        dgains = [torch.empty_like(p) for p in self.gains]
        dweights = [None] * len(weights)
        for i in reversed(range(len(self.seams))):
            gate, post, gain = seams[i]
            dgate, dpost, dgain = dgains[1 + 3 * i:4 + 3 * i]
            dx, dout = self._new(), self._new()
            self.seams[i].backward(dy, total[i + 1], outs[i], dx, dout, dsum=dtotal, gate=gate,
                                   gamma_post=post, gamma=gain, dgate=dgate, dgamma_post=dpost,
                                   dgamma=dgain)
            z = zs[i].float()
            sig = z.sigmoid()
            dweights[2 * i + 1] = dout.T.contiguous() @ (z * sig).to(dtype)
            dz = (dout @ weights[2 * i + 1]).float() * (sig * (1 + z * (1 - sig)))
            dz = dz.to(dtype)
            dweights[2 * i] = dz.T.contiguous() @ ys[i]
            dy, dtotal = dz @ weights[2 * i], dx
        dx = self._new()
        self.norm.backward(dy, total[0], None, dx, None, dsum=dtotal, gamma=self.gains[0],
                           dgamma=dgains[0])
        # the table's gradient as the embedding joins that as the output's
        self.embed.backward(ids, dx, dtable, accumulate=True)
        return loss, dweights, [dtable] + dgains

    def step(self, ids, targets, lr: float = 0.01) -> float:
        """One update from a batch; the loss before it."""
        self.t += 1
        loss, dweights, rest = self.gradients(ids, targets)
        for muon, dw in zip(self.muon, dweights):
            muon.step([dw.to(BF).view(-1)], lr)
        self.adam.gnorm(rest, self.sumsq)  # over ranks: all-reduce self.sumsq here
        self.adam.step(rest, lr, self.t, self.sumsq)
        return float(loss)


def train(steps: int = 40, tokens: int = 512, vocab: int = 1000, width: int = 256,
          hidden: int = 512) -> list[float]:
    """The losses of learning a fixed map from a token to the next."""
    model = TokenModel(tokens, vocab, width, hidden)
    g = torch.Generator(device="cuda").manual_seed(1)
    following = torch.randperm(vocab, device="cuda", generator=g)
    losses = []
    for _ in range(steps):
        ids = torch.randint(vocab, (tokens,), device="cuda", generator=g)
        losses.append(model.step(ids, following[ids]))
    return losses


if __name__ == "__main__":
    for i, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)):
        if i % 5 == 0:
            print(f"step {i:4d}  loss {loss:.4f}")
