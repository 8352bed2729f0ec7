"""A pre-norm feed-forward block trained with the library's operators: layer
norm (with the residual's gradient joined in its backward pass), Muon for the
two weight matrices, the AdamW shard step for the norm's gain and bias.  Two
ranks' micro-batches give the gradient contributions.

    python examples/muon_block.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sharded_mixed_precision_zero_amd as Z  # noqa: E402

BF = torch.bfloat16


class Block:
    """out = x + relu(LN(x) W1^T) W2^T over (tokens, width) bf16 tensors."""

    def __init__(self, tokens: int, width: int, hidden: int, ranks: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ranks, self.width = ranks, width
        self.norm = Z.ZeroLayerNorm(rows=tokens, cols=width, dtype=BF)
        self.muon, self.weights = [], []
        for rows, cols in ((hidden, width), (width, hidden)):
            n = rows * cols
            master = torch.randn(n, device="cuda", generator=g) * cols ** -0.5
            weight = master.to(BF)
            self.weights.append(weight.view(rows, cols))
            self.muon.append(Z.ZeroMuon(n_d=ranks, rows=rows, cols=cols, master=master,
                                        momentum=torch.zeros(n, device="cuda"), param_out=weight))
        # gain and bias, one after another
        self.affine = torch.cat([torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")])
        self.affine_bf = self.affine.to(BF)
        self.adam = Z.ZeroShard(phi=2 * width, n_d=ranks, r=0, shard_len=2 * width,
                                master=self.affine, m=torch.zeros_like(self.affine),
                                v=torch.zeros_like(self.affine), param_out=self.affine_bf)
        self.y, self.dx = (torch.empty(tokens, width, device="cuda", dtype=BF) for _ in range(2))
        self.t = 0

    def gradients(self, x, target):
        """The loss, and the bf16 gradients of W1, W2 and (gain, bias)."""
        gain, bias = self.affine_bf[:self.width], self.affine_bf[self.width:]
        w1, w2 = self.weights
        self.norm.forward(x, self.y, gamma=gain, beta=bias)
        z = self.y @ w1.T
        a = torch.relu(z)
        off = (x + a @ w2.T).float() - target.float()
        dout = (off * (2.0 / off.numel())).to(BF)
        dz = (dout @ w2) * (z > 0)
        dy = dz @ w1
        affine = torch.empty(2 * self.width, device="cuda", dtype=BF)
        # dx also takes dout, which reaches x past the block
        self.norm.backward(dy, x, self.dx, gamma=gain, dgamma=affine[:self.width],
                           dbeta=affine[self.width:], dsum=dout)
        grads = [dz.T.contiguous() @ self.y, dout.T.contiguous() @ a]
        return (off * off).mean(), [w.view(-1) for w in grads] + [affine]

    def step(self, batches, lr: float = 0.02) -> float:
        """One update from a batch (x, target) of each rank; the mean loss."""
        self.t += 1
        per_rank = [self.gradients(*b) for b in batches]
        for i, muon in enumerate(self.muon):
            muon.step([g[i] for _, g in per_rank], lr)
        self.adam.step([g[2] for _, g in per_rank], lr, self.t)
        return sum(float(loss) for loss, _ in per_rank) / len(per_rank)


def train(steps: int = 40, tokens: int = 512, width: int = 256, hidden: int = 1024,
          ranks: int = 2) -> list[float]:
    """The losses of fitting a block to another one of random weights."""
    block, teacher = (Block(tokens, width, hidden, ranks, seed=s) for s in (1, 2))
    g = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for _ in range(steps):
        batches = []
        for _ in range(ranks):
            x = torch.randn(tokens, width, device="cuda", generator=g).to(BF)
            y = torch.empty_like(x)
            teacher.norm.forward(x, y)
            batches.append((x, x + torch.relu(y @ teacher.weights[0].T) @ teacher.weights[1].T))
        losses.append(block.step(batches))
    return losses


if __name__ == "__main__":
    for i, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)):
        if i % 5 == 0:
            print(f"step {i:4d}  loss {loss:.4f}")
