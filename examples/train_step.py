"""Data-parallel training steps of a small next-token model on simulated ranks.

Every rank looks its tokens up (rra.embedding), normalises them
(rra.layer_norm), scores the next token with a linear head, and goes back
through rra.layer_norm_grad and rra.embedding_grad.  The ranks' gradients then
meet in the ring: the embedding's, mostly zero rows, with the sparse codec;
the head's and the norm's, in one flat bucket, uncompressed.  The averaged
gradients are clipped to a largest norm (rra.grad_clip) and applied.

    python examples/train_step.py [--steps 30] [--ranks 4]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_allreduce_compressed_gb300 as rra  # noqa: E402


class Model:
    """Weights, and one rank's buffers for activations and gradients."""

    def __init__(self, vocab, dim, tokens, ranks, seed=0, ff=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.dim, self.tokens, self.ranks, self.ff = vocab, dim, tokens, ranks, ff
        self.scale = math.sqrt(dim)
        self.table = torch.randn(vocab, dim, generator=g, device="cuda") * 0.02
        # gamma, beta and the head's weight in one flat bucket; the block's behind them
        n = 2 * dim + vocab * dim + 3 * ff * dim
        self.bucket = torch.zeros(n, device="cuda")
        self.gamma, self.beta, self.head = self.views(self.bucket)
        self.gamma.fill_(1.0)
        self.head.copy_(torch.randn(vocab, dim, generator=g, device="cuda") * 0.02)
        if ff:
            for w, fan in zip(self.block(self.bucket), (dim, dim, ff)):
                w.copy_(torch.randn(w.shape, generator=g, device="cuda") / math.sqrt(fan))
            self.saved = rra.Saved.empty(tokens, dim)
            self.gate, self.up = (rra.Saved.empty(tokens, ff) for _ in range(2))
            self.h, self.dh, self.dup = (torch.empty(tokens, ff, device="cuda") for _ in range(3))
        self.x = torch.empty(tokens, dim, device="cuda")
        self.y = torch.empty_like(self.x)
        self.mean, self.rstd = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.dtable = [torch.empty_like(self.table) for _ in range(ranks)]
        self.dbucket = [torch.empty_like(self.bucket) for _ in range(ranks)]
        self.norm = torch.empty(1, device="cuda")
        self.comm = rra.Comm(ranks, max(n, vocab * dim))

    def views(self, bucket):
        d = self.dim
        return bucket[:d], bucket[d:2 * d], bucket[2 * d:(2 + self.vocab) * d].view(self.vocab, d)

    def block(self, bucket):
        """The feed-forward block's gate, up (ff, dim) and down (dim, ff) weights."""
        d, n = self.dim, self.ff * self.dim
        gate, up, down = bucket[(2 + self.vocab) * d:].split(n)
        return gate.view(self.ff, d), up.view(self.ff, d), down.view(d, self.ff)

    def forward(self, inputs):
        """What the head scores."""
        rra.embedding(self.table, inputs, self.x, scale=self.scale)
        if not self.ff:
            rra.layer_norm(self.x, self.gamma, self.beta, self.y, self.mean, self.rstd)
            return self.y
        rra.layer_norm_save(self.x, self.gamma, self.beta, self.y, self.saved, self.mean, self.rstd)
        gate, up, down = self.block(self.bucket)
        rra.gated_ff(self.y, gate, up, self.h, self.gate, self.up)
        return torch.addmm(self.y, self.h, down.t())

    def backward(self, rank, dy):
        """From the gradient of forward's result: into x's, in dy's place, and the weights'."""
        dgamma, dbeta, _ = self.views(self.dbucket[rank])
        if not self.ff:
            rra.layer_norm_grad(dy, self.x, self.gamma, self.mean, self.rstd, dy, dgamma, dbeta)
            return
        gate, up, down = self.block(self.bucket)
        dgate, dup, ddown = self.block(self.dbucket[rank])
        torch.mm(dy, down, out=self.dh)
        # y and h again, out of 8 bits
        rra.layer_norm_restore(self.saved, self.y, self.gamma, self.beta, self.mean, self.rstd)
        dnorm = torch.empty_like(dy)
        rra.gated_ff_grad(self.dh, self.y, gate, up, self.gate, self.up, self.dh, self.dup,
                          dx=dnorm, dw_gate=dgate, dw_up=dup, h=self.h)
        torch.mm(dy.t(), self.h, out=ddown)
        dy += dnorm
        rra.layer_norm_saved_grad(dy, self.saved, self.gamma, self.mean, self.rstd, dy, dgamma,
                                  dbeta)

    def rank_gradients(self, rank, inputs, targets):
        """Forward and backward pass of one rank; returns its loss."""
        y = self.forward(inputs)
        logits = y @ self.head.t()
        logp = torch.log_softmax(logits, 1)
        at = torch.arange(self.tokens, device="cuda")
        loss = -logp[at, targets].mean()
        dlogits = logp.exp()
        dlogits[at, targets] -= 1
        dlogits /= self.tokens
        torch.mm(dlogits.t(), y, out=self.views(self.dbucket[rank])[2])
        dy = dlogits @ self.head
        self.backward(rank, dy)
        rra.embedding_grad(dy, inputs, self.dtable[rank], scale=self.scale)
        return loss

    def step(self, batches, lr, max_norm):
        """One step over every rank's (inputs, targets); returns the mean loss."""
        losses = [self.rank_gradients(r, *b) for r, b in enumerate(batches)]
        self.comm.ring_allreduce(self.dtable, self.dtable, rra.Codec("sparse", average=True))
        self.comm.ring_allreduce(self.dbucket, self.dbucket, rra.Codec("none", average=True))
        # every rank holds the same averages: rank 0's are clipped and applied
        grads = [self.dtable[0], self.dbucket[0]]
        rra.grad_clip(grads, grads, max_norm, self.norm)
        self.table.add_(grads[0], alpha=-lr)
        self.bucket.add_(grads[1], alpha=-lr)
        return torch.stack(losses).mean()


def batch(model, step, rank):
    """Tokens and the ones that follow them by a fixed rule."""
    g = torch.Generator(device="cuda").manual_seed(1000 * step + rank)
    inputs = torch.randint(0, model.vocab, (model.tokens,), generator=g, device="cuda")
    return inputs, (3 * inputs + 1) % model.vocab


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--ff", type=int, default=0, help="width of the feed-forward block (0: none)")
    a = ap.parse_args()
    m = Model(vocab=512, dim=256, tokens=1024, ranks=a.ranks, ff=a.ff)
    for s in range(a.steps):
        loss = m.step([batch(m, s, r) for r in range(a.ranks)], lr=2.0, max_norm=1.0)
        if s % 5 == 0 or s == a.steps - 1:
            print(f"step {s:3d}  loss {float(loss):.4f}  gradient norm {float(m.norm):.4f}")


if __name__ == "__main__":
    main()
