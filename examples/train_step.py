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

    def __init__(self, vocab, dim, tokens, ranks, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.dim, self.tokens, self.ranks = vocab, dim, tokens, ranks
        self.scale = math.sqrt(dim)
        self.table = torch.randn(vocab, dim, generator=g, device="cuda") * 0.02
        # gamma, beta and the head's weight in one flat bucket
        n = 2 * dim + vocab * dim
        self.bucket = torch.zeros(n, device="cuda")
        self.gamma, self.beta, self.head = self.views(self.bucket)
        self.gamma.fill_(1.0)
        self.head.copy_(torch.randn(vocab, dim, generator=g, device="cuda") * 0.02)
        self.x = torch.empty(tokens, dim, device="cuda")
        self.y = torch.empty_like(self.x)
        self.mean, self.rstd = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.dtable = [torch.empty_like(self.table) for _ in range(ranks)]
        self.dbucket = [torch.empty_like(self.bucket) for _ in range(ranks)]
        self.norm = torch.empty(1, device="cuda")
        self.comm = rra.Comm(ranks, max(n, vocab * dim))

    def views(self, bucket):
        d = self.dim
        return bucket[:d], bucket[d:2 * d], bucket[2 * d:].view(self.vocab, d)

    def rank_gradients(self, rank, inputs, targets):
        """Forward and backward pass of one rank; returns its loss."""
        rra.embedding(self.table, inputs, self.x, scale=self.scale)
        rra.layer_norm(self.x, self.gamma, self.beta, self.y, self.mean, self.rstd)
        logits = self.y @ self.head.t()
        logp = torch.log_softmax(logits, 1)
        at = torch.arange(self.tokens, device="cuda")
        loss = -logp[at, targets].mean()
        dlogits = logp.exp()
        dlogits[at, targets] -= 1
        dlogits /= self.tokens
        dgamma, dbeta, dhead = self.views(self.dbucket[rank])
        torch.mm(dlogits.t(), self.y, out=dhead)
        dy = dlogits @ self.head
        rra.layer_norm_grad(dy, self.x, self.gamma, self.mean, self.rstd, dy, dgamma, dbeta)
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
    a = ap.parse_args()
    m = Model(vocab=512, dim=256, tokens=1024, ranks=a.ranks)
    for s in range(a.steps):
        loss = m.step([batch(m, s, r) for r in range(a.ranks)], lr=2.0, max_norm=1.0)
        if s % 5 == 0 or s == a.steps - 1:
            print(f"step {s:3d}  loss {float(loss):.4f}  gradient norm {float(m.norm):.4f}")


if __name__ == "__main__":
    main()
