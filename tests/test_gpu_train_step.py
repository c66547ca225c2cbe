"""The training step of examples/train_step.py: embedding, layer norm, the ring
with its codecs and clipping together, against autograd in 64 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference_step(table, bucket, views, batches, scale, lr, max_norm):
    table, bucket = (t.double().requires_grad_() for t in (table, bucket))
    gamma, beta, head = views(bucket)
    losses = []
    for inputs, targets in batches:
        x = table[inputs] * scale
        mean = x.mean(1, keepdim=True)
        var = (x - mean).square().mean(1, keepdim=True)
        y = (x - mean) / (var + 1e-5).sqrt() * gamma + beta
        logp = torch.log_softmax(y @ head.t(), 1)
        losses.append(-logp.gather(1, targets[:, None]).mean())
    loss = torch.stack(losses).mean()
    loss.backward()
    norm = (table.grad.square().sum() + bucket.grad.square().sum()).sqrt()
    c = min(1.0, max_norm / (float(norm) + 1e-6))
    return (table - lr * c * table.grad).detach(), (bucket - lr * c * bucket.grad).detach(), norm


@pytest.mark.parametrize("ranks,max_norm", [(1, 1e9), (4, 0.05), (5, 0.05)])
def test_step_against_autograd(example, ranks, max_norm):
    torch.backends.cuda.matmul.allow_tf32 = False
    m = example.Model(vocab=100, dim=72, tokens=130, ranks=ranks)
    batches = [example.batch(m, 0, r) for r in range(ranks)]
    table, bucket, norm = reference_step(m.table, m.bucket, m.views, batches, m.scale, 0.5,
                                         max_norm)
    m.step(batches, lr=0.5, max_norm=max_norm)
    # fp32 sums of up to 130 * ranks terms, over three layers: 1e-5 of the largest
    assert abs(float(m.norm) / float(norm) - 1) < 1e-5
    for got, want in ((m.table, table), (m.bucket, bucket)):
        assert float((got.double() - want).abs().max()) < 1e-5 * float(want.abs().max())


def test_training_lowers_the_loss(example):
    m = example.Model(vocab=128, dim=64, tokens=512, ranks=2)
    losses = [float(m.step([example.batch(m, s, r) for r in range(2)], lr=2.0, max_norm=1.0))
              for s in range(40)]
    assert losses[-1] < 0.5 * losses[0]
