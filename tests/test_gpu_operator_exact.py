"""Sums of the training-step operators on whole numbers.  Every partial sum is
below 2^24, so the results are exact in any order of additions and one term
that is lost, doubled or misplaced shows."""
import math

import pytest
import torch

import ring_allreduce_compressed_gb300 as rra

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(shape, seed, most=4, dtype="f32", offset=0):
    shape = (shape,) if isinstance(shape, int) else tuple(shape)
    count = math.prod(shape)
    x = torch.randint(-most, most + 1, (offset + count,), generator=gen(seed), device="cuda")
    return x.to(DT[dtype])[offset:].view(shape)


# ---------------------------------------------------------------- embedding

def order(kind, n, vocab):
    k = torch.arange(n, device="cuda")
    if kind == "same":
        return k * 0 + vocab // 2
    if kind == "two":
        return (k % 2) * (vocab - 1)
    if kind == "falling":
        return (n - 1 - k) % vocab
    if kind == "text":  # frequencies fall with the number
        u = torch.rand(n, generator=gen(n), device="cuda", dtype=torch.float64)
        return (torch.exp(u * torch.log(torch.tensor(vocab + 1.0, device="cuda"))).floor().long()
                - 1).clamp(0, vocab - 1)
    return torch.randint(0, vocab, (n,), generator=gen(n + 1), device="cuda")


def check_embedding_grad(n, dim, vocab, kind, t="f32", out="f32", accumulate=False, index=None):
    d, tok = whole((n, dim), n + dim, 4, t), order(kind, n, vocab)
    base = whole((vocab, dim), 9, 4, out) if accumulate else torch.zeros(vocab, dim, device="cuda")
    want = base.double().index_add_(0, tok, d.double())
    dw = base.clone() if accumulate else torch.full((vocab, dim), 7.0, dtype=DT[out], device="cuda")
    rra.embedding_grad(d, tok if index is None else tok.to(index), dw, accumulate=accumulate)
    assert torch.equal(dw, want.to(DT[out]))


# one block to sixteen, one to eight pairs a thread, and the sort of more
@pytest.mark.parametrize("kind", ["same", "two", "falling", "text", "random"])
@pytest.mark.parametrize("n", [1, 33, 1024, 1025, 2048, 2049, 4097, 8193, 16_384, 16_385, 32_769,
                               65_537, 131_071, 131_072, 131_073, 262_145])
def test_embedding_grad_is_exact(n, kind):
    check_embedding_grad(n, 40, 1200, kind, "bf16")
    check_embedding_grad(n, 40, 1200, kind, "f16", "f16", index=torch.int32)


@pytest.mark.parametrize("kind", ["two", "text", "falling"])
@pytest.mark.parametrize("dim", [1, 7, 130, 513, 1032])
@pytest.mark.parametrize("n", [1500, 20_000])
def test_embedding_grad_widths_are_exact(n, dim, kind):
    check_embedding_grad(n, dim, 900, kind, "bf16", "bf16")
    check_embedding_grad(n, dim, 900, kind, "f32", accumulate=True)


@pytest.mark.parametrize("n", [5000, 131_072, 131_073])
@pytest.mark.parametrize("vocab", [2, 500, 30_000, 70_000])
def test_embedding_grad_vocabularies_are_exact(vocab, n):
    check_embedding_grad(n, 64, vocab, "text", "bf16")
    check_embedding_grad(n, 64, vocab, "random", "bf16", accumulate=True)


# ---------------------------------------------------------------- layer norm's weights

def check_weights(rows, dim, t, w, off=0, accumulate=False):
    """dgamma and dbeta with a mean of 0 and a deviation of 1, so that xh is x."""
    x, dy = whole((rows, dim), 1, 3, t, off), whole((rows, dim), 2, 3, t, off)
    zero, one = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dg, db = whole(dim, 3, 3, w), whole(dim, 4, 3, w)
    want_g, want_b = dg.double() * accumulate, db.double() * accumulate
    for lo in range(0, rows, 4096):
        xd, dyd = x[lo:lo + 4096].double(), dy[lo:lo + 4096].double()
        want_g += (xd * dyd).sum(0)
        want_b += dyd.sum(0)
    dx = torch.full_like(x, 9.0)
    rra.layer_norm_grad(dy, x, None, zero, one, dx, dg, db, accumulate=accumulate)
    assert torch.equal(dg, want_g.to(DT[w])) and torch.equal(db, want_b.to(DT[w]))
    # dx = dy - mean(dy) - x mean(dy x): sums exact, three roundings, one to dx's type
    xd, dyd = x.double(), dy.double()
    a, b = dyd.mean(1, keepdim=True), (dyd * xd).mean(1, keepdim=True)
    want = dyd - a - xd * b
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[t]
    tol = 8 * 2.0 ** -24 * (dyd.abs() + a.abs() + (xd * b).abs()) + u * want.abs() + 2.0 ** -24
    assert bool(((dx.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("t,w", [("f32", "f32"), ("f16", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,dim", [(1, 8), (151, 24), (5003, 40), (10_001, 256), (6001, 768),
                                      (5003, 1001), (10_001, 1032), (5003, 4096), (2500, 6152),
                                      (40_000, 8), (100_001, 63)])
def test_layer_norm_weights_are_exact(rows, dim, t, w):
    check_weights(rows, dim, t, w)
    check_weights(rows, dim, t, w, accumulate=True)


# rows that take the widest block, on 16-byte boundaries and off them, and rows
# that no block holds
@pytest.mark.parametrize("off", [0, 1, 3])
@pytest.mark.parametrize("t,dim", [("bf16", 12_296), ("bf16", 16_384), ("bf16", 12_289),
                                   ("bf16", 16_001), ("bf16", 16_370), ("bf16", 16_371),
                                   ("f16", 16_384), ("f16", 16_001), ("f16", 1001),
                                   ("f32", 6148), ("f32", 8192), ("f32", 7001), ("f32", 8186),
                                   ("f32", 8189), ("f32", 8190), ("f32", 8191), ("f32", 9000)])
def test_layer_norm_wide_rows_are_exact(t, dim, off):
    for rows in (1, 9, 700):
        check_weights(rows, dim, t, "f32", off)


# ---------------------------------------------------------------- means

@pytest.mark.parametrize("dims", [range(1, 1100), range(1100, 33_000, 373), (1 << 14, 1 << 15)])
def test_means_are_the_quotient_that_division_gives(dims):
    """Rows that a block holds divide by their length without a division
    instruction: the result is the division's, bit for bit."""
    for dim in dims:
        most = (1 << 23) // dim
        x = torch.randint(-most, most + 1, (40, dim), generator=gen(dim), device="cuda").float()
        m = torch.empty(40, device="cuda")
        rra.layer_norm(x, None, None, torch.empty_like(x), m)
        s = x.double().sum(1).float()
        assert torch.equal(m, s / torch.full_like(s, float(dim))), dim
