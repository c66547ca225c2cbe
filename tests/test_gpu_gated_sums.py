"""How far the sums of the gated feed-forward block's products may be off, on operands
of one sign, where whatever an instruction cuts off adds up: the bounds that the header gives.

An instruction adds 16 products to an fp32 sum.  It cuts every addend 25 bits below the
leading bit of the largest, less than 2^-25 of it each, and the result to 24 bits, less than
2^-23: 16 * 2^-25 + 2^-23 < 2^-20 of the sum of magnitudes at every 16 elements of k.  (The
leading bit goes by the operands' exponents, so subnormal ones count as the least normal number.)  Sums
of splits and warps are added with roundings of 2^-24, one for 128 elements or more, which
the bound has room for.  fp32: four such instructions of the largest parts of a slice of
64 elements, on that slice's part of the sum: 4 * 5 * 2^-23; those of the smaller parts come
before them, at 2^-6 of it; 2^-21 for the parts left out; a rounding of 2^-24 a slice.  With 16
rows or less, fp32: a rounding for every 51 elements, and 15 more."""
import pytest
import torch

import ring_allreduce_compressed_gb300 as rra
from test_gpu_operators import DT, U, gen, randn

pytestmark = pytest.mark.gpu


def bound(k, t):
    return 2.0 ** -18 + U * k / 32 if t == "f32" else U * (-(-k // 16) * 16)


def positive(shape, seed, t):
    """[1, 2), all bits of the type in use."""
    return (1 + torch.rand(shape, generator=gen(seed), device="cuda")).to(DT[t])


def weights_grad(dh, x):
    """dh^T x in fp32: the gradient of w_gate where gate and up are 1."""
    ff, dim = dh.shape[1], x.shape[1]
    one, w = torch.ones_like(dh), torch.zeros(ff, dim, dtype=dh.dtype, device="cuda")
    dgate, dup = torch.empty_like(dh), torch.empty_like(dh)
    dw = torch.empty(ff, dim, device="cuda")
    rra.gated_ff_grad(dh, x, w, w, one, one, dgate, dup, dw_gate=dw, act="relu")
    assert torch.equal(dgate, dh)
    return dw


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,ff,dim", [(1, 40, 64), (16, 40, 64), (100, 136, 72),
                                         (1000, 2048, 2048), (8192, 2048, 2304), (20_000, 64, 256)])
def test_sums_of_one_sign(rows, ff, dim, t):
    """Many results (few splits along the rows) and few (many splits)."""
    dh, x = positive((rows, ff), 1, t), positive((rows, dim), 2, t)
    got = weights_grad(dh, x)[:64].double()
    want = dh[:, :64].double().t() @ x.double()
    assert ((got - want).abs() <= bound(rows, t) * want).all()


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("j", range(-3, 8))
def test_small_addends_behind_a_large_one(j, t):
    """2^24, and 128 times 16 products of just below 2^(1-j): the sum's last place is 2."""
    rows, ff, dim = 16 * 129, 2048, 2304
    dh = torch.ones(rows, ff, dtype=DT[t], device="cuda")
    x = torch.full((rows, dim), (2 - 2.0 ** -6) * 2.0 ** -j, dtype=DT[t], device="cuda")
    dh[:16] = 0
    dh[0] = x[0] = 2.0 ** 12
    got = weights_grad(dh, x).double()
    want = 2.0 ** 24 + 16 * 128 * (2 - 2.0 ** -6) * 2.0 ** -j
    assert ((got - want).abs() <= bound(rows, t) * want).all()


@pytest.mark.parametrize("rows", [1, 2, 40, 1000])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("both", [False, True])
def test_sums_of_subnormal_numbers(both, t, rows):
    """One operand, or both, down to the type's least number."""
    least = torch.finfo(DT[t]).tiny
    def tiny(shape, seed):  # noqa: E306
        e = torch.rand(shape, generator=gen(seed + 9), device="cuda", dtype=torch.float64)
        v = torch.randn(shape, generator=gen(seed), device="cuda", dtype=torch.float64)
        return (v * least * 2.0 ** torch.floor(16 * e - 10)).to(DT[t])
    dh = tiny((rows, 200), 1)
    # (products of two subnormal numbers of bf16 are no fp32 numbers)
    x = tiny((rows, 520), 2) if both and t == "f16" else randn((rows, 520), 2, 1.0, t)
    got, want = weights_grad(dh, x).double(), dh.double().t() @ x.double()
    size = dh.double().abs().clamp(min=least).t() @ x.double().abs().clamp(min=least)
    assert ((got - want).abs() <= bound(rows, t) * size + 2.0 ** -149).all()
    if rows == 1 and t == "f16":
        assert torch.equal(got, want)


@pytest.mark.parametrize("dim", [7, 64, 1000, 8192])
@pytest.mark.parametrize("rows", [1, 9, 16, 17, 200])
def test_sums_of_the_forward_pass(rows, dim):
    """gate and up of fp32, which show their sums; both kernels."""
    x, wg, wu = positive((rows, dim), 1, "f32"), positive((300, dim), 2, "f32"), \
        positive((300, dim), 3, "f32")
    h, gate, up = (torch.empty(rows, 300, device="cuda") for _ in range(3))
    rra.gated_ff(x, wg, wu, h, gate, up, act="relu")
    for got, w in ((gate, wg), (up, wu)):
        want = x.double() @ w.double().t()
        assert ((got.double() - want).abs() <= bound(dim, "f32") * want).all()


def test_sums_of_dx():
    """k is both halves: 2 ff."""
    rows, ff, dim = 300, 2000, 520
    dh, w = positive((rows, ff), 1, "f32"), [positive((ff, dim), s, "f32") for s in (2, 3)]
    one = torch.ones_like(dh)
    dgate, dup, dx = torch.empty_like(dh), torch.empty_like(dh), torch.empty(rows, dim, device="cuda")
    rra.gated_ff_grad(dh, None, *w, one, one, dgate, dup, dx=dx, act="relu")
    want = dh.double() @ (w[0].double() + w[1].double())
    assert ((dx.double() - want).abs() <= bound(2 * ff, "f32") * want).all()
