"""Where the gated feed-forward block's results lie: every output at a place of its own,
with guards on both sides; and its weights' gradients as a whole."""
import math

import pytest
import torch

import ring_allreduce_compressed_gb300 as rra
from test_gpu_gated_ff import check_ff, check_ff_grad, grad_inputs, weights
from test_gpu_operators import DT, TINY, U, UT, randn

pytestmark = pytest.mark.gpu

GUARD = 40  # elements


class Place:
    """Room for an output, `offset` elements behind a 16-byte boundary, between two guards."""

    def __init__(self, shape, t, offset, fill=9.0):
        n = math.prod(shape)
        self.whole = torch.full((2 * GUARD + offset + n,), fill, dtype=t, device="cuda")
        self.out = self.whole[GUARD + offset:GUARD + offset + n].view(shape)
        self.ends = (self.whole[:GUARD + offset], self.whole[GUARD + offset + n:])
        self.fill = fill

    def untouched(self):
        return all(bool((e == self.fill).all()) for e in self.ends)


def moved(v, offset):
    """The same values, `offset` elements behind a 16-byte boundary."""
    to = torch.empty(offset + v.numel(), dtype=v.dtype, device="cuda")[offset:].view(v.shape)
    return to.copy_(v)


@pytest.mark.parametrize("t,wt", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                  ("bf16", "f32")])
@pytest.mark.parametrize("keep", ["full", "bits8"])
@pytest.mark.parametrize("rows,dim,ff", [(150, 64, 136), (33, 72, 137), (70, 129, 264),
                                         (200, 51, 333), (2, 5, 7)])
def test_ff_grad_into_every_place(rows, dim, ff, keep, t, wt):
    """The same bits as into arrays of their own, whose results are checked in 64 bits, and
    nothing around them."""
    dh, x, w, kept = grad_inputs(rows, dim, ff, t, keep)
    want = check_ff_grad(dh, x, w, kept, wt=DT[wt])
    want = [*want[:4], *want[4]]
    shapes = [(rows, ff)] * 3 + [(rows, dim)] + [(ff, dim)] * 2
    for off in range(1, 9):
        # another offset for every output, and for the inputs
        at = [Place(s, DT[wt if i > 3 else t], (off + 3 * i) % 8 + (i == 1))
              for i, s in enumerate(shapes)]
        dgate, dup, h, dx, dwg, dwu = (p.out for p in at)
        place = lambda v: moved(v, (off + 5) % 9)  # noqa: E731
        rra.gated_ff_grad(place(dh), place(x), place(w[0]), place(w[1]),
                          *(k if isinstance(k, rra.Saved) else place(k) for k in kept), dgate, dup,
                          dx=dx, dw_gate=dwg, dw_up=dwu, h=h)
        for p, v in zip(at, want):
            assert torch.equal(p.out, v)
            assert p.untouched()


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim,ff", [(3, 40, 136), (40, 72, 137), (70, 129, 264), (200, 51, 333)])
def test_ff_into_every_place(rows, dim, ff, t):
    """h, gate and up whole; then codes and exponents between guards of their own."""
    x, w = randn((rows, dim), 1, 1.0, t), weights(dim, ff, t)
    h0, kept0 = check_ff(x, *w, keep="full")
    for off in range(1, 9):
        at = [Place((rows, ff), DT[t], (off + 3 * i) % 9) for i in range(3)]
        rra.gated_ff(x, *w, *(p.out for p in at))
        for p, v in zip(at, (h0, *kept0)):
            assert torch.equal(p.out, v)
            assert p.untouched()
    nb = -(-ff // 128)
    _, saved0 = check_ff(x, *w, keep="bits8")
    for off in range(1, 9):
        exps = [Place((rows, nb), torch.int8, off + i, 77) for i in range(2)]
        codes = [Place((rows, nb * 128), torch.int8, -GUARD % 16, 77) for _ in range(2)]  # aligned
        h = Place((rows, ff), DT[t], 9 - off)
        rra.gated_ff(x, *w, h.out, *(rra.Saved(e.out, c.out, ff) for e, c in zip(exps, codes)))
        assert torch.equal(h.out, h0)
        for e, c, s in zip(exps, codes, saved0):
            assert torch.equal(e.out, s.exps) and torch.equal(c.out, s.codes)
        assert all(p.untouched() for p in [*exps, *codes, h])


@pytest.mark.parametrize("t,wt", [("f32", "f32"), ("f16", "f32"), ("bf16", "f32"),
                                  ("bf16", "bf16")])
@pytest.mark.parametrize("rows,dim,ff", [(300, 264, 520), (8192, 512, 768), (8192, 136, 40),
                                         (20_000, 1024, 2048)])
def test_ff_grad_weights_as_a_whole(rows, dim, ff, t, wt):
    """Far nearer as a whole than its worst element may be.  An instruction cuts the sum
    towards zero, by 0.75 * 2^-24 of it in the mean, which grows as the root of k: k / 32 such
    units of the result at most, below 16 * sqrt(k) of them up to k = 2^18; what is cut of the
    products goes both ways and stays below sqrt(k / 16) units."""
    dh, x, w, kept = grad_inputs(rows, dim, ff, t, "bits8")
    dgate, dup = torch.empty_like(dh), torch.empty_like(dh)
    dw = [torch.empty(ff, dim, dtype=DT[wt], device="cuda") for _ in range(2)]
    rra.gated_ff_grad(dh, x, *w, *kept, dgate, dup, dw_gate=dw[0], dw_up=dw[1])
    for got, d in zip(dw, (dgate, dup)):
        want = d.double().t() @ x.double()
        off = (got.double() - want).norm()
        assert off <= (UT[DT[wt]] + 16 * math.sqrt(rows + 8) * U) * want.norm() + \
            TINY[DT[wt]] * math.sqrt(want.numel())
