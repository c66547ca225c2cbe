"""The activations of the gated feed-forward block and their derivatives where
the activation's argument or the logistic function leaves fp32's range."""
import pytest
import torch

import ring_allreduce_compressed_gb300 as rra
from saved_util import act, saved_of, values
from test_gpu_operators import DT, UT

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
FAR = {"f32": (1e3, 1e9, 1e13, 1.2e13, 2e13, 1e20, 1e30), "bf16": (1e3, 1e9, 1e13, 2e13, 1e20, 1e30),
       "f16": (1e3, 2e4)}


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("keep", ["full", "bits8"])
@pytest.mark.parametrize("name", ACTS)
def test_slopes_far_out_are_0_or_1(name, keep, t):
    """A row for each magnitude, up to the largest finite one, its signs in turn: the slope is 0
    below zero and 1 above, the activation 0 and g, and nothing is NaN."""
    far = FAR[t] + (torch.finfo(DT[t]).max,)
    rows, ff, dim = len(far), 200, 40
    gate = torch.tensor(far, dtype=torch.float64, device="cuda")[:, None].repeat(1, ff)
    gate[:, 1::2] *= -1
    gate = gate.to(DT[t])
    up, dh = torch.ones_like(gate), torch.ones_like(gate)
    kept = [saved_of(v.double()) for v in (gate, up)] if keep == "bits8" else [gate, up]
    g = values(kept[0]) if keep == "bits8" else gate.double()
    x = torch.ones(rows, dim, dtype=DT[t], device="cuda")
    w = [torch.ones(ff, dim, dtype=DT[t], device="cuda") for _ in range(2)]
    dgate, dup, h = (torch.full_like(dh, 9.0) for _ in range(3))
    dw = [torch.full_like(v, 9.0) for v in w]
    rra.gated_ff_grad(dh, x, *w, *kept, dgate, dup, dw_gate=dw[0], dw_up=dw[1], h=h, act=name)
    assert torch.equal(dgate, (g > 0).to(DT[t]))
    for got in (dup, h):  # (what 8 bits stand for is a number of each type)
        assert torch.equal(got, g.clamp(min=0).to(DT[t]))
    # columns of negative gates alone: no gradient, and none of it NaN
    assert (dw[0][1::2] == 0).all() and (dw[1][1::2] == 0).all()
    assert (dw[0][::2] == rows).all()


# silu's argument, and sums of two numbers of 8 bits whose gelu_tanh has such an argument
EDGE = {"silu": [(-87.0, 0.0), (-87.5, 0.0), (-88.0, 0.0), (-88.5, 0.0)],
        "gelu_tanh": [(-9.75, 0.0), (-10.0, -0.015625), (-10.0, -0.03125), (-10.0, -0.046875)]}


@pytest.mark.parametrize("rows", [4, 300])
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_quotients_of_large_denominators(name, rows):
    """1 + e^-z between 2^126 and 2^128: the logistic function is below the normal numbers of
    fp32, and the activation is one of bf16 (some 2^-121).

    e^-z misses by 2 + 1.2 |z| units of its last place, 2^-23 each, z by 4 roundings, which count
    |z| times, the quotient by 2 units and by half of fp32's least number of 2^-128: in all
    less than (2 + 1.2 * 89) * 2^-23 + 4 * 89 * 2^-24 + 2^-20 < 2^-14 of the result."""
    pairs = EDGE[name]
    x = torch.tensor([[a, b, 1.0] for a, b in pairs], device="cuda").bfloat16()
    x = x.repeat(rows // len(pairs), 1)
    wg = torch.tensor([[1.0, 1.0, 0.0]] * 5, device="cuda").bfloat16()
    wu = torch.tensor([[0.0, 0.0, 1.0]] * 5, device="cuda").bfloat16()
    h = torch.empty(rows, 5, dtype=torch.bfloat16, device="cuda")
    rra.gated_ff(x, wg, wu, h, act=name)
    want = act(name, x.double() @ wg.double().t())[0]
    assert (want < -2.0 ** -125).all()
    assert ((h.double() - want).abs() <= (UT[torch.bfloat16] + 2.0 ** -14) * want.abs()).all()


def test_slopes_of_large_denominators():
    """The same for silu's derivative, from gates kept whole and in 8 bits."""
    gate = torch.tensor([[-87.0, -87.5, -88.0, -88.5]], device="cuda").bfloat16().repeat(3, 50)
    dh, up = torch.ones_like(gate), torch.ones_like(gate)
    x, w = torch.ones_like(gate[:, :8]), torch.ones(200, 8, device="cuda").bfloat16()
    for kept in ((gate, up), tuple(saved_of(v.double()) for v in (gate, up))):
        dgate, dup = torch.empty_like(dh), torch.empty_like(dh)
        rra.gated_ff_grad(dh, x, w, w, *kept, dgate, dup)
        g = values(kept[0]) if isinstance(kept[0], rra.Saved) else gate.double()
        a, slope, _ = act("silu", g)
        for got, want in ((dgate, slope), (dup, a)):
            err = (UT[torch.bfloat16] + 2.0 ** -14) * want.abs()
            assert ((got.double() - want).abs() <= err).all()
