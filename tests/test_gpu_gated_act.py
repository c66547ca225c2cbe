"""The activations of the gated feed-forward block and their derivatives where
the activation's argument or the logistic function leaves fp32's range."""
import pytest
import torch

import ring_allreduce_compressed_gb300 as rra
from saved_util import saved_of, values
from test_gpu_operators import DT

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
