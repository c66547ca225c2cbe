"""What the header says of the training-step operators at the ends of their
contract: infinite limits, tokens outside the table, captures elsewhere, and
calls that begin while the kernels ahead of them still write."""
import math

import pytest
import torch

import ring_allreduce_compressed_gb300 as rra

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, dtype="f32"):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(DT[dtype])


# ---------------------------------------------------------------- clipping

@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("n", [1000, 200_003])
@pytest.mark.parametrize("limit", [1.0, math.inf])
def test_grad_clip_factor_of_an_infinite_norm_is_zero(n, p, limit):
    """Whatever the limit is, an infinite one too."""
    g, norm = randn(n, 1), torch.empty(1, device="cuda")
    g[5] = math.inf
    out = torch.full_like(g, 9.0)
    rra.grad_clip([g], [out], limit, norm, norm_type=p)
    assert float(norm) == math.inf
    assert math.isnan(float(out[5]))  # 0 times infinity
    out[5] = 0
    assert (out == 0).all()


@pytest.mark.parametrize("n", [1000, 200_003])
def test_grad_clip_without_a_limit_changes_nothing(n):
    g, norm = randn(n, 1), torch.empty(1, device="cuda")
    out = torch.zeros_like(g)
    rra.grad_clip([g], [out], math.inf, norm)
    assert torch.equal(out, g)


# ---------------------------------------------------------------- lookup

@pytest.mark.parametrize("scale", [-2.0, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype,dim", [("f32", 24), ("f32", 7), ("f16", 64), ("bf16", 1024),
                                       ("bf16", 33)])
def test_embedding_of_tokens_outside_the_table_is_zero_for_every_scale(dtype, dim, scale):
    w = randn((10, dim), 1, dtype).abs() + 1
    t = torch.tensor([0, -1, 9, 10, 1 << 40, 3], device="cuda")
    out = torch.full((6, dim), 9.0, dtype=DT[dtype], device="cuda")
    rra.embedding(w, t, out, scale=scale)
    bits = out.view(torch.int32 if dtype == "f32" else torch.int16)
    for k, v in enumerate(t.tolist()):
        if 0 <= v < 10:
            want = (w[v].float() * scale).to(DT[dtype])
            assert torch.equal(out[k], want) or (torch.isnan(want).all()
                                                 and torch.isnan(out[k]).all())
        else:
            assert (bits[k] == 0).all()  # +0
