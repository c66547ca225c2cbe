"""What the header says of the training-step operators at the ends of their
contract: infinite limits, tokens outside the table, captures elsewhere, and
calls that begin while the kernels ahead of them still write."""
import ctypes
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


# ---------------------------------------------------------------- captures

def new_stream():
    """A stream that no other test has used, and the function that destroys it."""
    rt = torch.cuda.cudart()
    handle = ctypes.c_void_p()
    assert int(rt.cudaStreamCreate(ctypes.addressof(handle))) == 0
    st = torch.cuda.ExternalStream(handle.value)
    return st, lambda: rt.cudaStreamDestroy(handle.value)


def test_scratch_grows_while_another_stream_is_captured():
    """The capture goes on as if nothing had been."""
    d = torch.ones(20_000, 64, device="cuda")
    t = torch.arange(20_000, device="cuda") % 10
    dw, y = torch.empty(10, 64, device="cuda"), torch.zeros(4, device="cuda")
    want = torch.full((10, 64), 2000.0, device="cuda")
    rra.embedding_grad(d, t, dw)  # kernels are loaded
    dw.zero_()
    st, destroy = new_stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y.add_(1.0)
        rra.embedding_grad(d, t, dw, stream=st)  # the new stream's first call
        y.add_(1.0)
    st.synchronize()
    assert torch.equal(dw, want)
    graph.replay()
    torch.cuda.synchronize()
    assert (y == 2).all()
    destroy()


def test_sparse_codec_s_scratch_grows_while_another_stream_is_captured():
    x = randn(9_000_001, 3)
    x = torch.where(x > 1, x, torch.zeros_like(x))
    hdr, back = torch.empty(2, dtype=torch.int32, device="cuda"), torch.zeros_like(x)
    vals, idx = torch.empty_like(x), torch.empty(x.numel(), dtype=torch.int32, device="cuda")
    y = torch.zeros(4, device="cuda")
    rra.sparse_encode(x, 0.5, hdr, vals, idx)  # kernels are loaded
    rra.sparse_decode(hdr, vals, idx, x.numel(), back)
    nnz = int((x != 0).sum())
    st, destroy = new_stream()
    torch.cuda.synchronize()
    rra.sparse_encode(x[:5], 0.5, hdr, vals, idx, stream=st)
    rra.sparse_decode(hdr, vals, idx, 5, back, stream=st)
    back.zero_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y.add_(1.0)
        rra.sparse_encode(x, 0.5, hdr, vals, idx, stream=st)
        rra.sparse_decode(hdr, vals, idx, x.numel(), back, stream=st)
        y.add_(1.0)
    st.synchronize()
    assert hdr.tolist() == [1, nnz] and torch.equal(back, x)
    graph.replay()
    torch.cuda.synchronize()
    assert (y == 2).all()
    destroy()


def test_streams_that_come_and_go():
    """A stream may be destroyed while its last call runs; the next one, often
    of the same handle, has a scratch that the old call does not write."""
    problems = []
    for seed, (n, vocab, dim) in enumerate([(50_000, 100, 512), (3000, 2000, 64)]):
        t = torch.randint(0, vocab, (n,), generator=gen(seed), device="cuda")
        d = torch.randint(-8, 9, (n, dim), generator=gen(seed), device="cuda").float()
        problems.append((t, d, torch.zeros(vocab, dim, device="cuda").index_add_(0, t, d)))
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for t, d, want in problems:
            st, destroy = new_stream()
            got.append(torch.empty_like(want))
            torch.cuda.synchronize()
            rra.embedding_grad(d, t, got[-1], stream=st)
            destroy()
        torch.cuda.synchronize()
        for o, (_, _, want) in zip(got, problems):
            assert torch.equal(o, want)


# ---------------------------------------------------------------- early starts

@pytest.mark.parametrize("rows,dim", [(40, 1024), (2000, 1024), (300, 8192)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_behind_one_another_read_what_was_written_last(rows, dim, dtype):
    """Every result differs from what its buffer held and from the last turn's,
    so a value that is read too early shows.  Sums of whole numbers and factors
    that are powers of two: all of it is exact."""
    dt = DT[dtype]
    t = torch.randint(0, rows, (3 * rows,), generator=gen(1), device="cuda")
    count = torch.bincount(t, minlength=rows).double()[:, None]
    most = float(count.max())
    table = torch.zeros(rows, dim, dtype=dt, device="cuda")
    dw = torch.empty(rows, dim, device="cuda")
    x = torch.empty(3 * rows, dim, dtype=dt, device="cuda")
    y, clipped = torch.empty_like(x), torch.empty_like(dw)
    norm, norm2 = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    mean, rstd = torch.empty(3 * rows, device="cuda"), torch.empty(3 * rows, device="cuda")
    # +1 and -1 in turn: rows of mean 0 whose square is the turn's
    sign = torch.ones(dim, device="cuda")
    sign[1::2] = -1
    for k in range(1, 13):
        a = float(k % 7 + 1)
        m = most * a
        dw.fill_(-5.0)
        torch.mul(sign.to(dt), a, out=table[0])
        table.copy_(table[0].expand_as(table).clone())
        rra.embedding(table, t, x, scale=2.0)                       # 2 a sign
        rra.embedding_grad(x, t, dw, scale=0.5)                     # count a sign
        rra.grad_clip([dw], [clipped], m / 4, norm2, norm_type=math.inf, eps=0.0)
        rra.grad_norm([dw], norm, norm_type=math.inf)               # a max(count)
        rra.layer_norm(x, None, None, y, mean, rstd, eps=0.0)
        rra.grad_clip([dw], [dw], m / 2, norm2, norm_type=math.inf, eps=0.0)
        got = [v.clone() for v in (x, dw, clipped, norm, norm2, y, mean, rstd)]
        x.fill_(7.0)
        y.fill_(7.0)
        clipped.fill_(7.0)
        want_dw = count * a * sign.double()
        assert torch.equal(got[0].double(), 2 * a * sign.double().expand_as(x)), k
        assert torch.equal(got[1].double(), want_dw / 2), k
        assert torch.equal(got[2].double(), want_dw / 4), k
        assert float(got[3]) == m and float(got[4]) == m, k
        assert (got[6] == 0).all(), k
        # a square root and one product away from 1
        assert float((got[5].double() - sign.double()).abs().max()) <= (
            2.0 ** -20 if dtype == "f32" else 2.0 ** -8), k
        assert float((got[7].double() * 2 * a - 1).abs().max()) <= 2.0 ** -20, k
