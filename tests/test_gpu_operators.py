"""The training-step operators against plain formulas in 64 bits.

Tolerances come from the roundings that the formulas need: u = 2^-24 for every
fp32 operation, over sums as long as a kernel's longest chain of additions can
be, and one rounding of the result to its type (2^-11 for fp16, 2^-8 for bf16,
2^-25 absolute below fp16's normal numbers)."""
import math

import pytest
import torch

import ring_allreduce_compressed_gb300 as rra

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
UT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
PAIRS = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, std=1.0, dtype="f32", offset=0):
    """Normal numbers; offset: elements before the tensor in its allocation."""
    shape = (shape,) if isinstance(shape, int) else tuple(shape)
    n = math.prod(shape)
    x = (torch.randn(offset + n, generator=gen(seed), device="cuda") * std).to(DT[dtype])
    return x[offset:].view(shape)


def close(got, want, tol, what=""):
    """|got - want| <= tol elementwise; want and tol in 64 bits."""
    g = got.double()
    assert torch.isfinite(g).all(), what
    over = (g - want).abs() - tol
    assert float(over.max()) <= 0 if g.numel() else True, \
        f"{what}: {int((over > 0).sum())} of {g.numel()} off, by up to {float(over.max()):.3g}"


def rounded(want, dtype, err):
    """Tolerance of a value with fp32 error `err` that is rounded to dtype once."""
    return err * (1 + UT[dtype]) + want.abs() * UT[dtype] + TINY[dtype]


# ---------------------------------------------------------------- gradient norm, clipping

CHAIN = 128  # more fp32 additions in a row than any accumulator makes for these sizes

LISTS = [
    [("f32", 1, 0)],
    [("f16", 7, 0)],
    [("f32", 4096, 0)],
    [("bf16", 8, 1), ("f32", 3, 1), ("f16", 9, 3)],
    [("f32", 0, 0), ("f32", 8192, 0), ("bf16", 0, 0), ("f16", 16384 + 3, 0)],
    [("bf16", 100_003, 5), ("f32", 8191, 2), ("f16", 1, 7), ("bf16", 16385, 0)],
    [("f32", 1_000_003, 3)],
    [("f16", 2_000_001, 1), ("bf16", 70_001, 0)],
]


def make_list(spec, std=1e-3):
    return [randn(n, 10 + k, std, t, off) for k, (t, n, off) in enumerate(spec)]


def exact_norm(grads, p):
    flat = torch.cat([g.double().reshape(-1) for g in grads])
    if p == 2:
        return float((flat * flat).sum().sqrt())
    return float(flat.abs().sum() if p == 1 else (flat.abs().max() if flat.numel() else 0))


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("spec", LISTS)
def test_grad_norm(spec, p):
    grads, norm = make_list(spec), torch.empty(1, device="cuda")
    rra.grad_norm(grads, norm, norm_type=p)
    want = exact_norm(grads, p)
    assert abs(float(norm) - want) <= (0 if p == math.inf else CHAIN * U) * want


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("place", ["apart", "shifted", "in place"])
@pytest.mark.parametrize("spec", LISTS)
def test_grad_clip(spec, p, place):
    grads, norm = make_list(spec), torch.empty(1, device="cuda")
    n = exact_norm(grads, p)
    limit = float(torch.tensor(0.3 * n))
    want = [g.double() * min(1.0, limit / (n + 1e-6)) for g in grads]
    if place == "in place":
        outs = grads
    else:
        more = 1 if place == "shifted" else 0
        outs = [torch.full((off + more + k,), 7.0, dtype=DT[t], device="cuda")[off + more:]
                for t, k, off in spec]
    rra.grad_clip(grads, outs, limit, norm, norm_type=p)
    assert abs(float(norm) - n) <= CHAIN * U * n
    for o, w in zip(outs, want):
        close(o, w, rounded(w, o.dtype, w.abs() * (CHAIN + 4) * U), place)


@pytest.mark.parametrize("in_place", [False, True])
def test_grad_clip_below_the_limit_changes_nothing(in_place):
    grads = make_list(LISTS[5])
    keep = [g.clone() for g in grads]
    outs = grads if in_place else [torch.zeros_like(g) for g in grads]
    norm = torch.empty(1, device="cuda")
    rra.grad_clip(grads, outs, 1e6, norm)
    for o, k in zip(outs, keep):
        assert torch.equal(o, k)


@pytest.mark.parametrize("scale", [1e-40, 1e-30, 1e-20, 1e20, 1e35])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_norm_keeps_the_whole_range(scale, dtype):
    g = (torch.randn(5003, generator=gen(3), device="cuda", dtype=torch.float64) * scale).to(
        DT[dtype])
    norm = torch.empty(1, device="cuda")
    rra.grad_norm([g], norm)
    want = exact_norm([g], 2)
    assert abs(float(norm) - want) <= CHAIN * U * want + 2.0 ** -149


def test_grad_norm_of_large_and_small_values_together():
    g = torch.full((4096,), 1e-25, device="cuda")
    g[100] = 3e30
    g[2000] = 4e30
    norm = torch.empty(1, device="cuda")
    rra.grad_norm([g], norm)
    assert abs(float(norm) / 5e30 - 1) <= CHAIN * U


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("at", [0, 4097, 9999])
def test_grad_norm_of_nan_and_infinity(p, at):
    norm = torch.empty(1, device="cuda")
    g = randn(10_000, 1)
    g[at] = -math.inf
    rra.grad_norm([randn(10, 2), g], norm, norm_type=p)
    assert float(norm) == math.inf
    g[at // 2] = math.nan
    rra.grad_norm([randn(10, 2), g], norm, norm_type=p)
    assert math.isnan(float(norm))
    out = torch.zeros_like(g)
    rra.grad_clip([g], [out], 1.0, norm, norm_type=p)
    assert torch.isnan(out).all()


def test_grad_clip_of_an_infinite_norm():
    g = randn(1000, 1)
    g[5] = math.inf
    out, norm = torch.empty_like(g), torch.empty(1, device="cuda")
    rra.grad_clip([g], [out], 1.0, norm)
    assert math.isnan(float(out[5]))
    out[5] = 0
    assert (out == 0).all()


def test_grad_clip_of_zeros_and_of_nothing():
    g, norm = torch.zeros(33, device="cuda"), torch.full((1,), 5.0, device="cuda")
    rra.grad_clip([g], [g], 0.0, norm, eps=0.0)
    assert float(norm) == 0 and (g == 0).all()
    norm.fill_(5.0)
    rra.grad_clip([], [], 1.0, norm)
    assert float(norm) == 0
    norm.fill_(5.0)
    rra.grad_norm([g[:0]], norm)
    assert float(norm) == 0
    x = randn(100, 4)
    rra.grad_clip([x], [x], 0.0, norm)
    assert (x == 0).all()


@pytest.mark.parametrize("count", [33, 511, 512, 513, 1300])
def test_grad_clip_of_many_tensors(count):
    sizes = [(k * 37) % 501 for k in range(count)]
    flat = randn(sum(sizes), 8, dtype="bf16")
    grads = list(torch.split(flat, sizes))
    norm, out = torch.empty(1, device="cuda"), torch.zeros_like(flat)
    n = exact_norm([flat], 2)
    rra.grad_clip(grads, list(torch.split(out, sizes)), n / 2, norm)
    want = flat.double() * ((n / 2) / (n + 1e-6))
    assert abs(float(norm) - n) <= CHAIN * U * n
    close(out, want, rounded(want, out.dtype, want.abs() * (CHAIN + 4) * U))


def test_grad_clip_on_a_stream_in_a_graph_and_twice_alike():
    grads = make_list(LISTS[7])
    outs = [torch.zeros_like(g) for g in grads]
    norm = torch.empty(1, device="cuda")
    rra.grad_clip(grads, outs, 0.5, norm)
    first, n0 = [o.clone() for o in outs], norm.clone()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    rra.grad_clip(grads, outs, 0.5, norm, stream=st)  # the stream's scratch
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        rra.grad_clip(grads, outs, 0.5, norm)
    for _ in range(3):
        for o in outs:
            o.zero_()
        norm.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, n0)
        for o, f in zip(outs, first):
            assert torch.equal(o, f)


def test_scratch_does_not_grow_during_a_capture():
    """A first call that needs scratch inside a capture is refused and leaves
    the capture usable."""
    st = torch.cuda.Stream()
    x = torch.zeros(1, 1 << 22, device="cuda")  # needs more than a new stream's scratch
    w, m, norm = x[0].clone(), torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        with pytest.raises(rra.RRAError) as e:
            rra.layer_norm_grad(x, x, None, m, m, None, None, w)
        assert e.value.code == rra.RRA_ERR_INVALID
        norm.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm) == 1.0


def test_grad_clip_beyond_32_bits():
    """A tensor of more than 2^31 elements whose last ones alone are not zero."""
    n = (1 << 31) + 5
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = torch.tensor([2.0, -1.0, 2.0])
    norm = torch.empty(1, device="cuda")
    rra.grad_clip([g], [g], 1.5, norm, eps=0.0)
    assert float(norm) == 3.0
    assert g[-4:].tolist() == [0.0, 1.0, -0.5, 1.0] and int((g != 0).sum()) == 3


# ---------------------------------------------------------------- embedding

DIMS = [1, 3, 8, 33, 64, 513, 1024, 2050, 4104]


def tokens(n, vocab, seed, index=torch.int64):
    u = torch.rand(n, generator=gen(seed), device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1)).floor() - 1).clamp(0, vocab - 1).to(index)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 700])
@pytest.mark.parametrize("dim", DIMS)
def test_embedding(dim, n, dtype):
    vocab = 301
    w = randn((vocab, dim), 5, 0.02, dtype)
    t = tokens(n, vocab, 6, torch.int32 if n == 5 else torch.int64)
    out = torch.full((n, dim), 9.0, dtype=DT[dtype], device="cuda")
    rra.embedding(w, t, out, scale=3.7)
    want = (w[t.long()].float() * torch.tensor(3.7, device="cuda")).to(DT[dtype])
    assert torch.equal(out, want)  # one product, one rounding


@pytest.mark.parametrize("woff,ooff", [(1, 0), (0, 1), (2, 4), (3, 3)])
def test_embedding_of_misaligned_buffers(woff, ooff):
    w = randn((50, 64), 5, dtype="bf16", offset=woff)
    t = tokens(77, 50, 6).view(7, 11)
    out = torch.zeros(ooff + 77 * 64, dtype=torch.bfloat16, device="cuda")[ooff:].view(7, 11, 64)
    rra.embedding(w, t, out, scale=0.5)
    assert torch.equal(out, w[t] * 0.5)


def test_embedding_of_tokens_outside_the_table():
    w = randn((10, 24), 1)
    t = torch.tensor([0, -1, 9, 10, 1 << 40, -(1 << 40), 3], device="cuda")
    out = torch.full((7, 24), 9.0, device="cuda")
    rra.embedding(w, t, out)
    for k, v in enumerate(t.tolist()):
        assert torch.equal(out[k], w[v] if 0 <= v < 10 else torch.zeros(24, device="cuda"))
    rra.embedding(w, t[:0], out[:0])  # no tokens


def test_embedding_beyond_32_bits():
    """A table of more than 2^31 elements."""
    vocab, dim = (1 << 21) + 3, 1024
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    w[-1] = randn(dim, 2, dtype="bf16")
    out = torch.zeros(3, dim, dtype=torch.bfloat16, device="cuda")
    rra.embedding(w, torch.tensor([vocab - 1, 0, vocab - 2], device="cuda"), out)
    assert torch.equal(out[0], w[-1]) and (out[1:] == 0).all()
    dw = torch.full((vocab, dim), 2.0, dtype=torch.bfloat16, device="cuda")
    rra.embedding_grad(w[-3:], torch.tensor([vocab - 1, vocab - 1, vocab - 2], device="cuda"), dw)
    assert (dw[:-2] == 0).all() and (dw[-1] == 0).all() and torch.equal(dw[-2], w[-1])


def test_embedding_grad_of_rows_beyond_32_bits():
    """More than 2^31 elements of dout, in many tokens."""
    n, dim = (1 << 21) + 3, 1024
    d = torch.zeros(n, dim, dtype=torch.bfloat16, device="cuda")
    d[-2:] = randn((2, dim), 2, dtype="bf16")
    t = torch.arange(n, device="cuda", dtype=torch.int32) % 1000
    t[-1] = t[0] = 1000
    dw = torch.full((1001, dim), 2.0, device="cuda")
    rra.embedding_grad(d, t, dw)
    assert torch.equal(dw[1000], d[-1].float())
    assert torch.equal(dw[(n - 2) % 1000], d[-2].float())
    assert int((dw != 0).any(1).sum()) == 2


def check_embedding_grad(dout, t, vocab, out, scale, padding=None, accumulate=False, offset=0):
    dim = dout.shape[-1]
    old = randn((vocab, dim), 77, 0.5, out, offset)
    dw = old.clone() if offset == 0 else old
    base = old.double()
    rra.embedding_grad(dout, t, dw, scale=scale, padding_idx=padding, accumulate=accumulate)
    v = t.reshape(-1).long()
    on = (v >= 0) & (v < vocab)
    if padding is not None:
        on &= v != padding
    v, d = v[on], dout.reshape(-1, dim)[on].double()
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, v, d) * scale
    mag = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, v, d.abs())
    terms = torch.bincount(v, minlength=vocab)[:, None]
    err = (terms + 2) * U * mag * abs(scale)
    if accumulate:
        want = want + base
        err = torch.where(terms > 0, err + U * want.abs(), 0.0)
        close(dw, want, torch.where(terms > 0, rounded(want, DT[out], err), 0.0))
    else:
        close(dw, want, torch.where(terms > 0, rounded(want, DT[out], err), 0.0))
    return dw


@pytest.mark.parametrize("din,dout", PAIRS)
@pytest.mark.parametrize("dim", DIMS)
def test_embedding_grad(dim, din, dout):
    check_embedding_grad(randn((700, dim), 5, dtype=din), tokens(700, 301, 6), 301, dout, 3.7)


@pytest.mark.parametrize("n", [0, 1, 2, 31, 33, 1023, 1025, 4095, 4096, 4097, 8193, 131_072,
                               131_073, 200_000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_grad_lengths(n, accumulate):
    t = tokens(n, 5000, n, torch.int32)
    check_embedding_grad(randn((n, 40), 5, dtype="bf16"), t, 5000, "f32", 0.5, padding=0,
                         accumulate=accumulate)


@pytest.mark.parametrize("n", [1, 33, 70, 200, 1000])
@pytest.mark.parametrize("dim", [1, 3, 6, 513, 1030])
def test_embedding_grad_odd_widths(n, dim):
    check_embedding_grad(randn((n, dim), 5), tokens(n, 50, 3), 50, "f32", 1.0)
    check_embedding_grad(randn((n, dim), 5, dtype="bf16"), tokens(n, 50, 3), 50, "bf16", 1.0)


@pytest.mark.parametrize("vocab", [1, 2, 255, 256, 257, 65_535, 65_536, 70_000, 1 << 18,
                                   (1 << 24) + 5])
def test_embedding_grad_vocabularies(vocab):
    n = 3000
    t = torch.randint(0, vocab, (n,), generator=gen(1), device="cuda")
    t[5] = vocab - 1
    t[6] = 0
    check_embedding_grad(randn((n, 8), 5), t, vocab, "f32", 1.0)


@pytest.mark.parametrize("kind", ["same", "distinct", "falling", "two", "none"])
@pytest.mark.parametrize("n", [700, 20_000])
@pytest.mark.parametrize("dim", [40, 520])
def test_embedding_grad_orders(kind, n, dim):
    k = torch.arange(n, device="cuda")
    t = {"same": k * 0 + 17, "distinct": k, "falling": n - 1 - k, "two": (k % 2) * (n - 1),
         "none": k * 0 - 1}[kind]
    check_embedding_grad(randn((n, dim), 5, dtype="f16"), t, n, "f16", 0.25)
    check_embedding_grad(randn((n, dim), 5, dtype="f16"), t, n, "f32", 0.25, padding=17,
                         accumulate=True)


def test_embedding_grad_of_tokens_outside_the_table():
    t = torch.tensor([0, -1, 9, 10, 1 << 40, -(1 << 40), 3, 3, 1 << 32], device="cuda")
    check_embedding_grad(randn((9, 24), 5), t, 10, "f32", 1.0)
    check_embedding_grad(randn((9, 24), 5), t, 10, "f32", 1.0, padding=3)


@pytest.mark.parametrize("offset", [1, 2, 4])
def test_embedding_grad_of_misaligned_buffers(offset):
    t = tokens(600, 90, 3).view(20, 30)
    check_embedding_grad(randn((20, 30, 64), 5, dtype="bf16", offset=offset), t, 90, "bf16", 2.0)
    check_embedding_grad(randn((20, 30, 64), 5, dtype="bf16"), t, 90, "bf16", 2.0, offset=offset)


def test_embedding_grad_gives_equal_bits():
    t = tokens(30_000, 2000, 3)
    d = randn((30_000, 256), 5)
    a, b = torch.empty(2000, 256, device="cuda"), torch.empty(2000, 256, device="cuda")
    rra.embedding_grad(d, t, a)
    for _ in range(3):
        b.fill_(9)
        rra.embedding_grad(d, t, b)
        assert torch.equal(a, b)


def test_embedding_grad_against_differences():
    """The loss sum(out * c) is linear in the table: its difference quotient is
    exact up to rounding."""
    w = torch.randn(20, 6, generator=gen(1), device="cuda", dtype=torch.float64)
    t, c = tokens(50, 20, 2), randn((50, 6), 3)
    dw = torch.empty(20, 6, device="cuda")
    rra.embedding_grad(c, t, dw, scale=1.5)
    v = torch.randn(20, 6, generator=gen(4), device="cuda", dtype=torch.float64)

    def loss(a):
        return float((1.5 * a[t] * c.double()).sum())
    slope = (loss(w + 1e-3 * v) - loss(w - 1e-3 * v)) / 2e-3
    assert abs(slope - float((dw.double() * v).sum())) <= 64 * U * float(
        (1.5 * v[t] * c.double()).abs().sum())


# ---------------------------------------------------------------- layer norm

NORM_DIMS = [1, 2, 7, 32, 100, 128, 255, 1000, 1024, 2048, 4096, 5001, 8192, 12_288, 16_384,
             20_000, 40_003]


def chain(dim):
    """Most fp32 additions in a row of a kernel's sum over a row."""
    return 40 + dim / 128


def exact_norm_rows(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    var = (x - mean).square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    xh = (x - mean) * rstd
    g = gamma.double() if gamma is not None else 1.0
    b = beta.double() if beta is not None else 0.0
    return xh * g + b, mean, rstd, xh


def check_layer_norm(x, gamma, beta, eps=1e-5, y=None):
    dim = x.shape[-1]
    rows = x.numel() // dim
    want, mean, rstd, xh = exact_norm_rows(x, gamma, beta, eps)
    mag = x.double().abs().mean(-1, keepdim=True)
    y = torch.full_like(x, 9.0) if y is None else y
    m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    rra.layer_norm(x, gamma, beta, y, m, r, eps=eps)
    k = chain(dim)
    dm = k * U * mag                       # of the mean
    dr = rstd * ((k / 2 + 6) * U + (dm * rstd) ** 2)
    close(m.view_as(mean), mean, dm + 2.0 ** -149, "mean")
    close(r.view_as(rstd), rstd, dr, "rstd")
    g = gamma.double().abs() if gamma is not None else 1.0
    err = (xh.abs() * (dr / rstd + 4 * U) + rstd * dm * 2) * g + 2 * U * want.abs()
    close(y, want, rounded(want, y.dtype, err), "y")
    return m, r


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("dim", NORM_DIMS)
def test_layer_norm(dim, t, w):
    x = randn((5, dim), 1, 1.5, t) + 0.25
    check_layer_norm(x, randn(dim, 2, 0.1, w) + 1, randn(dim, 3, 0.1, w))


@pytest.mark.parametrize("rows", [1, 2, 31, 1000, 4001])
@pytest.mark.parametrize("dim", [48, 768])
def test_layer_norm_rows(rows, dim):
    check_layer_norm(randn((rows, dim), 1, dtype="bf16"), randn(dim, 2), randn(dim, 3))


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("rows,dim", [(10_001, 1032), (5003, 4096), (2500, 6152), (1300, 16_384)])
def test_layer_norm_of_many_long_rows(rows, dim, t, w):
    check_layer_norm(randn((rows, dim), 1, 1.5, t) + 0.25, randn(dim, 2, 0.1, w) + 1,
                     randn(dim, 3, 0.1, w))
    check_layer_norm_grad(randn((rows, dim), 4, dtype=t), randn((rows, dim), 1, 1.5, t) + 0.25,
                          randn(dim, 2, 0.1, w) + 1)
    x = randn((rows, dim), 1, 1.5, t)
    y = torch.empty_like(x)
    rra.layer_norm(x, None, None, y)
    rra.layer_norm(x, None, None, x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("gamma,beta", [(False, False), (True, False), (False, True)])
def test_layer_norm_without_weights(gamma, beta):
    check_layer_norm(randn((3, 4, 260), 1), randn(260, 2) if gamma else None,
                     randn(260, 3) if beta else None)


@pytest.mark.parametrize("dim", [64, 1000, 5000, 40_000])
def test_layer_norm_in_place_and_without_statistics(dim):
    x, g, b = randn((37, dim), 1, dtype="f16"), randn(dim, 2), randn(dim, 3)
    y = torch.empty_like(x)
    rra.layer_norm(x, g, b, y)
    z = x.clone()
    rra.layer_norm(z, g, b, z)
    assert torch.equal(y, z)
    check_layer_norm(x, g, b)


@pytest.mark.parametrize("dim", [8, 1024, 3001, 30_000])
def test_layer_norm_of_constant_rows_and_far_means(dim):
    """Rows without variance, and rows whose mean is far above their spread."""
    x = torch.full((3, dim), 3.0, device="cuda")
    y, m, r = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    rra.layer_norm(x, None, None, y, m, r, eps=1e-5)
    assert (m == 3).all() and (y == 0).all()
    close(r, torch.full((3,), 1e-5 ** -0.5, dtype=torch.float64, device="cuda"), 4e-7 * 320)
    check_layer_norm(randn((4, dim), 1) + 1000.0, None, None)


@pytest.mark.parametrize("dim", [100, 5000, 40_000])
def test_layer_norm_carries_nan_in_its_row_alone(dim):
    x = randn((3, dim), 1)
    x[1, 7] = math.nan
    y = torch.empty_like(x)
    rra.layer_norm(x, None, None, y)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all()


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("dim", [64, 2048])
def test_layer_norm_of_misaligned_buffers(offset, dim):
    x = randn((9, dim), 1, dtype="bf16", offset=offset)
    y = torch.empty(offset + 9 * dim, dtype=torch.bfloat16, device="cuda")[offset:].view(9, dim)
    g, b = randn(dim, 2, offset=offset), randn(dim, 3, offset=1)
    check_layer_norm(x, g, b, y=y)
    check_layer_norm_grad(randn((9, dim), 4, dtype="bf16"), x, g)
    check_layer_norm_grad(x, randn((9, dim), 4, dtype="bf16"), g)


def test_layer_norm_grad_of_rows_at_every_phase():
    """Rows of every length modulo 16 bytes, buffers that begin at every place
    between two 16-byte boundaries, equal and different ones."""
    for t in ("bf16", "f32"):
        for dim in (9, 62, 63, 515, 1001):
            for off in range(0, 8 if t == "bf16" else 4):
                for rows in (1, 7, 400):
                    x, dy = (randn((rows, dim), s, 1.0, t, off) for s in (1, 4))
                    dx = torch.full((off + rows * dim + 1,), 9.0, dtype=DT[t],
                                    device="cuda")
                    check_layer_norm_grad(dy, x, randn(dim, 2),
                                          dx=dx[off:off + rows * dim].view(rows, dim))
                    assert (dx[:off] == 9).all() and dx[-1] == 9
            check_layer_norm_grad(randn((50, dim), 4, 1.0, t, 1), randn((50, dim), 1, 1.0, t),
                                  randn(dim, 2))


def check_layer_norm_grad(dy, x, gamma, eps=1e-5, accumulate=False, wt=None, dx=None):
    dim = x.shape[-1]
    rows = x.numel() // dim
    xd = x.double().reshape(rows, dim)
    mean = xd.mean(1).float()
    rstd = (xd.var(1, unbiased=False) + eps).rsqrt().float()
    rs, dyd = rstd.double()[:, None], dy.double().reshape(rows, dim)
    xh = (xd - mean.double()[:, None]) * rs
    w = dyd * (gamma.double() if gamma is not None else 1.0)
    a, b = w.mean(1, keepdim=True), (w * xh).mean(1, keepdim=True)
    want = rs * (w - a - xh * b)
    k = chain(dim)
    err = 2 * rs * (4 * U * (w.abs() + a.abs() + (xh * b).abs())
                    + k * U * w.abs().mean(1, keepdim=True)
                    + xh.abs() * (k + 4) * U * (w * xh).abs().mean(1, keepdim=True))
    wt = wt or (gamma.dtype if gamma is not None else x.dtype)
    dg, db = (randn(dim, s, 0.1).to(wt) for s in (50, 51))
    want_g, want_b = (dyd * xh).sum(0), dyd.sum(0)
    err_g, err_b = ((rows + 8) * U * v.abs().sum(0) for v in (dyd * xh, dyd))
    if accumulate:
        want_g, want_b = want_g + dg.double(), want_b + db.double()
        err_g, err_b = err_g + U * want_g.abs(), err_b + U * want_b.abs()
    dx = torch.full_like(x, 9.0) if dx is None else dx
    rra.layer_norm_grad(dy, x, gamma, mean, rstd, dx, dg, db, accumulate=accumulate)
    close(dx.reshape(rows, dim), want, rounded(want, dx.dtype, err), "dx")
    close(dg, want_g, rounded(want_g, wt, err_g), "dgamma")
    close(db, want_b, rounded(want_b, wt, err_b), "dbeta")
    return mean, rstd, dg, db


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("dim", NORM_DIMS)
def test_layer_norm_grad(dim, t, w):
    check_layer_norm_grad(randn((9, dim), 4, dtype=t), randn((9, dim), 1, 1.5, t) + 0.25,
                          randn(dim, 2, 0.1, w) + 1)


@pytest.mark.parametrize("rows", [0, 1, 2, 31, 151, 153, 1000, 6001])
@pytest.mark.parametrize("dim", [8, 48, 768, 1001])
@pytest.mark.parametrize("accumulate", [False, True])
def test_layer_norm_grad_rows(rows, dim, accumulate):
    check_layer_norm_grad(randn((rows, dim), 4, dtype="bf16"), randn((rows, dim), 1, dtype="bf16"),
                          randn(dim, 2), accumulate=accumulate)


@pytest.mark.parametrize("over", ["dy", "x"])
@pytest.mark.parametrize("dim", [64, 2000, 40_000])
def test_layer_norm_grad_in_place(over, dim):
    dy, x, g = randn((40, dim), 4), randn((40, dim), 1), randn(dim, 2)
    check_layer_norm_grad(dy.clone(), x.clone(), g)
    check_layer_norm_grad(dy, x, g, dx=dy if over == "dy" else x)


def test_layer_norm_grad_of_parts():
    """Each output alone is what it is with the others."""
    dy, x, g = randn((70, 500), 4), randn((70, 500), 1), randn(500, 2)
    mean, rstd, dg, db = check_layer_norm_grad(dy, x, g)
    dx = torch.empty_like(x)
    rra.layer_norm_grad(dy, x, g, mean, rstd, dx, None, None)
    for k in range(3):
        outs = [torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)]
        asked = [o if i == k else None for i, o in enumerate(outs)]
        rra.layer_norm_grad(dy, x, g, mean, rstd, *asked)
        assert torch.equal(outs[k], (dx, dg, db)[k])
    check_layer_norm_grad(dy, x, None)


def test_layer_norm_grad_gives_equal_bits():
    dy, x, g = randn((5000, 1024), 4, dtype="bf16"), randn((5000, 1024), 1, dtype="bf16"), \
        randn(1024, 2)
    first = None
    for _ in range(4):
        _, _, dg, db = check_layer_norm_grad(dy, x, g)
        first = first or (dg, db)
        assert torch.equal(dg, first[0]) and torch.equal(db, first[1])


@pytest.mark.parametrize("dim", [6, 300])
def test_layer_norm_grad_against_differences(dim):
    """Directional derivatives of sum(y * dy) in x, gamma and beta by central
    differences in 64 bits."""
    x, dy = randn((4, dim), 1), randn((4, dim), 4)
    g, b = randn(dim, 2) + 1, randn(dim, 3)
    m, r = check_layer_norm(x, g, b)
    dx, dg, db = torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)
    rra.layer_norm_grad(dy, x, g, m, r, dx, dg, db)

    def loss(x, g, b):
        return (exact_norm_rows(x, g, b, 1e-5)[0] * dy.double()).sum()
    args = [x.double(), g.double(), b.double()]
    for k, grad in enumerate((dx, dg, db)):
        v = torch.randn(args[k].shape, generator=gen(9), device="cuda", dtype=torch.float64)
        up, down = list(args), list(args)
        h = 1e-5
        up[k], down[k] = args[k] + h * v, args[k] - h * v
        slope = float((loss(*up) - loss(*down)) / (2 * h))
        got = float((grad.double() * v).sum())
        # h^2 truncation is below 1e-8; the kernel's sums have (dim + 40) roundings
        assert abs(slope - got) <= (dim + 40) * U * float((grad.double() * v).abs().sum()) + 1e-5


def test_layer_norm_beyond_32_bits():
    rows, dim = (1 << 19) + 1, 4096
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    x[-1] = randn(dim, 1, dtype="bf16")
    y, m, r = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows,
                                                                               device="cuda")
    rra.layer_norm(x, None, None, y, m, r)
    want = exact_norm_rows(x[-1:], None, None, 1e-5)[0]
    close(y[-1:], want, rounded(want, y.dtype, (chain(dim) + 8) * U * (want.abs() + 1)))
    assert (y[:-1] == 0).all()
    dg = torch.empty(dim, dtype=torch.bfloat16, device="cuda")
    dx = y
    rra.layer_norm_grad(x, x, None, m, r, dx, dg, None)
    xh, d = exact_norm_rows(x[-1:], None, None, 1e-5)[3], x[-1:].double()
    g = (d * xh)[0]
    close(dg, g, rounded(g, dg.dtype, (chain(dim) + 16) * U * (g.abs() + 1)))


# ---------------------------------------------------------------- streams, refusals

def test_operators_on_streams_of_their_own():
    """Calls on two streams at once keep their scratch apart."""
    t, d = tokens(20_000, 3000, 1), randn((20_000, 128), 2)
    want = torch.empty(3000, 128, device="cuda")
    rra.embedding_grad(d, t, want)
    outs = [torch.empty_like(want) for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for k, o in enumerate(outs):
        rra.embedding_grad(d, t, o, stream=streams[k % 2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_operators_in_a_graph():
    """Captured calls, replayed on new inputs, give the eager calls' bits."""
    t, d = tokens(9000, 700, 1), randn((9000, 256), 2, dtype="bf16")
    x, g = randn((500, 768), 3), randn(768, 4)
    dw = torch.empty(700, 256, device="cuda")
    y, m, r = torch.empty_like(x), torch.empty(500, device="cuda"), torch.empty(500, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)
    out, norm = torch.empty_like(dw), torch.empty(1, device="cuda")
    results = (dw, y, m, r, dx, dg, db, out, norm)

    def step():
        rra.embedding_grad(d, t, dw)
        rra.layer_norm(x, g, None, y, m, r)
        rra.layer_norm_grad(y, x, g, m, r, dx, dg, db)
        rra.grad_clip([dw, dg, db], [out, dg, db], 1.0, norm)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()  # the stream's scratch
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for seed in (5, 6):
        t.copy_(tokens(9000, 700, seed))
        x.copy_(randn((500, 768), seed))
        step()
        want = [v.clone() for v in results]
        for v in results:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for v, w in zip(results, want):
            assert torch.equal(v, w)


def test_operators_in_a_graph_of_two_streams():
    """Captured behind copies, a fork and a join, calls wait for what they read."""
    src, x = randn((64, 512), 3), torch.empty(64, 512, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    t, dw = tokens(3000, 64, 1), torch.empty(64, 512, device="cuda")
    d, norm = randn((3000, 512), 2), torch.empty(1, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (main, side):  # the streams' scratch
        rra.embedding_grad(d, t, dw, stream=st)
        rra.grad_norm([dw], norm, stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        x.copy_(src)
        dw.zero_()
        side.wait_stream(main)
        rra.embedding_grad(d, t, dw, stream=side)
        rra.layer_norm(x, None, None, y)
        x.fill_(0.0)  # y has been read from x
        main.wait_stream(side)
        rra.grad_norm([y, dw], norm)
        rra.embedding(dw, t[:64], z)
    for seed in (7, 8):
        src.copy_(randn((64, 512), seed))
        want_y, want_dw = torch.empty_like(y), torch.empty_like(dw)
        rra.layer_norm(src, None, None, want_y)
        rra.embedding_grad(d, t, want_dw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(dw, want_dw)
        assert torch.equal(z, dw[t[:64]])
        n = exact_norm([y, dw], 2)
        assert abs(float(norm) - n) <= CHAIN * U * n


def test_operators_right_behind_other_kernels():
    """A call that starts early still reads what is written just before it."""
    x, w = torch.empty(2000, 1024, device="cuda"), torch.empty(2000, 1024, device="cuda")
    y, out, norm = torch.empty_like(x), torch.empty_like(x), torch.empty(1, device="cuda")
    t = torch.arange(2000, device="cuda").flip(0).contiguous()
    for k in range(20):
        w.fill_(float(k))
        rra.embedding(w, t, x)
        rra.embedding_grad(x, t, w)
        rra.grad_clip([w], [w], 1e30, norm)
        rra.embedding(w, t, out)
        rra.layer_norm(out, None, None, y)
        assert torch.equal(out, torch.full_like(out, float(k)))
        assert (y == 0).all()


def test_refusals_of_the_binding():
    x, t = randn((4, 8), 1), torch.zeros(4, dtype=torch.int64, device="cuda")
    norm = torch.empty(1, device="cuda")
    with pytest.raises(ValueError):
        rra.grad_norm([x.t()], norm)
    with pytest.raises(TypeError):
        rra.grad_norm([x.double()], norm)
    with pytest.raises(TypeError):
        rra.grad_norm([x], norm.double())
    with pytest.raises(ValueError):
        rra.grad_clip([x], [], 1.0, norm)
    with pytest.raises(ValueError):
        rra.grad_clip([x], [x[:2]], 1.0, norm)
    with pytest.raises(TypeError):
        rra.grad_clip([x], [x.half()], 1.0, norm)
    with pytest.raises(rra.RRAError):
        rra.grad_clip([x], [x], -1.0, norm)
    with pytest.raises(TypeError):
        rra.embedding(x, t.float(), torch.empty(4, 8, device="cuda"))
    with pytest.raises(ValueError):
        rra.embedding(x, t, torch.empty(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        rra.embedding_grad(x[:3], t, x.clone())
    with pytest.raises(rra.RRAError):
        rra.embedding_grad(x, t, x.half())
    with pytest.raises(ValueError):
        rra.layer_norm(x, x[0, :7], None, x)
    with pytest.raises(rra.RRAError):
        rra.layer_norm(x, None, None, x, eps=-1.0)
    with pytest.raises(rra.RRAError):
        rra.layer_norm_grad(x, x, None, norm.expand(4).contiguous(), norm.expand(4).contiguous(),
                            None, None, None)
