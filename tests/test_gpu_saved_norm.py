"""Layer norm that keeps its input in 8 bits, its restoring and its gradient,
against plain formulas in 64 bits (tolerances as in test_gpu_operators.py); codes
and exponents bit for bit."""
import math

import pytest
import torch

import ring_allreduce_compressed_gb300 as rra
from saved_util import encode, saved_of, values
from test_gpu_operators import (DT, NORM_DIMS, PAIRS, U, chain, close, exact_norm_rows, gen, randn,
                                rounded)

pytestmark = pytest.mark.gpu


def check_save(x, gamma, beta, eps=1e-5, y=None, saved=None):
    dim = x.shape[-1]
    rows = x.numel() // dim
    want, mean, rstd, xh = exact_norm_rows(x, gamma, beta, eps)
    mag = x.double().abs().mean(-1, keepdim=True)
    codes = encode(x.double().reshape(rows, dim))
    y = torch.full_like(x, 9.0) if y is None else y
    saved = saved or rra.Saved.empty(rows, dim)
    saved.exps.fill_(77)
    saved.codes.fill_(77)
    m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    rra.layer_norm_save(x, gamma, beta, y, saved, m, r, eps=eps)
    k = chain(dim)
    dm = k * U * mag
    dr = rstd * ((k / 2 + 6) * U + (dm * rstd) ** 2)
    close(m.view_as(mean), mean, dm + 2.0 ** -149, "mean")
    close(r.view_as(rstd), rstd, dr, "rstd")
    g = gamma.double().abs() if gamma is not None else 1.0
    err = (xh.abs() * (dr / rstd + 4 * U) + rstd * dm * 2) * g + 2 * U * want.abs()
    close(y, want, rounded(want, y.dtype, err), "y")
    assert torch.equal(saved.exps, codes[0])
    assert torch.equal(saved.codes, codes[1])
    return saved, m, r


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("dim", NORM_DIMS + [127, 129, 256, 257, 1025, 32_768, 32_769])
def test_save(dim, t, w):
    x = randn((5, dim), 1, 1.5, t) + 0.25
    check_save(x, randn(dim, 2, 0.1, w) + 1, randn(dim, 3, 0.1, w))


@pytest.mark.parametrize("rows", [1, 2, 31, 1000, 4001])
@pytest.mark.parametrize("dim", [16, 48, 136, 768, 2056])
def test_save_rows(rows, dim):
    check_save(randn((rows, dim), 1, dtype="bf16"), randn(dim, 2), randn(dim, 3))


@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
@pytest.mark.parametrize("dim", [9, 64, 515, 1001, 2048])
def test_save_of_misaligned_buffers(offset, dim):
    for t in ("bf16", "f32"):
        x = randn((9, dim), 1, dtype=t, offset=offset)
        y = torch.full((offset + 9 * dim + 1,), 9.0, dtype=DT[t], device="cuda")
        check_save(x, randn(dim, 2, offset=offset), randn(dim, 3, offset=1),
                   y=y[offset:-1].view(9, dim))
        assert (y[:offset] == 9).all() and y[-1] == 9


@pytest.mark.parametrize("dim", [64, 1000, 5000, 40_000])
def test_save_in_place(dim):
    x, g, b = randn((37, dim), 1, dtype="f16"), randn(dim, 2), randn(dim, 3)
    y, s = torch.empty_like(x), [rra.Saved.empty(37, dim) for _ in range(2)]
    st = [torch.empty(37, device="cuda") for _ in range(4)]
    rra.layer_norm_save(x, g, b, y, s[0], *st[:2])
    z = x.clone()
    rra.layer_norm_save(z, g, b, z, s[1], *st[2:])
    assert torch.equal(y, z) and torch.equal(st[0], st[2]) and torch.equal(st[1], st[3])
    assert torch.equal(s[0].exps, s[1].exps) and torch.equal(s[0].codes, s[1].codes)


@pytest.mark.parametrize("dim", [5, 130, 3000])
def test_save_of_ends_of_the_range(dim):
    """Zeros, subnormals, the largest numbers, ties, values that round past 127."""
    rows = []
    base = randn((1, dim), 3)[0]
    for scale in (0.0, 2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 2.0 ** -122, 2.0 ** -119, 1e-20,
                  1.0, 1e20, 2.0 ** 120):
        rows.append(base * scale)
    top = torch.full((dim,), 3.4e38, device="cuda")
    top[::2] = -2.0 ** 127
    rows.append(top)
    ties = torch.arange(dim, device="cuda", dtype=torch.float32) % 128 + 0.5
    rows += [ties, -ties, 127.75 * torch.ones(dim, device="cuda")]
    x = torch.stack(rows)
    s, m, r = rra.Saved.empty(len(rows), dim), *(torch.empty(len(rows), device="cuda")
                                                 for _ in range(2))
    rra.layer_norm_save(x, None, None, torch.empty_like(x), s, m, r)
    e, c = encode(x.double())
    assert torch.equal(s.exps, e) and torch.equal(s.codes, c)
    back = torch.empty_like(x)
    rra.layer_norm_restore(s, back)
    assert torch.equal(back.double(), values(s))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim", [100, 300, 5000, 40_000])
def test_values_that_are_not_finite_spoil_their_block_alone(dim, bad):
    x = randn((3, dim), 1)
    x[1, dim - 1] = bad
    s, m, r = rra.Saved.empty(3, dim), *(torch.empty(3, device="cuda") for _ in range(2))
    y = torch.empty_like(x)
    rra.layer_norm_save(x, None, None, y, s, m, r)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[::2]).all()
    e, c = encode(x.double())
    assert torch.equal(s.exps, e) and torch.equal(s.codes, c)
    rra.layer_norm_restore(s, y)
    first = (dim - 1) // 128 * 128
    assert torch.isnan(y[1, first:]).all() and torch.isfinite(y[1, :first]).all()
    assert torch.isfinite(y[::2]).all()


def test_codes_are_the_codecs():
    """rra_bfp_encode writes the same bytes for rows of whole blocks, and
    rra_bfp_decode reads any rows."""
    x = randn((7, 384), 1, dtype="bf16")
    s, m, r = rra.Saved.empty(7, 384), *(torch.empty(7, device="cuda") for _ in range(2))
    rra.layer_norm_save(x, None, None, torch.empty_like(x), s, m, r)
    exps, mants = torch.empty(21, dtype=torch.int8, device="cuda"), \
        torch.empty(7 * 384, dtype=torch.int8, device="cuda")
    rra.bfp_encode(x, 8, exps, mants)
    assert torch.equal(s.exps.view(-1), exps) and torch.equal(s.codes.view(-1), mants)
    x = randn((5, 300), 2)
    s, m, r = rra.Saved.empty(5, 300), *(torch.empty(5, device="cuda") for _ in range(2))
    rra.layer_norm_save(x, None, None, torch.empty_like(x), s, m, r)
    out, seen = torch.empty(5 * 384, device="cuda"), torch.empty(5, 300, device="cuda")
    rra.bfp_decode(s.exps, s.codes, 5 * 384, 8, out)
    rra.layer_norm_restore(s, seen)
    assert torch.equal(out.view(5, 384)[:, :300], seen)
    assert (out.view(5, 384)[:, 300:] == 0).all()


# ---------------------------------------------------------------- restore

def check_restore(x, t, gamma=None, beta=None, mean=None, rstd=None, y=None):
    s = saved_of(x.double())
    v = values(s)
    m = mean.double()[:, None] if mean is not None else 0.0
    rs = rstd.double()[:, None] if rstd is not None else torch.ones_like(v[:, :1])
    g = gamma.double() if gamma is not None else torch.ones_like(v[0])
    b = beta.double() if beta is not None else 0.0
    xh = (v - m) * rs
    want = xh * g + b
    y = torch.full(x.shape, 9.0, dtype=DT[t], device="cuda") if y is None else y
    rra.layer_norm_restore(s, y, gamma, beta, mean, rstd)
    # v is exact; a difference, two products and a sum, one of them fused perhaps
    err = 4 * U * ((xh * g).abs() + want.abs())
    close(y, want, rounded(want, y.dtype, err), "y")


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("dim", NORM_DIMS + [127, 129, 257])
def test_restore(dim, t, w):
    x = randn((5, dim), 1, 1.5, t) + 0.25
    check_restore(x, t, randn(dim, 2, 0.1, w) + 1, randn(dim, 3, 0.1, w), randn(5, 4),
                  randn(5, 5).abs())


@pytest.mark.parametrize("rows", [1, 33, 1000, 6001])
@pytest.mark.parametrize("dim", [1, 24, 136, 1001, 2048])
def test_restore_rows(rows, dim):
    x = randn((rows, dim), 1)
    check_restore(x, "bf16", randn(dim, 2), None, randn(rows, 4), None)
    check_restore(x, "f32")
    check_restore(x, "f16", None, randn(dim, 2), None, randn(rows, 4))


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_restore_at_every_place(t):
    for dim in (9, 64, 515):
        for off in range(8):
            y = torch.full((off + 7 * dim + 1,), 9.0, dtype=DT[t], device="cuda")
            check_restore(randn((7, dim), 1), t, randn(dim, 2, offset=off), randn(dim, 3),
                          randn(7, 4), randn(7, 5), y=y[off:-1].view(7, dim))
            assert (y[:off] == 9).all() and y[-1] == 9


# ---------------------------------------------------------------- gradient

def check_saved_grad(dy, x, gamma, accumulate=False, wt=None, dx=None):
    dim = x.shape[-1]
    rows = x.numel() // dim
    xd = x.double().reshape(rows, dim)
    s = saved_of(xd)
    mean = xd.mean(1).float()
    rstd = (xd.var(1, correction=0) + 1e-5).rsqrt().float()
    rs, dyd = rstd.double()[:, None], dy.double().reshape(rows, dim)
    xh = (values(s) - mean.double()[:, None]) * rs
    w = dyd * (gamma.double() if gamma is not None else 1.0)
    a, b = w.mean(1, keepdim=True), (w * xh).mean(1, keepdim=True)
    want = rs * (w - a - xh * b)
    k = chain(dim)
    err = 2 * rs * (4 * U * (w.abs() + a.abs() + (xh * b).abs())
                    + k * U * w.abs().mean(1, keepdim=True)
                    + xh.abs() * (k + 4) * U * (w * xh).abs().mean(1, keepdim=True))
    wt = wt or (gamma.dtype if gamma is not None else x.dtype)
    dg, db = (randn(dim, s_, 0.1).to(wt) for s_ in (50, 51))
    want_g, want_b = (dyd * xh).sum(0), dyd.sum(0)
    err_g, err_b = ((rows + 8) * U * v.abs().sum(0) for v in (dyd * xh, dyd))
    if accumulate:
        want_g, want_b = want_g + dg.double(), want_b + db.double()
        err_g, err_b = err_g + U * want_g.abs(), err_b + U * want_b.abs()
    dx = torch.full_like(dy, 9.0) if dx is None else dx
    rra.layer_norm_saved_grad(dy, s, gamma, mean, rstd, dx, dg, db, accumulate=accumulate)
    close(dx.reshape(rows, dim), want, rounded(want, dx.dtype, err), "dx")
    close(dg, want_g, rounded(want_g, wt, err_g), "dgamma")
    close(db, want_b, rounded(want_b, wt, err_b), "dbeta")
    return s, mean, rstd, dg, db


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("dim", NORM_DIMS + [127, 129, 257, 12_289])
def test_saved_grad(dim, t, w):
    check_saved_grad(randn((9, dim), 4, dtype=t), randn((9, dim), 1, 1.5, t) + 0.25,
                     randn(dim, 2, 0.1, w) + 1)


@pytest.mark.parametrize("rows", [0, 1, 2, 31, 151, 153, 1000, 6001])
@pytest.mark.parametrize("dim", [1, 8, 48, 768, 1001])
@pytest.mark.parametrize("accumulate", [False, True])
def test_saved_grad_rows(rows, dim, accumulate):
    check_saved_grad(randn((rows, dim), 4, dtype="bf16"), randn((rows, dim), 1, dtype="bf16"),
                     randn(dim, 2), accumulate=accumulate)


@pytest.mark.parametrize("t,w", PAIRS)
@pytest.mark.parametrize("rows,dim", [(10_001, 1032), (5003, 4096), (2500, 6152), (1300, 16_384),
                                      (3001, 1001)])
def test_saved_grad_of_many_long_rows(rows, dim, t, w):
    x = randn((rows, dim), 1, 1.5, t) + 0.25
    check_saved_grad(randn((rows, dim), 4, dtype=t), x, randn(dim, 2, 0.1, w) + 1)
    check_save(x, randn(dim, 2, 0.1, w) + 1, randn(dim, 3, 0.1, w))


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_saved_grad_at_every_place(t):
    for dim in (9, 62, 64, 515, 1001):
        for off in range(8):
            for rows in (1, 7, 400):
                dy = randn((rows, dim), 4, 1.0, t, off)
                dx = torch.full((off + rows * dim + 1,), 9.0, dtype=DT[t], device="cuda")
                check_saved_grad(dy, randn((rows, dim), 1), randn(dim, 2, offset=off),
                                 dx=dx[off:-1].view(rows, dim))
                assert (dx[:off] == 9).all() and dx[-1] == 9
        check_saved_grad(randn((50, dim), 4, 1.0, t, 1), randn((50, dim), 1), randn(dim, 2))


@pytest.mark.parametrize("dim", [64, 2000, 2001, 40_000])
def test_saved_grad_in_place(dim):
    dy = randn((40, dim), 4)
    check_saved_grad(dy, randn((40, dim), 1), randn(dim, 2), dx=dy)


@pytest.mark.parametrize("dim", [500, 20_000])
def test_saved_grad_of_parts(dim):
    dy, x, g = randn((70, dim), 4), randn((70, dim), 1), randn(dim, 2)
    s, mean, rstd, dg, db = check_saved_grad(dy, x, g)
    dx = torch.empty_like(x)
    rra.layer_norm_saved_grad(dy, s, g, mean, rstd, dx, None, None)
    for k in range(3):
        outs = [torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)]
        asked = [o if i == k else None for i, o in enumerate(outs)]
        rra.layer_norm_saved_grad(dy, s, g, mean, rstd, *asked)
        assert torch.equal(outs[k], (dx, dg, db)[k])
    check_saved_grad(dy, x, None)


@pytest.mark.parametrize("rows,dim", [(5000, 1024), (3001, 1001)])
def test_saved_grad_gives_equal_bits(rows, dim):
    dy, x, g = randn((rows, dim), 4, dtype="bf16"), randn((rows, dim), 1, dtype="bf16"), \
        randn(dim, 2)
    first = None
    for _ in range(4):
        _, _, _, dg, db = check_saved_grad(dy, x, g)
        first = first or (dg, db)
        assert torch.equal(dg, first[0]) and torch.equal(db, first[1])


@pytest.mark.parametrize("dim", [6, 300])
def test_saved_grad_against_differences(dim):
    """Of an input that 8 bits hold exactly: directional derivatives of sum(y * dy)
    in x, gamma and beta by central differences in 64 bits."""
    x = torch.randint(-127, 128, (4, dim), generator=gen(1), device="cuda").float() / 64
    x[:, ::128] = 1.5  # every block's exponent is 0
    dy, g, b = randn((4, dim), 4), randn(dim, 2) + 1, randn(dim, 3)
    s, m, r = check_save(x, g, b)
    assert torch.equal(values(s), x.double())
    dx, dg, db = torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)
    rra.layer_norm_saved_grad(dy, s, g, m, r, dx, dg, db)

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


def test_saved_norm_beyond_32_bits():
    rows, dim = (1 << 19) + 1, 4096
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    x[-1] = randn(dim, 1, dtype="bf16")
    s = rra.Saved.empty(rows, dim)
    m, r = (torch.empty(rows, device="cuda") for _ in range(2))
    y = torch.empty_like(x)
    rra.layer_norm_save(x, None, None, y, s, m, r)
    want = exact_norm_rows(x[-1:], None, None, 1e-5)[0]
    close(y[-1:], want, rounded(want, y.dtype, (chain(dim) + 8) * U * (want.abs() + 1)))
    assert (y[:-1] == 0).all()
    e, c = encode(x[-1:].double())
    assert torch.equal(s.exps[-1:], e) and torch.equal(s.codes[-1:], c)
    assert (s.exps[:-1] == -126).all() and int(s.codes[:-1].count_nonzero()) == 0
    y.fill_(9)
    rra.layer_norm_restore(s, y)
    assert torch.equal(y[-1:].double(), values(rra.Saved(e, c, dim))) and (y[:-1] == 0).all()
    dg = torch.empty(dim, device="cuda")
    rra.layer_norm_saved_grad(x, s, dg.fill_(1.0), m, r, y, None, dg.clone())
    assert (y[:-1] == 0).all()


def test_saved_norm_on_a_stream_and_in_a_graph():
    x, g, b = randn((500, 1000), 1, dtype="bf16"), randn(1000, 2), randn(1000, 3)
    dy = randn((500, 1000), 4, dtype="bf16")
    s, m, r = rra.Saved.empty(500, 1000), *(torch.empty(500, device="cuda") for _ in range(2))
    outs = [torch.empty_like(x) for _ in range(3)] + [torch.empty_like(g) for _ in range(2)]

    def calls(**kw):
        rra.layer_norm_save(x, g, b, outs[0], s, m, r, **kw)
        rra.layer_norm_restore(s, outs[1], g, b, m, r, **kw)
        rra.layer_norm_saved_grad(dy, s, g, m, r, outs[2], outs[3], outs[4], **kw)
    calls()
    first = [o.clone() for o in outs + [s.exps, s.codes]]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls(stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        calls()
    for _ in range(3):
        for o in outs + [s.exps, s.codes]:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, f in zip(outs + [s.exps, s.codes], first):
            assert torch.equal(o, f)
