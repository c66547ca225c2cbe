"""The gated feed-forward block and its gradient against plain formulas in 64
bits.

Tolerances: a product over k terms is within k (and 8 for how the pieces are joined)
units U = 2^-24 of the sum of magnitudes, twice that where a step cuts instead of
rounding; the activations' bounds stand in saved_util.py; a result is rounded to its
type once.  What is rounded before it is multiplied again (dgate and dup) is taken as
the call returned it."""
import math

import pytest
import torch

import ring_allreduce_compressed_gb300 as rra
from saved_util import act, act_errors, power, saved_of, values
from test_gpu_operators import DT, TINY, U, UT, close, gen, randn, rounded

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
# rows, dim, ff
SIZES = [(1, 1, 1), (1, 8, 8), (3, 5, 7), (33, 64, 129), (128, 128, 256), (257, 96, 640),
         (64, 1000, 72), (5, 2048, 1024), (130, 4096, 264), (1000, 256, 1032), (300, 513, 1001),
         (16, 72, 4000), (17, 520, 128), (255, 64, 127), (513, 40, 392)]


def products(k, size):
    """Error of sums of k products whose magnitudes add up to size."""
    return 2 * (k + 8) * U * size


def check_kept(got, want, err):
    """gate or up as it was kept."""
    if isinstance(got, rra.Saved):
        v = values(got)
        step = power(got.exps.long() - 6).repeat_interleave(128, 1)[:, :got.dim]
        m = (v / step).abs()
        # half a step, or a whole one where 127.5 to 128 went to 127
        assert ((v - want).abs() <= step * torch.where(m == 127, 1.0, 0.5) + err).all()
        rows, nb = got.exps.shape
        codes = got.codes.view(rows, nb, 128)
        top = codes.int().abs().amax(2)
        nil = torch.nn.functional.pad(want.abs(), (0, -got.dim % 128)).view(rows, nb, 128).amax(2) \
            < 2.0 ** -120
        assert (nil | (top >= 63)).all()  # no exponent above the block's
        assert (got.codes[:, got.dim:] == 0).all()
    else:
        close(got, want, rounded(want, got.dtype, err), "kept")


def check_ff(x, wg, wu, name="silu", keep="none", h=None):
    dim, ff = x.shape[-1], wg.shape[0]
    rows = x.numel() // dim
    xd, gd, ud = x.double().reshape(rows, dim), wg.double(), wu.double()
    g, u = xd @ gd.t(), xd @ ud.t()
    eg, eu = (products(dim, xd.abs() @ w.abs().t()) for w in (gd, ud))
    a, _, _ = act(name, g)
    # the activations' slopes are below 1.13
    ea = 1.13 * eg + act_errors(name, g)[0] * (1 + 1e-3)
    want = a * u
    err = ea * (u.abs() + eu) + a.abs() * eu + 2 * U * want.abs()
    h = torch.full(x.shape[:-1] + (ff,), 9.0, dtype=x.dtype, device="cuda") if h is None else h
    kept = [None, None]
    if keep == "full":
        kept = [torch.full_like(h, 9.0) for _ in range(2)]
    elif keep == "bits8":
        kept = [rra.Saved.empty(rows, ff) for _ in range(2)]
        for k in kept:
            k.exps.fill_(77)
            k.codes.fill_(77)
    rra.gated_ff(x, wg, wu, h, *kept, act=name)
    close(h.view(rows, ff), want, rounded(want, h.dtype, err), "h")
    # as a whole far nearer: errors of sums do not all point one way
    off = (h.double().view(rows, ff) - want).norm()
    assert off <= (UT[h.dtype] + 16 * math.sqrt(dim + 8) * U) * (want.norm() + g.norm()) + \
        TINY[h.dtype] * math.sqrt(want.numel())
    for k, w, e in zip(kept, (g, u), (eg, eu)):
        if k is not None:
            check_kept(k if keep == "bits8" else k.view(rows, ff), w, e)
    return h, kept


def weights(dim, ff, t, offset=0):
    return [randn((ff, dim), s, 1 / math.sqrt(dim), t, offset) for s in (2, 3)]


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("keep", ["none", "full", "bits8"])
@pytest.mark.parametrize("rows,dim,ff", SIZES)
def test_ff(rows, dim, ff, keep, t):
    check_ff(randn((rows, dim), 1, 1.0, t), *weights(dim, ff, t), keep=keep,
             name=ACTS[(rows + ff) % 4])


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", ACTS)
def test_ff_activations(name, t):
    """Far from zero, too."""
    x = randn((40, 64), 1, 1.0, t)
    x[::4] *= 30
    check_ff(x, *weights(64, 200, t), name=name, keep="full")


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65,
                                  96, 127, 128, 129, 192, 256, 257])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_ff_of_few_rows(rows, t):
    check_ff(randn((rows, 1024), 1, 1.0, t), *weights(1024, 1152, t), keep="full")
    check_ff(randn((rows, 264), 1, 1.0, t), *weights(264, 1000, t), name="gelu", keep="bits8")


@pytest.mark.parametrize("rows,dim,ff", [(1, 4096, 16_384), (48, 2048, 8192), (1024, 1024, 4096),
                                         (2000, 2048, 5000), (700, 4104, 2056)])
def test_ff_of_large_sizes(rows, dim, ff):
    check_ff(randn((rows, dim), 1, 1.0, "bf16"), *weights(dim, ff, "bf16"),
             keep="bits8" if rows > 50 else "none")


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,ff", [(20, 64, 136), (200, 72, 300)])
def test_ff_at_every_place(rows, dim, ff, t):
    for off in range(1, 9):
        h = torch.full((off + rows * ff + 1,), 9.0, dtype=DT[t], device="cuda")
        check_ff(randn((rows, dim), 1, 1.0, t, off), *weights(dim, ff, t, 9 - off),
                 h=h[off:-1].view(rows, ff))
        assert (h[:off] == 9).all() and h[-1] == 9


def test_ff_leading_dimensions_and_no_rows():
    x, w = randn((2, 3, 64), 1), weights(64, 40, "f32")
    h = torch.empty(2, 3, 40, device="cuda")
    gate, up = torch.empty_like(h), rra.Saved.empty(6, 40)
    rra.gated_ff(x, *w, h, gate, up)
    flat = torch.empty(6, 40, device="cuda")
    rra.gated_ff(x.view(6, 64), *w, flat)
    assert torch.equal(h.view(6, 40), flat)
    rra.gated_ff(x.view(6, 64)[:0], *w, flat[:0])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [3, 300])
def test_ff_carries_nan_and_infinity_in_their_row(rows, t):
    x, w = randn((rows, 64), 1, 1.0, t), weights(64, 200, t)
    clean = torch.empty(rows, 200, dtype=DT[t], device="cuda")
    rra.gated_ff(x, *w, clean)
    for bad in (math.nan, math.inf):
        x[1, 5] = bad
        h, kept = torch.empty_like(clean), [rra.Saved.empty(rows, 200) for _ in range(2)]
        rra.gated_ff(x, *w, h, *kept)
        assert not torch.isfinite(h[1]).any()
        others = [r for r in range(rows) if r != 1]
        assert torch.equal(h[others], clean[others])
        for k in kept:
            assert (k.exps[1] == -128).all() and (k.codes[1] == 0).all()
            assert (k.exps[others] > -126).all()


def test_ff_gives_equal_bits():
    for rows, dim, ff in ((1, 2048, 3000), (40, 2048, 3000), (1000, 1024, 1024)):
        x, w = randn((rows, dim), 1, 1.0, "bf16"), weights(dim, ff, "bf16")
        first = None
        for _ in range(5):
            h = torch.full((rows, ff), 9.0, dtype=torch.bfloat16, device="cuda")
            rra.gated_ff(x, *w, h)
            first = h if first is None else first
            assert torch.equal(h, first)


# ---------------------------------------------------------------- gradient

def grad_inputs(rows, dim, ff, t, keep, offset=0):
    x, dh = randn((rows, dim), 1, 1.0, t, offset), randn((rows, ff), 4, 0.1, t, offset)
    kept = [randn((rows, ff), s, 1.0, t, offset) for s in (5, 6)]
    if keep == "bits8":
        kept = [saved_of(k.double()) for k in kept]
    return dh, x, weights(dim, ff, t, offset), kept


def check_ff_grad(dh, x, w, kept, name="silu", wt=None, accumulate=False, outs=None, places=None):
    """outs: which of dx, dw_gate, dw_up, h to ask for; places: where dgate, dup, h go."""
    outs = outs or ("dx", "dwg", "dwu", "h")
    (rows, ff), dim, t = dh.shape, x.shape[1], dh.dtype
    g, u = (values(k) if isinstance(k, rra.Saved) else k.double() for k in kept)
    d, xd, wd = dh.double(), x.double(), [v.double() for v in w]
    a, slope, _ = act(name, g)
    ea, es = act_errors(name, g)
    wt = wt or t
    dw = [randn((ff, dim), s, 0.1).to(wt) for s in (50, 51)]
    old = [v.double() for v in dw]
    dx = torch.full_like(x, 9.0)
    if places is None:
        places = [torch.full_like(dh, 9.0) for _ in range(3)]
    dgate, dup, h = places
    rra.gated_ff_grad(dh, x, *w, *kept, dgate, dup, dx=dx if "dx" in outs else None,
                      dw_gate=dw[0] if "dwg" in outs else None,
                      dw_up=dw[1] if "dwu" in outs else None, h=h if "h" in outs else None,
                      act=name, accumulate=accumulate)
    for got, want, err in ((dgate, d * u * slope, (d * u).abs() * es),
                           (dup, d * a, d.abs() * ea), (h, a * u, u.abs() * ea)):
        if got is not h or "h" in outs:
            close(got, want, rounded(want, t, err + 3 * U * want.abs()), "elementwise")
    parts = [dgate.double(), dup.double()]
    if "dx" in outs:
        want = parts[0] @ wd[0] + parts[1] @ wd[1]
        size = parts[0].abs() @ wd[0].abs() + parts[1].abs() @ wd[1].abs()
        close(dx, want, rounded(want, t, products(2 * ff, size)), "dx")
        off = (dx.double() - want).norm()
        assert off <= (UT[t] + 16 * math.sqrt(2 * ff + 8) * U) * want.norm() + TINY[t] * rows * dim
    else:
        assert (dx == 9).all()
    for k, key in enumerate(("dwg", "dwu")):
        if key not in outs:
            assert torch.equal(dw[k].double(), old[k])
            continue
        want = parts[k].t() @ xd
        err = products(rows, parts[k].abs().t() @ xd.abs())
        if accumulate:
            want = want + old[k]
            err = err + U * want.abs()
        close(dw[k], want, rounded(want, wt, err), key)
    return dgate, dup, h, dx, dw


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("keep", ["full", "bits8"])
@pytest.mark.parametrize("rows,dim,ff", SIZES)
def test_ff_grad(rows, dim, ff, keep, t):
    dh, x, w, kept = grad_inputs(rows, dim, ff, t, keep)
    check_ff_grad(dh, x, w, kept, name=ACTS[(rows + ff) % 4])


@pytest.mark.parametrize("t,wt", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"),
                                  ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,dim,ff", [(300, 264, 520), (77, 51, 130)])
def test_ff_grad_types(rows, dim, ff, accumulate, t, wt):
    dh, x, w, kept = grad_inputs(rows, dim, ff, t, "bits8")
    check_ff_grad(dh, x, w, kept, wt=DT[wt], accumulate=accumulate)


@pytest.mark.parametrize("rows,dim,ff", [(1024, 1024, 4096), (2000, 2048, 5000), (700, 4104, 2056),
                                         (8192, 512, 768)])
def test_ff_grad_of_large_sizes(rows, dim, ff):
    dh, x, w, kept = grad_inputs(rows, dim, ff, "bf16", "bits8")
    check_ff_grad(dh, x, w, kept)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_ff_grad_activations(name, t):
    dh, x, w, kept = grad_inputs(50, 40, 200, t, "full")
    kept[0][::4] *= 8  # far from zero
    kept[0][1] = 0
    check_ff_grad(dh, x, w, kept, name=name)


@pytest.mark.parametrize("outs", [("dx",), ("dwg",), ("dwu",), ("h",), (), ("dwg", "dwu"),
                                  ("dx", "dwu")])
def test_ff_grad_of_parts(outs):
    dh, x, w, kept = grad_inputs(200, 136, 264, "bf16", "bits8")
    whole = check_ff_grad(dh, x, w, kept)
    part = check_ff_grad(dh, x, w, kept, outs=outs or ("none",))
    for k, key in enumerate(("dgate", "dup", "h", "dx")):
        if key in outs or k < 2:
            assert torch.equal(part[k], whole[k])
    for k, key in enumerate(("dwg", "dwu")):
        if key in outs:
            assert torch.equal(part[4][k], whole[4][k])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("ff", [264, 333])
def test_ff_grad_in_place(ff, t):
    """dgate, dup and h in the places of dh, gate and up, in any order."""
    for order in ((0, 1, 2), (1, 2, 0), (2, 0, 1), (0, 2, 1)):
        dh, x, w, kept = grad_inputs(100, 72, ff, t, "full")
        apart = check_ff_grad(dh, x, w, kept)
        inputs = [dh, kept[0], kept[1]]
        outs = [inputs[k] for k in order]
        dx, dw = torch.empty_like(x), [torch.empty_like(v) for v in w]
        rra.gated_ff_grad(dh, x, *w, *kept, outs[0], outs[1], dx=dx, dw_gate=dw[0], dw_up=dw[1],
                          h=outs[2])
        for got, want in zip([*outs, dx], apart[:4]):
            assert torch.equal(got, want)
        for got, want in zip(dw, apart[4]):
            assert torch.equal(got, want)
    dh, x, w, kept = grad_inputs(100, 72, ff, t, "bits8")
    apart = check_ff_grad(dh, x, w, kept)
    up, h = torch.empty_like(dh), torch.empty_like(dh)
    rra.gated_ff_grad(dh, x, *w, *kept, dh, up, h=h)
    assert torch.equal(dh, apart[0]) and torch.equal(up, apart[1]) and torch.equal(h, apart[2])


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_ff_grad_at_every_place(t):
    for off in range(1, 9):
        dh, x, w, kept = grad_inputs(150, 64, 136, t, "full", off)
        check_ff_grad(dh, x, w, kept)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_ff_grad_of_no_rows(accumulate, t):
    dh, x, w, kept = grad_inputs(4, 64, 40, t, "bits8")
    dw = [torch.full_like(v, 3.0) for v in w]
    kept = [rra.Saved(k.exps[:0], k.codes[:0], 40) for k in kept]
    rra.gated_ff_grad(dh[:0], x[:0], *w, *kept, dh[:0], dh[:0].clone(), dw_gate=dw[0], dw_up=dw[1],
                      accumulate=accumulate)
    for v in dw:
        assert (v == (3.0 if accumulate else 0.0)).all()


def test_ff_grad_gives_equal_bits():
    dh, x, w, kept = grad_inputs(3000, 520, 1032, "bf16", "bits8")
    first = None
    for _ in range(4):
        got = check_ff_grad(dh, x, w, kept)
        got = [*got[:4], *got[4]]
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_ff_grad_against_differences(name):
    """Directional derivatives of sum(h * dh) in x and the weights by central
    differences in 64 bits; gate and up of the framework's own forward pass, kept whole."""
    rows, dim, ff = 7, 20, 30
    x, w, dh = randn((rows, dim), 1), weights(dim, ff, "f32"), randn((rows, ff), 4)
    h, kept = check_ff(x, *w, name=name, keep="full")
    _, _, _, dx, _ = check_ff_grad(dh, x, w, kept, name=name)
    dw = [torch.empty_like(v) for v in w]
    rra.gated_ff_grad(dh, x, *w, *kept, torch.empty_like(dh), torch.empty_like(dh), dw_gate=dw[0],
                      dw_up=dw[1], act=name)

    def loss(x, wg, wu):
        return (act(name, x @ wg.t())[0] * (x @ wu.t()) * dh.double()).sum()
    args = [x.double(), w[0].double(), w[1].double()]
    for k, grad in enumerate((dx, dw[0], dw[1])):
        v = torch.randn(args[k].shape, generator=gen(9), device="cuda", dtype=torch.float64)
        step = 1e-5
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + step * v, args[k] - step * v
        slope = float((loss(*up) - loss(*down)) / (2 * step))
        got = float((grad.double() * v).sum())
        # truncation and 64-bit rounding below 1e-5; sums of 2 ff terms, gate and up off by
        # dim + 8 units, the activations by 100: all first-order in U
        assert abs(slope - got) <= 400 * U * float((grad.double() * v).abs().sum()) + 1e-5


@pytest.mark.parametrize("t,rows,dim,ff", [("bf16", 40, 520, 1032), ("bf16", 1000, 520, 1032),
                                           ("f32", 100, 64, 96), ("f16", 100, 63, 97)])
def test_ff_on_a_stream_and_in_a_graph(t, rows, dim, ff):
    dh, x, w, kept = grad_inputs(rows, dim, ff, t, "bits8")
    outs = [torch.empty_like(dh) for _ in range(4)] + [torch.empty_like(x)] + \
        [torch.empty_like(v) for v in w]

    def calls(**kw):
        rra.gated_ff(x, *w, outs[0], **kw)
        rra.gated_ff_grad(dh, x, *w, *kept, outs[1], outs[2], h=outs[3], dx=outs[4],
                          dw_gate=outs[5], dw_up=outs[6], **kw)
    calls()
    first = [o.clone() for o in outs]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls(stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        calls()
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, f in zip(outs, first):
            assert torch.equal(o, f)


# ---------------------------------------------------------------- few tiles, many slices

@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim,ff", [(300, 2056, 130), (20, 4096, 264), (65, 1000, 129),
                                         (257, 8192, 64), (70, 385, 257)])
def test_ff_split_along_k(rows, dim, ff, t):
    """Few results of long sums."""
    x, w = randn((rows, dim), 1, 1.0, t), weights(dim, ff, t)
    h, _ = check_ff(x, *w, keep="bits8", name="gelu_tanh")
    again, _ = check_ff(x, *w, keep="full", name="gelu_tanh")
    assert torch.equal(h, again)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,ff", [(40, 72, 5000), (300, 500, 2064), (5000, 72, 40),
                                         (2100, 264, 130), (129, 130, 131)])
def test_ff_grad_split_along_k(rows, dim, ff, t):
    dh, x, w, kept = grad_inputs(rows, dim, ff, t, "bits8")
    first = check_ff_grad(dh, x, w, kept)
    for _ in range(3):
        again = check_ff_grad(dh, x, w, kept)
        assert torch.equal(first[3], again[3])
        for a, b in zip(first[4], again[4]):
            assert torch.equal(a, b)


def test_ff_of_sizes_around_the_tiles():
    """Every remainder that an end of a tile, of a slice, of a block of codes can have."""
    for rows in (31, 65, 127, 129, 255, 257, 385):
        for dim, ff in ((63, 127), (64, 128), (65, 129), (72, 136), (128, 264), (200, 392)):
            x, w = randn((rows, dim), rows, 1.0, "bf16"), weights(dim, ff, "bf16")
            check_ff(x, *w, keep="bits8" if (rows + ff) % 2 else "full")


@pytest.mark.parametrize("keep", ["full", "bits8"])
def test_ff_beyond_32_bits(keep):
    """More than 2^31 elements of h, whose last rows alone are not zero."""
    rows, dim, ff = 131_100, 64, 16_384
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    x[-3:] = randn((3, dim), 1, 1.0, "bf16")
    w = weights(dim, ff, "bf16")
    h = torch.full((rows, ff), 9.0, dtype=torch.bfloat16, device="cuda")
    kept = [rra.Saved.empty(rows, ff) if keep == "bits8" else torch.full_like(h, 9.0)
            for _ in range(2)]
    rra.gated_ff(x, *w, h, *kept)
    tail = torch.empty(300, ff, dtype=torch.bfloat16, device="cuda")
    rra.gated_ff(x[-300:], *w, tail)
    assert torch.equal(h[-300:], tail) and int(torch.count_nonzero(h[:-3])) == 0
    dh = torch.zeros_like(h)
    dh[-3:] = randn((3, ff), 4, 0.1, "bf16")
    dx, dw = torch.full_like(x, 9.0), [torch.full_like(v, 9.0) for v in w]
    rra.gated_ff_grad(dh, x, *w, *kept, dh, h, dx=dx, dw_gate=dw[0], dw_up=dw[1])
    g, u = (values(k)[-3:] if keep == "bits8" else k[-3:].double() for k in
            ([rra.Saved(k.exps[-3:], k.codes[-3:], ff) if keep == "bits8" else k for k in kept]))
    d = randn((3, ff), 4, 0.1, "bf16").double()
    a, slope, _ = act("silu", g)
    close(h[-3:], d * a, rounded(d * a, h.dtype, d.abs() * act_errors("silu", g)[0]
                                 + 3 * U * (d * a).abs()), "dup")
    for k, part in enumerate((dh, h)):
        want = part[-3:].double().t() @ x[-3:].double()
        close(dw[k], want, rounded(want, dw[k].dtype, products(
            11, part[-3:].double().abs().t() @ x[-3:].double().abs())), "dw")
    assert int(torch.count_nonzero(dx[:-3])) == 0 and torch.isfinite(dx[-3:]).all()


# ---------------------------------------------------------------- streams, scratch

def test_ff_scratch_does_not_grow_during_a_capture():
    st = torch.cuda.Stream()
    x, w = randn((100, 999), 1), weights(999, 2001, "f32")  # operands laid out anew
    h, mark = torch.empty(100, 2001, device="cuda"), torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        with pytest.raises(rra.RRAError) as e:
            rra.gated_ff(x, *w, h)
        assert e.value.code == rra.RRA_ERR_INVALID
        mark.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert float(mark) == 1.0


def test_ff_on_two_streams_at_once():
    """Calls that use scratch (copies of operands, splits) side by side."""
    cases = []
    for k, (rows, dim, ff, t) in enumerate([(300, 2056, 130, "bf16"), (200, 999, 257, "f32"),
                                            (40, 72, 5000, "bf16"), (333, 513, 301, "f16")]):
        dh, x, w, kept = grad_inputs(rows, dim, ff, t, "bits8")
        outs = [torch.empty_like(dh) for _ in range(3)] + [torch.empty_like(x)] + \
            [torch.empty_like(v) for v in w]
        cases.append((dh, x, w, kept, outs))

    def call(case, st=None):
        dh, x, w, kept, outs = case
        rra.gated_ff(x, *w, outs[0], stream=st)
        rra.gated_ff_grad(dh, x, *w, *kept, outs[1], outs[2], dx=outs[3], dw_gate=outs[4],
                          dw_up=outs[5], stream=st)
    want = []
    for c in cases:
        call(c)
        torch.cuda.synchronize()
        want.append([o.clone() for o in c[4]])
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        for c in cases:
            for o in c[4]:
                o.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for c, st in zip(cases, streams):
                call(c, st)
        torch.cuda.synchronize()
        for c, ws in zip(cases, want):
            for o, v in zip(c[4], ws):
                assert torch.equal(o, v)


def test_ff_calls_behind_one_another_and_behind_their_inputs_writers():
    """Inputs written right before the call on its stream, outputs read right behind it."""
    for rows, dim, ff, t in ((1, 2048, 4096, "bf16"), (300, 520, 1032, "bf16"), (33, 65, 129, "f32")):
        x, w = randn((rows, dim), 1, 1.0, t), weights(dim, ff, t)
        want = [torch.empty(rows, ff, dtype=DT[t], device="cuda") for _ in range(2)]
        other = randn((rows, dim), 9, 1.0, t)
        for v, o in zip((x, other), want):
            rra.gated_ff(v, *w, o)
            torch.cuda.synchronize()
        inp, h, seen = torch.empty_like(x), torch.empty_like(want[0]), []
        for k in range(20):
            inp.copy_(x if k % 2 == 0 else other)
            rra.gated_ff(inp, *w, h)
            seen.append(h.clone())
        for k, s in enumerate(seen):
            assert torch.equal(s, want[k % 2])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,ff", [(40, 72, 300), (300, 520, 1032)])
def test_ff_grad_carries_nan_where_it_belongs(rows, dim, ff, t):
    """A block of codes that is not finite: its row of dx, its columns of the weights'
    gradients, and nothing else."""
    dh, x, w, kept = grad_inputs(rows, dim, ff, t, "bits8")
    kept[0].exps[3, 1] = -128
    kept[0].codes[3, 128:256] = 0
    dgate, dup, h = (torch.empty_like(dh) for _ in range(3))
    dx, dw = torch.empty_like(x), [torch.empty_like(v) for v in w]
    rra.gated_ff_grad(dh, x, *w, *kept, dgate, dup, dx=dx, dw_gate=dw[0], dw_up=dw[1], h=h)
    for v in (dgate, dup, h):
        bad = torch.zeros_like(v, dtype=torch.bool)
        bad[3, 128:256] = True
        assert torch.equal(torch.isnan(v), bad)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[3] = True
    assert torch.equal(torch.isnan(dx).all(1), bad) and torch.equal(torch.isnan(dx).any(1), bad)
    for v in dw:
        bad = torch.zeros(ff, dtype=torch.bool, device="cuda")
        bad[128:256] = True
        assert torch.equal(torch.isnan(v).all(1), bad) and torch.equal(torch.isnan(v).any(1), bad)


def test_ff_first_call_of_a_process_in_a_capture():
    """Calls that need no scratch may be captured without having been made before."""
    import subprocess
    import sys
    code = """
import torch, ring_allreduce_compressed_gb300 as rra
x = torch.randn(300, 64, device="cuda").bfloat16()
w = [torch.randn(128, 64, device="cuda").bfloat16() for _ in range(2)]
h, few = torch.zeros(300, 128, device="cuda").bfloat16(), torch.zeros(3, 128, device="cuda").bfloat16()
s, m, r = rra.Saved.empty(300, 64), *(torch.empty(300, device="cuda") for _ in range(2))
y = torch.empty_like(x)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    rra.gated_ff(x, *w, h)
    rra.gated_ff(x[:3], *w, few)
    rra.layer_norm_save(x, None, None, y, s, m, r)
    rra.layer_norm_restore(s, y)
g.replay()
torch.cuda.synchronize()
want = torch.nn.functional.silu(x.float() @ w[0].float().t()) * (x.float() @ w[1].float().t())
for got, ref in ((h, want), (few, want[:3])):
    assert float((got.float() - ref).norm() / ref.norm()) < 1e-2
assert float((y.float() - x.float()).norm() / x.float().norm()) < 2e-2
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_ff_in_two_threads_at_once():
    """Two threads with a stream each, scratch that grows among the calls."""
    import threading
    jobs = []
    for k, t in enumerate(("bf16", "f32")):
        sizes = [(100 + 50 * k, 99, 301), (200, 515, 129), (300, 1030, 257)]
        jobs.append([(randn((r, d), 1, 1.0, t), weights(d, f, t)) for r, d, f in sizes])
    want = [[torch.empty(x.shape[0], w[0].shape[0], dtype=x.dtype, device="cuda") for x, w in j]
            for j in jobs]
    for j, ws in zip(jobs, want):
        for (x, w), o in zip(j, ws):
            rra.gated_ff(x, *w, o)
    torch.cuda.synchronize()
    errors = []

    def work(j, ws):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    for (x, w), o in zip(j, ws):
                        h = torch.empty_like(o)
                        rra.gated_ff(x, *w, h)
                        assert torch.equal(h, o)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
