"""A feed-forward block whose activations are held in 8 bits, as examples/train_step.py
runs it: norm, gated projections and their gradients together, against formulas in 64
bits that read the same 8 bits."""
import importlib.util
import os

import pytest
import torch

import ring_allreduce_compressed_gb300 as rra
from saved_util import act, encode, values
from test_gpu_gated_ff import check_kept

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def normed(x, gamma, beta):
    mean = x.mean(1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + 1e-5).sqrt()
    return (x - mean) * rstd * gamma + beta, mean, rstd


def gradients(m, inputs, targets):
    """Loss and gradients of one rank in 64 bits.  Forward as the formulas have it; backward
    with what the model's codes stand for."""
    t = {k: getattr(m, k).double() for k in ("table", "bucket")}
    gamma, beta, head = m.views(t["bucket"])
    wg, wu, wd = m.block(t["bucket"])
    x = t["table"][inputs] * m.scale
    y, mean, rstd = normed(x, gamma, beta)
    g, u = y @ wg.t(), y @ wu.t()
    z = y + (act("silu", g)[0] * u) @ wd.t()
    logp = torch.log_softmax(z @ head.t(), 1)
    at = torch.arange(m.tokens, device="cuda")
    loss = -logp[at, targets].mean()
    dlogits = logp.exp()
    dlogits[at, targets] -= 1
    dlogits /= m.tokens
    dz = dlogits @ head
    grad = dict(head=dlogits.t() @ z)
    # what was kept: within half a step (a whole one at the clamp) of x, g and u
    check_kept(m.saved, x, 1e-6 * x.abs().max())
    check_kept(m.gate, g, 1e-5 * g.abs().max())
    check_kept(m.up, u, 1e-5 * u.abs().max())
    xh = (values(m.saved) - mean) * rstd
    yr, gr, ur = xh * gamma + beta, values(m.gate), values(m.up)
    a, slope, _ = act("silu", gr)
    dh = dz @ wd
    dgate, dup = dh * ur * slope, dh * a
    grad["gate"], grad["up"] = dgate.t() @ yr, dup.t() @ yr
    grad["down"] = dz.t() @ (a * ur)
    dy = dz + dgate @ wg + dup @ wu
    w = dy * gamma
    dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    grad["gamma"], grad["beta"] = (dy * xh).sum(0), dy.sum(0)
    grad["table"] = torch.zeros_like(t["table"]).index_add_(0, inputs, dx) * m.scale
    return loss, grad


@pytest.mark.parametrize("dim,ff,tokens", [(72, 200, 130), (64, 96, 40), (33, 257, 300)])
def test_gradients_of_a_rank(example, dim, ff, tokens):
    torch.backends.cuda.matmul.allow_tf32 = False
    m = example.Model(vocab=100, dim=dim, tokens=tokens, ranks=1, ff=ff)
    inputs, targets = example.batch(m, 0, 0)
    loss = m.rank_gradients(0, inputs, targets)
    want_loss, want = gradients(m, inputs, targets)
    assert abs(float(loss) / float(want_loss) - 1) < 1e-5
    dgamma, dbeta, dhead = m.views(m.dbucket[0])
    dg, du, dd = m.block(m.dbucket[0])
    got = dict(gamma=dgamma, beta=dbeta, head=dhead, gate=dg, up=du, down=dd, table=m.dtable[0])
    # fp32 sums of up to `tokens`, `ff` and `dim` terms over six products in a row: 1e-5 of the
    # largest, as in test_gpu_train_step.py
    for k, v in want.items():
        assert float((got[k].double() - v).abs().max()) < 1e-5 * float(v.abs().max()), k


def test_steps_run_with_several_ranks_and_change_every_weight(example):
    m = example.Model(vocab=100, dim=64, tokens=200, ranks=3, ff=160)
    before = m.bucket.clone(), m.table.clone()
    for s in range(3):
        loss = m.step([example.batch(m, s, r) for r in range(3)], lr=0.1, max_norm=1.0)
        assert torch.isfinite(loss) and torch.isfinite(m.norm).all()
    for w, v in zip(m.views(m.bucket) + m.block(m.bucket),
                    m.views(before[0]) + m.block(before[0])):
        assert torch.isfinite(w).all() and not torch.equal(w, v)
    assert not torch.equal(m.table, before[1])


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
def test_block_in_16_bits_captured_and_replayed(t):
    """The block's calls one behind the other in a graph, on new inputs each time."""
    rows, dim, ff = 300, 264, 520
    gen = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(t)
    x, dy = randn(rows, dim), randn(rows, dim, std=0.1)
    gamma, beta = randn(dim, std=0.1) + 1, randn(dim, std=0.1)
    wg, wu = randn(ff, dim, std=dim ** -0.5), randn(ff, dim, std=dim ** -0.5)
    dh = randn(rows, ff, std=0.1)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    saved, gate, up = rra.Saved.empty(rows, dim), rra.Saved.empty(rows, ff), \
        rra.Saved.empty(rows, ff)
    y, yr, dn, dx = (torch.empty_like(x) for _ in range(4))
    h, hr, dg, du = (torch.empty_like(dh) for _ in range(4))
    dwg, dwu, dgamma, dbeta = (torch.empty_like(v) for v in (wg, wu, gamma, beta))
    outs = [y, yr, dn, dx, h, hr, dg, du, dwg, dwu, dgamma, dbeta, saved.codes, saved.exps,
            gate.codes, gate.exps, up.codes, up.exps]

    def calls():
        rra.layer_norm_save(x, gamma, beta, y, saved, mean, rstd)
        rra.gated_ff(y, wg, wu, h, gate, up)
        rra.layer_norm_restore(saved, yr, gamma, beta, mean, rstd)
        rra.gated_ff_grad(dh, yr, wg, wu, gate, up, dg, du, dx=dn, dw_gate=dwg, dw_up=dwu, h=hr)
        rra.layer_norm_saved_grad(dn, saved, gamma, mean, rstd, dx, dgamma, dbeta)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        calls()  # the stream's scratch
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        calls()
    for k in range(3):
        x.copy_(randn(rows, dim))
        dh.copy_(randn(rows, ff, std=0.1))
        torch.cuda.synchronize()
        calls()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
        e, c = encode(x.double())
        assert torch.equal(saved.exps, e) and torch.equal(saved.codes, c)
