"""Host-side refusals of the training-step operators: every bad argument is
turned down before any CUDA call, so these run without a GPU.  Addresses are
plain numbers that nothing reads."""
import ctypes as C

import pytest

import ring_allreduce_compressed_gb300 as rra

INV, UNS = rra.RRA_ERR_INVALID, rra.RRA_ERR_UNSUPPORTED
A, B, D, E = 1 << 20, 2 << 20, 3 << 20, 4 << 20  # far apart
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    rra.build()
    return rra.lib()


def _list(ptrs, counts, dtypes):
    n = len(ptrs)
    return (C.c_void_p * n)(*ptrs), (C.c_size_t * n)(*counts), (C.c_int * n)(*dtypes)


@pytest.mark.parametrize("ptrs,counts,dtypes,kind,norm", [
    ([A], [8], [0], 0, None),           # no place for the norm
    ([A], [8], [0], 3, E),              # unknown norm
    ([A], [8], [3], 0, E),              # unknown type
    ([None], [8], [0], 0, E),           # a gradient without an address
    ([A + 2], [8], [0], 0, E),          # an fp32 gradient at an odd half-word
    ([A], [(1 << 40) + 1], [1], 0, E),  # too many elements
    ([A], [8], [0], 0, A + 28),         # the norm inside a gradient
    ([A], [8], [0], 0, E + 2),          # the norm at an odd half-word
])
def test_grad_norm_refuses(lib, ptrs, counts, dtypes, kind, norm):
    p, c, d = _list(ptrs, counts, dtypes)
    assert lib.rra_grad_norm(p, c, d, len(ptrs), kind, norm, None) == INV


def test_grad_norm_refuses_missing_arrays(lib):
    p, c, d = _list([A], [8], [0])
    assert lib.rra_grad_norm(None, c, d, 1, 0, E, None) == INV
    assert lib.rra_grad_norm(p, None, d, 1, 0, E, None) == INV
    assert lib.rra_grad_norm(p, c, None, 1, 0, E, None) == INV
    assert lib.rra_grad_norm(p, c, d, -1, 0, E, None) == INV


@pytest.mark.parametrize("out,max_norm,eps", [
    (None, 1.0, 1e-6), (A + 4, 1.0, 1e-6), (A + 31, 1.0, 1e-6), (B, -1.0, 1e-6), (B, NAN, 1e-6),
    (B, 1.0, -1e-6), (B, 1.0, NAN), (B, 1.0, INF),
])
def test_grad_clip_refuses(lib, out, max_norm, eps):
    p, c, d = _list([A], [8], [0])
    o = (C.c_void_p * 1)(out)
    assert lib.rra_grad_clip(p, o, c, d, 1, 0, max_norm, eps, E, None) == INV


def test_grad_clip_refuses_missing_outputs(lib):
    p, c, d = _list([A], [8], [0])
    assert lib.rra_grad_clip(p, None, c, d, 1, 0, 1.0, 1e-6, E, None) == INV


GOOD = dict(weight=A, tokens=B, n=4, vocab=8, dim=16, dtype=0, index=1, out=D)


@pytest.mark.parametrize("bad", [
    dict(weight=None), dict(tokens=None), dict(out=None), dict(vocab=0), dict(dim=0),
    dict(vocab=1 << 31), dict(n=1 << 31), dict(dim=(1 << 32) + 1), dict(dtype=3), dict(index=2),
    dict(weight=A + 2), dict(tokens=B + 4), dict(out=D + 1),
    dict(out=A + 16), dict(out=B + 16),  # over the table, over the tokens
])
def test_embedding_refuses(lib, bad):
    a = dict(GOOD, **bad)
    assert lib.rra_embedding(a["weight"], a["tokens"], a["n"], a["vocab"], a["dim"], a["dtype"],
                             a["index"], 1.0, a["out"], None) == INV


@pytest.mark.parametrize("bad,code", [
    (dict(dout=None), INV), (dict(tokens=None), INV), (dict(dw=None), INV), (dict(vocab=0), INV),
    (dict(dim=0), INV), (dict(n=1 << 31), INV), (dict(vocab=1 << 31), INV), (dict(t=5), INV),
    (dict(index=-1), INV), (dict(wt=-1), INV), (dict(dw=A + 4), INV), (dict(dw=B), INV),
    (dict(dout=A + 1), INV), (dict(t=0, wt=1), UNS), (dict(t=1, wt=2), UNS),
])
def test_embedding_grad_refuses(lib, bad, code):
    a = dict(dict(dout=A, tokens=B, n=4, vocab=8, dim=16, t=0, index=1, dw=D, wt=0), **bad)
    assert lib.rra_embedding_grad(a["dout"], a["tokens"], a["n"], a["vocab"], a["dim"], a["t"],
                                  a["index"], 1.0, -1, a["dw"], a["wt"], 0, None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), INV), (dict(y=None), INV), (dict(dim=0), INV), (dict(dim=(1 << 31) + 1), INV),
    (dict(rows=(1 << 40) + 1), INV), (dict(t=3), INV), (dict(wt=3), INV), (dict(eps=-1.0), INV),
    (dict(eps=NAN), INV), (dict(y=A + 16), INV), (dict(y=D), INV), (dict(mean=A), INV),
    (dict(x=A + 1), INV), (dict(mean=D + 66), INV), (dict(t=0, wt=1), UNS), (dict(t=2, wt=1), UNS),
])
def test_layer_norm_refuses(lib, bad, code):
    a = dict(dict(x=A, gamma=D, beta=D + 4096, rows=4, dim=16, t=0, wt=0, eps=1e-5, y=B, mean=E,
                  rstd=E + 64), **bad)
    assert lib.rra_layer_norm(a["x"], a["gamma"], a["beta"], a["rows"], a["dim"], a["t"], a["wt"],
                              a["eps"], a["y"], a["mean"], a["rstd"], None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(dy=None), INV), (dict(x=None), INV), (dict(mean=None), INV), (dict(rstd=None), INV),
    (dict(dim=0), INV), (dict(dx=None, dg=None, db=None), INV), (dict(dx=A + 16), INV),
    (dict(dg=E + 1024), INV), (dict(db=B), INV), (dict(dg=A), INV), (dict(dx=D), INV),
    (dict(t=3), INV), (dict(wt=4), INV), (dict(t=1, wt=2), UNS), (dict(t=0, wt=2), UNS),
])
def test_layer_norm_grad_refuses(lib, bad, code):
    a = dict(dict(dy=A, x=B, gamma=D, mean=D + 4096, rstd=D + 8192, rows=4, dim=16, t=0, wt=0,
                  dx=E, dg=E + 4096, db=E + 8192), **bad)
    if bad.get("dg") == E + 1024:
        a["db"] = E + 1024 + 32  # dgamma and dbeta share bytes
    assert lib.rra_layer_norm_grad(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["rows"],
                                   a["dim"], a["t"], a["wt"], a["dx"], a["dg"], a["db"], 0,
                                   None) == code


def test_binding_refuses_what_is_not_a_cuda_tensor():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        rra.grad_norm([x], torch.zeros(1))
    with pytest.raises(ValueError):
        rra.grad_norm([], torch.zeros(1), norm_type=3)
    with pytest.raises(ValueError):
        rra.embedding(x, torch.zeros(2, dtype=torch.int64), torch.zeros(2, 8))
    with pytest.raises(ValueError):
        rra.layer_norm(x, None, None, x)


def test_norm_and_index_constants_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                             "include", "rra.h")).read()
    for name in ("RRA_NORM_L2", "RRA_NORM_L1", "RRA_NORM_INF", "RRA_I32", "RRA_I64"):
        assert int(re.search(rf"\b{name} = (\d+)", text).group(1)) == getattr(rra, name)
