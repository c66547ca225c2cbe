"""Arguments that the operators with activations in 8 bits have to turn down before
any CUDA call.  Addresses are plain numbers that nothing reads."""
import pytest
import torch

import ring_allreduce_compressed_gb300 as rra

OK, INV, UNS = rra.RRA_OK, rra.RRA_ERR_INVALID, rra.RRA_ERR_UNSUPPORTED
A, B, C, D, E, F, G, H = (k << 24 for k in range(1, 9))  # far apart
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    rra.build()
    return rra.lib()


def save(lib, **given):
    a = dict(dict(x=A, gamma=B, beta=B + 4096, rows=4, dim=16, t=0, wt=0, eps=1e-5, y=C, exps=D,
                  codes=E, mean=F, rstd=G), **given)
    return lib.rra_layer_norm_save(a["x"], a["gamma"], a["beta"], a["rows"], a["dim"], a["t"],
                                   a["wt"], a["eps"], a["y"], a["exps"], a["codes"], a["mean"],
                                   a["rstd"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), INV), (dict(y=None), INV), (dict(exps=None), INV), (dict(codes=None), INV),
    (dict(mean=None), INV), (dict(rstd=None), INV), (dict(dim=0), INV),
    (dict(dim=(1 << 31) + 1), INV), (dict(rows=(1 << 40) + 1), INV),
    (dict(rows=1 << 40, dim=1 << 31), INV), (dict(rows=1 << 40, dim=1), INV),
    (dict(t=3), INV), (dict(wt=-1), INV), (dict(eps=-1.0), INV), (dict(eps=NAN), INV),
    (dict(x=A + 2), INV), (dict(y=C + 1), INV), (dict(gamma=B + 2), INV), (dict(codes=E + 8), INV),
    (dict(mean=F + 2), INV), (dict(y=A + 4), INV), (dict(exps=A), INV), (dict(exps=A + 255), INV),
    (dict(codes=C), INV), (dict(codes=C - 512 + 16), INV), (dict(codes=D - 496), INV),
    (dict(mean=G + 12), INV), (dict(rstd=B + 60), INV), (dict(exps=B + 4096), INV),
    (dict(mean=E + 508), INV), (dict(t=1, wt=2), UNS), (dict(t=0, wt=1), UNS),
])
def test_save_refuses(lib, bad, code):
    assert save(lib, **bad) == code


def test_empty_calls_are_valid(lib):
    assert save(lib, rows=0, x=None, y=None, exps=None, codes=None, mean=None, rstd=None) == OK
    assert restore(lib, rows=0, exps=None, codes=None, y=None) == OK
    assert gated(lib, rows=0, x=None, h=None) == OK


def restore(lib, **given):
    a = dict(dict(exps=A, codes=B, mean=C, rstd=D, gamma=E, beta=F, rows=4, dim=16, t=0, wt=0, y=G),
             **given)
    return lib.rra_layer_norm_restore(a["exps"], a["codes"], a["mean"], a["rstd"], a["gamma"],
                                      a["beta"], a["rows"], a["dim"], a["t"], a["wt"], a["y"],
                                      None)


@pytest.mark.parametrize("bad,code", [
    (dict(exps=None), INV), (dict(codes=None), INV), (dict(y=None), INV), (dict(dim=0), INV),
    (dict(t=9), INV), (dict(codes=B + 1), INV), (dict(y=G + 2), INV), (dict(mean=C + 1), INV),
    (dict(y=B), INV), (dict(y=B + 508), INV), (dict(y=A), INV), (dict(y=C), INV), (dict(y=D), INV),
    (dict(y=E + 60), INV), (dict(y=F), INV), (dict(t=2, wt=1), UNS),
])
def test_restore_refuses(lib, bad, code):
    assert restore(lib, **bad) == code


def saved_grad(lib, **given):
    a = dict(dict(dy=A, exps=B, codes=C, gamma=D, mean=E, rstd=E + 4096, rows=4, dim=16, t=0, wt=0,
                  dx=F, dgamma=G, dbeta=H), **given)
    return lib.rra_layer_norm_saved_grad(a["dy"], a["exps"], a["codes"], a["gamma"], a["mean"],
                                         a["rstd"], a["rows"], a["dim"], a["t"], a["wt"], a["dx"],
                                         a["dgamma"], a["dbeta"], 0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dy=None), INV), (dict(exps=None), INV), (dict(codes=None), INV), (dict(mean=None), INV),
    (dict(rstd=None), INV), (dict(dx=None, dgamma=None, dbeta=None), INV), (dict(dim=0), INV),
    (dict(codes=C + 4), INV), (dict(dx=F + 2), INV), (dict(dgamma=G + 2), INV),
    (dict(dx=A + 4), INV), (dict(dx=C), INV), (dict(dx=B), INV), (dict(dx=D), INV),
    (dict(dgamma=A), INV), (dict(dgamma=C + 508), INV), (dict(dbeta=G), INV), (dict(dbeta=F), INV),
    (dict(dx=A, dgamma=A + 16), INV), (dict(dgamma=E), INV), (dict(dy=D, dx=D), INV),
    (dict(t=1, wt=2), UNS),
])
def test_saved_grad_refuses(lib, bad, code):
    assert saved_grad(lib, **bad) == code


def gated(lib, **given):
    a = dict(dict(x=A, wg=B, wu=C, rows=4, dim=16, ff=32, t=0, act=0, h=D, ge=None, gate=None,
                  ue=None, up=None), **given)
    return lib.rra_gated_ff(a["x"], a["wg"], a["wu"], a["rows"], a["dim"], a["ff"], a["t"],
                            a["act"], a["h"], a["ge"], a["gate"], a["ue"], a["up"], None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(wg=None), dict(wu=None), dict(h=None), dict(dim=0), dict(ff=0), dict(t=3),
    dict(act=4), dict(act=-1), dict(rows=1 << 31), dict(dim=1 << 31), dict(ff=1 << 31),
    dict(rows=(1 << 31) - 1, dim=(1 << 31) - 1), dict(x=A + 2), dict(wg=B + 1), dict(h=D + 2),
    dict(ge=E), dict(ue=E), dict(ge=E, gate=F + 8), dict(gate=F + 2), dict(ue=E, up=F + 4),
    dict(h=A), dict(h=B + 2044), dict(h=C), dict(gate=D), dict(gate=E, up=E + 508),
    dict(ge=E, gate=E), dict(ge=E, gate=F, ue=E + 3, up=G), dict(ge=A, gate=F),
    dict(ge=E, gate=F, ue=F + 511, up=G), dict(ge=E, gate=C, ue=F, up=G),
])
def test_gated_ff_refuses(lib, bad):
    assert gated(lib, **bad) == INV


def gated_grad(lib, **given):
    a = dict(dict(dh=A, x=B, wg=C, wu=C + 65536, ge=None, gate=D, ue=None, up=D + 65536, rows=4,
                  dim=16, ff=32, t=0, act=0, dg=E, du=E + 65536, h=E + 131072, dx=F, dwg=G, dwu=H,
                  dwt=0), **given)
    return lib.rra_gated_ff_grad(a["dh"], a["x"], a["wg"], a["wu"], a["ge"], a["gate"], a["ue"],
                                 a["up"], a["rows"], a["dim"], a["ff"], a["t"], a["act"], a["dg"],
                                 a["du"], a["h"], a["dx"], a["dwg"], a["dwu"], a["dwt"], 0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dh=None), INV), (dict(gate=None), INV), (dict(up=None), INV), (dict(dg=None), INV),
    (dict(du=None), INV), (dict(x=None), INV), (dict(wg=None), INV), (dict(wu=None), INV),
    (dict(dim=0), INV), (dict(ff=0), INV), (dict(t=7), INV), (dict(dwt=7), INV), (dict(act=9), INV),
    (dict(ge=G + 4096), INV), (dict(ue=G + 4096), INV),  # one of the two in 8 bits
    (dict(ge=G + 65536, ue=G + 70000, gate=D + 4), INV), (dict(dg=E + 1), INV),
    (dict(dg=A + 16), INV), (dict(dg=D - 16), INV), (dict(du=E), INV), (dict(h=E + 65536 + 4), INV),
    (dict(dg=B), INV), (dict(dg=C), INV), (dict(dx=A), INV), (dict(dx=B), INV), (dict(dx=C), INV),
    (dict(dx=E), INV), (dict(dwg=B), INV), (dict(dwg=F), INV), (dict(dwu=G), INV),
    (dict(dwu=D), INV), (dict(dwg=E + 131072), INV),
    (dict(ge=G + 65536, ue=G + 70000, dg=D), INV),  # in the place of codes
    (dict(ge=G + 65536, ue=G + 70000, t=1, dwt=1, ff=64, dg=D), INV),  # of the same size
    (dict(t=1, dwt=2), UNS), (dict(t=0, dwt=1), UNS),
])
def test_gated_ff_grad_refuses(lib, bad, code):
    assert gated_grad(lib, **bad) == code


def test_saved_checks_its_shapes():
    def z(*shape):
        return torch.zeros(shape, dtype=torch.int8)
    rra.Saved(z(3, 2), z(3, 256), 129)
    for exps, codes, dim in ((z(3, 1), z(3, 256), 129), (z(3, 2), z(3, 129), 129),
                             (z(2, 2), z(3, 256), 129), (z(6), z(3, 256), 129),
                             (z(3, 2), z(768), 256), (z(3, 2), z(3, 256), 128)):
        with pytest.raises(ValueError):
            rra.Saved(exps, codes, dim)
    s = rra.Saved.empty(3, 200, device="cpu")
    assert s.exps.shape == (3, 2) and s.codes.shape == (3, 256) and s.dim == 200


def test_python_checks_before_any_call():
    x, w = torch.zeros(2, 8), torch.zeros(4, 8)
    s = rra.Saved.empty(2, 4, device="cpu")
    with pytest.raises(ValueError, match="act"):
        rra.gated_ff(x, w, w, x, act="tanh")
    with pytest.raises(ValueError, match="w_gate"):
        rra.gated_ff(x, w[0], w, x)
    with pytest.raises(ValueError, match="CUDA"):
        rra.gated_ff(x, w, w, x)
    with pytest.raises(ValueError, match="CUDA"):
        rra.gated_ff_grad(x, x, w, w, s, s, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        rra.layer_norm_save(x, None, None, x, s, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        rra.layer_norm_restore(s, x)
    with pytest.raises(ValueError, match="CUDA"):
        rra.layer_norm_saved_grad(x, s, None, x, x, x, None, None)
