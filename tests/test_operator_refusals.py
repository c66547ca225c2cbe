"""Arguments that the training-step operators have to turn down before any CUDA
call.  Addresses are plain numbers that nothing reads."""
import ctypes as C

import pytest

import ring_allreduce_compressed_gb300 as rra

INV = rra.RRA_ERR_INVALID
A, B, D, E = 1 << 20, 2 << 20, 3 << 20, 4 << 20  # far apart


@pytest.fixture(scope="module")
def lib():
    rra.build()
    return rra.lib()


def layer_norm(lib, **given):
    a = dict(dict(x=A, gamma=D, beta=D + 4096, rows=4, dim=16, t=0, wt=0, eps=1e-5, y=B, mean=E,
                  rstd=E + 64), **given)
    return lib.rra_layer_norm(a["x"], a["gamma"], a["beta"], a["rows"], a["dim"], a["t"], a["wt"],
                              a["eps"], a["y"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("bad", [
    dict(mean=D), dict(mean=D + 60), dict(rstd=D + 12), dict(mean=D + 4096), dict(rstd=D + 4096 + 60),
    dict(rstd=D - 12),
])
def test_layer_norm_refuses_statistics_over_the_weights(lib, bad):
    assert layer_norm(lib, **bad) == INV
