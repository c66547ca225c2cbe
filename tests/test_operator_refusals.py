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


# Products of sizes that are each in range can pass 64 bits, and what is left of
# them then says nothing about overlaps.
def test_operators_refuse_arrays_beyond_any_memory(lib):
    most = (1 << 31) - 1
    assert lib.rra_embedding(A, B, 4, most, 1 << 32, 0, 1, 1.0, D, None) == INV
    assert lib.rra_embedding(A, B, most, 8, 1 << 32, 0, 1, 1.0, D, None) == INV
    assert lib.rra_embedding_grad(A, B, 4, most, 1 << 32, 0, 1, 1.0, -1, D, 0, 0, None) == INV
    assert lib.rra_embedding_grad(A, B, most, 8, 1 << 32, 1, 1, 1.0, -1, D, 0, 0, None) == INV
    assert layer_norm(lib, rows=1 << 40, dim=1 << 31, mean=None, rstd=None) == INV
    assert lib.rra_layer_norm_grad(A, B, None, D, E, 1 << 40, 1 << 22, 0, 0, None, None, E + 4096,
                                   0, None) == INV
