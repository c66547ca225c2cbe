"""Activations in 8 bits and the gated activations, from their definitions in 64
bits: shared by the tests of the operators that keep and read them."""
import math

import torch

import ring_allreduce_compressed_gb300 as rra

BLOCK = 128
U = 2.0 ** -24


def power(n):
    """2^n for whole n from -1022 on, by its bits (torch.pow may miss by a last place)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def normal(g):
    """The normal distribution, without cancellation far below zero."""
    return torch.special.erfc(-g / math.sqrt(2)) / 2


def encode(x):
    """exps (rows, blocks) and codes (rows, blocks * 128) of the rows of x: the exponent of a
    block's largest magnitude; the nearest whole numbers of 2^(e-6), ties to even, within +-127;
    a block that is not finite throughout: -128 and zeros."""
    rows, dim = x.shape
    nb = -(-dim // BLOCK)
    b = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=x.device)
    b[:, :dim] = x
    b = b.view(rows, nb, BLOCK)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    e = torch.where(bad | (top == 0), torch.full_like(top, -126.0),
                    torch.floor(torch.log2(top.clamp(min=1e-300, max=1e300))))
    # log2 may round to a whole number from below it, or from above
    e = torch.where(top < power(e), e - 1, torch.where(top >= power(e + 1), e + 1, e))
    e = torch.where(bad, torch.full_like(e, -126.0), e).clamp(min=-126)
    m = torch.round(b * power(6 - e)[:, :, None]).clamp(-127, 127)
    e = torch.where(bad, torch.full_like(e, -128.0), e)
    m = torch.where(bad[:, :, None], torch.zeros_like(m), m)
    return e.to(torch.int8), m.to(torch.int8).view(rows, nb * BLOCK)


def values(saved):
    """What a Saved stands for, in 64 bits."""
    rows, nb = saved.exps.shape
    e = saved.exps.double()
    unit = torch.where(e == -128, torch.full_like(e, math.nan), power(e - 6))
    m = saved.codes.view(rows, nb, BLOCK).double() * unit[:, :, None]
    return m.view(rows, nb * BLOCK)[:, :saved.dim]


def saved_of(x):
    """x (rows, dim) as a Saved, made from the definition."""
    return rra.Saved(*encode(x), x.shape[1])


def act(name, g):
    """a(g), a'(g) and the argument of the logistic function, in 64 bits."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).double(), torch.zeros_like(g)
    if name == "gelu":
        p = normal(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi), torch.zeros_like(g)
    k = math.sqrt(8 / math.pi)
    z = g if name == "silu" else k * (g + 0.044715 * g ** 3)
    dz = 1.0 if name == "silu" else k * (1 + 3 * 0.044715 * g * g)
    s = torch.sigmoid(z)
    return g * s, s * (1 + g * torch.sigmoid(-z) * dz), z


def act_errors(name, g):
    """Bounds of the errors of a fp32 evaluation of a and a' at the fp32 number g.
    The fast exponential misses by 2 + 1.2 |z| units of its last place, z has some
    4 roundings, the quotient 2 units: 2 (24 + 8 |z|) U of s, relatively, covers both
    ways of evaluating.  1 - s misses by that share of s, and every product by U."""
    a, slope, z = act(name, g)
    if name == "relu":
        return torch.zeros_like(g), torch.zeros_like(g)
    tiny = 2.0 ** -120 * (1 + g.abs())
    if name == "gelu":  # the distribution within 5 units, the density 2 + 1.2 g^2 / 2
        p = normal(g)
        dens = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        return 16 * U * a.abs() + tiny, 16 * U * p + g.abs() * dens * (16 + 8 * g * g) * U + tiny
    d = 2 * (24 + 8 * z.abs()) * U
    dz = 1.0 if name == "silu" else math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g * g)
    s = torch.sigmoid(z)
    return d * a.abs() + tiny, 2 * d * s * (1 + g.abs() * dz) + tiny * dz
