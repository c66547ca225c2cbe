"""What is measured of a feed-forward block whose activations are held in 8 bits: layer norm that
saves its input, its restoring and its gradient from there, and the gated projections with their
gradient."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
BLOCK = 128  # elements that share an exponent
MOST_PRODUCT = 8192 * 4096 * 16384  # rows * dim * ff of one drawn case
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def listed():
    return [
        # a few rows, one step of decoding: the call's own latency
        dict(name="save_step", op="save", rows=32, dim=1024, dtype="f16", weight="f16"),
        # a training batch's forward pass
        dict(name="save_batch", op="save", rows=16_384, dim=4096, dtype="bf16", weight="bf16"),
        # rows of an odd width, fp32
        dict(name="restore_ragged", op="restore", rows=3001, dim=1001, dtype="f32",
             weight="f32"),
        # a training batch, before its backward pass
        dict(name="restore_batch", op="restore", rows=16_384, dim=4096, dtype="bf16",
             weight="bf16"),
        # an fp32 model with odd sizes
        dict(name="norm_grad_ragged", op="norm_grad", rows=3001, dim=1001, dtype="f32",
             weight="f32"),
        # a training batch's backward pass
        dict(name="norm_grad_batch", op="norm_grad", rows=16_384, dim=4096, dtype="bf16",
             weight="f32"),
        # one token: the weights are read for it alone
        dict(name="ff_token", op="ff", rows=1, dim=4096, ff=16_384, dtype="bf16", act="silu",
             save="none"),
        # one step of decoding many sequences
        dict(name="ff_tokens", op="ff", rows=48, dim=2048, ff=8192, dtype="f16", act="gelu_tanh",
             save="none"),
        # an fp32 model with odd sizes, gate and up kept in 8 bits and looked at
        dict(name="ff_ragged", op="ff", rows=333, dim=513, ff=1001, dtype="f32", act="gelu",
             save="bits8"),
        # a training batch's forward pass, gate and up kept as they are
        dict(name="ff_batch", op="ff", rows=8192, dim=4096, ff=16_384, dtype="bf16", act="silu",
             save="full"),
        # odd sizes, from 8 bits
        dict(name="ff_grad_ragged", op="ff_grad", rows=333, dim=513, ff=1001, dtype="f16",
             act="gelu", save="bits8"),
        # a training batch's backward pass, from 8 bits
        dict(name="ff_grad_batch", op="ff_grad", rows=8192, dim=4096, ff=16_384, dtype="bf16",
             act="silu", save="bits8"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm; about every second one odd."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["save", "restore", "norm_grad", "ff", "ff", "ff_grad"])
    if op in ("ff", "ff_grad"):
        dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
        most = MOST_PRODUCT // 256 if dtype == "f32" else MOST_PRODUCT
        rows = _spread(rng, 1, 8192)
        dim = rng.choice([_spread(rng, 16, 4096), 64 * rng.randint(1, 64)])
        top = max(16, min(16_384, most // (rows * dim)))
        ff = rng.choice([_spread(rng, 16, top), max(16, top // 64 * 64 // rng.randint(1, 4))])
        save = rng.choice(["none", "full", "bits8"] if op == "ff" else ["full", "bits8", "bits8"])
        return dict(op=op, rows=rows, dim=dim, ff=ff, dtype=dtype, act=rng.choice(ACTS), save=save)
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    dim = rng.choice([_spread(rng, 2, 16_384), 64 * rng.randint(1, 128)])
    rows = _spread(rng, 1, min(131_072, (1 << 26) // dim))
    return dict(op=op, rows=rows, dim=dim, dtype=dtype, weight=rng.choice([dtype, "f32"]))


# ---------------------------------------------------------------- activations in 8 bits

def _blocks(x):
    """Rows cut into blocks of 128, the last one filled up with zeros."""
    rows, dim = x.shape
    return torch.nn.functional.pad(x, (0, -dim % BLOCK)).view(rows, -1, BLOCK)


def _power(n):
    """2^n for whole n from -126 to 127, by its bits: pow() may miss by a last place."""
    return ((n.int() + 127) << 23).view(torch.float32)


def _encode(x):
    """Exponents and codes of the rows of x (fp32): one exponent per block."""
    b = _blocks(x)
    top = b.abs().amax(2)
    e = (top.view(torch.int32) >> 23).clamp(min=1) - 127
    m = (b * _power(-e).unsqueeze(2) * 64).round().clamp(-127, 127)
    return e.to(torch.int8), m.to(torch.int8).view(x.shape[0], -1)


def _decode(exps, codes, dim):
    """The values, fp32: m * 2^(e - 6)."""
    m = codes.view(exps.shape[0], exps.shape[1], BLOCK).float()
    return (m / 64 * _power(exps).unsqueeze(2)).view(exps.shape[0], -1)[:, :dim]


# ---------------------------------------------------------------- inputs

def _normal(shape, gen, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _room(rows, dim):
    """Places for the exponents and codes of an activation."""
    n = -(-dim // BLOCK)
    return (torch.empty(rows, n, device="cuda", dtype=torch.int8),
            torch.empty(rows, n * BLOCK, device="cuda", dtype=torch.int8))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, rows, dim, dtype = case["op"], case["rows"], case["dim"], TYPES[case["dtype"]]
    s = dict(op=op, dim=dim, dtype=dtype)
    if op in ("save", "restore", "norm_grad"):
        wtype = TYPES[case["weight"]]
        x = (torch.randn(rows, dim, generator=gen, device="cuda") * 1.5 + 0.25).to(dtype)
        s["gamma"] = (1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(wtype)
        if op != "norm_grad":
            s["beta"] = _normal(dim, gen, 0.1, wtype)
            s["y"] = torch.empty_like(x)
        if op == "save":
            s["x"] = x
            s["exps"], s["codes"] = _room(rows, dim)
            s["mean"], s["rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
            return s
        # what the forward pass has left
        s["exps"], s["codes"] = _encode(x.float())
        s["mean"] = x.double().mean(1).float()
        s["rstd"] = (x.double().var(1, unbiased=False) + EPS).rsqrt().float()
        if op == "norm_grad":
            s["dy"] = _normal((rows, dim), gen, 1e-2, dtype)
            s["dx"] = torch.empty_like(x)
            s["dgamma"], s["dbeta"] = (torch.empty_like(s["gamma"]) for _ in range(2))
        return s
    ff, s["act"], s["save"] = case["ff"], case["act"], case["save"]
    s["ff"] = ff
    s["x"] = _normal((rows, dim), gen, 1.0, dtype)
    s["wg"], s["wu"] = (_normal((ff, dim), gen, 1 / math.sqrt(dim), dtype) for _ in range(2))
    if op == "ff":
        s["h"] = torch.empty(rows, ff, device="cuda", dtype=dtype)
        if s["save"] == "full":
            s["gate"], s["up"] = (torch.empty_like(s["h"]) for _ in range(2))
        elif s["save"] == "bits8":
            s["gate"], s["up"] = (_room(rows, ff) for _ in range(2))
            # a code of 8 bits is a number of 16 bits
            s["seen"] = [torch.empty(rows, ff, device="cuda", dtype=torch.bfloat16)
                         for _ in range(2)]
        return s
    # what the forward pass has left, and the gradient that comes back
    for name in ("gate", "up"):
        v = _normal((rows, ff), gen, 1.0, dtype)
        s[name] = v if s["save"] == "full" else _encode(v.float())
    s["dh"] = _normal((rows, ff), gen, 1e-2, dtype)
    s["dgate"], s["dup"], s["h"] = (torch.empty_like(s["dh"]) for _ in range(3))
    s["dx"] = torch.empty_like(s["x"])
    s["dwg"], s["dwu"] = torch.empty_like(s["wg"]), torch.empty_like(s["wu"])
    return s


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    import ring_allreduce_compressed_gb300 as rra
    op = s["op"]
    if op == "save":
        rra.layer_norm_save(s["x"], s["gamma"], s["beta"], s["y"],
                            rra.Saved(s["exps"], s["codes"], s["dim"]), s["mean"], s["rstd"],
                            eps=EPS)
        return s["y"], s["exps"], s["codes"], s["mean"], s["rstd"]
    if op == "restore":
        rra.layer_norm_restore(rra.Saved(s["exps"], s["codes"], s["dim"]), s["y"], s["gamma"],
                               s["beta"], s["mean"], s["rstd"])
        return s["y"]
    if op == "norm_grad":
        rra.layer_norm_saved_grad(s["dy"], rra.Saved(s["exps"], s["codes"], s["dim"]), s["gamma"],
                                  s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"])
        return s["dx"], s["dgamma"], s["dbeta"]
    gate, up = s.get("gate"), s.get("up")
    if s["save"] == "bits8":
        gate, up = rra.Saved(*gate, s["ff"]), rra.Saved(*up, s["ff"])
    if op == "ff":
        rra.gated_ff(s["x"], s["wg"], s["wu"], s["h"], gate, up, act=s["act"])
        if s["save"] == "none":
            return s["h"]
        if s["save"] == "full":
            return s["h"], gate, up
        rra.layer_norm_restore(gate, s["seen"][0])
        rra.layer_norm_restore(up, s["seen"][1])
        return s["h"], s["seen"][0], s["seen"][1]
    rra.gated_ff_grad(s["dh"], s["x"], s["wg"], s["wu"], gate, up, s["dgate"], s["dup"],
                      dx=s["dx"], dw_gate=s["dwg"], dw_up=s["dwu"], h=s["h"], act=s["act"])
    return s["dgate"], s["dup"], s["h"], s["dx"], s["dwg"], s["dwu"]


# ---------------------------------------------------------------- plain forms

def _act(name, g):
    """The activation and its derivative, in the type of g."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if name == "silu":
        t = 1 / (1 + torch.exp(-g))
        return g * t, t * (1 + g * (1 - t))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k, c = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k * (g + c * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * c * g * g)


def _kept(s, name):
    """Gate or up as the backward pass has it, fp32."""
    return s[name].float() if s["save"] == "full" else _decode(*s[name], s["ff"])


def _run_plain(s):
    op, dtype = s["op"], s["dtype"]
    if op in ("ff", "ff_grad"):
        x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
        if op == "ff":
            gate, up = x @ wg.t(), x @ wu.t()
            h = (_act(s["act"], gate)[0] * up).to(dtype)
            if s["save"] == "none":
                return h
            if s["save"] == "full":
                return h, gate.to(dtype), up.to(dtype)
            return (h,) + tuple(_decode(*_encode(v), s["ff"]).to(torch.bfloat16)
                                for v in (gate, up))
        gate, up, dh = _kept(s, "gate"), _kept(s, "up"), s["dh"].float()
        a, slope = _act(s["act"], gate)
        dgate, dup = dh * up * slope, dh * a
        return ((dgate.to(dtype), dup.to(dtype), (a * up).to(dtype),
                 (dgate @ wg + dup @ wu).to(dtype), (dgate.t() @ x).to(dtype),
                 (dup.t() @ x).to(dtype)))
    gamma = s["gamma"].float()
    if op == "save":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = xc * rstd * gamma + s["beta"].float()
        exps, codes = _encode(x)
        return y.to(dtype), exps, codes, mean.reshape(-1), rstd.reshape(-1)
    rstd = s["rstd"].unsqueeze(1)
    xh = (_decode(s["exps"], s["codes"], s["dim"]) - s["mean"].unsqueeze(1)) * rstd
    if op == "restore":
        return (xh * gamma + s["beta"].float()).to(dtype)
    dy = s["dy"].float()
    w = dy * gamma
    dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    return (dx.to(dtype), (dy * xh).sum(0).to(s["gamma"].dtype),
            dy.sum(0).to(s["gamma"].dtype))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    op, rows, dim, es = case["op"], case["rows"], case["dim"], _size(case["dtype"])
    if op in ("ff", "ff_grad"):
        ff = case["ff"]
        kept = {"none": 0, "full": es, "bits8": 1 + 1 / BLOCK}[case["save"]] * 2 * rows * ff
        if op == "ff":  # (the values that stand for 8 bits are read and written besides)
            seen = 2 * rows * ff * (3 + 1 / BLOCK) if case["save"] == "bits8" else 0
            return {"bytes": (rows * dim + 2 * ff * dim + rows * ff) * es + kept + seen,
                    "flops": 4 * rows * ff * dim + 8 * rows * ff}
        return {"bytes": (2 * rows * dim + 4 * ff * dim + 4 * rows * ff) * es + kept,
                "flops": 8 * rows * ff * dim + 16 * rows * ff}
    n, ws = rows * dim, _size(case["weight"])
    if op == "save":
        return {"bytes": n * (2 * es + 1 + 1 / BLOCK) + 2 * dim * ws + 8 * rows, "flops": 9 * n}
    if op == "restore":
        return {"bytes": n * (es + 1 + 1 / BLOCK) + 2 * dim * ws + 8 * rows, "flops": 5 * n}
    return {"bytes": n * (2 * es + 1 + 1 / BLOCK) + 3 * dim * ws + 8 * rows, "flops": 13 * n}


# ---------------------------------------------------------------- in 64 bits

def _exact_power(n):
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_codes(x):
    """Exponents and codes of x, from the definition: the exponent of a block's largest magnitude,
    and the nearest whole numbers of its 64ths."""
    rows, dim = x.shape
    n = -(-dim // BLOCK)
    b = torch.zeros(rows, n * BLOCK, dtype=torch.float64, device=x.device)
    b[:, :dim] = x
    top = b.abs().reshape(rows, n, BLOCK).max(2).values
    e = torch.where(top > 0, torch.frexp(top).exponent - 1, -126).clamp(min=-126)
    unit = _exact_power(e.long() - 6).repeat_interleave(BLOCK, 1)
    return e.to(torch.int8), torch.clamp(torch.round(b / unit), -127, 127).to(torch.int8)


def _exact_values(exps, codes, dim):
    unit = _exact_power(exps.long() - 6)
    return (codes.double() * unit.repeat_interleave(BLOCK, 1))[:, :dim]


def _exact_act(name, g):
    if name == "relu":
        return torch.where(g > 0, g, 0.0), torch.where(g > 0, 1.0, 0.0).double()
    if name == "silu":
        t = torch.sigmoid(g)
        return g * t, t + g * t * torch.sigmoid(-g)
    if name == "gelu":
        cdf = torch.erfc(-g / math.sqrt(2)) / 2
        return g * cdf, cdf + g * torch.exp(-g * g / 2 - 0.5 * math.log(2 * math.pi))
    # 1 + tanh(z) is twice the logistic function of 2 z
    z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    t = torch.sigmoid(z)
    return g * t, t + g * t * torch.sigmoid(-z) * math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("ff", "ff_grad"):
        x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
        if op == "ff":
            gate, up = torch.mm(x, wg.mT), torch.mm(x, wu.mT)
            h = _exact_act(s["act"], gate)[0] * up
            if s["save"] == "none":
                return h
            if s["save"] == "full":
                return h, gate, up
            # a value next to a border between two codes may be given either
            return h, None, None
        gate, up = (s[k].double() if s["save"] == "full" else _exact_values(*s[k], s["ff"])
                    for k in ("gate", "up"))
        a, slope = _exact_act(s["act"], gate)
        dh = s["dh"].double()
        dup, dgate = torch.mul(dh, a), torch.mul(dh, up).mul(slope)
        return (dgate, dup, a * up, torch.addmm(torch.mm(dup, wu), dgate, wg),
                torch.mm(dgate.mT, x), torch.mm(dup.mT, x))
    gamma = s["gamma"].double()
    if op == "save":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], gamma)
        exps, codes = _exact_codes(x)
        return y, exps, codes, mean, rstd
    rstd = s["rstd"].double()[:, None]
    v = _exact_values(s["exps"], s["codes"], s["dim"])
    xh = torch.addcmul(-s["mean"].double()[:, None] * rstd, v, rstd)
    if op == "restore":
        return torch.addcmul(s["beta"].double(), xh, gamma)
    dy = s["dy"].double()
    a = dy @ gamma / s["dim"]
    b = torch.einsum("rd,rd,d->r", dy, xh, gamma) / s["dim"]
    dx = rstd * (dy * gamma - a[:, None] - xh * b[:, None])
    return dx, torch.einsum("rd,rd->d", dy, xh), dy.sum(0)
