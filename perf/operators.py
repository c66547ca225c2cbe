"""What is measured of the training-step operators around the ring: the gradient norm with
clipping, the embedding lookup with its gradient, and layer norm with its gradient."""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NORMS = {"l2": 2, "l1": 1, "inf": math.inf}
EPS_CLIP = 1e-6
EPS_NORM = 1e-5
MOST_BYTES = 2_250_000_000  # of one drawn case's gradients: below the largest listed one's


def listed():
    return [
        # one small parameter's gradient, fp32: the call's own latency
        dict(name="clip_small", op="clip", total=4096, buckets=1, dtype="f32", norm="l2", offset=0),
        # the 25 MiB fp16 gradient bucket of the compressed ring
        dict(name="clip_bucket", op="clip", total=13_107_200, buckets=1, dtype="f16", norm="l2",
             offset=0),
        # a whole model's gradients: bf16 buckets of uneven, odd sizes, every fourth one fp32
        dict(name="clip_model", op="clip", total=1_000_000_000, buckets=40, dtype="mixed",
             norm="l2", offset=0),
        # lookup of a few tokens, one step of decoding
        dict(name="embed_step", op="embed", tokens=16, vocab=32_000, dim=4096, dtype="bf16",
             index="i64"),
        # lookup of a training batch
        dict(name="embed_batch", op="embed", tokens=32_768, vocab=128_000, dim=2048, dtype="bf16",
             index="i64"),
        # a small table with an odd width, fp32, with a padding token
        dict(name="embed_grad_small", op="embed_grad", tokens=200, vocab=1000, dim=513,
             dtype="f32", out="f32", index="i64", padding=0),
        # a training batch, bf16 gradients
        dict(name="embed_grad_batch", op="embed_grad", tokens=16_384, vocab=50_000, dim=2048,
             dtype="bf16", out="bf16", index="i64", padding=-1),
        # a long batch over a large vocabulary, bf16 activations, fp32 weight gradients
        dict(name="embed_grad_long", op="embed_grad", tokens=131_072, vocab=128_000, dim=1024,
             dtype="bf16", out="f32", index="i32", padding=-1),
        # a few rows, one step of decoding
        dict(name="norm_step", op="norm", rows=32, dim=1024, dtype="f16", weight="f16"),
        # a training batch's activations
        dict(name="norm_batch", op="norm", rows=16_384, dim=4096, dtype="bf16", weight="bf16"),
        # an fp32 model with odd sizes
        dict(name="norm_grad_ragged", op="norm_grad", rows=3001, dim=1001, dtype="f32",
             weight="f32"),
        # a training batch's backward pass
        dict(name="norm_grad_batch", op="norm_grad", rows=16_384, dim=4096, dtype="bf16",
             weight="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm; about every second one odd."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["clip", "embed", "embed_grad", "embed_grad", "norm", "norm_grad"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "clip":
        dtype = rng.choice(["f32", "f16", "bf16", "mixed"])
        most = MOST_BYTES // {"f32": 4, "mixed": 3}.get(dtype, 2)
        total = _spread(rng, 1, most)
        return dict(op=op, total=total, buckets=rng.randint(1, min(48, total)), dtype=dtype,
                    norm=rng.choice(["l2", "l2", "l1", "inf"]), offset=rng.choice([0, 0, 1]))
    index = rng.choice(["i32", "i64"])
    if op in ("embed", "embed_grad"):
        dim = rng.choice([_spread(rng, 1, 8192), 64 * rng.randint(1, 96)])
        tokens = _spread(rng, 1, min(262_144, (1 << 27) // dim))
        vocab = _spread(rng, 2, min(200_000, (1 << 27) // dim))
        if op == "embed":
            return dict(op=op, tokens=tokens, vocab=vocab, dim=dim, dtype=dtype, index=index)
        return dict(op=op, tokens=tokens, vocab=vocab, dim=dim, dtype=dtype,
                    out=rng.choice([dtype, "f32"]), index=index, padding=rng.choice([-1, -1, 0]))
    dim = rng.choice([_spread(rng, 2, 16_384), 64 * rng.randint(1, 128)])
    rows = _spread(rng, 1, min(131_072, (1 << 26) // dim))
    return dict(op=op, rows=rows, dim=dim, dtype=dtype, weight=rng.choice([dtype, "f32"]))


def _buckets(case):
    """(count, dtype name) of every gradient bucket: uneven sizes that add up to the total."""
    n, total = case["buckets"], case["total"]
    share = np.random.RandomState(n).uniform(0.5, 1.5, n)
    ends = np.floor(np.cumsum(share) / share.sum() * total).astype(np.int64)
    ends[-1] = total
    counts = np.diff(ends, prepend=0).tolist()
    kinds = ["f32" if i % 4 == 3 else "bf16" for i in range(n)] if case["dtype"] == "mixed" \
        else [case["dtype"]] * n
    return list(zip(counts, kinds))


def _normal(shape, gen, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _tokens(case, gen):
    """Token numbers as text has them: the frequency falls with the number (log-uniform)."""
    u = torch.rand(case["tokens"], generator=gen, device="cuda", dtype=torch.float64)
    t = torch.exp(u * math.log(case["vocab"] + 1)).floor().long() - 1
    t = t.clamp(0, case["vocab"] - 1)
    return t.to(torch.int32 if case["index"] == "i32" else torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(op=op)
    if op == "clip":
        std, total, off = 1e-3, case["total"], case["offset"]
        kinds = _buckets(case)
        s["grads"] = [_normal(off + n, gen, std, TYPES[k])[off:] for n, k in kinds]
        s["outs"] = [torch.empty(off + n, device="cuda", dtype=TYPES[k])[off:] for n, k in kinds]
        s["norm"] = torch.empty(1, device="cuda")
        s["kind"] = case["norm"]
        # half of what the norm is expected to be: the gradients are clipped
        s["max_norm"] = {"l2": 0.5 * std * math.sqrt(total), "l1": 0.4 * std * total,
                         "inf": 2 * std}[case["norm"]]
        return s
    if op in ("embed", "embed_grad"):
        s["tokens"] = _tokens(case, gen)
        s["scale"] = math.sqrt(case["dim"])
        dtype = TYPES[case["dtype"]]
        if op == "embed":
            s["weight"] = _normal((case["vocab"], case["dim"]), gen, 0.02, dtype)
            s["out"] = torch.empty(case["tokens"], case["dim"], device="cuda", dtype=dtype)
        else:
            s["dout"] = _normal((case["tokens"], case["dim"]), gen, 1e-2, dtype)
            s["dweight"] = torch.empty(case["vocab"], case["dim"], device="cuda",
                                       dtype=TYPES[case["out"]])
            s["padding"] = case["padding"] if case["padding"] >= 0 else None
        return s
    rows, dim, dtype, wtype = case["rows"], case["dim"], TYPES[case["dtype"]], TYPES[case["weight"]]
    s["x"] = (torch.randn(rows, dim, generator=gen, device="cuda") * 1.5 + 0.25).to(dtype)
    s["gamma"] = (1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(wtype)
    if op == "norm":
        s["beta"] = _normal(dim, gen, 0.1, wtype)
        s["y"] = torch.empty_like(s["x"])
        s["mean"] = torch.empty(rows, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        return s
    # what the forward pass has left for the backward pass
    x = s["x"].double()
    s["mean"] = x.mean(1).float()
    s["rstd"] = (x.var(1, unbiased=False) + EPS_NORM).rsqrt().float()
    s["dy"] = _normal((rows, dim), gen, 1e-2, dtype)
    s["dx"] = torch.empty_like(s["x"])
    s["dgamma"] = torch.empty_like(s["gamma"])
    s["dbeta"] = torch.empty_like(s["gamma"])
    return s


def _run_own(s):
    import ring_allreduce_compressed_gb300 as rra
    op = s["op"]
    if op == "clip":
        rra.grad_clip(s["grads"], s["outs"], s["max_norm"], s["norm"], norm_type=NORMS[s["kind"]],
                      eps=EPS_CLIP)
        return [s["norm"]] + s["outs"]
    if op == "embed":
        rra.embedding(s["weight"], s["tokens"], s["out"], scale=s["scale"])
        return s["out"]
    if op == "embed_grad":
        rra.embedding_grad(s["dout"], s["tokens"], s["dweight"], scale=s["scale"],
                           padding_idx=s["padding"])
        return s["dweight"]
    if op == "norm":
        rra.layer_norm(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], eps=EPS_NORM)
        return s["y"], s["mean"], s["rstd"]
    rra.layer_norm_grad(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"],
                        s["dbeta"])
    return s["dx"], s["dgamma"], s["dbeta"]


def _run_plain(s):
    op = s["op"]
    if op == "clip":
        if s["kind"] == "l2":
            norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
        elif s["kind"] == "l1":
            norm = torch.stack([g.float().abs().sum() for g in s["grads"]]).sum()
        else:
            norm = torch.stack([g.float().abs().max() for g in s["grads"]]).max()
        c = (s["max_norm"] / (norm + EPS_CLIP)).clamp(max=1.0)
        return [norm.reshape(1)] + [(g.float() * c).to(g.dtype) for g in s["grads"]]
    if op == "embed":
        return (s["weight"][s["tokens"].long()].float() * s["scale"]).to(s["weight"].dtype)
    if op == "embed_grad":
        rows = s["dout"].float() * s["scale"]
        if s["padding"] is not None:
            rows = rows * (s["tokens"] != s["padding"]).float().unsqueeze(1)
        dw = torch.zeros(s["dweight"].shape, device="cuda")
        return dw.index_add_(0, s["tokens"], rows).to(s["dweight"].dtype)
    x, gamma = s["x"].float(), s["gamma"].float()
    if op == "norm":
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + EPS_NORM).rsqrt()
        y = xc * rstd * gamma + s["beta"].float()
        return y.to(s["x"].dtype), mean.reshape(-1), rstd.reshape(-1)
    rstd = s["rstd"].unsqueeze(1)
    xh = (x - s["mean"].unsqueeze(1)) * rstd
    dy = s["dy"].float()
    w = dy * gamma
    dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    return (dx.to(s["x"].dtype), (dy * xh).sum(0).to(s["gamma"].dtype),
            dy.sum(0).to(s["gamma"].dtype))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _distinct(case):
    """Expected number of different tokens among the drawn ones."""
    v = np.arange(case["vocab"], dtype=np.float64)
    p = np.log1p(1 / (v + 1)) / math.log(case["vocab"] + 1)
    return float(-np.expm1(case["tokens"] * np.log1p(-p)).sum())


def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    op = case["op"]
    if op == "clip":
        return {"bytes": 2 * sum(n * _size(k) for n, k in _buckets(case)) + 4,
                "flops": 3 * case["total"]}
    if op in ("embed", "embed_grad"):
        n, d = case["tokens"], case["dim"]
        ids = n * (4 if case["index"] == "i32" else 8)
        if op == "embed":
            return {"bytes": ids + (_distinct(case) + n) * d * _size(case["dtype"]),
                    "flops": n * d}
        return {"bytes": ids + n * d * _size(case["dtype"])
                + case["vocab"] * d * _size(case["out"]), "flops": n * d}
    rows, dim, es, ws = case["rows"], case["dim"], _size(case["dtype"]), _size(case["weight"])
    if op == "norm":
        return {"bytes": 2 * rows * dim * es + 2 * dim * ws + 8 * rows, "flops": 7 * rows * dim}
    return {"bytes": 3 * rows * dim * es + 3 * dim * ws + 8 * rows, "flops": 12 * rows * dim}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "clip":
        mags = [torch.linalg.vector_norm(g.double(), NORMS[s["kind"]]) for g in s["grads"]]
        norm = torch.linalg.vector_norm(torch.stack(mags), NORMS[s["kind"]])
        c = min(1.0, s["max_norm"] / (float(norm) + EPS_CLIP))
        return [norm.reshape(1)] + [g.double() * c for g in s["grads"]]
    if op == "embed":
        return torch.index_select(s["weight"], 0, s["tokens"]).double() * s["scale"]
    if op == "embed_grad":
        keep = torch.nonzero(s["tokens"] != (-1 if s["padding"] is None else s["padding"]))[:, 0]
        dw = torch.zeros(s["dweight"].shape, device="cuda", dtype=torch.float64)
        return dw.index_put_((s["tokens"][keep].long(),), s["dout"][keep].double() * s["scale"],
                             accumulate=True)
    x, gamma = s["x"].double(), s["gamma"].double()
    if op == "norm":
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS_NORM)
        y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], gamma)
        return y, mean, rstd
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    xh = (x - s["mean"].double()[:, None]) * rstd
    a = dy @ gamma / x.shape[1]
    b = torch.einsum("rd,rd,d->r", dy, xh, gamma) / x.shape[1]
    dx = rstd * (dy * gamma - a[:, None] - xh * b[:, None])
    return dx, torch.einsum("rd,rd->d", dy, xh), dy.sum(0)
