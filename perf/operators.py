"""Timing cases of the training-side operators of an MoE block.

Layer norm and its gradient, the load-balance loss of the router and its
gradient, SiLU*mul with an 8-bit checkpoint of its input and the gradient that
reads it back, and the experts' weight gradient.  Each case runs in a plain form
(elementary torch operations in 32 bits, rounded once at the end) or, with
``own`` set, through the calls of this package.

    listed()             the named cases
    draw(rng)            one more case of the same ranges
    prepare(case, seed)  what a program holds before the call, on the GPU
    run(state)           one pass and its outputs
    exact(case, seed)    the same outputs from the definitions in 64 bits
    work(case)           the bytes and operations a pass cannot do without
"""
import math

import torch

own = False

EPS = 1e-5
COEFFICIENT = 0.01
BLOCK = 128                        # columns of a checkpoint row that share one exponent
MIN_EXP, MAX_EXP = -100, 119       # a checkpoint's exponents; stored as exponent + 127
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode batch's norm in front of the router: a call's latency
        dict(name="norm decode", op="norm", T=16, D=5120, dtype="bf16", valid=16),
        # the norm of a padded prefill batch
        dict(name="norm padded", op="norm", T=16384, D=4096, dtype="bf16", valid=11000),
        # its gradient in a training step on 8192 tokens
        dict(name="norm grad train", op="norm_grad", T=8192, D=5120, dtype="bf16", valid=8192),
        # an fp32 model of an odd width on an odd number of tokens
        dict(name="norm grad odd f32", op="norm_grad", T=1003, D=2051, dtype="f32", valid=1003),
        # sigmoid scores of a small step, as the framework's router leaves them
        dict(name="balance small", op="balance", T=128, E=16, top_k=1, kind="scores", dtype="bf16", valid=128),
        # softmax router of many fine-grained experts over a large batch, fp32 logits
        dict(name="balance large", op="balance", T=65536, E=128, top_k=8, kind="softmax", dtype="f32", valid=65536),
        # the gradient for a padded batch's sigmoid logits
        dict(name="balance grad padded", op="balance_grad", T=16384, E=128, top_k=4, kind="sigmoid", dtype="bf16",
             valid=11000),
        # SiLU*mul of fine-grained experts, 4096 tokens at top 8, keeping its input in 8 bits
        dict(name="silu checkpoint", op="silu", a=32768, H=2048, valid=32768),
        # the gradient that reads it back; also a small ragged one
        dict(name="silu grad", op="silu_grad", a=32768, H=2048, valid=32768),
        dict(name="silu grad ragged", op="silu_grad", a=517, H=1456, valid=451),
        # weight gradient of w2 of the fine-grained layer: 128 experts of very uneven load, bound by the write
        dict(name="weight grad w2", op="weight_grad", a=32768, E=128, N=7168, K=2048, skew="zipf", ckpt=False),
        # weight gradient of w13 of 16 large experts, 512 rows each, from the 8-bit rows: bound by the products
        dict(name="weight grad w13 8-bit", op="weight_grad", a=8192, E=16, N=16384, K=5120, skew="uniform", ckpt=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _valid(rng, n):
    return n if rng.random() < 0.6 else rng.randint(max(1, n // 2), n)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "balance", "balance_grad", "silu", "silu_grad", "weight_grad",
                     "weight_grad"])
    if op in ("norm", "norm_grad"):
        T = _log_int(rng, 1, 16384)
        D = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            D = max(16, D // 16 * 16)
        return dict(op=op, T=T, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]), valid=_valid(rng, T))
    if op in ("balance", "balance_grad"):
        T = _log_int(rng, 1, 65536)
        E = _log_int(rng, 2, 256)
        # fewer than all experts are chosen: with all of them the loss is constant and its gradient zero
        return dict(op=op, T=T, E=E, top_k=rng.randint(1, max(1, min(8, E // 2))),
                    kind=rng.choice(["scores", "softmax", "sigmoid"]), dtype=rng.choice(["bf16", "f32"]),
                    valid=_valid(rng, T))
    if op in ("silu", "silu_grad"):
        a = _log_int(rng, 1, 32768)
        return dict(op=op, a=a, H=_log_int(rng, 4, 256) * 16, valid=_valid(rng, a))
    while True:
        a = _log_int(rng, 1, 32768)
        E = _log_int(rng, 1, 128)
        N, K = _log_int(rng, 4, 512) * 16, _log_int(rng, 4, 512) * 16
        if 2 * E * N * K <= 3.7e9 and 2 * a * N * K <= 1.3e12:
            return dict(op=op, a=a, E=E, N=N, K=K, skew=rng.choice(["uniform", "zipf", "empty"]),
                        ckpt=rng.random() < 0.5)


# ------------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _count(n):
    return torch.tensor([n], dtype=torch.int32, device="cuda")


def _activations(g, T, D, dt):
    """Rows of unequal size on channels of unequal offset, as a residual stream has them."""
    size = torch.exp(0.5 * _randn(g, T, 1))
    return (_randn(g, T, D) * size + 0.3 * _randn(g, D)).to(dt)


def _router_input(g, c):
    logits = _randn(g, c["T"], c["E"]) + _randn(g, c["E"])      # some experts are preferred
    if c["kind"] == "scores":
        logits = torch.sigmoid(logits)
    return logits.to(_DTYPES[c["dtype"]])


def _blocks(v):
    """[a, W] -> [a, blocks, 128], the last block filled up with zeros."""
    a, w = v.shape
    return torch.nn.functional.pad(v, (0, -w % BLOCK)).view(a, -1, BLOCK)


def _pack(v):
    """e4m3 codes [a, W] and exponent bytes [a, blocks] of fp32 rows."""
    b = _blocks(v)
    f, p = torch.frexp(b.abs().amax(-1))                          # max = f * 2^p, f in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(f > 0, p - 9 + (f > 0.875), MIN_EXP).clamp(MIN_EXP, MAX_EXP)
    q = b * torch.exp2(-e.float())[..., None]
    codes = q.clamp(-448, 448).view(len(v), -1)[:, : v.shape[1]].contiguous().to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _unpack(codes, exps):
    b = _blocks(codes.float())
    return (b * torch.exp2(exps.float() - 127)[..., None]).view(len(codes), -1)[:, : codes.shape[1]]


def _expert_counts(c, g):
    """Rows per expert: even, Zipf-like, or even with every third expert empty; they add up to a."""
    w = torch.rand(c["E"], generator=g, device="cuda") * 0.2 + 0.9
    if c["skew"] == "zipf":
        w = 1.0 / (1 + torch.randperm(c["E"], generator=g, device="cuda")).float()
    elif c["skew"] == "empty":
        w[1::3] = 0
    ends = (torch.cumsum(w.double(), 0) / w.double().sum() * c["a"]).round().to(torch.int64)
    return torch.diff(ends, prepend=ends.new_zeros(1)).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    op = c["op"]
    if op in ("norm", "norm_grad"):
        dt, T, D = _DTYPES[c["dtype"]], c["T"], c["D"]
        s["x"] = _activations(g, T, D, dt)
        s["gamma"] = (1 + 0.1 * _randn(g, D)).to(dt)
        s["beta"] = (0.1 * _randn(g, D)).to(dt)
        s["valid"] = _count(c["valid"])
        s["out"] = torch.zeros(T, D, dtype=dt, device="cuda")
        s["mean"], s["rstd"] = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
        if op == "norm_grad":
            s["dy"] = _randn(g, T, D).to(dt)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, correction=0) + EPS).rsqrt().float()
    elif op in ("balance", "balance_grad"):
        s["scores"] = _router_input(g, c)
        s["valid"] = _count(c["valid"])
        if op == "balance_grad":
            s["counts"] = _counts(s["scores"][: c["valid"]].float(), c["top_k"])
            s["dloss"] = 1 + torch.rand(1, generator=g, device="cuda")
            s["out"] = torch.zeros_like(s["scores"])
    elif op == "silu":
        a, H = c["a"], c["H"]
        s["y"] = (1.5 * _randn(g, a, 2 * H)).to(torch.bfloat16)
        s["valid"] = _count(c["valid"])
        s["z"] = torch.zeros(a, H, dtype=torch.bfloat16, device="cuda")
        s["codes"] = torch.zeros(a, 2 * H, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s["exps"] = torch.zeros(a, 2 * -(-H // BLOCK), dtype=torch.uint8, device="cuda")
    elif op == "silu_grad":
        a, H = c["a"], c["H"]
        y = (1.5 * _randn(g, a, 2 * H)).to(torch.bfloat16).float()
        (c0, e0), (c1, e1) = _pack(y[:, :H]), _pack(y[:, H:])
        s["codes"] = torch.cat([c0.view(torch.uint8), c1.view(torch.uint8)], 1).view(torch.float8_e4m3fn)
        s["exps"] = torch.cat([e0, e1], 1)
        s["dz"] = (0.1 * _randn(g, a, H)).to(torch.bfloat16)
        s["valid"] = _count(c["valid"])
        s["dy"] = torch.zeros(a, 2 * H, dtype=torch.bfloat16, device="cuda")
        s["z"] = torch.zeros(a, H, dtype=torch.bfloat16, device="cuda")
    else:
        s["dy"] = (0.05 * _randn(g, c["a"], c["N"])).to(torch.bfloat16)
        x = _randn(g, c["a"], c["K"]).to(torch.bfloat16)
        if c["ckpt"]:
            s["codes"], s["exps"] = _pack(x.float())
        else:
            s["x"] = x
        s["counts"] = _expert_counts(c, g)
        s["rows"] = s["counts"].tolist()     # the plain form's split of the rows
    return s


# ------------------------------------------------------------------- plain forms

def _counts(v, k):
    """Per-expert counts of the k largest of each row, equal values to the lower expert, and their sum."""
    E = v.shape[1]
    top = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k].reshape(-1)
    n = torch.zeros(E + 1, dtype=torch.int32, device=v.device)
    n.index_add_(0, top, torch.ones_like(top, dtype=torch.int32))
    n[E] = top.numel()
    return n


def _probs(v, kind):
    if kind == "softmax":
        p = torch.exp(v - v.amax(1, keepdim=True))
    elif kind == "sigmoid":
        p = 1 / (1 + torch.exp(-v))
    else:
        p = v
    total = p.sum(1, keepdim=True)
    return p, total


def _plain_norm(s, c):
    n = c["valid"]
    x = s["x"][:n].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    s["out"][:n], s["mean"][:n], s["rstd"][:n] = y.to(s["out"].dtype), mean, rstd
    return [s["out"], s["mean"], s["rstd"]]


def _plain_norm_grad(s, c):
    n = c["valid"]
    dy, x = s["dy"][:n].float(), s["x"][:n].float()
    xh = (x - s["mean"][:n, None]) * s["rstd"][:n, None]
    g = dy * s["gamma"].float()
    dx = s["rstd"][:n, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    s["out"][:n] = dx.to(s["out"].dtype)
    return [s["out"], (dy * xh).sum(0), dy.sum(0)]


def _plain_balance(s, c):
    v = s["scores"][: c["valid"]].float()
    counts = _counts(v, c["top_k"])
    p, total = _probs(v, c["kind"])
    mean_p = (p / total).mean(0)
    f = counts[:-1].float() * (c["E"] / (c["top_k"] * c["valid"]))
    return [(COEFFICIENT * (f * mean_p).sum()).reshape(1), counts, mean_p]


def _plain_balance_grad(s, c):
    n = c["valid"]
    v = s["scores"][:n].float()
    f = s["counts"][:-1].float() * (c["E"] / (c["top_k"] * n))
    p, total = _probs(v, c["kind"])
    q = p / total
    d = (f - (q * f).sum(1, keepdim=True)) / total * (COEFFICIENT / n * s["dloss"])
    if c["kind"] == "softmax":
        d = d * p
    elif c["kind"] == "sigmoid":
        d = d * p * (1 - p)
    s["out"][:n] = d.to(s["out"].dtype)
    return s["out"]


def _plain_silu(s, c):
    n, H = c["valid"], c["H"]
    y = s["y"][:n].float()
    y0, y1 = y[:, :H], y[:, H:]
    s["z"][:n] = (y0 / (1 + torch.exp(-y0)) * y1).to(torch.bfloat16)
    (c0, e0), (c1, e1) = _pack(y0), _pack(y1)
    codes = s["codes"].view(torch.uint8)
    codes[:n, :H], codes[:n, H:] = c0.view(torch.uint8), c1.view(torch.uint8)
    s["exps"][:n] = torch.cat([e0, e1], 1)
    return [s["z"], s["codes"], s["exps"]]


def _plain_silu_grad(s, c):
    n, H = c["valid"], c["H"]
    nb = -(-H // BLOCK)
    y0 = _unpack(s["codes"][:n, :H], s["exps"][:n, :nb])
    y1 = _unpack(s["codes"][:n, H:], s["exps"][:n, nb:])
    dz = s["dz"][:n].float()
    sg = 1 / (1 + torch.exp(-y0))
    s["dy"][:n, :H] = (dz * y1 * sg * (1 + y0 * (1 - sg))).to(torch.bfloat16)
    s["dy"][:n, H:] = (dz * y0 * sg).to(torch.bfloat16)
    s["z"][:n] = (y0 * sg * y1).to(torch.bfloat16)
    return [s["dy"], s["z"]]


def _plain_weight_grad(s, c):
    x = _unpack(s["codes"], s["exps"]) if c["ckpt"] else s["x"].float()
    dy = s["dy"].float()
    dw = torch.empty(c["E"], c["N"], c["K"], dtype=torch.bfloat16, device="cuda")
    for w, a, b in zip(dw, dy.split(s["rows"]), x.split(s["rows"])):
        w.copy_(a.T @ b)
    return dw


_PLAIN = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, balance=_plain_balance, balance_grad=_plain_balance_grad,
              silu=_plain_silu, silu_grad=_plain_silu_grad, weight_grad=_plain_weight_grad)


# --------------------------------------------------------------- the package's calls

def _own(s, c):
    from moe_token_routing_index_gb300 import binding as mb

    op = c["op"]
    kinds = dict(scores=mb.MOE_BALANCE_SCORES, softmax=mb.MOE_BALANCE_SOFTMAX, sigmoid=mb.MOE_BALANCE_SIGMOID) \
        if op.startswith("balance") else None
    if op == "norm":
        return list(mb.moe_layer_norm(s["x"], s["gamma"], s["beta"], s["valid"], eps=EPS, out=s["out"],
                                      mean=s["mean"], rstd=s["rstd"]))
    if op == "norm_grad":
        return list(mb.moe_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["valid"],
                                               out=s["out"]))
    if op == "balance":
        return list(mb.moe_balance_loss(s["scores"], c["top_k"], s["valid"], kind=kinds[c["kind"]],
                                        coefficient=COEFFICIENT))
    if op == "balance_grad":
        return mb.moe_balance_loss_backward(s["scores"], s["counts"], c["top_k"], s["valid"], kind=kinds[c["kind"]],
                                            coefficient=COEFFICIENT, dloss=s["dloss"], out=s["out"])
    if op == "silu":
        z, ck = mb.moe_silu_mul_checkpoint(s["y"], valid_rows=s["valid"], out=s["z"],
                                           checkpoint=mb.Checkpoint(s["codes"], s["exps"], halves=2))
        return [z, ck.codes, ck.exponents]
    if op == "silu_grad":
        return list(mb.moe_silu_mul_backward(mb.Checkpoint(s["codes"], s["exps"], halves=2), s["dz"],
                                             valid_rows=s["valid"], out=s["dy"], z=s["z"]))
    x = mb.Checkpoint(s["codes"], s["exps"]) if c["ckpt"] else s["x"]
    return mb.moe_grouped_weight_grad(s["dy"], x, s["counts"])


def run(state):
    c = state["case"]
    return _own(state, c) if own else _PLAIN[c["op"]](state, c)


# ------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    c, s, op = case, prepare(case, seed), case["op"]
    n = c.get("valid")
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], s["gamma"].double())
        keep = (torch.arange(c["T"], device="cuda") < n).double()
        return [y * keep[:, None], mean * keep, rstd * keep]
    if op == "norm_grad":
        keep = (torch.arange(c["T"], device="cuda") < n).double()[:, None]
        dy, r = s["dy"].double() * keep, s["rstd"].double()[:, None]
        xh = r * (s["x"].double() - s["mean"].double()[:, None])
        g = dy * s["gamma"].double()
        along = torch.einsum("td,td->t", g, xh)[:, None] / c["D"]
        return [r * (g - g.sum(1, keepdim=True) / c["D"] - along * xh), torch.einsum("td,td->d", dy, xh), dy.sum(0)]
    if op in ("balance", "balance_grad"):
        v, E, k = s["scores"][:n].double(), c["E"], c["top_k"]
        weight = v if c["kind"] == "scores" else torch.exp(v) if c["kind"] == "softmax" else torch.sigmoid(v)
        q = weight / weight.sum(1, keepdim=True)
        if op == "balance":
            # an expert is among the k largest when fewer than k come before it in (value, index) order
            kth = torch.topk(v, k, dim=1).values[:, -1:]
            tied = v == kth
            room = k - (v > kth).sum(1, keepdim=True)
            chosen = (v > kth) | (tied & (torch.cumsum(tied, 1) <= room))
            f = chosen.double().mean(0) * E / k
            counts = torch.cat([chosen.sum(0), chosen.sum().reshape(1)]).to(torch.int32)
            return [(COEFFICIENT * torch.dot(f, q.mean(0))).reshape(1), counts, q.mean(0)]
        f = s["counts"][:E].double() * E / (k * n)
        inner = f[None] - (q @ f)[:, None]
        slope = {"scores": 1 / weight.sum(1, keepdim=True), "softmax": q, "sigmoid": q * torch.sigmoid(-v)}[c["kind"]]
        d = torch.zeros(c["T"], E, dtype=torch.float64, device="cuda")
        d[:n] = COEFFICIENT / n * s["dloss"].double() * slope * inner
        return d
    if op == "silu":
        H = c["H"]
        y = s["y"].double()
        y[n:] = 0
        z = y[:, :H] * torch.sigmoid(y[:, :H]) * y[:, H:]
        halves = torch.nn.functional.pad(y.view(c["a"], 2, H), (0, -H % BLOCK)).view(c["a"], 2, -1, BLOCK)
        top = halves.abs().amax(-1)
        e = torch.ceil(torch.log2(torch.clamp(top, min=2.0**-90) / 448))
        e = torch.where(top > 448 * 2.0**e, e + 1, torch.where(top <= 448 * 2.0 ** (e - 1), e - 1, e))
        e = torch.where(top > 0, e, torch.full_like(e, MIN_EXP))
        codes = (halves / (2.0**e)[..., None]).float().to(torch.float8_e4m3fn).double()
        codes = codes.view(c["a"], 2, -1)[:, :, :H].reshape(c["a"], 2 * H)
        exps = (e + 127).to(torch.uint8).view(c["a"], -1)
        exps[n:] = 0
        return [z, codes, exps]
    if op == "silu_grad":
        H, nb = c["H"], s["exps"].shape[1] // 2
        scale = torch.repeat_interleave(2.0 ** (s["exps"].double() - 127), BLOCK, dim=1).view(c["a"], 2, nb * BLOCK)
        y0, y1 = (s["codes"].double().view(c["a"], 2, H) * scale[:, :, :H]).unbind(1)
        dz = s["dz"].double()
        keep = (torch.arange(c["a"], device="cuda") < n).double()[:, None]
        sg = torch.sigmoid(y0)
        slope = sg + y0 * sg * torch.sigmoid(-y0)
        return [torch.cat([dz * y1 * slope, dz * y0 * sg], 1) * keep, y0 * sg * y1 * keep]
    if c["ckpt"]:
        scale = torch.repeat_interleave(2.0 ** (s["exps"].double() - 127), BLOCK, dim=1)[:, : c["K"]]
        x = s["codes"].double() * scale
    else:
        x = s["x"].double()
    dw = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device="cuda")
    start = 0
    for e, rows in enumerate(s["rows"]):
        torch.mm(s["dy"][start:start + rows].double().T, x[start:start + rows], out=dw[e])
        start += rows
    return dw


# ---------------------------------------------------------------------------- work

def work(case):
    c = case
    op = c["op"]
    if op in ("norm", "norm_grad"):
        n, D = c["valid"], c["D"]
        e = _DTYPES[c["dtype"]].itemsize
        if op == "norm":
            return {"bytes": 2 * n * D * e + 2 * D * e + 8 * n, "flops": 8 * n * D}
        return {"bytes": 3 * n * D * e + D * e + 8 * n + 8 * D, "flops": 14 * n * D}
    if op in ("balance", "balance_grad"):
        n, E = c["valid"], c["E"]
        e = _DTYPES[c["dtype"]].itemsize
        if op == "balance":
            return {"bytes": n * E * e + 8 * E + 8, "flops": 5 * n * E}
        return {"bytes": 2 * n * E * e + 4 * E + 8, "flops": 9 * n * E}
    if op in ("silu", "silu_grad"):
        n, H = c["valid"], c["H"]
        exps = 2 * n * -(-H // BLOCK)
        if op == "silu":
            return {"bytes": n * H * (4 + 2 + 2) + exps, "flops": 10 * n * H}
        return {"bytes": n * H * (2 + 2 + 4 + 2) + exps, "flops": 12 * n * H}
    a, E, N, K = c["a"], c["E"], c["N"], c["K"]
    x = a * K + a * -(-K // BLOCK) if c["ckpt"] else 2 * a * K
    return {"bytes": 2 * a * N + x + 2 * E * N * K + 4 * E, "flops": 2 * a * N * K}
