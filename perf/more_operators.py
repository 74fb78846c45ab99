"""Timing cases of the experts' gated feed-forward block in training and of the update of its weights.

The block's forward (gate and up projection, activation, product, down projection) that keeps
what its gradient needs, the gradient of its data path, the orthogonalisation of a batch of
matrices by Newton-Schulz products, and the momentum update of weights that applies it.  Each
case runs in a plain form (elementary torch operations in 32 bits, rounded once at the end) or,
with ``own`` set, through the calls of this package.

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

STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)   # of an odd quintic that drives singular values towards 1
EPS = 1e-7
MU, LR, DECAY = 0.95, 0.02, 0.01
BF16 = torch.bfloat16
_DTYPES = {"bf16": BF16, "f32": torch.float32}


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest layer's training step: what a call costs besides its work
        dict(name="gated tiny", op="gated", a=64, E=8, D=256, H=512, act="silu", skew="uniform", valid=64),
        # a decode batch through 16 large experts with the other activation: one read of the weights
        dict(name="gated decode gelu", op="gated", a=128, E=16, D=5120, H=8192, act="gelu", skew="uniform", valid=128),
        # 4096 tokens at top 8 on 128 fine-grained experts, loads as uneven as a router leaves them
        dict(name="gated fine-grained", op="gated", a=32768, E=128, D=7168, H=2048, act="silu", skew="zipf",
             valid=32768),
        # a few odd rows on small experts, with rows behind the last expert's
        dict(name="gated grad ragged", op="gated_grad", a=517, E=5, D=272, H=208, act="gelu", skew="empty", valid=451),
        # 8192 tokens at top 1 on 16 large experts, 512 rows each
        dict(name="gated grad large", op="gated_grad", a=8192, E=16, D=5120, H=8192, act="silu", skew="uniform",
             valid=8192),
        # a padded batch at top 4 on 128 experts, about 344 rows each
        dict(name="gated grad padded", op="gated_grad", a=65536, E=128, D=4096, H=1536, act="silu", skew="uniform",
             valid=44000),
        # one router's gradient: a flat matrix, many short steps
        dict(name="orthogonal router", op="orthogonal", B=1, N=128, K=7168, dtype="bf16"),
        # fp32 gradients of odd sizes
        dict(name="orthogonal odd f32", op="orthogonal", B=3, N=517, K=1003, dtype="f32"),
        # down projections of 8 fine-grained experts
        dict(name="orthogonal w2", op="orthogonal", B=8, N=7168, K=2048, dtype="bf16"),
        # the smallest layer's gate and up projections
        dict(name="update tiny", op="update", B=16, N=512, K=256, dtype="bf16"),
        # gate and up projections of 8 fine-grained experts
        dict(name="update w13", op="update", B=16, N=2048, K=7168, dtype="bf16"),
        # down projections of two large experts, fp32 gradients summed over micro-batches
        dict(name="update w2 large f32", op="update", B=2, N=5120, K=8192, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated_grad", "orthogonal", "update"])
    while True:
        if op in ("gated", "gated_grad"):
            a, E = _log_int(rng, 1, 65536), _log_int(rng, 1, 128)
            D, H = _log_int(rng, 4, 512) * 16, _log_int(rng, 4, 512) * 16
            valid = a if rng.random() < 0.6 else rng.randint(max(1, a // 2), a)
            if 3 * E * D * H <= 5.6e9 and 6 * valid * D * H <= 2.9e12:
                return dict(op=op, a=a, E=E, D=D, H=H, act=rng.choice(["silu", "gelu"]),
                            skew=rng.choice(["uniform", "zipf", "empty"]), valid=valid)
        else:
            B, N, K = _log_int(rng, 1, 64), _log_int(rng, 16, 8192), _log_int(rng, 16, 8192)
            c = dict(op=op, B=B, N=N, K=K, dtype=rng.choice(["bf16", "f32"]))
            if B * N * K <= 2.4e8 and _iteration_flops(c) <= 1e13:
                return c


# ------------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _expert_counts(c, g):
    """Rows per expert: even, Zipf-like, or even with every third expert empty; they add up to `valid`."""
    w = torch.rand(c["E"], generator=g, device="cuda") * 0.2 + 0.9
    if c["skew"] == "zipf":
        w = 1.0 / (1 + torch.randperm(c["E"], generator=g, device="cuda")).float()
    elif c["skew"] == "empty":
        w[1::3] = 0
    ends = (torch.cumsum(w.double(), 0) / w.double().sum() * c["valid"]).round().to(torch.int64)
    return torch.diff(ends, prepend=ends.new_zeros(1)).to(torch.int32)


def _gradient(g, c):
    """Gradients of a batch of matrices: a few strong directions over a weaker rest, rows of unequal size."""
    B, N, K = c["B"], c["N"], c["K"]
    r = min(24, N, K)
    strength = 1 / (1 + torch.arange(r, device="cuda").float())
    v = (_randn(g, B, N, r) * strength) @ _randn(g, B, r, K)
    v = (v + 0.2 * _randn(g, B, N, K)) * torch.exp(0.4 * _randn(g, B, N, 1))
    return (1e-3 * v).to(_DTYPES[c["dtype"]])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] in ("gated", "gated_grad"):
        a, E, D, H = c["a"], c["E"], c["D"], c["H"]
        s["w13"] = _randn(g, E, 2 * H, D, dtype=BF16).mul_(1 / math.sqrt(D))
        s["w2"] = _randn(g, E, D, H, dtype=BF16).mul_(1 / math.sqrt(H))
        s["counts"] = _expert_counts(c, g)
        s["rows"] = s["counts"].tolist()     # the plain form's split of the rows
        zeros = lambda *shape: torch.zeros(*shape, dtype=BF16, device="cuda")
        s["y"] = zeros(a, 2 * H)
        if c["op"] == "gated":
            s["x"] = _randn(g, a, D, dtype=BF16)
            s["out"] = zeros(a, D)
        else:
            s["y"].copy_(_randn(g, a, 2 * H, dtype=BF16).mul_(1.5))
            s["dout"] = (0.1 * _randn(g, a, D)).to(BF16)
            s["dx"], s["dy"], s["z"] = zeros(a, D), zeros(a, 2 * H), zeros(a, H)
    else:
        s["grad"] = _gradient(g, c)
        if c["op"] == "orthogonal":
            s["out"] = torch.zeros(c["B"], c["N"], c["K"], dtype=BF16, device="cuda")
        else:
            s["w"] = _randn(g, c["B"], c["N"], c["K"], dtype=BF16).mul_(0.02)
            s["momentum"] = 5 * _gradient(g, c).float()
    return s


# ------------------------------------------------------------------- plain forms

def _activation(v, act):
    """act(v) and its slope: v * sigmoid(v), or the tanh form of the Gaussian error unit."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return v * s, s * (1 + v * (1 - s))
    k = math.sqrt(2 / math.pi)
    t = 1 - 2 / (1 + torch.exp(2 * k * (v + 0.044715 * v * v * v)))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


def _grouped(x, w, rows):
    """Each expert's rows times its own matrix: x_e @ w[e]^T."""
    return torch.cat([a @ m.float().T for a, m in zip(x.split(rows), w)])


def _plain_gated(s, c):
    n, H = c["valid"], c["H"]
    y = _grouped(s["x"][:n].float(), s["w13"], s["rows"])
    z = _activation(y[:, :H], c["act"])[0] * y[:, H:]
    s["y"][:n] = y.to(BF16)
    s["out"][:n] = _grouped(z, s["w2"], s["rows"]).to(BF16)
    return [s["out"], s["y"]]


def _plain_gated_grad(s, c):
    n, H = c["valid"], c["H"]
    y = s["y"][:n].float()
    y0, y1 = y[:, :H], y[:, H:]
    dz = _grouped(s["dout"][:n].float(), s["w2"].transpose(1, 2), s["rows"])
    f, slope = _activation(y0, c["act"])
    dy = torch.cat([dz * y1 * slope, dz * f], 1)
    s["dx"][:n] = _grouped(dy, s["w13"].transpose(1, 2), s["rows"]).to(BF16)
    s["dy"][:n] = dy.to(BF16)
    s["z"][:n] = (f * y1).to(BF16)
    return [s["dx"], s["dy"], s["z"]]


def _plain_orthogonalise(u):
    """The quintic of X = u / |u|, STEPS times, on the shorter side's products."""
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if tall else u
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if tall else x


def _plain_orthogonal(s, c):
    s["out"].copy_(_plain_orthogonalise(s["grad"].float()))
    return s["out"]


def _plain_update(s, c):
    g = s["grad"].float()
    s["momentum"].mul_(MU).add_(g)
    o = _plain_orthogonalise(g + MU * s["momentum"])
    w = s["w"].float()
    s["w"].copy_(w - LR * (DECAY * w + o))
    return [s["w"], s["momentum"]]


_PLAIN = dict(gated=_plain_gated, gated_grad=_plain_gated_grad, orthogonal=_plain_orthogonal, update=_plain_update)


# --------------------------------------------------------------- the package's calls

def _own(s, c):
    from moe_token_routing_index_gb300 import binding as mb

    op = c["op"]
    if op in ("gated", "gated_grad"):
        act = mb.MOE_ACT_SILU if c["act"] == "silu" else mb.MOE_ACT_GELU
        if op == "gated":
            return list(mb.moe_gated_mlp(s["x"], s["w13"], s["w2"], s["counts"], activation=act, y=s["y"],
                                         out=s["out"]))
        return list(mb.moe_gated_mlp_backward(s["dout"], s["y"], s["w13"], s["w2"], s["counts"], activation=act,
                                              out=s["dx"], dy=s["dy"], z=s["z"]))
    if op == "orthogonal":
        return mb.moe_orthogonalize(s["grad"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS, out=s["out"])
    mb.moe_muon_update(s["w"], s["grad"], s["momentum"], lr=LR, mu=MU, nesterov=True, weight_decay=DECAY, steps=STEPS,
                       coefficients=COEFFICIENTS, eps=EPS)
    return [s["w"], s["momentum"]]


def run(state):
    c = state["case"]
    return _own(state, c) if own else _PLAIN[c["op"]](state, c)


# ------------------------------------------------------------------------- 64 bits

def _exact_act(v, act):
    """(act(v), act'(v)) in 64 bits: both are v * sigmoid(u(v)), with u = v or an odd cubic."""
    if act == "silu":
        u, du = v, torch.ones_like(v)
    else:
        r = math.sqrt(8 / math.pi)
        u, du = torch.addcmul(r * v, v * v, v, value=r * 0.044715), r + 3 * r * 0.044715 * v * v
    p = torch.sigmoid(u)
    return v * p, torch.addcmul(p, v * p * torch.sigmoid(-u), du)


def _exact_orthogonalise(u):
    """The iteration in Horner's form on the smaller of the two products with the transpose."""
    x = u / (torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True) + EPS)
    a, b, c = COEFFICIENTS
    right = u.shape[1] > u.shape[2]
    eye = torch.eye(min(u.shape[1:]), dtype=torch.float64, device=u.device).expand(len(u), -1, -1)
    for _ in range(STEPS):
        m = torch.einsum("bki,bkj->bij", x, x) if right else torch.einsum("bik,bjk->bij", x, x)
        p = torch.baddbmm(eye, torch.baddbmm(eye, m, eye, beta=b, alpha=c), m, beta=a)
        x = torch.bmm(x, p) if right else torch.bmm(p, x)
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op in ("gated", "gated_grad"):
        H, start = c["H"], 0
        wide = lambda cols: torch.zeros(c["a"], cols, dtype=torch.float64, device="cuda")
        out, y, z = wide(c["D"]), wide(2 * H), wide(H)
        for e, rows in enumerate(s["rows"]):
            at = slice(start, start + rows)
            start += rows
            if rows == 0:
                continue
            w13, w2 = s["w13"][e].double(), s["w2"][e].double()
            if op == "gated":
                y[at] = torch.einsum("rd,nd->rn", s["x"][at].double(), w13)
                out[at] = torch.einsum("rh,dh->rd", _exact_act(y[at, :H], c["act"])[0] * y[at, H:], w2)
            else:
                kept = s["y"][at].double()
                dz = torch.mm(s["dout"][at].double(), w2)
                f, slope = _exact_act(kept[:, :H], c["act"])
                y[at, :H] = dz * kept[:, H:] * slope
                y[at, H:] = dz * f
                z[at] = f * kept[:, H:]
                out[at] = torch.mm(y[at], w13)
        return [out, y] if op == "gated" else [out, y, z]
    g = s["grad"].double()
    if op == "orthogonal":
        return _exact_orthogonalise(g)
    m = torch.add(g, s["momentum"].double(), alpha=MU)
    o = _exact_orthogonalise(torch.add(g, m, alpha=MU))
    return [s["w"].double() * (1 - LR * DECAY) - LR * o, m]


# ---------------------------------------------------------------------------- work

def _iteration_flops(c):
    """Of the products: the two that are symmetric need one half of their elements."""
    m, n = min(c["N"], c["K"]), max(c["N"], c["K"])
    return STEPS * c["B"] * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)


def work(case):
    c = case
    if c["op"] in ("gated", "gated_grad"):
        n, D, H = c["valid"], c["D"], c["H"]
        full = c["E"] - len(range(1, c["E"], 3)) if c["skew"] == "empty" else c["E"]
        weights = 2 * 3 * min(full, n) * D * H
        # forward: x, y and the output; gradient: its input, y, dy, z and dx
        rows = 2 * n * (2 * D + 2 * H) if c["op"] == "gated" else 2 * n * (2 * D + 5 * H)
        return {"bytes": weights + rows + 4 * c["E"], "flops": 6 * n * D * H}
    e, size = _DTYPES[c["dtype"]].itemsize, c["B"] * c["N"] * c["K"]
    # gradient and result; for an update also the momentum and the weights, read and written
    return {"bytes": size * (e + 2 if c["op"] == "orthogonal" else e + 8 + 4), "flops": _iteration_flops(c)}
