"""Plain 64-bit forms of the gated feed-forward block and of the orthogonalised update (tests only),
with the bounds that follow from the operators' own roundings."""
from __future__ import annotations

import math

import torch

HALF16 = 2.0 ** -8        # half a bf16 step, relative
HALF_FP16 = 2.0 ** -11    # half an fp16 step, relative
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def act(v: torch.Tensor, kind: str) -> torch.Tensor:
    u = v if kind == "silu" else math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)
    return v * torch.sigmoid(u)


def slope(v: torch.Tensor, kind: str) -> torch.Tensor:
    """act'(v) by autograd, in 64 bits."""
    v = v.detach().clone().requires_grad_()
    return torch.autograd.grad(act(v, kind).sum(), v)[0]


def experts(counts, a: int):
    """(expert, rows) of each expert's rows, cut at a."""
    start = 0
    for e, c in enumerate(counts):
        end = min(a, start + max(0, c))
        yield e, slice(start, end)
        start = end


def forward(x, w13, w2, counts, kind: str):
    """(out, y) and the largest errors that the kernels' roundings allow, all [a, .] in 64 bits; rows of no expert
    are zero.  fp32 sums of n products: n 2^-22 of the sum of their sizes (tensor cores may cut, not round)."""
    x, w13, w2 = x.double(), w13.double(), w2.double()
    H, D = w2.shape[2], w2.shape[1]
    a = len(x)
    y, ey = torch.zeros(a, 2 * H).double(), torch.zeros(a, 2 * H).double()
    out, eo = torch.zeros(a, D).double(), torch.zeros(a, D).double()
    for e, at in experts(counts, a):
        y[at] = x[at] @ w13[e].T
        acc = D * 2.0 ** -22 * (x[at].abs() @ w13[e].abs().T)        # of y before its rounding
        ey[at] = HALF16 * y[at].abs() + acc
        y0, y1 = y[at][:, :H], y[at][:, H:]
        f = act(y0, kind)
        z = f * y1
        # the gate's own arithmetic: sigmoid within 2^-20 (1 + |v|) of itself, slopes of act below 1.2
        ez = (1.2 * acc[:, :H] + 2.0 ** -20 * (1 + y0.abs()) * f.abs()) * y1.abs() + f.abs() * acc[:, H:]
        ez = ez * 1.01 + HALF16 * z.abs()
        out[at] = z @ w2[e].T
        eo[at] = HALF16 * out[at].abs() + 1.01 * (ez @ w2[e].abs().T) + H * 2.0 ** -22 * (z.abs() @ w2[e].abs().T)
    return out, y, eo + 1e-30, ey + 1e-30


def backward(dout, y, w13, w2, counts, kind: str):
    """(dx, dy, z) from the kept y, and the largest errors, as in forward."""
    dout, y, w13, w2 = dout.double(), y.double(), w13.double(), w2.double()
    H, D = w2.shape[2], w2.shape[1]
    a = len(dout)
    dy, edy = torch.zeros(a, 2 * H).double(), torch.zeros(a, 2 * H).double()
    z, dx, edx = torch.zeros(a, H).double(), torch.zeros(a, D).double(), torch.zeros(a, D).double()
    ez = torch.zeros(a, H).double()
    for e, at in experts(counts, a):
        dz = dout[at] @ w2[e]
        acc = D * 2.0 ** -22 * (dout[at].abs() @ w2[e].abs())
        y0, y1 = y[at][:, :H], y[at][:, H:]
        f, s = act(y0, kind), slope(y0, kind)
        own = 2.0 ** -20 * (1 + y0.abs())
        dy[at] = torch.cat([dz * y1 * s, dz * f], 1)
        # the slope's parts may cancel: its own error is absolute, in the size of 1 + |y0| parts of p
        small = torch.cat([acc * (y1 * s).abs() + dz.abs() * y1.abs() * own * (1 + y0.abs()),
                           acc * f.abs() + dz.abs() * own * f.abs()], 1)
        edy[at] = HALF16 * dy[at].abs() + 1.01 * small
        z[at] = f * y1
        ez[at] = HALF16 * z[at].abs() + own * z[at].abs()
        dx[at] = dy[at] @ w13[e]
        edx[at] = HALF16 * dx[at].abs() + 1.01 * (edy[at] @ w13[e].abs()) + 2 * H * 2.0 ** -22 * (dy[at].abs() @ w13[e].abs())
    return dx, dy, z, edx + 1e-30, edy + 1e-30, ez + 1e-30


# ------------------------------------------------------------ orthogonalisation

def _first(g, eps):
    g = g.double()
    return g / (torch.sqrt((g * g).sum((-2, -1), keepdim=True)) + eps)


def orthogonalize(g, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7, half: bool = False):
    """[B, N, K] in 64 bits; half: with the products' operands rounded to fp16 (scaled by 2^10) as the kernels
    round them, and nothing else."""
    a, b, c = coefficients
    tall = g.shape[-2] > g.shape[-1]
    x = _first(g, eps)
    x = x.transpose(-2, -1) if tall else x
    r = (lambda t: (t * 1024).half().double() / 1024) if half else (lambda t: t)
    for _ in range(steps):
        xh = r(x)
        m = r(xh @ xh.transpose(-2, -1))
        x = a * x + r(b * m + c * (m @ m)) @ xh
    return x.transpose(-2, -1) if tall else x


def one_step_error(g, coefficients=COEFFICIENTS, eps: float = 1e-7):
    """The largest error, element by element, of one step with operands in fp16, X in 22 bits and fp32 sums.
    (fp16's least step, 2^-24, is 2^-34 after the scaling.)"""
    a, b, c = coefficients
    tall = g.shape[-2] > g.shape[-1]
    x = _first(g, eps)
    x = x.transpose(-2, -1) if tall else x
    n, m_side = x.shape[-1], x.shape[-2]
    tiny, h = 2.0 ** -35, HALF_FP16 * 1.01
    dx = h * x.abs() + tiny
    ax, at = x.abs(), x.abs().transpose(-2, -1)
    gram = x @ x.transpose(-2, -1)
    dg = h * gram.abs() + tiny + 1.01 * (dx @ at + ax @ dx.transpose(-2, -1)) + n * 2.0 ** -22 * (ax @ at)
    ag = gram.abs()
    p = b * gram + c * (gram @ gram)
    dp = h * p.abs() + tiny + abs(b) * dg + abs(c) * (1.01 * (dg @ ag + ag @ dg) + m_side * 2.0 ** -22 * (ag @ ag))
    out = a * x + p @ x
    d = 1.01 * (dp @ ax + p.abs() @ dx) + m_side * 2.0 ** -22 * (p.abs() @ ax) + abs(a) * (2.0 ** -20 * ax + tiny)
    d = d + HALF16 * out.abs() * 1.01 + 1e-30
    return (out.transpose(-2, -1), d.transpose(-2, -1)) if tall else (out, d)
