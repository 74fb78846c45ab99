"""The training operators in 64 bits, from their definitions (torch on the CPU), and the input
generators that their tests share.  Nothing here calls the library."""
from __future__ import annotations

import torch

BLOCK = 128


def gen(seed: int) -> torch.Generator:
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- layer norm

def layer_norm(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * gamma.double()
    return (y if beta is None else y + beta.double()), mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd):
    dy, x = dy.double(), x.double()
    xh = (x - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy * gamma.double()
    dx = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# -------------------------------------------------------------- balance loss

def top_counts(a, k):
    """counts[E + 1] of the k largest of each row, equal values to the lower index."""
    chosen = a.double().sort(dim=1, descending=True, stable=True).indices[:, :k]
    counts = torch.zeros(a.shape[1] + 1, dtype=torch.int32)
    counts[:-1] = torch.bincount(chosen.reshape(-1), minlength=a.shape[1])
    counts[-1] = a.shape[0] * k
    return counts


def weights(a, kind):
    """Unnormalised probabilities in 64 bits, kind in "scores", "softmax", "sigmoid"."""
    a = a.double()
    if kind == "softmax":
        m = a.amax(1, keepdim=True)
        return torch.exp(a - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return torch.sigmoid(a) if kind == "sigmoid" else a


def probs(a, kind):
    w = weights(a, kind)
    s = w.sum(1, keepdim=True)
    return torch.where(s > 0, w / s, torch.zeros_like(w))


def balance_loss(a, kind, counts, k, coefficient):
    """(loss, mean_probs) of the rows a [n, E]."""
    n, E = a.shape
    if n == 0:
        return torch.zeros((), dtype=torch.float64), torch.zeros(E, dtype=torch.float64)
    mean = probs(a, kind).mean(0)
    f = counts[:E].double() * E / (k * n)
    return coefficient * (f * mean).sum(), mean


def balance_loss_backward(a, kind, counts, k, coefficient, dloss):
    """(gradient, its scale for error bounds): |f| + q in the place of f - q."""
    n, E = a.shape
    w, f = weights(a, kind), counts[:E].double() * E / (k * max(n, 1))
    s = w.sum(1, keepdim=True)
    p = torch.where(s > 0, w / s, torch.zeros_like(w))
    q = (p * f).sum(1, keepdim=True)
    if kind == "scores":
        slope = torch.where(s > 0, 1 / s, torch.zeros_like(s)).expand_as(w)
    elif kind == "softmax":
        slope = p
    else:
        slope = p * torch.sigmoid(-a.double())
    c = coefficient * dloss / max(n, 1)
    return c * (f - q) * slope, abs(c) * (f + q) * slope


# --------------------------------------------------------------- checkpoints

def pack(v):
    """(codes float8 [a, W], exponents uint8) of bf16 rows, block by block by search over the exponents."""
    a, W = v.shape
    v = v.double()
    codes = torch.zeros(a, W, dtype=torch.float64)
    exps = torch.zeros(a, -(-W // BLOCK), dtype=torch.uint8)
    for b in range(exps.shape[1]):
        blk = v[:, b * BLOCK:(b + 1) * BLOCK]
        m = torch.where(torch.isfinite(blk), blk.abs(), torch.zeros_like(blk)).amax(1)
        e = torch.full((a,), -100.0, dtype=torch.float64)
        while bool(((m > 448 * 2.0 ** e) & (e < 119)).any()):
            e = torch.where((m > 448 * 2.0 ** e) & (e < 119), e + 1, e)
        q = (blk / (2.0 ** e)[:, None]).clamp(-448, 448)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = torch.where(torch.isfinite(blk), q, torch.full_like(q, float("nan")))
        exps[:, b] = (e + 127).to(torch.uint8)
    return codes.float().to(torch.float8_e4m3fn), exps


def unpack(codes, exps):
    scale = torch.repeat_interleave(2.0 ** (exps.double() - 127), BLOCK, dim=1)[:, : codes.shape[1]]
    return codes.double() * scale


def silu_mul(y0, y1):
    return y0 * torch.sigmoid(y0) * y1


def silu_mul_backward(y0, y1, dz):
    """(dy0, dy1) in 64 bits."""
    s = torch.sigmoid(y0)
    return dz * y1 * s * (1 + y0 * (1 - s)), dz * y0 * s


# ------------------------------------------------------------- weight gradient

def weight_grad(dy, x, counts):
    """(dw [E, N, K], sum of |terms|) in 64 bits."""
    E = len(counts)
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(dw)
    at = 0
    for e, c in enumerate(counts):
        a, b = dy[at:at + c].double(), x[at:at + c].double()
        dw[e], mag[e] = a.T @ b, a.abs().T @ b.abs()
        at += c
    return dw, mag
