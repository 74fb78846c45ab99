"""A training step of one pre-norm MoE block on one GPU: out = x + MoE(layer_norm(x)).

    block = MoETrainBlock(top_k, w13, w2, router, gamma, beta)
    out, saved = block.forward(x, num_valid_tokens)
    grads = block.backward(saved, dout)             # dx and the gradient of every parameter

The forward is the routed-expert forward of MoELayer behind a layer norm, with scores as input
weights; it adds the router's balance loss and keeps, for the backward, the norm's statistics and
two 8-bit checkpoints: the experts' input rows and the SiLU*mul input.  Between forward and
backward a routed row so holds D + 2H bytes (and an exponent per 128 of them) instead of the
2D + 6H bytes of its bf16 input, SiLU*mul input and output.

  backward, for the gradient dout of out:
    do   = rows of dout by expert                         moe_gather_scale (unit scores)
    dz   = do w2                                          moe_grouped_gemm, w2 transposed
    dy,z = SiLU*mul gradient at the checkpoint            moe_silu_mul_backward
    dw2  = do^T z,  dw13 = dy^T x                         moe_grouped_weight_grad (x: the checkpoint)
    dxr  = dy w13                                         moe_grouped_gemm, w13 transposed
    scores: the routed rows' part, plus the balance loss  moe_balance_loss_backward (accumulate)
    logits again, for the sigmoid's slope                 moe_dense_gemm
    router: dlogits^T n and dlogits router                moe_grouped_weight_grad, moe_dense_gemm
    dn   = sum of score * dxr over a token's rows + ...   moe_topk_finalize
    dx, dgamma, dbeta                                     moe_layer_norm_backward (+ dout)

With fused=True the experts' gated block is moe_gated_mlp and its data path's gradient
moe_gated_mlp_backward: y is kept in bf16 (4H bytes a routed row instead of 2H), dz, dy, z and
dxr are two launches, and the weights are read as they lie (no transposed copies of w13 and w2).

update(grads, lr) moves the weights: w13's projections, w2 and the router by their orthogonalised
momentum (moe_muon_update), gamma and beta along their gradients.

    python -m moe_token_routing_index_gb300.training [--config tiny] [--steps 20] [--fused]
                                                     [--optimizer sgd|muon] [--lr 0.1]

trains a block of a workload's shape on a fixed random target and prints the loss and the time
of a step.
"""
from __future__ import annotations

import argparse
import time
from dataclasses import dataclass

import torch

from . import binding as mb
from . import workloads

__all__ = ["MoETrainBlock", "Saved"]


@dataclass
class Saved:
    """What the forward leaves for the backward."""

    x: torch.Tensor
    n: torch.Tensor                  # layer norm of x
    mean: torch.Tensor
    rstd: torch.Tensor
    num_valid: torch.Tensor | None
    scores: torch.Tensor
    route: dict
    rows: mb.Checkpoint              # the experts' input rows
    y: mb.Checkpoint | torch.Tensor  # the input of SiLU*mul: two halves in 8 bits, or bf16 (fused)
    balance_loss: torch.Tensor       # fp32 [1]


class MoETrainBlock:
    """w13 [E, 2H, D], w2 [E, D, H], router [E, D] and gamma, beta [D], all bf16 on the GPU; E a
    multiple of 16 for the router's gradient.  After the weights changed in place,
    refresh_weights() brings the transposed copies of the data gradients up to date."""

    def __init__(self, top_k: int, w13, w2, router, gamma, beta, *, balance: float = 0.01, eps: float = 1e-5,
                 fused: bool = False):
        self.E, n2, self.D = w13.shape
        self.H = n2 // 2
        if w2.shape != (self.E, self.D, self.H) or router.shape != (self.E, self.D):
            raise ValueError("w13 [E, 2H, D], w2 [E, D, H] and router [E, D] must fit together")
        if self.E % 16:
            raise ValueError("the router's gradient needs a multiple of 16 experts")
        self.top_k, self.balance, self.eps, self.fused = top_k, balance, eps, fused
        self.momentum = {}
        self.w13, self.w2, self.router, self.gamma, self.beta = w13, w2, router, gamma, beta
        self.refresh_weights()

    def refresh_weights(self):
        if not self.fused:
            self.w13_t = self.w13.transpose(1, 2).contiguous()
            self.w2_t = self.w2.transpose(1, 2).contiguous()
        self.router_t = self.router.t().contiguous()

    def forward(self, x: torch.Tensor, num_valid_tokens: torch.Tensor | None = None):
        """x [T, D] bf16 -> (out [T, D], Saved).  Rows past the valid count pass through."""
        k, valid = self.top_k, num_valid_tokens
        n, mean, rstd = mb.moe_layer_norm(x, self.gamma, self.beta, valid, eps=self.eps)
        scores, r = mb.moe_router_route(n, self.router, k, valid, with_weights=True)
        counts = r["counts"]
        rows = counts[self.E:]
        loss, _, _ = mb.moe_balance_loss(scores, k, valid, coefficient=self.balance, counts=counts)
        xr = mb.moe_gather_scale(n, r["token_indices"], r["expert_indices"], scores, rows, inv_rows=r["inv_rows"],
                                 top_k=k)
        if self.fused:
            o, y8 = mb.moe_gated_mlp(xr, self.w13, self.w2, counts)
        else:
            y = mb.moe_grouped_gemm(xr, self.w13, counts)
            z, y8 = mb.moe_silu_mul_checkpoint(y, self.H, rows)
            o = mb.moe_grouped_gemm(z, self.w2, counts)
        out = mb.moe_scatter_add(x.clone(), o, r["token_indices"], r["inv_rows"], k, rows)
        x8 = mb.moe_checkpoint_pack(xr, rows)
        return out, Saved(x, n, mean, rstd, valid, scores, r, x8, y8, loss)

    def backward(self, s: Saved, dout: torch.Tensor, dloss: torch.Tensor | None = None) -> dict:
        """Gradients of sum(out * dout) + dloss * balance_loss (dloss: fp32 [1] on the device, None: 1):
        dict(x, w13, w2, router, gamma, beta); gamma and beta fp32, the others bf16."""
        E, k, r, valid = self.E, self.top_k, s.route, s.num_valid
        counts, ti, ei, inv = r["counts"], r["token_indices"], r["expert_indices"], r["inv_rows"]
        rows, T = counts[E:], s.x.shape[0]
        do = mb.moe_gather_scale(dout, ti, ei, None, rows, inv_rows=inv, top_k=k)
        if self.fused:
            dxr, dy, z = mb.moe_gated_mlp_backward(do, s.y, self.w13, self.w2, counts)
        else:
            dz = mb.moe_grouped_gemm(do, self.w2_t, counts)
            dy, z = mb.moe_silu_mul_backward(s.y, dz, rows)
            dxr = mb.moe_grouped_gemm(dy, self.w13_t, counts)
        dw2 = mb.moe_grouped_weight_grad(do, z, counts, E=E)
        dw13 = mb.moe_grouped_weight_grad(dy, s.rows, counts, E=E)
        dscores = self._score_gradient(s, dxr)
        mb.moe_balance_loss_backward(s.scores, counts, k, valid, coefficient=self.balance, dloss=dloss, out=dscores,
                                     accumulate=True)
        # the sigmoid's slope from the logits: of a score near 1, bf16 holds little of what it leaves to 1
        logits = mb.moe_dense_gemm(s.n, self.router, valid).float()
        dlogits = (dscores.float() * torch.sigmoid(logits) * torch.sigmoid(-logits)).to(torch.bfloat16)
        tokens = valid if valid is not None else torch.full((1,), T, dtype=torch.int32, device=s.x.device)
        drouter = mb.moe_grouped_weight_grad(dlogits, s.n, tokens, E=1)[0]
        through_router = mb.moe_dense_gemm(dlogits, self.router_t, valid)
        dn = mb.moe_topk_finalize(dxr, r["topk_weights"].view(T, k), inv.view(T, k), through_router, valid)
        dx, dgamma, dbeta = mb.moe_layer_norm_backward(dn, s.x, self.gamma, s.mean, s.rstd, valid, residual_grad=dout,
                                                       out=dout.clone() if valid is not None else None)
        return dict(x=dx, w13=dw13, w2=dw2, router=drouter, gamma=dgamma, beta=dbeta)

    def update(self, grads: dict, lr: float, *, mu: float = 0.95, weight_decay: float = 0.0, lr_scale=None):
        """One update of all weights, in place.  Each expert's gate and up projection, its down projection and
        the router move by lr * sqrt(max(1, rows / columns)) along their orthogonalised momentum and shrink by
        lr * weight_decay; gamma and beta move by lr along their gradients.  lr_scale: fp32 [1] on the device that
        multiplies lr, None: 1."""
        for name, w in (("w13", self.w13.view(2 * self.E, self.H, self.D)), ("w2", self.w2), ("router", self.router)):
            if name not in self.momentum:
                self.momentum[name] = torch.zeros(w.shape, dtype=torch.float32, device=w.device)
            # (moe_muon_update decays by its rate times weight_decay: the shape's factor is taken out of that again)
            N, K = w.shape[-2:]
            factor = max(1.0, N / K) ** 0.5
            mb.moe_muon_update(w, grads[name].view(w.shape), self.momentum[name], lr=lr * factor, mu=mu,
                               weight_decay=weight_decay / factor, lr_scale=lr_scale)
        for name in ("gamma", "beta"):
            step = lr * grads[name] if lr_scale is None else lr * lr_scale * grads[name]
            w = getattr(self, name)
            w.copy_(w.float() - step)
        self.refresh_weights()

    def _score_gradient(self, s: Saved, dxr: torch.Tensor) -> torch.Tensor:
        """d scores[t, e] = <dxr[row], n[t]> for the routed rows (t, e), zero elsewhere; bf16 [T, E]."""
        r, T = s.route, s.x.shape[0]
        live = torch.arange(T * self.top_k, device=dxr.device) < r["counts"][self.E]
        t = torch.where(live, r["token_indices"], T).long()     # rows past the count go to a spare row
        e = torch.where(live, r["expert_indices"], 0).long()
        dot = torch.einsum("rd,rd->r", dxr, s.n[t.clamp(max=T - 1)])
        d = torch.zeros(T + 1, self.E, dtype=torch.bfloat16, device=dxr.device)
        d[t, e] = torch.where(live, dot, torch.zeros_like(dot))
        return d[:T]


def _train_step(block: MoETrainBlock, x, target, valid, n: int, optimizer: str, lr: float):
    """One step on the first n tokens towards the target; returns (out - target, what the forward kept)."""
    out, saved = block.forward(x, valid)
    err = out.float() - target.float()
    err[n:] = 0
    grads = block.backward(saved, err.to(torch.bfloat16))
    if optimizer == "muon":  # (the orthogonalised matrices have no scale; the vectors' gradients are sums over n tokens)
        block.update(dict(grads, gamma=grads["gamma"].float() / n, beta=grads["beta"].float() / n), lr)
    else:
        for name in ("w13", "w2", "router", "gamma", "beta"):
            w = getattr(block, name)
            w.copy_(w.float() - lr / n * grads[name].float())
        block.refresh_weights()
    return err, saved


def _main():
    ap = argparse.ArgumentParser(description="train one MoE block on a fixed random target")
    ap.add_argument("--config", default="tiny", choices=sorted(workloads.CONFIGS))
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.1)
    ap.add_argument("--fused", action="store_true", help="the experts' block and its gradient in fused kernels")
    ap.add_argument("--optimizer", default="sgd", choices=("sgd", "muon"))
    a = ap.parse_args()
    cfg = workloads.CONFIGS[a.config]
    E = -(-cfg.E // 16) * 16
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    bf = torch.bfloat16
    block = MoETrainBlock(cfg.top_k, (rnd(E, 2 * cfg.H, cfg.D) / cfg.D ** 0.5).to(bf),
                          (rnd(E, cfg.D, cfg.H) / cfg.H ** 0.5).to(bf), (rnd(E, cfg.D) / cfg.D ** 0.5).to(bf),
                          torch.ones(cfg.D, dtype=bf, device="cuda"), torch.zeros(cfg.D, dtype=bf, device="cuda"), fused=a.fused)
    x, target = rnd(cfg.T, cfg.D).to(bf), rnd(cfg.T, cfg.D).to(bf)
    valid = None if cfg.Tv is None else torch.tensor([cfg.Tv], dtype=torch.int32, device="cuda")
    n = cfg.valid_tokens
    for step in range(a.steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        err, saved = _train_step(block, x, target, valid, n, a.optimizer, a.lr)
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t0) * 1e3
        print(f"step {step}: mean square error {float(err.square().sum()) / (n * cfg.D):.4f}, balance loss "
              f"{float(saved.balance_loss):.5f}, {ms:.2f} ms", flush=True)


if __name__ == "__main__":
    _main()
