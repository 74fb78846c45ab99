"""A whole training step of an MoE block against 64-bit autograd over the same routing.

Bound: the block's intermediates are bf16 (2^-9 each, about ten on the way), and the weight and
SiLU*mul gradients read e4m3 values, each within 2^-4 of itself and, spread evenly below that,
3.6% in the mean; two of them meet in a product.  The norm of a gradient's error is so held to
8% of the gradient's, and the output's, which has no 8-bit value in it, to 2%."""
import pytest
import torch

from tests import train_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _block(E, D, H, k, seed=0):
    from moe_token_routing_index_gb300.training import MoETrainBlock

    g = ref.gen(seed)
    p = dict(w13=torch.randn(E, 2 * H, D, generator=g) / D ** 0.5, w2=torch.randn(E, D, H, generator=g) / H ** 0.5,
             router=torch.randn(E, D, generator=g) / D ** 0.5, gamma=1 + 0.1 * torch.randn(D, generator=g),
             beta=0.1 * torch.randn(D, generator=g))
    p = {n: v.to(BF16) for n, v in p.items()}
    return MoETrainBlock(k, *(p[n].cuda() for n in ("w13", "w2", "router", "gamma", "beta")), balance=0.5), p


def _reference(x, p, chosen, H, k, coef, dout, dloss):
    """Autograd in 64 bits with the experts that were chosen; returns (out, loss, gradients)."""
    leaf = {n: v.double().requires_grad_() for n, v in dict(p, x=x).items()}
    x, E = leaf["x"], p["router"].shape[0]
    xc = x - x.mean(1, keepdim=True)
    n = xc / torch.sqrt((xc * xc).mean(1, keepdim=True) + 1e-5) * leaf["gamma"] + leaf["beta"]
    s = torch.sigmoid(n @ leaf["router"].T)
    out = x
    for e in range(E):
        xe = n * s[:, e:e + 1]
        y = xe @ leaf["w13"][e].T
        z = y[:, :H] * torch.sigmoid(y[:, :H]) * y[:, H:]
        out = out + (z @ leaf["w2"][e].T) * chosen[:, e:e + 1]
    f = chosen.double().sum(0) * E / (k * len(x))
    loss = coef * (f * (s / s.sum(1, keepdim=True)).mean(0)).sum()
    ((out * dout.double()).sum() + dloss * loss).backward()
    return out.detach(), loss.detach(), {n: v.grad for n, v in leaf.items()}


def _near(got, want, rel, what):
    err = float((got.cpu().double() - want).norm() / want.norm())
    assert err <= rel, f"{what}: {err:.4f} of its norm"


@pytest.mark.parametrize("T,E,D,H,k,valid", [(64, 16, 256, 128, 2, None), (37, 16, 128, 144, 1, None),
                                             (200, 32, 272, 96, 4, 131), (1, 16, 64, 32, 3, None)])
def test_training_step(T, E, D, H, k, valid):
    from moe_token_routing_index_gb300 import binding as mb

    block, p = _block(E, D, H, k)
    x = (torch.randn(T, D, generator=ref.gen(1)) + 0.2).to(BF16)
    dout = torch.randn(T, D, generator=ref.gen(2)).to(BF16)
    n = T if valid is None else valid
    nv = None if valid is None else torch.tensor([valid], dtype=torch.int32, device="cuda")
    out, saved = block.forward(x.cuda(), nv)
    grads = block.backward(saved, dout.cuda(), torch.tensor([1.5], device="cuda"))
    assert mb.device_error() == 0
    r = saved.route
    chosen = torch.zeros(T, E, dtype=torch.bool)
    rows = n * k
    chosen[r["token_indices"][:rows].cpu().long(), r["expert_indices"][:rows].cpu().long()] = True
    want, loss, g = _reference(x[:n], p, chosen[:n], H, k, 0.5, dout[:n], 1.5)
    _near(out[:n], want, 0.02, "out")
    assert abs(float(saved.balance_loss) - float(loss)) <= 0.02 * float(loss)
    assert torch.equal(out[n:].cpu(), x[n:]) and torch.equal(grads["x"][n:].cpu(), dout[n:])
    for name in ("w13", "w2", "router", "gamma", "beta"):
        _near(grads[name], g[name], 0.08, name)
    _near(grads["x"][:n], g["x"], 0.08, "x")


def test_block_refuses_what_does_not_fit():
    from moe_token_routing_index_gb300.training import MoETrainBlock

    z = lambda *s: torch.zeros(*s, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        MoETrainBlock(2, z(8, 64, 32), z(8, 32, 32), z(8, 32), z(32), z(32))          # 8 experts
    with pytest.raises(ValueError):
        MoETrainBlock(2, z(16, 64, 32), z(16, 32, 64), z(16, 32), z(32), z(32))


@pytest.mark.parametrize("at", [4.0, 7.0, -7.0])
def test_gradients_of_confident_scores(at):
    """Every expert's logit near `at`, where a score leaves little to 1 or to 0: the router's gradient still
    follows from what it leaves (logits are bf16: 2^-9 of them, below 2% of such a slope)."""
    E, D, H, k, T = 16, 256, 64, 2, 96
    block, p = _block(E, D, H, k, seed=3)
    u = torch.randn(D, generator=ref.gen(4))
    p["beta"] = u.to(BF16)
    p["router"] = (at * u / u.square().sum() + 0.3 * torch.randn(E, D, generator=ref.gen(5)) / D ** 0.5).to(BF16)
    block.beta.copy_(p["beta"])
    block.router.copy_(p["router"])
    block.refresh_weights()
    x = torch.randn(T, D, generator=ref.gen(1)).to(BF16)
    dout = torch.randn(T, D, generator=ref.gen(2)).to(BF16)
    out, saved = block.forward(x.cuda())
    grads = block.backward(saved, dout.cuda(), torch.tensor([1.5], device="cuda"))
    r = saved.route
    chosen = torch.zeros(T, E, dtype=torch.bool)
    chosen[r["token_indices"].cpu().long(), r["expert_indices"].cpu().long()] = True
    want, _, g = _reference(x, p, chosen, H, k, 0.5, dout, 1.5)
    _near(out, want, 0.02, "out")
    for name in ("router", "w13", "w2", "gamma", "beta", "x"):
        _near(grads[name], g[name], 0.08, name)
