"""The weights' update of the training block, with the kernels replaced by their definition, so that it runs
without a GPU."""
import pytest
import torch

from tests import gated_ref as ref
from tests.test_streams import mb  # noqa: F401  (a fixture)

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("w13", "w2", "router", "gamma", "beta")


def _muon(w, grad, momentum, *, lr, mu=0.95, nesterov=True, weight_decay=0.0, lr_scale=None):
    """moe_muon_update's definition (include/moe_train.h), in 64 bits and rounded once."""
    momentum.copy_(mu * momentum.double() + grad.double())
    u = grad.double() + mu * momentum.double() if nesterov else momentum.double()
    r = lr * (1.0 if lr_scale is None else float(lr_scale))
    shape = (1, *w.shape)[-3:]
    w.copy_((1 - r * weight_decay) * w.double() - r * ref.orthogonalize(u.view(shape)).view(w.shape))
    return w


def _block(E, D, H, seed=0):
    from moe_token_routing_index_gb300.training import MoETrainBlock

    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    block = MoETrainBlock(2, r(E, 2 * H, D).to(BF16), r(E, D, H).to(BF16), r(E, D).to(BF16), (1 + 0.1 * r(D)).to(BF16),
                          (0.1 * r(D)).to(BF16), fused=True)
    return block, {n: r(*getattr(block, n).shape) for n in NAMES}


@pytest.mark.parametrize("D,H", [(96, 32), (32, 96), (64, 64)])
def test_decay_goes_by_the_rate_alone(mb, monkeypatch, D, H):  # noqa: F811
    """w = (1 - lr wd) w - lr sqrt(max(1, rows / columns)) X: a matrix's shape scales its step, not its decay.
    Held to one bf16 rounding, and 1e-6 for the 32 bits of rates."""
    from moe_token_routing_index_gb300 import training

    monkeypatch.setattr(training.mb, "moe_muon_update", _muon)
    E, lr, decay = 16, 0.05, 4.0
    block, grads = _block(E, D, H)
    before = {n: getattr(block, n).double() for n in NAMES}
    block.update(grads, lr, mu=0.9, weight_decay=decay, lr_scale=torch.tensor([0.5]))
    for name, shape in (("w13", (2 * E, H, D)), ("w2", (E, D, H)), ("router", (1, E, D))):
        rate = 0.5 * lr
        u = 1.9 * grads[name].double().view(shape)
        want = (1 - rate * decay) * before[name].view(shape)
        want = want - rate * max(1.0, shape[1] / shape[2]) ** 0.5 * ref.orthogonalize(u)
        off = (getattr(block, name).double().view(shape) - want).abs()
        assert bool((off <= (ref.HALF16 + 1e-6) * want.abs() + 1e-6).all()), name


@pytest.mark.parametrize("optimizer", ["sgd", "muon"])
def test_a_step_of_the_command_takes_the_mean_over_tokens(mb, monkeypatch, optimizer):  # noqa: F811
    """The gradients of a step are sums over its tokens: gamma and beta move by lr times their mean, and what is
    orthogonalised moves as it would for any multiple of its gradient.  One bf16 rounding each."""
    from moe_token_routing_index_gb300 import training

    monkeypatch.setattr(training.mb, "moe_muon_update", _muon)
    E, D, H, T, n, lr = 16, 64, 32, 80, 75, 0.1
    block, grads = _block(E, D, H, seed=1)
    grads = {name: n * g for name, g in grads.items()}
    before = {name: getattr(block, name).double() for name in NAMES}
    x, target = torch.randn(T, D).to(BF16), torch.randn(T, D).to(BF16)
    handed = []
    monkeypatch.setattr(block, "forward", lambda x, valid: (x.clone(), "kept"))
    monkeypatch.setattr(block, "backward", lambda saved, dout: handed.append(dout) or grads)
    err, saved = training._train_step(block, x, target, None, n, optimizer, lr)
    want_err = x.float() - target.float()
    want_err[n:] = 0
    assert saved == "kept" and torch.equal(err, want_err) and torch.equal(handed[0], want_err.to(BF16))
    for name in ("gamma", "beta") if optimizer == "muon" else NAMES:
        want = before[name] - lr * grads[name].double() / n
        off = (getattr(block, name).double() - want).abs()
        assert bool((off <= (ref.HALF16 + 1e-6) * want.abs() + 1e-6).all()), name


@pytest.mark.gpu
@pytest.mark.parametrize("D,H", [(96, 32), (192, 144)])
def test_decay_of_the_kernels(D, H):
    """Without a gradient only the decay is left: half of each weight, to the bit."""
    block, grads = _block(16, D, H, seed=2)
    for name in NAMES:
        setattr(block, name, getattr(block, name).cuda())
    before = {n: getattr(block, n).clone() for n in NAMES}
    zero = {n: torch.zeros_like(g, dtype=F32 if n in ("gamma", "beta") else BF16, device="cuda") for n, g in grads.items()}
    block.update(zero, 0.25, weight_decay=2.0)
    for name in ("w13", "w2", "router"):
        assert torch.equal(getattr(block, name), before[name] * 0.5), name
    assert torch.equal(block.gamma, before["gamma"]) and torch.equal(block.beta, before["beta"])


@pytest.mark.gpu
@pytest.mark.parametrize("options", [[], ["--fused"]])
def test_command_stays_finite(monkeypatch, capsys, options):
    """Ten steps with the default rate."""
    import math
    import sys

    from moe_token_routing_index_gb300 import training

    monkeypatch.setattr(sys, "argv", ["training", "--config", "tiny", "--steps", "10", "--optimizer", "muon", *options])
    training._main()
    lines = capsys.readouterr().out.strip().splitlines()
    errors = [float(line.split("error ")[1].split(",")[0]) for line in lines]
    assert len(errors) == 10 and all(math.isfinite(e) for e in errors)
