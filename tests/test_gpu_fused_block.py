"""The training block with its experts in the fused kernels, and its update, as they are used together.

Bounds: the block's intermediates are bf16, about ten on the way, each off by 1.7e-3 of its norm (2^-8 at
most, spread evenly), so by 0.6% in all where they add up as squares do; held to 3%.  w13's gradient reads
the experts' rows in 8 bits (3.6% of their norm) and is held to 8%, the output to 2%."""
import sys

import pytest
import torch

from tests import gated_ref
from tests import train_ref as ref
from tests.test_gpu_training import BF16, _near, _reference

pytestmark = pytest.mark.gpu


def _block(E, D, H, k, seed=0, fused=True):
    from moe_token_routing_index_gb300.training import MoETrainBlock

    g = ref.gen(seed)
    p = dict(w13=torch.randn(E, 2 * H, D, generator=g) / D ** 0.5, w2=torch.randn(E, D, H, generator=g) / H ** 0.5,
             router=torch.randn(E, D, generator=g) / D ** 0.5, gamma=1 + 0.1 * torch.randn(D, generator=g),
             beta=0.1 * torch.randn(D, generator=g))
    p = {n: v.to(BF16) for n, v in p.items()}
    return MoETrainBlock(k, *(p[n].cuda() for n in ("w13", "w2", "router", "gamma", "beta")), balance=0.5, fused=fused), p


@pytest.mark.parametrize("T,E,D,H,k,valid", [(64, 16, 256, 128, 2, None), (37, 16, 128, 144, 1, None),
                                             (200, 32, 272, 96, 4, 131), (1, 16, 64, 32, 3, None)])
def test_training_step(T, E, D, H, k, valid):
    from moe_token_routing_index_gb300 import binding as mb

    block, p = _block(E, D, H, k)
    assert not hasattr(block, "w13_t") and not hasattr(block, "w2_t")
    x = (torch.randn(T, D, generator=ref.gen(1)) + 0.2).to(BF16)
    dout = torch.randn(T, D, generator=ref.gen(2)).to(BF16)
    n = T if valid is None else valid
    nv = None if valid is None else torch.tensor([valid], dtype=torch.int32, device="cuda")
    out, saved = block.forward(x.cuda(), nv)
    grads = block.backward(saved, dout.cuda(), torch.tensor([1.5], device="cuda"))
    assert mb.device_error() == 0
    r = saved.route
    chosen = torch.zeros(T, E, dtype=torch.bool)
    chosen[r["token_indices"][:n * k].cpu().long(), r["expert_indices"][:n * k].cpu().long()] = True
    want, _, g = _reference(x[:n], p, chosen[:n], H, k, 0.5, dout[:n], 1.5)
    _near(out[:n], want, 0.02, "out")
    assert torch.equal(out[n:].cpu(), x[n:]) and torch.equal(grads["x"][n:].cpu(), dout[n:])
    for name in ("w2", "router", "gamma", "beta"):
        _near(grads[name], g[name], 0.03, name)
    _near(grads["w13"], g["w13"], 0.08, "w13")
    _near(grads["x"][:n], g["x"], 0.03, "x")


def test_update_after_a_step():
    """Forward, backward, weight gradients and the update in a row: the weights move as the formulas say for the
    gradients that came out, each projection for itself, and the next step sees them."""
    from moe_token_routing_index_gb300 import binding as mb

    E, D, H, k, T, lr = 16, 96, 64, 2, 64, 0.02
    block, _ = _block(E, D, H, k, seed=1)
    x = torch.randn(T, D, generator=ref.gen(3)).to(BF16).cuda()
    dout = torch.randn(T, D, generator=ref.gen(4)).to(BF16).cuda()
    momentum = {}
    for step in range(3):
        before = {n: getattr(block, n).clone() for n in ("w13", "w2", "router", "gamma", "beta")}
        out, saved = block.forward(x)
        grads = block.backward(saved, dout)
        block.update(grads, lr, mu=0.9, weight_decay=0.1, lr_scale=torch.tensor([0.5], device="cuda"))
        for name, shape in (("w13", (2 * E, H, D)), ("w2", (E, D, H)), ("router", (1, E, D))):
            g = grads[name].double().cpu().view(shape)
            m = 0.9 * momentum.get(name, torch.zeros(shape).double()) + g
            momentum[name] = m
            u = g + 0.9 * m
            exact, half = gated_ref.orthogonalize(u), gated_ref.orthogonalize(u, half=True)
            rate = 0.5 * lr * max(1.0, shape[1] / shape[2]) ** 0.5
            w0 = before[name].double().cpu().view(shape)
            want = w0 * (1 - 0.1 * rate) - rate * exact
            got = getattr(block, name).double().cpu().view(shape)
            for b in range(shape[0]):
                # 1.5 times what fp16 operands allow, the momentum's fp32 roundings, the weights' bf16
                most = rate * (1.5 * float((half[b] - exact[b]).norm()) + 1e-4 * float(exact[b].norm()))
                off = float((got[b] - want[b]).norm())
                assert off <= most + 1.01 * gated_ref.HALF16 * float(want[b].norm()), (name, b)
        for name in ("gamma", "beta"):
            want = before[name].double() - 0.5 * lr * grads[name].double()
            off = (getattr(block, name).double() - want).abs()
            assert bool((off <= 1.01 * gated_ref.HALF16 * want.abs() + 1e-6).all()), name
        assert torch.equal(block.router_t, block.router.t())
    assert mb.device_error() == 0


def test_a_captured_training_step():
    """A whole step in a CUDA graph gives the bytes of the same step run by itself."""
    E, D, H, k, T = 16, 64, 48, 2, 80
    x = torch.randn(T, D, generator=ref.gen(5)).to(BF16).cuda()
    dout = torch.randn(T, D, generator=ref.gen(6)).to(BF16).cuda()
    eager, _ = _block(E, D, H, k, seed=2)
    block, _ = _block(E, D, H, k, seed=2)

    def step(b):
        out, saved = b.forward(x)
        b.update(b.backward(saved, dout), 0.01)
        return out

    for _ in range(2):
        want = step(eager)
    step(block)                                     # momentum exists, kernels are loaded
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(block)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for name in ("w13", "w2", "router", "gamma", "beta"):
        assert torch.equal(getattr(block, name), getattr(eager, name)), name


@pytest.mark.parametrize("options", [["--fused"], ["--fused", "--optimizer", "muon", "--lr", "0.02"],
                                     ["--optimizer", "muon"]])
def test_command_runs(monkeypatch, capsys, options):
    from moe_token_routing_index_gb300 import training

    monkeypatch.setattr(sys, "argv", ["training", "--config", "tiny", "--steps", "2", *options])
    training._main()
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 2 and all("mean square error" in line and "nan" not in line for line in lines)
