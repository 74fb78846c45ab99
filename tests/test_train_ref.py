"""The 64-bit definitions that the GPU tests compare with: each gradient against central differences
of its forward, the checkpoint format against its own bounds."""
import pytest
import torch

from tests import train_ref as ref


def _difference(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


# central differences in 64 bits: truncation h^2 ~ 1e-12, rounding 1e-16 / h ~ 1e-10 of the loss
DIFF_TOL = 1e-7


def test_layer_norm_gradient_is_the_difference():
    g = ref.gen(0)
    x = torch.randn(5, 37, generator=g, dtype=torch.float64) + 0.5
    gamma, beta = torch.randn(2, 37, generator=g, dtype=torch.float64)
    dy = torch.randn(5, 37, generator=g, dtype=torch.float64)
    _, mean, rstd = ref.layer_norm(x, gamma, beta, 1e-5)
    dx, dgamma, dbeta = ref.layer_norm_backward(dy, x, gamma, mean, rstd)
    for var, grad, f in ((x, dx, lambda v: (ref.layer_norm(v, gamma, beta, 1e-5)[0] * dy).sum()),
                         (gamma, dgamma, lambda v: (ref.layer_norm(x, v, beta, 1e-5)[0] * dy).sum()),
                         (beta, dbeta, lambda v: (ref.layer_norm(x, gamma, v, 1e-5)[0] * dy).sum())):
        d = torch.randn(var.shape, generator=g, dtype=torch.float64)
        assert abs(_difference(f, var, d) - (grad * d).sum()) < DIFF_TOL * (1 + (grad * d).abs().sum())


@pytest.mark.parametrize("kind", ["scores", "softmax", "sigmoid"])
def test_balance_gradient_is_the_difference(kind):
    g = ref.gen(1)
    a = torch.randn(6, 9, generator=g, dtype=torch.float64)
    if kind == "scores":
        a = torch.sigmoid(a)
    counts = ref.top_counts(a, 2)
    grad, _ = ref.balance_loss_backward(a, kind, counts, 2, 0.3, 1.7)
    d = torch.randn(6, 9, generator=g, dtype=torch.float64)
    diff = _difference(lambda v: 1.7 * ref.balance_loss(v, kind, counts, 2, 0.3)[0], a, d)
    assert abs(diff - (grad * d).sum()) < DIFF_TOL * (1 + (grad * d).abs().sum())


def test_silu_mul_gradient_is_the_difference():
    g = ref.gen(2)
    y0, y1, dz, d0, d1 = (2 * torch.randn(5, 4, 32, generator=g, dtype=torch.float64)).unbind(0)
    g0, g1 = ref.silu_mul_backward(y0, y1, dz)
    diff = _difference(lambda t: (ref.silu_mul(y0 + t * d0, y1 + t * d1) * dz).sum(),
                       torch.zeros((), dtype=torch.float64), 1.0)
    want = (g0 * d0 + g1 * d1).sum()
    assert abs(diff - want) < DIFF_TOL * (1 + (g0 * d0).abs().sum() + (g1 * d1).abs().sum())


def test_balanced_router_has_the_coefficient_as_its_loss():
    a = torch.eye(8).repeat(4, 1)
    counts = ref.top_counts(a, 1)
    assert counts.tolist() == [4] * 8 + [32]
    assert ref.balance_loss(a, "scores", counts, 1, 0.25)[0].item() == pytest.approx(0.25, abs=1e-15)


def test_checkpoint_keeps_each_value_within_half_a_code():
    v = (torch.randn(7, 272, generator=ref.gen(3)) * torch.logspace(-6, 6, 7)[:, None]).to(torch.bfloat16)
    codes, exps = ref.pack(v)
    kept = ref.unpack(codes, exps)
    assert torch.equal(kept.to(torch.bfloat16).double(), kept)        # bf16 holds what was kept
    scale = torch.repeat_interleave(2.0 ** (exps.double() - 127), 128, dim=1)[:, :272]
    # e4m3 has 4 significant bits, subnormals in steps of 2^-9
    assert torch.all((kept - v.double()).abs() <= torch.maximum(v.double().abs() * 2.0 ** -4, scale * 2.0 ** -10))
