"""The gated block and its gradient where every product's reduction is longer than 512, as at the sizes that
matter: ragged loads, columns that end inside a tile, rows of no expert."""
import pytest
import torch

from tests import gated_ref as ref
from tests.test_gpu_gated import BF16, _counts, _filled, _kind, _make, _mb, _within

pytestmark = pytest.mark.gpu

CASES = [(700, 1040, 528, [300, 0, 257, 100]), (90, 640, 1056, [33, 1, 50]), (600, 784, 560, [0, 600]),
         (40, 528, 1296, [1, 0, 3, 0, 30])]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("a,D,H,counts", CASES)
def test_forward(a, D, H, counts, kind):
    mb = _mb()
    x, w13, w2, _ = _make(a, len(counts), D, H, seed=20)
    n = sum(counts)
    x[n:] = float("nan")
    y, z, out = _filled(a, 2 * H), _filled(a, H), _filled(a, D)
    mb.moe_gated_mlp(x.cuda(), w13.cuda(), w2.cuda(), _counts(counts), activation=_kind(kind), y=y, z=z, out=out)
    assert mb.device_error() == 0
    x[n:] = 0
    want, wy, eo, ey = ref.forward(x, w13, w2, counts, kind)
    _within(y, wy, ey, n, "y")
    _within(out, want, eo, n, "out")
    assert all(bool((t[n:] == 7).all()) for t in (y, z, out))


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("a,D,H,counts", CASES)
def test_backward(a, D, H, counts, kind, codes):
    """From y in bf16, or from 8-bit rows at the values that they hold."""
    mb = _mb()
    _, w13, w2, dout = _make(a, len(counts), D, H, seed=21)
    kept = held = (1.5 * torch.randn(a, 2 * H, generator=torch.Generator().manual_seed(22))).to(BF16)
    n = sum(counts)
    if codes:
        _, kept = mb.moe_silu_mul_checkpoint(held.cuda(), H)
        scale = torch.exp2(kept.exponents.double().cpu() - 127)
        nb = scale.shape[1] // 2
        held = kept.codes.double().cpu().view(a, 2, H) * scale.view(a, 2, nb).repeat_interleave(128, 2)[:, :, :H]
        held = held.reshape(a, 2 * H)
    else:
        kept = kept.cuda()
        kept[n:] = float("inf")
    dx, dy, z = _filled(a, D), _filled(a, 2 * H), _filled(a, H)
    mb.moe_gated_mlp_backward(dout.cuda(), kept, w13.cuda(), w2.cuda(), _counts(counts), activation=_kind(kind), out=dx,
                              dy=dy, z=z)
    assert mb.device_error() == 0
    wx, wy, wz, ex, ey, ez = ref.backward(dout, held, w13, w2, counts, kind)
    _within(dy, wy, ey, n, "dy")
    _within(z, wz, ez, n, "z")
    _within(dx, wx, ex, n, "dx")
    assert all(bool((t[n:] == 7).all()) for t in (dx, dy, z))
