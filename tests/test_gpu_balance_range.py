"""The balance loss of rows whose weights add up to very little or to more than fp32 holds: the
distribution over experts is the one of the definition, as for any other row."""
import pytest
import torch

from tests import train_ref as ref
from tests.test_gpu_train import EXP, _check_balance, _close, _kind, _mb

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# every layout of tokens and experts over lanes: widths, and few and many tokens
SHAPES = [(70, 5, 2), (70, 24, 3), (45, 61, 8), (45, 128, 8), (40, 200, 4), (30, 500, 8), (30, 700, 3), (8300, 61, 8),
          (8300, 100, 2)]


def _sigmoid_rows(T, E, dtype):
    """Logits of every size below zero, rows of one size and rows that mix them, some experts masked."""
    g = ref.gen(T + E)
    a = torch.randn(T, E, generator=g)
    for i, at in enumerate((-90, -100, -120, -32, -34, -300, -650, -88, -104)):
        a[i::11] += at
    a[4::11, 0] = -20.0                                    # one of them far above the others
    a[9::11, ::2] -= 60
    a[2::11, E - 1] = float("-inf")
    a[10::22] = float("-inf")                              # nothing left: p = 0
    a[21::22] = torch.finfo(dtype).min                     # masked by the lowest value: p = 0, too
    return a.to(dtype)


def _score_rows(T, E, dtype):
    """Scores down to the subnormal numbers and up to sums beyond the largest fp32 number."""
    g = ref.gen(T + 2 * E)
    a = 0.1 + 0.9 * torch.rand(T, E, generator=g)
    for i, size in enumerate((1e-39, 1e-38, 3e38, 1e-30, 1e30, 1e-37, 2.0 ** -100, 2.0 ** 100)):
        a[i::9] *= size
    a[3::9, 1:] = 0
    a[17::18] = 0
    return a.to(dtype)


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("kind", ["scores", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_balance_loss_of_tiny_and_huge_rows(T, E, k, kind, dtype):
    mb = _mb()
    a = (_sigmoid_rows if kind == "sigmoid" else _score_rows)(T, E, dtype)
    for valid in (T, T - 3):
        _check_balance(mb, a, a.cuda(), kind, k, valid)
    _check_balance(mb, a, a.cuda(), kind, k, T, counts_in=ref.top_counts(a, k).cuda())


@pytest.mark.parametrize("dtype,least", [(BF16, 2.0 ** -133), (F32, 2.0 ** -149)])
def test_balance_loss_of_the_least_scores(dtype, least):
    """Forward only: the gradient of such a row is past fp32's range."""
    mb = _mb()
    a = torch.full((33, 24), least, dtype=torch.float64)
    a[::2, :7] *= 3
    a = a.to(dtype)
    loss, counts, mean = mb.moe_balance_loss(a.cuda(), 2, kind=_kind(mb, "scores"))
    assert torch.equal(counts.cpu(), ref.top_counts(a, 2))
    wl, wm = ref.balance_loss(a, "scores", counts.cpu(), 2, 1.0)
    n = (33 + 1024) * 2.0 ** -24 + EXP
    _close(mean, wm, n * wm, "mean_probs")
    _close(loss[0], wl, n * wl, "loss")
    assert mb.device_error() == 0
