"""The experts' weight gradients on the GPU against 64-bit products.

Bound: each fp32 addition of the tensor cores or of a join is off by at most 2^-23 of the sum of
magnitudes (they may truncate), with at most one addition for each row and 64 more for the joins;
bf16 results have one bf16 step more."""
import pytest
import torch

from tests import train_ref as ref
from tests.helpers import sentinel_like

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _mb():
    from moe_token_routing_index_gb300 import binding

    return binding


def _data(counts, N, K, spare=0, seed=0):
    g = ref.gen(seed + N + K + sum(counts))
    a = sum(counts) + spare
    dy = torch.randn(a, N, generator=g).to(BF16)
    x = torch.randn(a, K, generator=g).to(BF16)
    dy[sum(counts):], x[sum(counts):] = float("nan"), float("inf")     # rows of no expert hold anything
    return dy, x, torch.tensor(counts, dtype=torch.int32).cuda()


def _check(got, dy, x, counts, extra=None):
    want, mag = ref.weight_grad(dy, x, counts)
    rows = torch.tensor(counts, dtype=torch.float64)[:, None, None]
    bound = (rows + 64) * 2.0 ** -23 * mag + want.abs() * (2.0 ** -8 if got.dtype == BF16 else 2.0 ** -23)
    if extra is not None:
        want, bound = want + extra.double(), bound + 2.0 ** -23 * (extra.double().abs() + want.abs())
    bad = ~((got.cpu().double() - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside the bound"


# rows: none, one, tile edges (16-row steps, 64-row blocks), long; sizes on both sides of the tiles
CASES = [([1], 16, 16), ([0], 64, 64), ([5, 0, 3], 48, 80), ([16, 17, 15, 1, 64, 65], 128, 256),
         ([63, 0, 0, 130, 2], 144, 272), ([300], 272, 528), ([0, 0, 0], 32, 32), ([129, 31], 512, 1024),
         ([7] * 40, 96, 64), ([1000, 3], 160, 48), ([4100], 128, 256), ([2, 260, 33], 400, 784)]


@pytest.mark.parametrize("counts,N,K", CASES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weight_grad(counts, N, K, dtype):
    mb = _mb()
    dy, x, c = _data(counts, N, K, spare=13)
    got = mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), c, dtype=dtype)
    _check(got, dy, x, counts)
    again = mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), c, out=sentinel_like(got.shape, dtype))
    assert torch.equal(got, again)
    assert mb.device_error() == 0


@pytest.mark.parametrize("counts,N,K", CASES)
def test_weight_grad_from_a_checkpoint(counts, N, K):
    """The same bytes as from the unpacked rows, which hold the checkpoint's values exactly."""
    mb = _mb()
    dy, x, c = _data(counts, N, K, spare=5)
    ck = mb.moe_checkpoint_pack(x.cuda())
    rows = mb.moe_checkpoint_unpack(ck)
    got = mb.moe_grouped_weight_grad(dy.cuda(), ck, c, dtype=F32)
    assert torch.equal(got, mb.moe_grouped_weight_grad(dy.cuda(), rows, c, dtype=F32))
    _check(got, dy, rows.cpu(), counts)
    assert mb.device_error() == 0


@pytest.mark.parametrize("counts,N,K", CASES)
def test_weight_grad_accumulates(counts, N, K):
    mb = _mb()
    dy, x, c = _data(counts, N, K)
    base = torch.randn(len(counts), N, K, generator=ref.gen(1))
    out = base.cuda()
    mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), c, out=out, accumulate=True)
    _check(out, dy, x, counts, base)
    for e, n in enumerate(counts):
        if n == 0:
            assert torch.equal(out[e].cpu(), base[e])
    assert mb.device_error() == 0


def test_weight_grad_keeps_experts_apart():
    """A NaN row reaches its own expert's gradient and no other, whatever step of rows it shares."""
    mb = _mb()
    counts = [5, 20, 3, 70, 1]
    dy, x, c = _data(counts, 64, 96)
    dy[5 + 4], x[5 + 20 + 1] = float("nan"), float("inf")      # experts 1 and 2
    got = mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), c, dtype=F32)
    clean = [0, 3, 4]
    assert got[1].isnan().all() and not got[2].isfinite().any() and got[clean].isfinite().all()
    want, _ = ref.weight_grad(dy, x, counts)
    assert torch.allclose(got[clean].cpu().double(), want[clean], atol=1e-4)


@pytest.mark.parametrize("counts", [list(range(1, 200)), [1, 16, 31, 32, 33, 47, 63, 65, 79, 81, 95, 96, 97, 113, 7],
                                    [3, 5, 190, 2, 191, 4, 192, 6, 193]])
@pytest.mark.parametrize("odd", [0, 1])
def test_weight_grad_of_every_length_between_poisoned_rows(counts, odd):
    """Every other expert's rows are NaN and infinite: wherever the others end, nothing of them comes in."""
    mb = _mb()
    dy, x, c = _data(counts, 144, 272, spare=3)
    clean = torch.zeros(sum(counts) + 3, dtype=torch.bool)
    row = 0
    for e, n in enumerate(counts):
        clean[row:row + n] = e % 2 == odd
        row += n
    pdy, px = dy.clone(), x.clone()
    pdy[~clean], px[~clean] = float("nan"), float("inf")
    got = mb.moe_grouped_weight_grad(pdy.cuda(), px.cuda(), c, dtype=F32)
    keep = list(range(odd, len(counts), 2))
    dy[~clean], x[~clean] = 0, 0
    _check(got[keep], dy[clean], x[clean], [counts[e] for e in keep])
    assert mb.device_error() == 0


def test_weight_grad_counts_on_the_device():
    """More counts than experts (counts[E] of the router), a negative count, a sum past the rows, no rows."""
    mb = _mb()
    dy, x, _ = _data([40], 32, 48)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    got = mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), i32([10, 30, 40]), E=2, dtype=F32)
    _check(got, dy, x, [10, 30])
    assert mb.device_error() == 0
    got = mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), i32([10, -4, 30]), dtype=F32)
    _check(got, dy, x, [10, 0, 30])
    assert mb.device_error() == mb.MOE_DEVERR_BAD_COUNT
    got = mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), i32([10, 2**31 - 1, 2**31 - 1]), dtype=F32)
    _check(got, dy, x, [10, 30, 0])
    assert mb.device_error() == mb.MOE_DEVERR_BAD_COUNT
    none = torch.empty(0, 32, dtype=BF16, device="cuda")
    got = mb.moe_grouped_weight_grad(none, torch.empty(0, 48, dtype=BF16, device="cuda"), i32([0, 0]),
                                     out=sentinel_like((2, 32, 48), BF16))
    assert not got.any() and mb.device_error() == 0


def test_weight_grad_many_experts():
    mb = _mb()
    counts = [(7 * e) % 5 for e in range(1024)]
    dy, x, c = _data(counts, 16, 32)
    _check(mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), c, dtype=F32), dy, x, counts)
    assert mb.device_error() == 0


def test_weight_grad_gradient_is_the_difference():
    """Along a random direction of the weights, the difference of sum(dy * (x w^T)) is <dw, direction>."""
    mb = _mb()
    counts = [21, 0, 50]
    dy, x, c = _data(counts, 48, 64)
    dw = mb.moe_grouped_weight_grad(dy.cuda(), x.cuda(), c, dtype=F32).cpu().double()
    w, d = torch.randn(2, 3, 48, 64, generator=ref.gen(3), dtype=torch.float64)
    owner = torch.repeat_interleave(torch.arange(3), torch.tensor(counts))
    f = lambda v: torch.einsum("rn,rnk,rk->", dy.double(), v[owner], x.double())
    diff = (f(w + 1e-4 * d) - f(w - 1e-4 * d)) / 2e-4
    _, mag = ref.weight_grad(dy, x, counts)
    assert abs(diff - (dw * d).sum()) <= 128 * 2.0 ** -23 * (mag * d.abs()).sum() + 1e-6


def test_weight_grad_python_refusals():
    mb = _mb()
    dy, x, c = _data([8], 32, 32)
    dy, x = dy.cuda(), x.cuda()
    with pytest.raises(TypeError):
        mb.moe_grouped_weight_grad(dy.float(), x, c)
    with pytest.raises(TypeError):
        mb.moe_grouped_weight_grad(dy, x, c.long())
    with pytest.raises(ValueError):
        mb.moe_grouped_weight_grad(dy, x[:4], c)
    with pytest.raises(ValueError):
        mb.moe_grouped_weight_grad(dy, x, c, E=2)
    with pytest.raises(ValueError):
        mb.moe_grouped_weight_grad(dy, x, c, accumulate=True)
    with pytest.raises(mb.MoEError):
        mb.moe_grouped_weight_grad(dy, x, c, out=torch.zeros(1, 32, 32, dtype=BF16, device="cuda"), accumulate=True)
    with pytest.raises(ValueError):
        mb.moe_grouped_weight_grad(dy, x, c, out=torch.empty(1, 32, 16, dtype=BF16, device="cuda"))


@pytest.mark.parametrize("counts,rows", [([10] + [0] * 31 + [2**31 - 1], [10] + [0] * 31 + [30]),
                                         ([2**31 - 1] * 70, [40] + [0] * 69),
                                         ([3] * 8 + [2**31 - 1] * 2 + [5] * 60, [3] * 8 + [16] + [0] * 61),
                                         ([7, -2**31] * 20, [7, 0] * 5 + [5, 0] + [0, 0] * 14)])
def test_weight_grad_from_a_checkpoint_of_oversized_counts(counts, rows):
    """Counts are cut where their sum passes the rows, however far it goes, for 8-bit rows as for bf16."""
    mb = _mb()
    dy, x, _ = _data([40], 32, 48)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    ck = mb.moe_checkpoint_pack(x.cuda())
    kept = mb.moe_checkpoint_unpack(ck)
    ws = torch.full((mb.moe_grouped_weight_grad_workspace_size(len(counts), 40, 32, 48, mb.MOE_DTYPE_E4M3),), 0xFF,
                    dtype=torch.uint8, device="cuda")                   # what was not unpacked is NaN
    got = mb.moe_grouped_weight_grad(dy.cuda(), ck, c, dtype=F32, workspace=ws)
    _check(got, dy, kept.cpu(), rows)
    assert mb.device_error() == mb.MOE_DEVERR_BAD_COUNT
