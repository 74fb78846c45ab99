"""Weight gradients of which a pair of CTAs computes many tiles: long and short experts by turns in its
two accumulators, experts cut into parts among others that are whole, more experts than are ordered.

The definition is evaluated in 64 bits on the GPU, an expert at a time; the bound is that of
tests/test_gpu_weight_grad.py."""
import pytest
import torch

from tests.test_gpu_train import BF16, F32, _mb

pytestmark = pytest.mark.gpu

LONG_AND_SHORT = [2000, 900, 300, 257, 256, 97, 5, 0, 1]
CASES = {
    # 81 tiles of each expert, about ten for each pair; the rows around 96-row stages and 256
    "long and short": (LONG_AND_SHORT, 2304, 2304),
    "ragged edges": ([1, 770, 0, 95, 96, 97, 400, 16, 17, 1300], 2320, 2288),
    "one long, many short": ([5000] + [3, 40, 0, 17, 33] * 6, 2560, 2048),
    "even": ([200, 201, 199, 208, 192, 193, 207, 195], 2304, 2304),
    # rows too few to cut; up to 256 experts and above, above 384 units
    "200 experts": ([(7 * e) % 9 for e in range(200)], 512, 528),
    "300 experts": ([(5 * e) % 7 for e in range(300)], 544, 512),
    "600 experts": ([(3 * e) % 4 for e in range(600)], 512, 512),
    # cut into parts: experts above and below a part's rows, more tiles than pairs
    "parts of 1824": ([5000, 100, 961, 960, 0, 1500, 30], 1024, 1024),
    "parts of 960": ([5000, 100, 961, 960, 0, 1919, 1920, 1921, 30] + [50, 0, 97] * 7, 512, 512),
    "one part more": ([959, 960, 961, 962, 4] * 4, 768, 272),
}


def _make(counts, N, K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    a = sum(counts) + 3
    dy = torch.randn(a, N, generator=g, device="cuda").to(BF16)
    x = torch.randn(a, K, generator=g, device="cuda").to(BF16)
    dy[sum(counts):], x[sum(counts):] = float("nan"), float("inf")
    return dy, x, torch.tensor(counts, dtype=torch.int32, device="cuda")


def _check(got, dy, x, counts, base=None):
    at, step = 0, 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -23
    for e, n in enumerate(counts):
        a, b = dy[at:at + n].double(), x[at:at + n].double()
        want, mag = a.T @ b, a.abs().T @ b.abs()
        bound = (n + 64) * 2.0 ** -23 * mag + want.abs() * step
        if base is not None:
            old = base[e].double()
            want, bound = want + old, bound + 2.0 ** -23 * (old.abs() + (want + old).abs())
        bad = ~((got[e].double() - want).abs() <= bound)
        assert not bad.any(), f"expert {e} of {n} rows: {int(bad.sum())} of {bad.numel()} outside the bound"
        at += n


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("form", ["bf16", "f32", "accumulate", "checkpoint"])
def test_weight_grad_of_many_tiles(name, form):
    mb = _mb()
    counts, N, K = CASES[name]
    dy, x, c = _make(counts, N, K, len(name))
    base, out = None, None
    if form == "accumulate":
        base = torch.randn(len(counts), N, K, device="cuda")
        out = base.clone()
    rows = x
    if form == "checkpoint":
        x = mb.moe_checkpoint_pack(x)
        rows = mb.moe_checkpoint_unpack(x)
    kw = dict(dtype=F32 if form != "bf16" else BF16, accumulate=base is not None)
    got = mb.moe_grouped_weight_grad(dy, x, c, out=out, **kw)
    _check(got, dy, rows, counts, base)
    again = mb.moe_grouped_weight_grad(dy, x, c, out=None if base is None else base.clone(), **kw)
    assert torch.equal(got, again)
    assert mb.device_error() == 0


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("name", ["ragged edges", "one long, many short", "parts of 960"])
def test_weight_grad_of_many_tiles_between_poisoned_rows(name, odd):
    """Every other expert's rows are NaN and infinite: nothing of them comes into the others'."""
    mb = _mb()
    counts, N, K = CASES[name]
    dy, x, c = _make(counts, N, K, 7)
    clean, at = [], 0
    for e, n in enumerate(counts):
        if e % 2 == odd:
            clean.append(e)
        else:
            dy[at:at + n], x[at:at + n] = float("nan"), float("inf")
        at += n
    got = mb.moe_grouped_weight_grad(dy, x, c)
    at = 0
    for e, n in enumerate(counts):
        if e in clean:
            _check(got[e:e + 1], dy[at:at + n], x[at:at + n], [n])
        at += n
    assert mb.device_error() == 0
