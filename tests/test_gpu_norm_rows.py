"""Layer norm of whole, aligned rows where a group of threads takes many of them, one after the
other: the rows' places on chip are used again and again, and the weights' gradients add up over them.

The bounds are those of a row and of a column's sum in the other tests of the norm; the definitions
are evaluated in 64 bits on the GPU."""
import pytest
import torch

from tests import train_ref as ref
from tests.helpers import is_sentinel, sentinel_like
from tests.test_gpu_train import BF16, F32, ROW, _i32, _mb, _norm_bound, _step

pytestmark = pytest.mark.gpu

# (rows, columns): more rows a group than twice the places of its ring, which are at most 6
SHAPES = [(14000, 640), (24000, 520), (5000, 4096), (2600, 7168), (900, 16384), (2200, 11008), (60000, 256),
          (34000, 512), (61000, 64)]


def _near(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("past", [0, 777])
def test_layer_norm_of_many_whole_rows(T, D, dtype, wdtype, past):
    mb = _mb()
    g = torch.Generator(device="cuda")
    g.manual_seed(T + D)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    n = T - past
    x = (rnd(T, D) * torch.exp(rnd(T, 1)) + rnd(1, D)).to(dtype)
    dy, res = rnd(T, D).to(dtype), rnd(T, D).to(dtype)
    gamma, beta = (1 + 0.2 * rnd(D)).to(wdtype), rnd(D).to(wdtype)
    x[n:], dy[n:], res[n:] = float("nan"), float("inf"), float("nan")
    valid = _i32(n) if past else None
    y, m, r, dx = sentinel_like((T, D), dtype), sentinel_like((T,), F32), sentinel_like((T,), F32), sentinel_like((T, D), dtype)
    mb.moe_layer_norm(x, gamma, beta, valid, eps=1e-3, out=y, mean=m, rstd=r)
    xv = x[:n]
    want, mean, rstd = ref.layer_norm(xv, gamma, beta, 1e-3)
    size = xv.double().abs().mean(1)
    _near(y[:n], want, _norm_bound(xv, gamma, beta, mean, rstd, dtype, want), "y")
    _near(m[:n], mean, ROW * size + 1e-30, "mean")
    _near(r[:n], rstd, ROW * rstd * (1 + (rstd * size) ** 2), "rstd")
    mean, rstd = mean.float(), rstd.float()
    full = lambda v: torch.cat([v, torch.full((past,), float("nan"), device="cuda")])
    _, dgamma, dbeta = mb.moe_layer_norm_backward(dy, x, gamma, full(mean), full(rstd), valid, residual_grad=res, out=dx)
    for t in (y, m, r, dx):
        assert is_sentinel(t[n:])
    wdx, wg, wb = ref.layer_norm_backward(dy[:n], xv, gamma, mean, rstd)
    wdx = wdx + res[:n].double()
    xh = ((xv.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs()
    a = dy[:n].double().abs()
    gg = a * gamma.double().abs()
    err = ROW * rstd.double()[:, None] * (gg + gg.mean(1, keepdim=True) + 2 * xh * (gg * xh).mean(1, keepdim=True))
    _near(dx[:n], wdx, _step(wdx, dtype) + err + 2.0 ** -23 * res[:n].double().abs(), "dx")
    bound = (T + 64) * 2.0 ** -24
    _near(dgamma, wg, bound * (a * xh).sum(0) + 1e-30, "dgamma")
    _near(dbeta, wb, bound * a.sum(0) + 1e-30, "dbeta")
    assert mb.device_error() == 0


@pytest.mark.parametrize("T,D", [(14000, 640), (5000, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_norm_of_many_rows_gives_the_same_bytes_again(T, D, dtype):
    mb = _mb()
    x, dy = torch.randn(T, D, device="cuda").to(dtype), torch.randn(T, D, device="cuda").to(dtype)
    gamma = torch.rand(D, device="cuda")
    first = mb.moe_layer_norm(x, gamma)
    grads = mb.moe_layer_norm_backward(dy, x, gamma, *first[1:])
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(first, mb.moe_layer_norm(x, gamma)))
        assert all(torch.equal(a, b) for a, b in zip(grads, mb.moe_layer_norm_backward(dy, x, gamma, *first[1:])))
