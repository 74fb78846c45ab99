"""Layer norm, balance loss and 8-bit checkpoints on the GPU against their definitions in 64 bits,
and their gradients against differences of the forward too.

Bounds.  A bf16 result is within one bf16 step (2^-8 of its value, twice its rounding) plus the fp32
error; an fp32 error is a count of 2^-24 roundings times the magnitudes summed:
  row sums      at most 16384 / 256 adds in a row and a tree: below 2^8 roundings, 2^-16
  column sums   at most one add for each token: T roundings
  exp           its argument's rounding is |x| log2(e) 2^-24 of the result, below 2^-17 for |x| <= 80
"""
import pytest
import torch

from tests import train_ref as ref
from tests.helpers import is_sentinel, sentinel_like

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ROW = 2.0 ** -16
EXP = 2.0 ** -17


def _mb():
    from moe_token_routing_index_gb300 import binding

    return binding


def _i32(n):
    return torch.tensor([n], dtype=torch.int32, device="cuda")


def _step(want, dtype):
    return want.abs() * 2.0 ** (-8 if dtype == BF16 else -23)


def _close(got, want, bound, what):
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, " \
                          f"worst {float(((got - want).abs() / bound.clamp(min=1e-300)).max()):.3g} of the bound"


# ---------------------------------------------------------------- layer norm

# one token to many; one column to the most; widths on both sides of every vector and tile width
NORM_SHAPES = [(1, 1), (1, 5120), (3, 7), (2, 16384), (5, 8), (33, 96), (64, 256), (9, 1000), (7, 2051), (130, 4096),
               (701, 640), (17, 7168), (3, 16376), (2, 16383), (1500, 64)]


def _norm_data(T, D, dtype, wdtype, seed=0, scale=1.0):
    g = ref.gen(seed + 31 * T + D)
    x = (scale * (torch.randn(T, D, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
                  + torch.randn(1, D, generator=g))).to(dtype)
    gamma = (1 + 0.2 * torch.randn(D, generator=g)).to(wdtype)
    beta = torch.randn(D, generator=g).to(wdtype)
    dy = torch.randn(T, D, generator=g).to(dtype)
    return x, gamma, beta, dy


def _norm_bound(x, gamma, beta, mean, rstd, dtype, y):
    xh = ((x.double() - mean[:, None]) * rstd[:, None]).abs()
    off = (rstd * x.double().abs().mean(1))[:, None]
    return _step(y, dtype) + ROW * (gamma.double().abs() * (xh + 1 + off) + (0 if beta is None else beta.double().abs()))


@pytest.mark.parametrize("T,D", NORM_SHAPES)
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_layer_norm(T, D, dtype, wdtype):
    mb = _mb()
    x, gamma, beta, _ = _norm_data(T, D, dtype, wdtype)
    for b in (beta, None):
        want, mean, rstd = ref.layer_norm(x, gamma, b, 1e-3)
        y, m, r = mb.moe_layer_norm(x.cuda(), gamma.cuda(), None if b is None else b.cuda(), eps=1e-3)
        _close(y, want, _norm_bound(x, gamma, b, mean, rstd, dtype, want), "y")
        _close(m, mean, ROW * x.double().abs().mean(1) + 1e-30, "mean")
        _close(r, rstd, ROW * rstd * (1 + (rstd * x.double().abs().mean(1)) ** 2), "rstd")
    assert mb.device_error() == 0


@pytest.mark.parametrize("T,D", NORM_SHAPES)
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_layer_norm_backward(T, D, dtype, wdtype):
    mb = _mb()
    x, gamma, beta, dy = _norm_data(T, D, dtype, wdtype, seed=5)
    _, mean, rstd = ref.layer_norm(x, gamma, beta, 1e-3)
    mean, rstd = mean.float(), rstd.float()
    res = torch.randn(T, D, generator=ref.gen(9)).to(dtype)
    dx, dgamma, dbeta = ref.layer_norm_backward(dy, x, gamma, mean, rstd)
    xh = ((x.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs()
    g = (dy.double() * gamma.double()).abs()
    err = ROW * rstd.double()[:, None] * (g + g.mean(1, keepdim=True) + 2 * xh * (g * xh).mean(1, keepdim=True))
    n = (T + 64) * 2.0 ** -24
    cu = [t.cuda() for t in (dy, x, gamma, mean, rstd)]
    for r in (None, res):
        want = dx if r is None else dx + r.double()
        a, b, c = mb.moe_layer_norm_backward(*cu, residual_grad=None if r is None else r.cuda())
        _close(a, want, _step(want, dtype) + err + (0 if r is None else 2.0 ** -23 * r.double().abs()), "dx")
        _close(b, dgamma, n * (dy.double().abs() * xh).sum(0) + 1e-30, "dgamma")
        _close(c, dbeta, n * dy.double().abs().sum(0) + 1e-30, "dbeta")
    a2, b2, c2 = mb.moe_layer_norm_backward(*cu, residual_grad=res.cuda(), with_beta=False)
    assert torch.equal(a2, a) and torch.equal(b2, b) and c2 is None       # the same bytes again
    assert mb.device_error() == 0


def test_layer_norm_gradient_is_the_difference():
    """The kernel's gradients along random directions against central differences of the definition."""
    mb = _mb()
    x, gamma, beta, dy = _norm_data(23, 777, F32, F32, seed=2)
    _, mean, rstd = mb.moe_layer_norm(x.cuda(), gamma.cuda(), beta.cuda())
    dx, dgamma, dbeta = mb.moe_layer_norm_backward(dy.cuda(), x.cuda(), gamma.cuda(), mean, rstd)
    f = lambda a, b, c: (ref.layer_norm(a, b, c, 1e-5)[0] * dy.double()).sum()
    args = [x.double(), gamma.double(), beta.double()]
    for i, grad in enumerate((dx, dgamma, dbeta)):
        d = torch.randn(args[i].shape, generator=ref.gen(i), dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-6 * d, args[i] - 1e-6 * d
        diff = (f(*up) - f(*down)) / 2e-6
        terms = grad.cpu().double() * d
        # mean and rstd carry fp32 errors into dx; each term of the sum is within 2^-14 of its scale
        assert abs(diff - terms.sum()) <= 2.0 ** -14 * terms.abs().sum()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_norm_strided_rows_and_valid_tokens(dtype):
    mb = _mb()
    for T, D, ld, off, valid in ((37, 256, 264, 0, 20), (37, 255, 301, 1, 36), (40, 640, 1280, 640, 40), (9, 96, 97, 3, 0),
                                 (300, 128, 160, 8, 177)):
        g = ref.gen(D + T)
        wide = torch.randn(T, ld + off, generator=g).to(dtype)
        x = wide[:, off:off + D]
        x[valid:] = float("nan")                       # rows past the count hold anything
        gamma, beta = torch.randn(D, generator=g), torch.randn(D, generator=g)
        dy = torch.randn(T, D, generator=g).to(dtype)
        dy[valid:] = float("inf")
        xc = wide.cuda()[:, off:off + D]
        y, m, r = (sentinel_like((T, D), dtype), sentinel_like((T,), F32), sentinel_like((T,), F32))
        mb.moe_layer_norm(xc, gamma.cuda(), beta.cuda(), _i32(valid), out=y, mean=m, rstd=r)
        assert is_sentinel(y[valid:]) and is_sentinel(m[valid:]) and is_sentinel(r[valid:])
        want, mean, rstd = ref.layer_norm(x[:valid], gamma, beta, 1e-5)
        _close(y[:valid], want, _norm_bound(x[:valid], gamma, beta, mean, rstd, dtype, want), "y")
        dx = sentinel_like((T, D), dtype)
        _, dgamma, dbeta = mb.moe_layer_norm_backward(dy.cuda(), xc, gamma.cuda(), m, r, _i32(valid), out=dx)
        assert is_sentinel(dx[valid:])
        wdx, wg, wb = ref.layer_norm_backward(dy[:valid], x[:valid], gamma, mean, rstd)
        xh = ((x[:valid].double() - mean[:, None]) * rstd[:, None]).abs()
        gg = (dy[:valid].double() * gamma.double()).abs()
        # the kernel's own mean and rstd: their errors enter xh
        err = 4 * ROW * rstd[:, None] * (gg + gg.mean(1, keepdim=True) + (2 * xh + 1) * (gg * (xh + 1)).mean(1, keepdim=True))
        _close(dx[:valid], wdx, _step(wdx, dtype) + err, "dx")
        n = (T + 64) * 2.0 ** -24 + ROW
        _close(dgamma, wg, n * (dy[:valid].double().abs() * (xh + 1)).sum(0) + 1e-30, "dgamma")
        _close(dbeta, wb, n * dy[:valid].double().abs().sum(0) + 1e-30, "dbeta")
    assert mb.device_error() == 0


# rows that start inside 16 bytes: widths on both sides of the pieces', one row a group to many
ODD_ROWS = [(305, 513), (1217, 519), (2000, 521), (310, 1001), (900, 2051), (2000, 2055), (700, 2601), (1300, 4097),
            (306, 5121), (305, 16383)]


@pytest.mark.parametrize("T,D", ODD_ROWS)
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_layer_norm_many_odd_rows(T, D, dtype, wdtype):
    test_layer_norm(T, D, dtype, wdtype)
    test_layer_norm_backward(T, D, dtype, wdtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D,gap,valid", [(640, 1003, 0, 640), (640, 1003, 8, 640), (1300, 515, 40, 1299),
                                           (1300, 2050, 8, 700), (1300, 2602, 8, 700), (400, 4097, 16, 0),
                                           (311, 777, 3, 310)])
def test_layer_norm_odd_rows_stay_in_their_memory(T, D, gap, valid, dtype):
    """Rows with gaps and NaN around them, outputs in the middle of a larger buffer that keeps its bytes."""
    mb = _mb()
    g = ref.gen(T + D + gap)
    wide = torch.full((T + 2, D + gap), float("nan")).to(dtype)
    wide[1:-1, :D] = torch.randn(T, D, generator=g).to(dtype)
    wide[1 + valid:] = float("nan")
    flat = torch.full((8 + T * (D + gap) + 8,), float("nan")).to(dtype)
    flat[8:-8] = wide[1:-1].reshape(-1)
    fc = flat.cuda()
    xc = fc[8:-8].view(T, D + gap)[:, :D]
    x = wide[1:1 + valid, :D]
    gamma, beta = torch.randn(D, generator=g), torch.randn(D, generator=g)
    dy = torch.full((8 + T * D + 8,), float("inf")).to(dtype)
    dy[8:8 + valid * D] = torch.randn(valid * D, generator=g).to(dtype)
    dyc, dy = dy.cuda()[8:-8].view(T, D), dy[8:8 + valid * D].view(valid, D)
    ys, dxs = sentinel_like((16 + T * D,), dtype), sentinel_like((16 + T * D,), dtype)
    y, dx = ys[8:-8].view(T, D), dxs[8:-8].view(T, D)
    _, m, r = mb.moe_layer_norm(xc, gamma.cuda(), beta.cuda(), _i32(valid), out=y)
    want, mean, rstd = ref.layer_norm(x, gamma, beta, 1e-5)
    _close(y[:valid], want, _norm_bound(x, gamma, beta, mean, rstd, dtype, want), "y")
    _, dgamma, dbeta = mb.moe_layer_norm_backward(dyc, xc, gamma.cuda(), m, r, _i32(valid), out=dx)
    for buf in (ys, dxs):
        assert is_sentinel(buf[:8]) and is_sentinel(buf[8 + valid * D:])
    wdx, wg, wb = ref.layer_norm_backward(dy, x, gamma, mean, rstd)
    xh = ((x.double() - mean[:, None]) * rstd[:, None]).abs()
    gg = (dy.double() * gamma.double()).abs()
    # the kernel's own mean and rstd: their errors enter xh
    err = 4 * ROW * rstd[:, None] * (gg + gg.mean(1, keepdim=True) + (2 * xh + 1) * (gg * (xh + 1)).mean(1, keepdim=True))
    _close(dx[:valid], wdx, _step(wdx, dtype) + err, "dx")
    n = (T + 64) * 2.0 ** -24 + ROW
    _close(dgamma, wg, n * (dy.double().abs() * (xh + 1)).sum(0) + 1e-30, "dgamma")
    _close(dbeta, wb, n * dy.double().abs().sum(0) + 1e-30, "dbeta")
    assert mb.device_error() == 0


def test_layer_norm_empty_constant_and_non_finite_rows():
    mb = _mb()
    gamma, beta = torch.full((48,), 2.0).cuda(), torch.full((48,), 0.5).cuda()
    # no tokens: zero weight gradients, nothing else
    e = torch.empty(0, 48, device="cuda")
    y, m, r = mb.moe_layer_norm(e, gamma, beta)
    dx, dg, db = mb.moe_layer_norm_backward(e, e, gamma, m, r)
    assert y.shape == (0, 48) and dx.shape == (0, 48) and not dg.any() and not db.any()
    # a constant row is beta; an infinite one is NaN and leaves its neighbours alone
    x = torch.randn(4, 48, generator=ref.gen(0))
    x[1] = 3.0
    x[2, 7] = float("inf")
    y, m, r = mb.moe_layer_norm(x.cuda(), gamma, beta)
    assert torch.equal(y[1].cpu(), torch.full((48,), 0.5)) and y[2].isnan().all()
    assert y[[0, 3]].isfinite().all()
    # values whose squares overflow in 16 bits, and a count outside [0, T]
    big = (x[[0, 3]] * 2.0 ** 40).to(BF16)
    y, _, _ = mb.moe_layer_norm(big.cuda(), gamma, beta, _i32(99))
    want, mean, rstd = ref.layer_norm(big, gamma.cpu(), beta.cpu(), 1e-5)
    _close(y, want, _norm_bound(big, gamma.cpu(), beta.cpu(), mean, rstd, BF16, want), "y")
    assert mb.device_error() == mb.MOE_DEVERR_BAD_COUNT


# -------------------------------------------------------------- balance loss

KINDS = ["scores", "softmax", "sigmoid"]
BALANCE_SHAPES = [(1, 1, 1), (1, 8, 8), (64, 8, 1), (130, 16, 2), (77, 33, 5), (300, 64, 6), (513, 128, 8), (40, 200, 3),
                  (257, 256, 8), (12, 512, 4), (9, 1000, 10), (20, 1024, 1), (4099, 12, 2)]


def _kind(mb, kind):
    return dict(scores=mb.MOE_BALANCE_SCORES, softmax=mb.MOE_BALANCE_SOFTMAX, sigmoid=mb.MOE_BALANCE_SIGMOID)[kind]


def _router(T, E, kind, dtype, seed=0):
    g = ref.gen(seed + T + 7 * E)
    a = 2 * torch.randn(T, E, generator=g) + torch.randn(E, generator=g)
    return (torch.sigmoid(a) if kind == "scores" else a).to(dtype)


def _check_balance(mb, a, ac, kind, k, valid, counts_in=None):
    """Forward and backward of the first `valid` rows of a (its device copy ac, any strides)."""
    E, coef = a.shape[1], 0.37
    rows = a[:valid]
    nv = None if valid == a.shape[0] else _i32(valid)
    loss, counts, mean = mb.moe_balance_loss(ac, k, nv, kind=_kind(mb, kind), coefficient=coef, counts=counts_in)
    if counts_in is None:
        assert torch.equal(counts.cpu(), ref.top_counts(rows, k))
    else:
        assert counts is counts_in
    wl, wm = ref.balance_loss(rows, kind, counts.cpu(), k, coef)
    n = (valid + 1024) * 2.0 ** -24 + EXP
    _close(mean, wm, n * wm + 1e-30, "mean_probs")
    _close(loss[0], wl, n * wl + 1e-30, "loss")
    dloss = torch.tensor([1.5])
    want, scale = ref.balance_loss_backward(rows, kind, counts.cpu(), k, coef, 1.5)
    bound = _step(want, a.dtype) + 2 * EXP * scale + 1e-38
    out = sentinel_like(a.shape, a.dtype)
    kw = dict(kind=_kind(mb, kind), coefficient=coef, dloss=dloss.cuda())
    mb.moe_balance_loss_backward(ac, counts, k, nv, out=out, **kw)
    _close(out[:valid], want, bound, "dscores")
    assert is_sentinel(out[valid:])
    base = torch.randn(a.shape, generator=ref.gen(4)).mul(coef / max(valid, 1)).to(a.dtype)
    acc = base.cuda()
    mb.moe_balance_loss_backward(ac, counts, k, nv, out=acc, accumulate=True, **kw)
    want = want + base[:valid].double()
    _close(acc[:valid], want, bound + _step(want, a.dtype) + 2.0 ** -23 * base[:valid].double().abs(), "accumulated")
    assert torch.equal(acc[valid:].cpu(), base[valid:])
    assert mb.device_error() == 0


@pytest.mark.parametrize("T,E,k", BALANCE_SHAPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_balance_loss(T, E, k, kind, dtype):
    mb = _mb()
    a = _router(T, E, kind, dtype)
    _check_balance(mb, a, a.cuda(), kind, k, T)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_balance_loss_strides_valid_counts(kind, dtype):
    mb = _mb()
    for T, E, k, valid in ((60, 24, 3, 41), (100, 130, 4, 1), (33, 16, 2, 0), (2000, 64, 6, 1999)):
        a = _router(T, E, kind, dtype, seed=3)
        a[valid:] = float("nan")
        wide = torch.full((T, E + 5), float("nan")).to(dtype)
        wide[:, 3:3 + E] = a
        _check_balance(mb, a, wide.cuda()[:, 3:3 + E], kind, k, valid)           # padded, unaligned rows
        _check_balance(mb, a, a.T.contiguous().cuda().T, kind, k, valid)         # expert-major
        counts = ref.top_counts(a[:valid], k).cuda()
        _check_balance(mb, a, a.cuda(), kind, k, valid, counts_in=counts)


@pytest.mark.parametrize("T,E,k,valid", [(8193, 33, 8, 8193), (9001, 61, 8, 9000), (8200, 128, 9, 8200),
                                         (12001, 128, 8, 11999), (8300, 100, 1, 8299)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_balance_loss_of_many_tokens(T, E, k, valid, kind, dtype):
    """Every third row of few different values, so that equal ones straddle the choice; masked experts
    in every fifth; NaN past the count."""
    mb = _mb()
    a = _router(T, E, kind, dtype, seed=6)
    a[::3] = (a[::3] * 4).round() / 4
    a[::5, E - 3:] = 0 if kind == "scores" else float("-inf")
    a[valid:] = float("nan")
    _check_balance(mb, a, a.cuda(), kind, k, valid)
    wide = torch.full((T, E + 3), float("nan")).to(dtype)
    wide[:, 1:1 + E] = a
    _check_balance(mb, a, wide.cuda()[:, 1:1 + E], kind, k, valid)


@pytest.mark.parametrize("T,E,k", [(700, 256, 8), (700, 255, 7), (300, 512, 8), (200, 700, 5), (100, 1024, 8),
                                   (64, 1024, 9)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_balance_counts_of_equal_scores(T, E, k, dtype):
    mb = _mb()
    a = (_router(T, E, "softmax", F32, seed=12) * 2).round().to(dtype)
    a[7] = float("-inf")
    a[9, 5:] = float("-inf")
    _check_balance(mb, a, a.cuda(), "softmax", k, T)


def test_balance_counts_are_the_routers():
    mb = _mb()
    for T, E, k in ((513, 128, 8), (64, 8, 1), (4096, 16, 2)):
        s = torch.sigmoid(torch.randn(T, E, generator=ref.gen(T))).to(BF16).cuda()   # many equal scores
        _, counts, _ = mb.moe_balance_loss(s, k)
        assert torch.equal(counts, mb.moe_route(s, k)["counts"])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_balance_masked_rows_and_experts(dtype):
    """-inf and the type's lowest value as masks, rows of them alone, scores that are all zero."""
    mb = _mb()
    low = torch.finfo(dtype).min
    a = _router(50, 40, "softmax", dtype, seed=8)
    a[:, 30:] = float("-inf")
    a[5] = float("-inf")                 # nothing left: p = 0
    a[6] = low                           # the lowest value everywhere: p uniform
    a[7, 1:] = low
    _check_balance(mb, a, a.cuda(), "softmax", 4, 50)
    s = _router(50, 40, "scores", dtype, seed=8)
    s[:, 30:] = 0
    s[5] = 0
    _check_balance(mb, s, s.cuda(), "scores", 4, 50)
    b = _router(50, 40, "sigmoid", dtype, seed=8)
    b[:, 30:] = float("-inf")
    b[5] = float("-inf")
    b[6, :3] = float("inf")
    _check_balance(mb, b, b.cuda(), "sigmoid", 4, 50)


@pytest.mark.parametrize("kind", KINDS)
def test_balance_gradient_is_the_difference(kind):
    mb = _mb()
    a = _router(37, 24, kind, F32, seed=1)
    _, counts, _ = mb.moe_balance_loss(a.cuda(), 3, kind=_kind(mb, kind))
    grad = mb.moe_balance_loss_backward(a.cuda(), counts, 3, kind=_kind(mb, kind)).cpu().double()
    d = torch.randn(37, 24, generator=ref.gen(2), dtype=torch.float64)
    f = lambda v: ref.balance_loss(v, kind, counts.cpu(), 3, 1.0)[0]
    diff = (f(a.double() + 1e-6 * d) - f(a.double() - 1e-6 * d)) / 2e-6
    _, scale = ref.balance_loss_backward(a, kind, counts.cpu(), 3, 1.0, 1.0)
    assert abs(diff - (grad * d).sum()) <= 2 * EXP * (scale * d.abs()).sum() + 1e-8


def test_balance_no_tokens_and_bad_count():
    mb = _mb()
    loss, counts, mean = mb.moe_balance_loss(torch.empty(0, 6, device="cuda"), 2)
    assert loss.item() == 0 and not counts.any() and not mean.any()
    assert mb.moe_balance_loss_backward(torch.empty(0, 6, device="cuda"), counts, 2).shape == (0, 6)
    assert mb.device_error() == 0
    a = _router(8, 6, "softmax", F32)
    loss, _, _ = mb.moe_balance_loss(a.cuda(), 2, _i32(-3), kind=mb.MOE_BALANCE_SOFTMAX)
    assert loss.item() == 0 and mb.device_error() == mb.MOE_DEVERR_BAD_COUNT


# --------------------------------------------------------------- checkpoints

CK_SHAPES = [(1, 16), (1, 2048), (3, 112), (5, 128), (7, 144), (33, 272), (64, 512), (130, 1456), (517, 80), (2, 16384)]


def _ck_rows(a, W, seed=0):
    """Rows of very different sizes, with zeros and the values that an 8-bit format handles specially."""
    g = ref.gen(seed + a + 3 * W)
    v = torch.randn(a, W, generator=g) * torch.exp2(torch.randint(-30, 30, (a, 1), generator=g).float())
    v[torch.rand(a, W, generator=g) < 0.05] = 0
    v = v.to(BF16)
    for i, special in enumerate((0.0, 448.0, 449.0, -1.75, 3.39e38, 1e-40, 2.0 ** -110)):
        if i < a:
            v[i, (5 * i) % W] = special
    if a > 2:
        v[2, :128] = 0
        v[a - 1, 0], v[a - 1, W // 2], v[a - 1, W - 1] = float("nan"), float("inf"), float("-inf")
    return v


def _same_codes(got, want):
    """Bit-equal codes; NaN codes of either sign are one value."""
    g, w = got.cpu().view(torch.uint8), want.view(torch.uint8)
    return bool(((g == w) | (((g & 0x7F) == 0x7F) & ((w & 0x7F) == 0x7F))).all())


def _same_bf16(got, want):
    got, want = got.cpu(), want.to(BF16)
    return bool(((got.view(torch.int16) == want.view(torch.int16)) | (got.isnan() & want.isnan())).all())


@pytest.mark.parametrize("a,W", CK_SHAPES)
def test_checkpoint_is_bit_exact(a, W):
    mb = _mb()
    v = _ck_rows(a, W)
    codes, exps = ref.pack(v)
    wide = torch.cat([v, v[:, :8]], 1).cuda()
    for x in (v.cuda(), wide[:, :W]):
        ck = mb.moe_checkpoint_pack(x)
        assert torch.equal(ck.exponents.cpu(), exps) and _same_codes(ck.codes, codes)
    assert _same_bf16(mb.moe_checkpoint_unpack(ck), ref.unpack(codes, exps))
    assert mb.device_error() == 0


@pytest.mark.parametrize("a,H", [(1, 16), (3, 112), (33, 272), (64, 512), (130, 1456), (5, 8192)])
def test_silu_mul_checkpoint_and_backward(a, H):
    mb = _mb()
    y = torch.cat([3 * torch.randn(a, H, generator=ref.gen(a)), _ck_rows(a, H, 1).float()], 1).to(BF16)
    y[0, :4] = torch.tensor([60.0, -60.0, 300.0, -300.0])
    yc = y.cuda()
    z, ck = mb.moe_silu_mul_checkpoint(yc)
    assert torch.equal(z.view(torch.int16), mb.moe_silu_mul(yc).view(torch.int16))
    nb = -(-H // 128)
    for i, half in enumerate((y[:, :H], y[:, H:])):
        codes, exps = ref.pack(half)
        assert torch.equal(ck.exponents[:, i * nb:(i + 1) * nb].cpu(), exps)
        assert _same_codes(ck.codes[:, i * H:(i + 1) * H].contiguous(), codes)
    dz = torch.randn(a, H, generator=ref.gen(3)).to(BF16)
    dy, z2 = mb.moe_silu_mul_backward(ck, dz.cuda())
    k0 = ref.unpack(ck.codes[:, :H].cpu(), ck.exponents[:, :nb].cpu())
    k1 = ref.unpack(ck.codes[:, H:].cpu(), ck.exponents[:, nb:].cpu())
    g0, g1 = ref.silu_mul_backward(k0, k1, dz.double())
    fine = torch.isfinite(k1) & torch.isfinite(k0)
    s = torch.sigmoid(k0)
    err0 = EXP * (dz.double() * k1).abs() * s * (1 + k0.abs())
    zero = torch.zeros((), dtype=torch.float64)
    for got, want, err in ((dy[:, :H], g0, err0), (dy[:, H:], g1, EXP * g1.abs()),
                           (z2, ref.silu_mul(k0, k1), EXP * (k0 * s * k1).abs())):
        over = want.abs() > 3.38e38             # past bf16's largest value: rounds to it or to infinity
        use = fine & ~over
        pick = lambda t: torch.where(use, t, zero)
        _close(torch.where(use.cuda(), got.double(), 0.0), pick(want), pick(_step(want, BF16) + err) + 2.0 ** -126, "silu")
    assert (dy[:, :H].cpu().isnan() == g0.isnan()).all() and (z2.cpu().isnan() == (k0 * s * k1).isnan()).all()
    dy2, none = mb.moe_silu_mul_backward(ck, dz.cuda(), with_z=False)
    assert none is None and torch.equal(dy2.view(torch.int16), dy.view(torch.int16))
    assert mb.device_error() == 0


@pytest.mark.parametrize("a,H,valid", [(9, 48, 4), (70, 272, 0), (33, 1456, 33), (400, 128, 399)])
def test_checkpoint_rows_past_the_count_are_untouched(a, H, valid):
    mb = _mb()
    y = torch.randn(a, 2 * H + 8, generator=ref.gen(a)).to(BF16).cuda()
    nb = -(-H // 128)
    n = _i32(valid)
    z = sentinel_like((a, H), BF16)
    ck = mb.Checkpoint(sentinel_like((a, 2 * H), torch.float8_e4m3fn), sentinel_like((a, 2 * nb), torch.uint8), 2)
    mb.moe_silu_mul_checkpoint(y[:, :2 * H], H, n, out=z, checkpoint=ck)
    full, fck = mb.moe_silu_mul_checkpoint(y[:, :2 * H], H)
    u8 = torch.uint8
    assert torch.equal(z[:valid], full[:valid]) and torch.equal(ck.exponents[:valid], fck.exponents[:valid])
    assert torch.equal(ck.codes[:valid].view(u8), fck.codes[:valid].view(u8))
    assert is_sentinel(z[valid:]) and is_sentinel(ck.codes[valid:]) and is_sentinel(ck.exponents[valid:])
    dz = torch.randn(a, H, generator=ref.gen(1)).to(BF16).cuda()
    dy, z2 = sentinel_like((a, 2 * H), BF16), sentinel_like((a, H), BF16)
    mb.moe_silu_mul_backward(ck, dz, n, out=dy, z=z2)
    fdy, fz = mb.moe_silu_mul_backward(fck, dz)
    assert torch.equal(dy[:valid], fdy[:valid]) and torch.equal(z2[:valid], fz[:valid])
    assert is_sentinel(dy[valid:]) and is_sentinel(z2[valid:])
    one = mb.Checkpoint(sentinel_like((a, H), torch.float8_e4m3fn), sentinel_like((a, nb), torch.uint8))
    mb.moe_checkpoint_pack(y[:, :H], n, checkpoint=one)
    assert is_sentinel(one.codes[valid:]) and is_sentinel(one.exponents[valid:])
    x = sentinel_like((a, H), BF16)
    mb.moe_checkpoint_unpack(one, n, out=x)
    assert is_sentinel(x[valid:]) and torch.equal(x[:valid], mb.moe_checkpoint_unpack(mb.moe_checkpoint_pack(y[:, :H]))[:valid])
    assert mb.device_error() == 0


def test_silu_gradient_is_the_difference():
    mb = _mb()
    y = 2 * torch.randn(6, 256, generator=ref.gen(5)).to(BF16)
    dz = torch.randn(6, 128, generator=ref.gen(6)).to(BF16)
    _, ck = mb.moe_silu_mul_checkpoint(y.cuda())
    dy, _ = mb.moe_silu_mul_backward(ck, dz.cuda())
    k = ref.unpack(ck.codes.cpu(), torch.cat([ck.exponents[:, :1], ck.exponents[:, 1:]], 1).cpu())
    d = torch.randn(6, 256, generator=ref.gen(7), dtype=torch.float64)
    f = lambda v: (ref.silu_mul(v[:, :128], v[:, 128:]) * dz.double()).sum()
    diff = (f(k + 1e-6 * d) - f(k - 1e-6 * d)) / 2e-6
    terms = dy.cpu().double() * d
    assert abs(diff - terms.sum()) <= 2.0 ** -8 * terms.abs().sum()          # dy is rounded to bf16


# ------------------------------------------------------------ streams, refusals

def test_operators_run_on_the_given_stream():
    """Inputs written on a side stream are read there, in order, without the caller synchronising."""
    mb = _mb()
    side = torch.cuda.Stream()
    x = torch.randn(2048, 1024, device="cuda").to(BF16)
    gamma = torch.ones(1024, device="cuda")
    want = mb.moe_layer_norm(x * 2 + 1, gamma)[0]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got, m, r = mb.moe_layer_norm(x * 2 + 1, gamma)
        back = mb.moe_layer_norm_backward(got, x * 2 + 1, gamma, m, r)
        loss = mb.moe_balance_loss(torch.sigmoid(x[:, :64].float()), 4)
        ck = mb.moe_checkpoint_pack(got)
        again = mb.moe_checkpoint_unpack(ck)
    x2 = x * 2 + 1
    explicit = mb.moe_layer_norm(x2, gamma, stream=torch.cuda.current_stream())[0]
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(explicit, want)
    assert torch.equal(back[1], mb.moe_layer_norm_backward(want, x2, gamma, m, r)[1])
    assert torch.equal(loss[0], mb.moe_balance_loss(torch.sigmoid(x[:, :64].float()), 4)[0])
    assert torch.equal(again, mb.moe_checkpoint_unpack(mb.moe_checkpoint_pack(want)))


def test_python_refusals():
    mb = _mb()
    x = torch.randn(8, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    v = torch.zeros(8, device="cuda")
    bf = x.to(BF16)
    with pytest.raises(TypeError):
        mb.moe_layer_norm(x.half(), w)
    with pytest.raises(TypeError):
        mb.moe_layer_norm(x.cpu(), w)
    with pytest.raises(ValueError):
        mb.moe_layer_norm(x, w[:32])
    with pytest.raises(ValueError):
        mb.moe_layer_norm(x.T, torch.ones(8, device="cuda"))          # columns are not dense
    with pytest.raises(ValueError):
        mb.moe_layer_norm(x, w, out=torch.empty(8, 32, device="cuda"))
    with pytest.raises(TypeError):
        mb.moe_layer_norm(x, w, w.to(BF16))
    with pytest.raises(TypeError):
        mb.moe_layer_norm(x, w, None, torch.tensor([4], device="cuda"))     # int64 count
    with pytest.raises(TypeError):
        mb.moe_layer_norm_backward(bf, x, w, v, v)
    with pytest.raises(ValueError):
        mb.moe_layer_norm_backward(x, x, w, v[:4], v)
    with pytest.raises(mb.MoEError):
        mb.moe_layer_norm(x, w, eps=-1.0)
    with pytest.raises(mb.MoEError):
        mb.moe_balance_loss(x, 65)
    with pytest.raises(TypeError):
        mb.moe_balance_loss(x.double(), 2)
    with pytest.raises(ValueError):
        mb.moe_balance_loss_backward(x, torch.zeros(5, dtype=torch.int32, device="cuda"), 2)
    with pytest.raises(ValueError):
        mb.moe_balance_loss_backward(x, torch.zeros(64, dtype=torch.int32, device="cuda"), 2, accumulate=True)
    with pytest.raises(TypeError):
        mb.moe_checkpoint_pack(x)
    with pytest.raises(mb.MoEError):
        mb.moe_checkpoint_pack(bf[:, :24])
    with pytest.raises(ValueError):
        mb.Checkpoint(torch.empty(8, 64, dtype=torch.float8_e4m3fn, device="cuda"),
                      torch.empty(8, 2, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mb.moe_silu_mul_backward(mb.moe_checkpoint_pack(bf), bf[:, :32].contiguous())   # one half
    with pytest.raises(ValueError):
        mb.moe_silu_mul_checkpoint(bf, 64)                             # two halves of 64 do not fit
