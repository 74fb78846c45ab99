"""The products over the whole GPU (a side above 128) at the arguments that the small matrices' tests use:
strides, odd bases, values that are not finite, other coefficients, the update in all types, batches.  References
in 64 bits, computed on the GPU; bounds as in the other tests of these operators."""
import pytest
import torch

from tests import gated_ref as ref
from tests.test_gpu_orthogonalize import BF16, F32, _check_five, _g, _mb

pytestmark = pytest.mark.gpu


def _within_one_step(got, g):
    want, bound = ref.one_step_error(g)
    assert float(((got.double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(200, 272), (272, 200), (203, 301), (301, 203)])
def test_strides_and_odd_bases(N, K, dtype):
    mb = _mb()
    big = _g(3, N + 5, -(-K // 8) * 8 + 40, dtype, seed=2).cuda()
    shifted = big[:, :N, 3:3 + K]                   # single elements, whatever K
    got = mb.moe_orthogonalize(shifted, steps=1)
    _within_one_step(got, shifted)
    assert torch.equal(mb.moe_orthogonalize(shifted[1], steps=1), got[1])
    apart = big[::2, :N, 8:8 + K]                   # 16-byte pieces where K is a multiple of 8
    whole = mb.moe_orthogonalize(apart.contiguous())
    assert torch.equal(mb.moe_orthogonalize(apart), whole)
    same = apart[:1].expand(3, -1, -1)              # one matrix three times: stride 0
    assert torch.equal(mb.moe_orthogonalize(same), whole[:1].expand(3, -1, -1))
    for head in (1, 8):                             # results off 32 bytes, by single elements
        flat = torch.full((2 * N * K + 2 * head,), 7.0, dtype=BF16, device="cuda")
        out = flat[head:-head].view(2, N, K)
        mb.moe_orthogonalize(apart, out=out)
        assert torch.equal(out, whole) and bool((flat[:head] == 7).all()) and bool((flat[-head:] == 7).all())
    assert mb.device_error() == 0


@pytest.mark.parametrize("N,K", [(200, 272), (301, 203)])
def test_zeros_nan_infinities_and_extreme_sizes(N, K):
    mb = _mb()
    g = _g(6, N, K, F32, seed=3)
    g[1] = 0
    g[2, 3, 5] = float("nan")
    g[4, 0, 0] = float("inf")
    got = mb.moe_orthogonalize(g.cuda())
    assert torch.equal(got[[0, 3, 5]], mb.moe_orthogonalize(g[[0, 3, 5]].cuda()))
    assert bool((got[1] == 0).all())
    assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[4]).all())
    base = (g[0] / g[0].abs().max()).to(F32)
    for e in (0, 40, 62, 100, 126):                 # squares whose sum overflows from about 2^60
        v = (base * 2.0 ** e)[None]
        _check_five(mb.moe_orthogonalize(v.cuda()), v.double())
    assert mb.device_error() == 0


def test_other_coefficients_and_steps():
    mb = _mb()
    cubic = (1.5, -0.5, 0.0)
    g = _g(2, 200, 272, F32, seed=4, strong=False).cuda()
    for steps in (1, 3, 12, 16):
        got = mb.moe_orthogonalize(g, steps=steps, coefficients=cubic).double()
        exact = ref.orthogonalize(g, steps, cubic)
        half = ref.orthogonalize(g, steps, cubic, half=True)
        assert float((got - exact).norm()) <= 1.5 * float((half - exact).norm()) + ref.HALF16 * float(exact.norm())
    assert mb.device_error() == 0


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("w_dtype,g_dtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("B,N,K", [(2, 256, 512), (2, 512, 256), (1, 301, 203), (3, 136, 1000), (1, 1100, 6144),
                                   (5, 2048, 1008)])
def test_update(B, N, K, w_dtype, g_dtype, nesterov):
    """One step element by element, five by their norm, with a rate that makes the step as large as the weights.

    One step: the bound of the product scaled by the rate.  u is in fp32, off by 2^-22 of itself at most, which the
    hundredth that the bound adds to fp16's half steps covers; the sum of weights and step is off by 2^-22 of
    its parts; one rounding of the weights."""
    mb = _mb()
    gen = torch.Generator().manual_seed(5)
    w = (0.02 * torch.randn(B, N, K, generator=gen)).to(w_dtype).cuda()
    g, m = _g(B, N, K, g_dtype, seed=6).cuda(), (2 * _g(B, N, K, F32, seed=7)).cuda()
    mu, lr, decay, lr_scale = 0.9, 1.5, 0.1, torch.tensor([0.5], device="cuda")
    rate, half_step = 0.75, 2.0 ** -24 if w_dtype == F32 else ref.HALF16
    m64 = mu * m.double() + g.double()
    u = g.double() + mu * m64 if nesterov else m64
    base = (1 - rate * decay) * w.double()
    args = dict(lr=lr, mu=mu, nesterov=nesterov, weight_decay=decay, lr_scale=lr_scale)
    got, moved = w.clone(), m.clone()
    mb.moe_muon_update(got, g, moved, steps=1, **args)
    assert bool(((moved.double() - m64).abs() <= 2.0 ** -23 * (m64.abs() + mu * m.double().abs())).all())
    x, bound = ref.one_step_error(u)
    want = base - rate * x
    bound = 1.01 * (rate * bound + 2.0 ** -22 * (base.abs() + rate * x.abs())) + 1.01 * half_step * want.abs()
    assert float(((got.double() - want).abs() - bound).max()) <= 0
    got, moved = w.clone(), m.clone()
    mb.moe_muon_update(got, g, moved, **args)
    exact, half = ref.orthogonalize(u), ref.orthogonalize(u, half=True)
    want = base - rate * exact
    for b in range(B):
        off = float((got[b].double() - want[b]).norm())
        most = rate * (1.5 * float((half[b] - exact[b]).norm()) + 1e-4 * float(exact[b].norm()))
        assert off <= most + 1.01 * half_step * float(want[b].norm()), b
    assert mb.device_error() == 0


def test_update_of_weights_that_start_anywhere():
    """Bases off 32 bytes: weights and results by single elements, gradient and momentum too."""
    mb = _mb()
    N, K = 256, 160
    place = lambda t, head: torch.cat([t.new_full((head,), 7.0), t.flatten(), t.new_full((5,), 7.0)])
    for w_dtype in (BF16, F32):
        w = (0.02 * torch.randn(N, K, generator=torch.Generator().manual_seed(8))).to(w_dtype).cuda()
        g, m = _g(1, N, K, BF16, seed=9)[0].cuda(), _g(1, N, K, F32, seed=10)[0].cuda()
        flat = [place(w, 1), place(g, 3), place(m, 1)]
        wv, gv, mv = (f[h:-5].view(N, K) for f, h in zip(flat, (1, 3, 1)))
        mb.moe_muon_update(wv, gv, mv, lr=1.0, mu=0.9, steps=1)
        m64 = 0.9 * m.double() + g.double()
        x, bound = ref.one_step_error((g.double() + 0.9 * m64)[None])
        want = w.double() - x[0]
        half_step = 2.0 ** -24 if w_dtype == F32 else ref.HALF16
        bound = 1.01 * (bound[0] + 2.0 ** -22 * (w.double().abs() + x[0].abs())) + 1.01 * half_step * want.abs()
        assert float(((wv.double() - want).abs() - bound).max()) <= 0
        assert all(bool((f[:h] == 7).all()) and bool((f[-5:] == 7).all()) for f, h in zip(flat, (1, 3, 1)))
    assert mb.device_error() == 0


@pytest.mark.parametrize("B,N,K", [(5, 600, 704), (4, 301, 203)])
def test_a_matrix_of_a_batch_and_by_itself(B, N, K):
    """Where A's reduction is not split and the first two steps are not one polynomial, whatever the batch: the
    same bytes alone and among others."""
    mb = _mb()
    g = _g(B, N, K, BF16, seed=11).cuda()
    whole = mb.moe_orthogonalize(g)
    for b in range(B):
        assert torch.equal(mb.moe_orthogonalize(g[b].clone()), whole[b])
    assert mb.device_error() == 0


# Batches of which A's reduction is not split, and the first two steps are worth a polynomial of their own.
MERGED = [(5, 1024, 2100), (2, 1500, 3300), (5, 2100, 1000), (3, 1301, 2403), (20, 512, 1500), (5, 2048, 1008)]


def _rounded(g, steps, coefficients, merged: bool):
    """The result in 64 bits with the products' operands in fp16 and nothing else; merged: of the polynomial that
    takes the first two steps at once."""
    a, b, c = coefficients
    half = lambda t: (t * 1024).half().double() / 1024
    turned = g.shape[1] > g.shape[2]
    x = ref._first(g, 1e-7)
    x = x.transpose(1, 2) if turned else x
    if merged:
        xh = half(x)
        m = half(xh @ xh.transpose(1, 2))
        p = half(b * m + c * (m @ m))
        t = half(a * m + m @ p)
        m2 = half(a * t + p @ t)
        p2 = half(b * m2 + c * (m2 @ m2))
        x = a * a * x + half(a * p + a * p2 + p2 @ p) @ xh
        steps -= 2
    for _ in range(steps):
        xh = half(x)
        m = half(xh @ xh.transpose(1, 2))
        x = a * x + half(b * m + c * (m @ m)) @ xh
    return x.transpose(1, 2) if turned else x


@pytest.mark.parametrize("B,N,K", MERGED)
def test_first_two_steps_as_one_polynomial(B, N, K):
    """Held to 1.5 times what that polynomial's own roundings do in 64 bits, and half a bf16 step."""
    mb = _mb()
    up = lambda n: -(-n // 16) * 16
    iterate, square = 2 * B * N * up(K), 2 * B * min(N, K) * up(min(N, K))
    # three iterates' halves and three square matrices: the third is the polynomial's
    assert 0 <= mb.moe_orthogonalize_workspace_size(B, N, K) - 3 * iterate - 3 * square < square

    def near(got, g, steps, coefficients, merged):
        exact = ref.orthogonalize(g, steps, coefficients)
        off = (got.double() - exact).flatten(1).norm(dim=1)
        most = 1.5 * (_rounded(g, steps, coefficients, merged) - exact).flatten(1).norm(dim=1)
        assert bool((off <= most + ref.HALF16 * exact.flatten(1).norm(dim=1)).all()), (steps, off, most)

    for strong in (True, False):
        g = _g(B, N, K, F32, seed=16, strong=strong).cuda()
        for steps in (1, 2, 3, 5):
            got = mb.moe_orthogonalize(g, steps=steps)
            near(got, g, steps, ref.COEFFICIENTS, steps > 1)
        for _ in range(10):
            assert torch.equal(mb.moe_orthogonalize(g), got)
        steep = (5.49, -9.85, 2.965)                # what the polynomial does not fit takes separate steps
        near(mb.moe_orthogonalize(g, steps=2, coefficients=steep), g, 2, steep, False)
    assert mb.device_error() == 0
