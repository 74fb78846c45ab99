"""Newton-Schulz orthogonalisation and the momentum update against 64-bit forms.

One step is held element by element to the bound of its roundings.  Over several steps the
worst case grows with the iteration's largest slope to the power of the steps and says
nothing, so five steps are held to what the same roundings do in 64 bits: no further from the
exact result than 1.5 times as far as that (its roundings fall otherwise where sums differ
in their last bits), plus the half bf16 step of the output."""
import pytest
import torch

from tests import gated_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

SHAPES = [(1, 1, 1), (2, 1, 7), (3, 17, 16), (1, 33, 257), (2, 300, 64), (1, 256, 256), (2, 517, 263), (1, 128, 1024),
          (1, 1024, 136), (5, 64, 96), (1, 257, 513)]


def _mb():
    from moe_token_routing_index_gb300 import binding

    return binding


def _g(B, N, K, dtype, seed=0, strong=True):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(B, N, K, generator=g)
    if strong:
        r = min(4, N, K)
        v = 0.2 * v + torch.randn(B, N, r, generator=g) @ torch.randn(B, r, K, generator=g)
    return (1e-3 * v).to(dtype)


def _check_five(got, g, scale=1.0, steps=5):
    exact = ref.orthogonalize(g, steps) * scale
    half = ref.orthogonalize(g, steps, half=True) * scale
    for b in range(len(g)):
        norm = float(exact[b].norm())
        off = float((got[b].cpu().double() - exact[b]).norm())
        most = 1.5 * float((half[b] - exact[b]).norm()) + ref.HALF16 * norm + 1e-30
        assert off <= most, f"matrix {b}: {off / norm:.3e} of its norm, allowed {most / norm:.3e}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,K", SHAPES)
def test_one_step(B, N, K, dtype):
    mb = _mb()
    g = _g(B, N, K, dtype)
    got = mb.moe_orthogonalize(g.cuda(), steps=1).cpu().double()
    want, bound = ref.one_step_error(g)
    over = (got - want).abs() - bound
    assert float(over.max()) <= 0, f"{float(over.max()):.3e} over its bound"
    assert mb.device_error() == 0


@pytest.mark.parametrize("strong", [True, False])
@pytest.mark.parametrize("B,N,K", SHAPES)
def test_five_steps(B, N, K, strong):
    mb = _mb()
    g = _g(B, N, K, F32, seed=1, strong=strong)
    _check_five(mb.moe_orthogonalize(g.cuda()), g)
    _check_five(mb.moe_orthogonalize(g.cuda(), scale=-0.5), g, -0.5)
    assert mb.device_error() == 0


def test_two_dimensions_strides_and_odd_bases():
    mb = _mb()
    big = _g(3, 70, 131, F32, seed=2).cuda()
    rows = big[:, :65, 3:100]                       # rows and matrices apart, base not 16-byte aligned
    whole = mb.moe_orthogonalize(rows.contiguous())
    assert torch.equal(mb.moe_orthogonalize(rows), whole)
    assert torch.equal(mb.moe_orthogonalize(rows[1]), whole[1])
    same = rows[:1].expand(3, -1, -1)               # one matrix three times: stride 0
    assert torch.equal(mb.moe_orthogonalize(same), whole[:1].expand(3, -1, -1))
    flat = torch.full((65 * 97 + 2,), 7.0, dtype=BF16, device="cuda")
    out = flat[1:-1].view(65, 97)
    mb.moe_orthogonalize(rows[0], out=out)
    assert torch.equal(out, whole[0]) and float(flat[0]) == 7 and float(flat[-1]) == 7
    half = big.to(BF16)[:, :65, 3:100]
    assert torch.equal(mb.moe_orthogonalize(half), mb.moe_orthogonalize(half.contiguous()))
    assert mb.device_error() == 0


def test_zeros_nan_infinities_and_extreme_sizes():
    """Each matrix for itself: zeros stay zeros, what is not finite is NaN in its own matrix, and the size
    of a matrix does not matter from 1e-4 of 1/eps to the largest fp32 (the norm is far above both)."""
    mb = _mb()
    g = _g(6, 40, 56, F32, seed=3)
    g[1] = 0
    g[2, 3, 5] = float("nan")
    g[4, 0, 0] = float("inf")
    got = mb.moe_orthogonalize(g.cuda())
    alone = mb.moe_orthogonalize(g[[0, 3, 5]].cuda())
    assert torch.equal(got[[0, 3, 5]], alone)
    assert bool((got[1] == 0).all())
    assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[4]).all())
    # a power of two changes no rounding but eps's part, which is 1e-7 of the norm at most
    base = (g[0] / g[0].abs().max()).to(F32)
    for e in (0, 40, 100, 126):
        _check_five(mb.moe_orthogonalize((base * 2.0 ** e)[None].cuda()), (base * 2.0 ** e)[None].double())
    assert mb.device_error() == 0


def test_other_coefficients_and_steps():
    mb = _mb()
    cubic = (1.5, -0.5, 0.0)
    g = _g(2, 48, 80, F32, seed=4, strong=False)
    for steps in (1, 3, 12, 16):
        got = mb.moe_orthogonalize(g.cuda(), steps=steps, coefficients=cubic).cpu().double()
        exact = ref.orthogonalize(g, steps, cubic)
        half = ref.orthogonalize(g, steps, cubic, half=True)
        assert float((got - exact).norm()) <= 1.5 * float((half - exact).norm()) + ref.HALF16 * float(exact.norm())
    # 16 steps of the cubic reach the nearest matrix with orthonormal rows: bf16 rounding and fp16 operands are left
    gram = got @ got.transpose(1, 2)
    assert float((gram - torch.eye(48).double()).abs().max()) < 0.02


@pytest.mark.parametrize("w_dtype,g_dtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("B,N,K,nesterov", [(1, 1, 3, True), (2, 40, 56, False), (3, 130, 33, True), (1, 300, 520, True),
                                            (2, 96, 480, False), (1, 100, 1500, True), (1, 2000, 64, True)])
def test_update(B, N, K, nesterov, w_dtype, g_dtype):
    mb = _mb()
    gen = torch.Generator().manual_seed(5)
    w = (0.02 * torch.randn(B, N, K, generator=gen)).to(w_dtype)
    g = _g(B, N, K, g_dtype, seed=6)
    m = (2 * _g(B, N, K, F32, seed=7)).float()
    mu, lr, decay = 0.9, 0.03, 0.1
    wd, md = w.cuda(), m.cuda()
    scale = torch.tensor([0.5], device="cuda")
    assert mb.moe_muon_update(wd, g.cuda(), md, lr=lr, mu=mu, nesterov=nesterov, weight_decay=decay, lr_scale=scale) is wd
    m64 = mu * m.double() + g.double()
    assert bool(((md.cpu().double() - m64).abs() <= 2.0 ** -23 * (m64.abs() + mu * m.double().abs())).all())
    u = g.double() + mu * m64 if nesterov else m64
    exact, half = ref.orthogonalize(u), ref.orthogonalize(u, half=True)
    want = (1 - 0.5 * lr * decay) * w.double() - 0.5 * lr * exact
    step = 2.0 ** -24 if w_dtype == F32 else ref.HALF16
    for b in range(B):
        off = float((wd[b].cpu().double() - want[b]).norm())
        most = 0.5 * lr * (1.5 * float((half[b] - exact[b]).norm()) + 1e-5 * float(exact[b].norm()))
        assert off <= most + 4 * step * float(want[b].norm()) if w_dtype == F32 else off <= most + 1.01 * step * float(
            want[b].norm())
    assert mb.device_error() == 0


def test_update_of_nothing_moves_only_by_decay():
    mb = _mb()
    w = torch.randn(2, 20, 30, generator=torch.Generator().manual_seed(8)).cuda()
    before = w.clone()
    zero = torch.zeros_like(w)
    mb.moe_muon_update(w, zero, zero.clone(), lr=0.1, weight_decay=0.0)
    assert torch.equal(w, before)
    mb.moe_muon_update(w, zero, zero.clone(), lr=0.5, weight_decay=0.5)
    assert torch.equal(w, before * 0.75)


@pytest.mark.parametrize("N,K", [(300, 200), (100, 1600)])
def test_same_bytes_again_captured_and_on_another_stream(N, K):
    mb = _mb()
    g = _g(2, N, K, BF16, seed=9).cuda()
    w0 = torch.randn(2, N, K, device="cuda").to(BF16)
    m0 = torch.randn(2, N, K, device="cuda")
    out = mb.moe_orthogonalize(g)
    w, m = w0.clone(), m0.clone()
    mb.moe_muon_update(w, g, m, lr=0.1)
    side = torch.cuda.Stream()
    w2, m2 = w0.clone(), m0.clone()
    side.wait_stream(torch.cuda.current_stream())
    out2 = mb.moe_orthogonalize(g, stream=side)
    mb.moe_muon_update(w2, g, m2, lr=0.1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(w, w2) and torch.equal(m, m2)
    # two captured graphs with a workspace of their own each, replayed by turns
    graphs = []
    for k in range(2):
        wk, mk, lr = w0.clone(), m0.clone(), torch.tensor([1.0], device="cuda")
        ws = torch.empty(mb.moe_orthogonalize_workspace_size(2, N, K), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mb.moe_muon_update(wk, g, mk, lr=0.1, lr_scale=lr, workspace=ws)
        graphs.append((graph, wk, mk, lr))
    for graph, wk, mk, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(wk, w) and torch.equal(mk, m) for _, wk, mk, _ in graphs)
    graph, wk, mk, lr = graphs[0]
    lr.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(wk, w) and not torch.equal(mk, m)      # a rate of zero: the momentum moves alone
    assert mb.device_error() == 0


def test_offsets_past_32_bits():
    """Matrices beyond 2^31 elements of a batch give the bytes that they give by themselves."""
    mb = _mb()
    B, N, K = 40, 8192, 8192
    g = torch.zeros(B, N, K, dtype=BF16, device="cuda")
    g[-1] = torch.randn(N, K, device="cuda").to(BF16)
    g[5] = g[-1]
    assert g.numel() > 2 ** 31
    out = mb.moe_orthogonalize(g, steps=1)
    alone = mb.moe_orthogonalize(g[-1], steps=1)
    assert torch.equal(out[-1], alone) and torch.equal(out[5], alone)
    assert not bool(out[-2].any()) and not bool(out[0].any())
    assert mb.device_error() == 0


def test_two_streams_at_once():
    mb = _mb()
    gs = [_g(9, 100, 7000, BF16, seed=19).cuda(), _g(3, 200, 330, BF16, seed=12).cuda(), _g(2, 700, 96, F32, seed=13).cuda(), _g(1, 64, 4096, F32, seed=14).cuda()]
    want = [mb.moe_orthogonalize(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [mb.moe_orthogonalize(g, stream=s) for g, s in zip(gs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    assert mb.device_error() == 0


@pytest.mark.parametrize("N,K", [(1, 20000), (20000, 1), (40, 30000), (16, 4000), (300, 9001)])
def test_long_and_flat(N, K):
    """Few tiles and a long reduction: A from parts of it."""
    mb = _mb()
    g = _g(1, N, K, F32, seed=15)
    got = mb.moe_orthogonalize(g.cuda(), steps=1).cpu().double()
    want, bound = ref.one_step_error(g)
    assert float(((got - want).abs() - bound).max()) <= 0
    _check_five(mb.moe_orthogonalize(g.cuda()), g)
    assert mb.device_error() == 0


@pytest.mark.parametrize("B,N,K", [(1, 1100, 6144), (2, 6100, 800), (3, 512, 7175)])
def test_two_steps_made_one(B, N, K):
    """Sizes at which the first two steps are one polynomial: the same iteration, at the same bounds.  What that
    polynomial's own roundings add to those of two steps is within the 1.5 of the bound (they are as large)."""
    mb = _mb()
    for strong in (True, False):
        g = _g(B, N, K, F32, seed=16, strong=strong)
        got = mb.moe_orthogonalize(g.cuda())
        _check_five(got, g)
        _check_five(mb.moe_orthogonalize(g.cuda(), steps=2), g, steps=2)
        _check_five(mb.moe_orthogonalize(g.cuda(), steps=3), g, steps=3)
    assert mb.device_error() == 0


@pytest.mark.parametrize("B,N,K,times", [(3, 512, 7168, 60), (2, 6100, 800, 20), (16, 512, 256, 60), (1, 1100, 6144, 20),
                                         (9, 128, 7168, 60), (1, 60, 1793, 60),
                                         (4, 1024, 2048, 30)])
def test_same_bytes_every_time(B, N, K, times):
    """A call's products follow one another inside one launch: what one stores has to be whole before the next
    reads it, whatever the timing, so that repeated calls give the same bytes."""
    mb = _mb()
    g = torch.randn(B, N, K, generator=torch.Generator().manual_seed(17)).cuda()
    ws = torch.empty(mb.moe_orthogonalize_workspace_size(B, N, K), dtype=torch.uint8, device="cuda")
    want = mb.moe_orthogonalize(g, workspace=ws).clone()
    for _ in range(times):
        assert torch.equal(mb.moe_orthogonalize(g, workspace=ws), want)
    assert mb.device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,K", [(1, 128, 448), (1, 128, 449), (2, 100, 900), (3, 64, 2000), (1, 65, 3585), (1, 128, 7168),
                                   (1, 7168, 128), (2, 1793, 60), (1, 3, 7000), (5, 128, 128), (1, 16, 16), (20, 33, 1000),
                                   (1, 128, 7169), (30, 90, 7000)])
def test_matrices_that_stay_on_the_chip(B, N, K, dtype):
    """Sides up to 128, over 1 to 16 CTAs; and sizes just past what fits."""
    mb = _mb()
    g = _g(B, N, K, dtype, seed=18)
    got = mb.moe_orthogonalize(g.cuda(), steps=1).cpu().double()
    want, bound = ref.one_step_error(g)
    assert float(((got - want).abs() - bound).max()) <= 0
    _check_five(mb.moe_orthogonalize(g.cuda()), g)
    assert mb.device_error() == 0


@pytest.mark.parametrize("N,K", [(40, 56), (200, 272), (203, 301)])
def test_eps_beside_a_norm_whose_square_overflows(N, K):
    """eps counts whatever the norm's size: here both are about 2^77."""
    mb = _mb()
    g = torch.randn(2, N, K, generator=torch.Generator().manual_seed(20)) * 2.0 ** 70
    eps = 2.0 ** 76
    got = mb.moe_orthogonalize(g.cuda(), steps=1, eps=eps).cpu().double()
    want, bound = ref.one_step_error(g, eps=eps)
    assert float(((got - want).abs() - bound).max()) <= 0
    assert mb.device_error() == 0
