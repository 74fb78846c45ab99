"""The experts' gated block and its gradient against 64-bit forms, at the bounds of their own roundings."""
import pytest
import torch

from tests import gated_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _mb():
    from moe_token_routing_index_gb300 import binding

    return binding


def _kind(name):
    mb = _mb()
    return mb.MOE_ACT_SILU if name == "silu" else mb.MOE_ACT_GELU


def _make(a, E, D, H, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return ((size * r(a, D)).to(BF16), (r(E, 2 * H, D) / D ** 0.5).to(BF16), (r(E, D, H) / H ** 0.5).to(BF16),
            (0.1 * r(a, D)).to(BF16))


def _counts(c):
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _filled(*shape):
    return torch.full(shape, 7.0, dtype=BF16, device="cuda")


def _within(got, want, bound, rows, what):
    got = got.cpu().double()
    assert torch.isfinite(got[:rows]).all(), what
    over = (got[:rows] - want[:rows]).abs() - bound[:rows]
    assert rows == 0 or float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} over its bound"


# rows of one expert below, at and above the parts of 256 rows and the steps of 32; columns that end inside
# a tile and inside a step of 64; experts without rows at either end; rows of no expert
CASES = [
    (1, 16, 16, [1]),
    (3, 32, 16, [0, 3, 0]),
    (33, 64, 32, [32, 1]),
    (64, 256, 512, [8, 9, 7, 0, 16, 1, 3, 20]),
    (300, 272, 208, [40, 0, 211, 2]),
    (600, 80, 144, [257, 300]),
    (530, 144, 272, [0, 513, 0]),
    (256, 128, 128, [256]),
    (40, 528, 400, [0, 0, 0]),
    (2100, 64, 48, [2049, 31]),
]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("a,D,H,counts", CASES)
def test_forward(a, D, H, counts, kind):
    mb = _mb()
    x, w13, w2, _ = _make(a, len(counts), D, H)
    n = sum(counts)
    x[n:] = float("nan")
    y, z, out = _filled(a, 2 * H), _filled(a, H), _filled(a, D)
    mb.moe_gated_mlp(x.cuda(), w13.cuda(), w2.cuda(), _counts(counts), activation=_kind(kind), y=y, z=z, out=out)
    assert mb.device_error() == 0
    x[n:] = 0
    want, wy, eo, ey = ref.forward(x, w13, w2, counts, kind)
    _within(y, wy, ey, n, "y")
    _within(out, want, eo, n, "out")
    for t in (y, z, out):
        assert bool((t[n:] == 7).all())
    again, none = mb.moe_gated_mlp(x.cuda(), w13.cuda(), w2.cuda(), _counts(counts), activation=_kind(kind), keep=False)
    assert none is None and torch.equal(again[:n], out[:n])


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("a,D,H,counts", CASES)
def test_backward(a, D, H, counts, kind):
    mb = _mb()
    _, w13, w2, dout = _make(a, len(counts), D, H, seed=1)
    yk = (1.5 * torch.randn(a, 2 * H, generator=torch.Generator().manual_seed(2))).to(BF16)
    n = sum(counts)
    dout[n:] = float("nan")
    yk[n:] = float("inf")
    dx, dy, z = _filled(a, D), _filled(a, 2 * H), _filled(a, H)
    args = (dout.cuda(), yk.cuda(), w13.cuda(), w2.cuda(), _counts(counts))
    mb.moe_gated_mlp_backward(*args, activation=_kind(kind), out=dx, dy=dy, z=z)
    assert mb.device_error() == 0
    dout[n:] = 0
    yk[n:] = 0
    wx, wy, wz, ex, ey, ez = ref.backward(dout, yk, w13, w2, counts, kind)
    _within(dy, wy, ey, n, "dy")
    _within(z, wz, ez, n, "z")
    _within(dx, wx, ex, n, "dx")
    for t in (dx, dy, z):
        assert bool((t[n:] == 7).all())
    dx2, dy2, none = mb.moe_gated_mlp_backward(*args, activation=_kind(kind), with_z=False)
    assert none is None and torch.equal(dx2[:n], dx[:n]) and torch.equal(dy2[:n], dy[:n])


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("a,D,H,counts", [(70, 64, 48, [33, 30]), (300, 272, 208, [40, 0, 211, 2])])
def test_backward_from_a_checkpoint(a, D, H, counts, kind):
    """From 8-bit rows: the gradient at the values that they hold."""
    mb = _mb()
    _, w13, w2, dout = _make(a, len(counts), D, H, seed=3)
    y = (torch.randn(a, 2 * H, generator=torch.Generator().manual_seed(4)) * torch.logspace(-3, 2, a)[:, None]).to(BF16)
    n = sum(counts)
    _, ck = mb.moe_silu_mul_checkpoint(y.cuda(), H)
    scale = torch.exp2(ck.exponents.double().cpu() - 127)
    nb = scale.shape[1] // 2
    held = ck.codes.double().cpu().view(a, 2, H) * scale.view(a, 2, nb).repeat_interleave(128, 2)[:, :, :H]
    held = held.reshape(a, 2 * H)
    dx, dy, z = mb.moe_gated_mlp_backward(dout.cuda(), ck, w13.cuda(), w2.cuda(), _counts(counts), activation=_kind(kind))
    assert mb.device_error() == 0
    wx, wy, wz, ex, ey, ez = ref.backward(dout, held, w13, w2, counts, kind)
    _within(dy, wy, ey, n, "dy")
    _within(z, wz, ez, n, "z")
    _within(dx, wx, ex, n, "dx")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gates_far_from_zero(kind):
    """Gates that are shut, open and beyond the range of exp and of the cubic: no NaN, the limits' values."""
    mb = _mb()
    D, H = 64, 64
    v = torch.tensor([-1e30, -1e20, -1e4, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 1e4, 1e20, 1e30])
    a = len(v)
    y = torch.ones(a, 2 * H)
    y[:, :H] = v[:, None]
    _, w13, w2, dout = _make(a, 1, D, H, seed=5)
    dx, dy, z = mb.moe_gated_mlp_backward(dout.cuda(), y.to(BF16).cuda(), w13.cuda(), w2.cuda(), _counts([a]),
                                          activation=_kind(kind))
    y0 = v.to(BF16).double()
    f = torch.where(y0 < -80, torch.zeros_like(y0), torch.where(y0 > 80, y0, ref.act(y0.clamp(-80, 80), kind)))
    s = torch.where(y0 < -80, torch.zeros_like(y0), torch.where(y0 > 80, torch.ones_like(y0),
                                                                  ref.slope(y0.clamp(-80, 80), kind)))
    dz = dout.double() @ w2[0].double()
    acc = D * 2.0 ** -22 * (dout.double().abs() @ w2[0].double().abs())
    got = dy.cpu().double()
    near = lambda g, w, e: bool(((g - w).abs() <= ref.HALF16 * w.abs() + e + 1e-30).all())
    # (what act leaves of 1e-7 of y0 below the limits' -80 is 1e-28 and less)
    assert near(got[:, :H], dz * s[:, None], acc * s[:, None].abs() + 2.0 ** -18 * dz.abs())
    assert near(got[:, H:], dz * f[:, None], (acc + 2.0 ** -18 * dz.abs()) * f[:, None].abs())
    assert near(z.cpu().double(), f[:, None].expand(a, H), 2.0 ** -18 * f[:, None].abs())
    assert mb.device_error() == 0


def test_counts_that_do_not_fit():
    """A negative count is empty and a sum past the rows is cut there; both are flagged."""
    mb = _mb()
    a, D, H = 50, 64, 48
    x, w13, w2, dout = _make(a, 3, D, H, seed=6)
    for counts in ([20, -5, 10], [20, 10, 400], [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]):
        cut = [max(0, c) for c in counts]
        n = min(a, sum(cut))
        y, out = _filled(a, 2 * H), _filled(a, D)
        mb.moe_gated_mlp(x.cuda(), w13.cuda(), w2.cuda(), _counts(counts), y=y, out=out)
        assert mb.device_error() == mb.MOE_DEVERR_BAD_COUNT
        want, wy, eo, ey = ref.forward(x, w13, w2, cut, "silu")
        _within(y, wy, ey, n, "y")
        _within(out, want, eo, n, "out")
        assert bool((out[n:] == 7).all()) and bool((y[n:] == 7).all())
        dx, dy, z = mb.moe_gated_mlp_backward(dout.cuda(), y, w13.cuda(), w2.cuda(), _counts(counts))
        assert mb.device_error() == mb.MOE_DEVERR_BAD_COUNT
        wx, _, _, ex, _, _ = ref.backward(dout[:n], y[:n].cpu(), w13, w2, cut, "silu")
        _within(dx, wx, ex, n, "dx")


def test_counts_of_the_router():
    """counts with the total behind the experts', as moe_route leaves them; no rows at all."""
    mb = _mb()
    x, w13, w2, _ = _make(24, 2, 32, 32, seed=7)
    out, y = mb.moe_gated_mlp(x.cuda(), w13.cuda(), w2.cuda(), _counts([10, 14, 24]))
    ref_out, ref_y = mb.moe_gated_mlp(x.cuda(), w13.cuda(), w2.cuda(), _counts([10, 14]))
    assert torch.equal(out, ref_out) and torch.equal(y, ref_y)
    empty = x[:0].cuda()
    out, y = mb.moe_gated_mlp(empty, w13.cuda(), w2.cuda(), _counts([0, 0]))
    assert out.shape == (0, 32) and y.shape == (0, 64)
    dx, dy, z = mb.moe_gated_mlp_backward(empty, y, w13.cuda(), w2.cuda(), _counts([0, 0]))
    assert dx.shape == (0, 32) and dy.shape == (0, 64) and z.shape == (0, 32)
    assert mb.device_error() == 0


def test_same_bytes_again_captured_and_on_another_stream():
    mb = _mb()
    x, w13, w2, dout = (t.cuda() for t in _make(700, 3, 192, 160, seed=8))
    counts = _counts([300, 5, 380])
    out, y = mb.moe_gated_mlp(x, w13, w2, counts)
    grads = mb.moe_gated_mlp_backward(dout, y, w13, w2, counts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, y2 = mb.moe_gated_mlp(x, w13, w2, counts, stream=side)
    g2 = mb.moe_gated_mlp_backward(dout, y2, w13, w2, counts, stream=side)
    torch.cuda.synchronize()
    n = 685
    same = lambda p, q: all(torch.equal(u[:n], v[:n]) for u, v in zip(p, q))
    assert same((out, y, *grads), (o2, y2, *g2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, y3 = mb.moe_gated_mlp(x, w13, w2, counts)
        g3 = mb.moe_gated_mlp_backward(dout, y3, w13, w2, counts)
    for _ in range(2):
        for t in (o3, y3, *g3):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same((out, y, *grads), (o3, y3, *g3))
    # other counts and inputs in the same buffers
    x.mul_(0.5)
    counts.copy_(_counts([0, 257, 100]))
    graph.replay()
    want, wy = mb.moe_gated_mlp(x, w13, w2, counts)
    torch.cuda.synchronize()
    assert torch.equal(o3[:357], want[:357]) and torch.equal(y3[:357], wy[:357])
    assert mb.device_error() == 0


def test_many_experts_with_few_rows():
    mb = _mb()
    E, D, H = 1024, 32, 16
    counts = [(7 * e) % 5 for e in range(E)]
    a = sum(counts) + 3
    x, w13, w2, dout = _make(a, E, D, H, seed=9)
    out, y = mb.moe_gated_mlp(x.cuda(), w13.cuda(), w2.cuda(), _counts(counts))
    dx, dy, z = mb.moe_gated_mlp_backward(dout.cuda(), y, w13.cuda(), w2.cuda(), _counts(counts))
    want, wy, eo, ey = ref.forward(x, w13, w2, counts, "silu")
    _within(out, want, eo, a - 3, "out")
    wx, wdy, wz, ex, edy, ez = ref.backward(dout[:a - 3], y[:a - 3].cpu(), w13, w2, counts, "silu")
    _within(dx, wx, ex, a - 3, "dx")
    _within(dy, wdy, edy, a - 3, "dy")
    assert mb.device_error() == 0


def test_offsets_past_32_bits():
    """Rows whose y lies beyond 2^31 elements, forward and backward, against the same rows by themselves."""
    mb = _mb()
    E, D, H, a = 2, 16, 4096, 300_000
    x, w13, w2, dout = _make(64, E, D, H, seed=10)
    x, dout = x.cuda().repeat(a // 64 + 1, 1)[:a].contiguous(), dout.cuda().repeat(a // 64 + 1, 1)[:a].contiguous()
    w13, w2 = w13.cuda(), w2.cuda()
    counts = _counts([100, a - 130])                # the last 30 rows are of no expert
    out, y = _filled(a, D), _filled(a, 2 * H)
    mb.moe_gated_mlp(x, w13, w2, counts, y=y, out=out)
    n = a - 30
    assert y.numel() > 2 ** 31
    tail = slice(n - 64, n)
    few = _counts([0, 64])
    want, wy = mb.moe_gated_mlp(x[tail].contiguous(), w13, w2, few)
    assert torch.equal(out[tail], want) and torch.equal(y[tail], wy)
    assert bool((y[n:] == 7).all()) and bool((out[n:] == 7).all())
    dx, dy, z = mb.moe_gated_mlp_backward(dout, y, w13, w2, counts, dy=_filled(a, 2 * H))
    wx, wdy, wz = mb.moe_gated_mlp_backward(dout[tail].contiguous(), wy, w13, w2, few)
    assert torch.equal(dx[tail], wx) and torch.equal(dy[tail], wdy) and torch.equal(z[tail], wz)
    assert bool((dy[n:] == 7).all())
    assert mb.device_error() == 0


def test_two_streams_at_once():
    mb = _mb()
    x, w13, w2, dout = (t.cuda() for t in _make(900, 4, 256, 320, seed=11))
    counts = [_counts([500, 0, 130, 270]), _counts([1, 600, 299, 0])]
    want = [mb.moe_gated_mlp(x, w13, w2, c) for c in counts]
    grads = [mb.moe_gated_mlp_backward(dout, y, w13, w2, c) for c, (_, y) in zip(counts, want)]
    streams = [torch.cuda.Stream() for _ in counts]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [mb.moe_gated_mlp(x, w13, w2, c, stream=s) for c, s in zip(counts, streams)]
        back = [mb.moe_gated_mlp_backward(dout, y, w13, w2, c, stream=s) for c, s, (_, y) in zip(counts, streams, got)]
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for p, q in zip(want, got) for u, v in zip(p, q))
    assert all(torch.equal(u, v) for p, q in zip(grads, back) for u, v in zip(p, q))
    assert mb.device_error() == 0
