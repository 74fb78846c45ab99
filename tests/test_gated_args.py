"""Refusals of the gated block's and the orthogonalised update's entry points and wrappers, and the streams
that their calls take their memory from.  Nothing is launched, so this runs without a GPU."""
import ctypes

import pytest
import torch

from tests import gated_ref as ref
from tests.test_streams import BF16, F32, I32, U8, World, _t, _tensors, mb  # noqa: F401  (mb: a fixture)
from tests.test_train_abi import FAKE, ODD, _sweep

OFF8 = ctypes.c_void_p(0x1008)
NAN, INF = float("nan"), float("inf")


def test_gated_refusals(mb):  # noqa: F811
    inv, uns, ok = mb.MOE_ERR_INVALID, mb.MOE_ERR_UNSUPPORTED, mb.MOE_OK
    fwd = dict(x=FAKE, w13=FAKE, w2=FAKE, counts=FAKE, E=4, a=64, D=64, H=32, act=0, y=None, z=FAKE, out=FAKE,
               stream=None)
    common = [(dict(w13=None), inv), (dict(w2=None), inv), (dict(counts=None), inv), (dict(E=0), inv), (dict(a=-1), inv),
              (dict(D=0), inv), (dict(H=0), inv), (dict(H=-16), inv), (dict(act=2), inv), (dict(act=-1), inv),
              (dict(E=1025), uns), (dict(D=72), uns), (dict(H=40), uns), (dict(w13=ODD), uns), (dict(w2=OFF8), uns),
              (dict(z=OFF8), uns), (dict(y=OFF8), uns)]
    _sweep(mb, mb.library().moe_gated_mlp, fwd, common + [
        (dict(x=None), inv), (dict(out=None), inv), (dict(z=None), inv), (dict(x=OFF8), uns), (dict(out=OFF8), uns),
        (dict(a=0, x=None, out=None, z=None), ok)])
    bwd = dict(dout=FAKE, y=FAKE, exps=None, w13=FAKE, w2=FAKE, counts=FAKE, E=4, a=64, D=64, H=32, act=1, dy=FAKE,
               z=None, dx=FAKE, stream=None)
    _sweep(mb, mb.library().moe_gated_mlp_backward, bwd, common + [
        (dict(dout=None), inv), (dict(y=None), inv), (dict(dy=None), inv), (dict(dx=None), inv), (dict(dy=OFF8), uns),
        (dict(dout=OFF8), uns), (dict(dx=OFF8), uns), (dict(a=0, dout=None, y=None, dy=None, dx=None), ok)])


def test_orthogonalize_refusals(mb):  # noqa: F811
    inv, uns, ok = mb.MOE_ERR_INVALID, mb.MOE_ERR_UNSUPPORTED, mb.MOE_OK
    n = ctypes.c_size_t(0)
    size = mb.library().moe_orthogonalize_workspace_size
    assert size(-1, 8, 8, ctypes.byref(n)) == inv and size(1, 8, 8, None) == inv
    assert size(1, 65536, 8, ctypes.byref(n)) == uns and size(65536, 8, 8, ctypes.byref(n)) == uns
    assert size(0, 8, 8, ctypes.byref(n)) == ok and n.value == 0
    assert size(2, 40, 56, ctypes.byref(n)) == ok and n.value == 0      # small ones need none
    assert size(2, 400, 560, ctypes.byref(n)) == ok and n.value > 0
    need = n.value
    c3 = lambda *v: (ctypes.c_float * 3)(*v)
    shared = [(dict(B=-1), inv), (dict(N=-1), inv), (dict(steps=0), inv), (dict(steps=17), inv), (dict(eps=0.0), inv),
              (dict(eps=NAN), inv), (dict(eps=INF), inv), (dict(ws=None), inv), (dict(nws=need - 1), mb.MOE_ERR_WORKSPACE),
              (dict(ws=ctypes.c_void_p(0x1010)), inv), (dict(K=65536), uns), (dict(coef=c3(NAN, 0, 0)), inv),
              (dict(coef=c3(5.0, 0.0, 0.0)), inv),              # leaves [0, 4)
              (dict(coef=c3(1.9, 0.0, 0.0), steps=3), inv)]   # grows step by step
    one = dict(g=FAKE, dtype=0, bs=400 * 560, rs=560, B=2, N=400, K=560, steps=5, coef=None, eps=1e-7, scale=1.0, out=FAKE,
               ws=FAKE, nws=need, stream=None)
    _sweep(mb, mb.library().moe_orthogonalize, one, shared + [
        (dict(g=None), inv), (dict(out=None), inv), (dict(dtype=2), inv), (dict(scale=INF), inv), (dict(bs=-1), inv),
        (dict(rs=-1), inv), (dict(g=ODD), uns), (dict(out=ODD), uns), (dict(N=0, g=None), ok)])
    two = dict(w=FAKE, wd=0, g=FAKE, gd=1, m=FAKE, B=2, N=400, K=560, mu=0.9, nesterov=1, lr=0.1, lrs=None, decay=0.0,
               steps=5, coef=None, eps=1e-7, ws=FAKE, nws=need, stream=None)
    _sweep(mb, mb.library().moe_muon_update, two, shared + [
        (dict(w=None), inv), (dict(g=None), inv), (dict(m=None), inv), (dict(wd=2), inv), (dict(gd=2), inv),
        (dict(mu=1.0), inv), (dict(mu=-0.1), inv), (dict(mu=NAN), inv), (dict(lr=NAN), inv), (dict(decay=INF), inv),
        (dict(w=ODD), uns), (dict(g=ctypes.c_void_p(0x1002)), uns), (dict(m=ctypes.c_void_p(0x1002)), uns),
        (dict(B=0, w=None), ok)])


def _calls(mb):  # noqa: F811
    E, D, H, a = 4, 64, 32, 16
    x, w13, w2, counts = _t(BF16, a, D), _t(BF16, E, 2 * H, D), _t(BF16, E, D, H), _t(I32, E)
    big = _t(BF16, 2, 200, 160)                 # (small matrices need no workspace)
    return dict(gated=lambda **s: mb.moe_gated_mlp(x, w13, w2, counts, **s),
                gated_grad=lambda **s: mb.moe_gated_mlp_backward(x, _t(BF16, a, 2 * H), w13, w2, counts, **s),
                orthogonal=lambda **s: mb.moe_orthogonalize(w13, **s),
                update=lambda **s: mb.moe_muon_update(big, big, _t(F32, 2, 200, 160), lr=0.1, **s))


@pytest.mark.parametrize("name", ["gated", "gated_grad", "orthogonal", "update"])
def test_a_call_takes_its_memory_from_the_stream_it_runs_on(mb, monkeypatch, name):  # noqa: F811
    world = World(monkeypatch, mb)
    result = _calls(mb)[name](stream=world.side)
    assert [s for _, s in world.launched] == [world.side.cuda_stream]
    assert world.allocated and {s.cuda_stream for _, s in world.allocated} == {world.side.cuda_stream}
    made = {id(t) for t, _ in world.allocated}
    got = [t for t in _tensors(mb, result) if id(t) in made]
    assert all(world.main in getattr(t, "recorded", []) for t in got) and (got or name == "update")
    world.allocated.clear()
    _calls(mb)[name]()
    assert {s.cuda_stream for _, s in world.allocated} == {world.main.cuda_stream}


def test_wrappers_refuse_what_does_not_fit(mb, monkeypatch):  # noqa: F811
    world = World(monkeypatch, mb)
    E, D, H, a = 4, 64, 32, 16
    x, w13, w2, counts = _t(BF16, a, D), _t(BF16, E, 2 * H, D), _t(BF16, E, D, H), _t(I32, E)
    y = _t(BF16, a, 2 * H)
    half = mb.Checkpoint(_t(torch.float8_e4m3fn, a, 2 * H), _t(U8, a, 1))
    wrong = [
        lambda: mb.moe_gated_mlp(x, w13, _t(BF16, E, H, D), counts),
        lambda: mb.moe_gated_mlp(x, _t(BF16, E, 2 * H + 1, D), w2, counts),
        lambda: mb.moe_gated_mlp(x, w13[0], w2, counts),
        lambda: mb.moe_gated_mlp(x, w13, w2, _t(I32, E - 1)),
        lambda: mb.moe_gated_mlp(x, w13, w2, _t(I32, 1, E)),
        lambda: mb.moe_gated_mlp(_t(BF16, a, D + 16), w13, w2, counts),
        lambda: mb.moe_gated_mlp(x, w13, w2, counts, y=_t(BF16, a, H)),
        lambda: mb.moe_gated_mlp(x, w13, w2, counts, out=_t(BF16, a + 1, D)),
        lambda: mb.moe_gated_mlp(x.t().contiguous().as_subclass(type(x)).t(), w13, w2, counts),
        lambda: mb.moe_gated_mlp_backward(x, _t(BF16, a, H), w13, w2, counts),
        lambda: mb.moe_gated_mlp_backward(x, half, w13, w2, counts),
        lambda: mb.moe_gated_mlp_backward(x, y, w13, w2, counts, dy=_t(BF16, a, H)),
        lambda: mb.moe_orthogonalize(_t(F32, 8)),
        lambda: mb.moe_orthogonalize(_t(F32, 8, 8), coefficients=(1.0, 2.0)),
        lambda: mb.moe_orthogonalize(_t(F32, 8, 8), out=_t(BF16, 8, 9)),
        lambda: mb.moe_orthogonalize(_t(F32, 8, 6).t()),
        lambda: mb.moe_muon_update(_t(F32, 8, 8), _t(F32, 8, 9), _t(F32, 8, 8), lr=0.1),
        lambda: mb.moe_muon_update(_t(F32, 8, 8), _t(F32, 8, 8), _t(F32, 1, 8, 8), lr=0.1),
        lambda: mb.moe_muon_update(_t(F32, 8, 8), _t(F32, 8, 8), _t(F32, 8, 8), lr=0.1, lr_scale=_t(F32, 0)),
        lambda: mb.moe_muon_update(_t(F32, 8, 6).t(), _t(F32, 6, 8), _t(F32, 6, 8), lr=0.1),
    ]
    for call in wrong:
        with pytest.raises(ValueError):
            call()
    types = [
        lambda: mb.moe_gated_mlp(x.float(), w13, w2, counts),
        lambda: mb.moe_gated_mlp(x, w13.float(), w2, counts),
        lambda: mb.moe_gated_mlp(x, w13, w2, counts.long()),
        lambda: mb.moe_gated_mlp(torch.ones(a, D, dtype=BF16), w13, w2, counts),
        lambda: mb.moe_gated_mlp_backward(x, y.float(), w13, w2, counts),
        lambda: mb.moe_orthogonalize(_t(torch.float16, 8, 8)),
        lambda: mb.moe_orthogonalize(torch.ones(8, 8)),
        lambda: mb.moe_orthogonalize(_t(F32, 8, 8), out=_t(F32, 8, 8)),
        lambda: mb.moe_orthogonalize(_t(F32, 200, 160), workspace=torch.ones(1 << 20, dtype=U8)),
        lambda: mb.moe_muon_update(_t(F32, 8, 8), _t(F32, 8, 8), _t(BF16, 8, 8), lr=0.1),
    ]
    for call in types:
        with pytest.raises(TypeError):
            call()
    assert not world.launched


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_reference_gradient_against_differences(kind):
    """The formula of the backward against central differences of the forward, in 64 bits."""
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    a, E, D, H, counts = 5, 2, 16, 16, [3, 2]
    x, w13, w2, dout = r(a, D), r(E, 2 * H, D) / 4, r(E, D, H) / 4, r(a, D)
    _, y, _, _ = ref.forward(x, w13, w2, counts, kind)
    dx, dy, z, *_ = ref.backward(dout, y, w13, w2, counts, kind)
    loss = lambda x_: float((ref.forward(x_, w13, w2, counts, kind)[0] * dout).sum())
    for _ in range(4):
        d = r(a, D)
        want = (loss(x + 1e-5 * d) - loss(x - 1e-5 * d)) / 2e-5
        assert abs(float((dx * d).sum()) - want) <= 1e-7 * (1 + abs(want))


def test_reference_iteration_reaches_orthonormal_rows():
    g = torch.randn(1, 12, 20, generator=torch.Generator().manual_seed(1))
    x = ref.orthogonalize(g, 40, (1.5, -0.5, 0.0))
    assert float((x @ x.transpose(1, 2) - torch.eye(12).double()).abs().max()) < 1e-10
    u, _, vh = torch.linalg.svd(g[0].double(), full_matrices=False)
    assert float((x[0] - u @ vh).abs().max()) < 1e-10


def test_a_tensor_of_another_device_is_refused(mb, monkeypatch):  # noqa: F811
    world = World(monkeypatch, mb)
    kind = type("Elsewhere", (type(_t(F32, 1)),), {"get_device": lambda self: 1})
    w = torch.ones(4, 8, 8).as_subclass(kind)
    with pytest.raises(ValueError):
        mb.moe_orthogonalize(w)
    with pytest.raises(ValueError):
        mb.moe_muon_update(_t(F32, 4, 8, 8), w, _t(F32, 4, 8, 8), lr=0.1)
    x, w13, w2, counts = _t(BF16, 16, 64), _t(BF16, 4, 64, 64), _t(BF16, 4, 64, 32), _t(I32, 4)
    with pytest.raises(ValueError):
        mb.moe_gated_mlp(x, w13.as_subclass(kind), w2, counts)
    with pytest.raises(ValueError):
        mb.moe_gated_mlp_backward(x.as_subclass(kind), _t(BF16, 16, 64), w13, w2, counts)
    assert not world.launched


def _device_cases(mb):  # noqa: F811
    """(a call of the arguments by name, each of its tensors): every pointer that the kernels get."""
    E, D, H, a = 4, 64, 32, 16
    rows = dict(w13=_t(BF16, E, 2 * H, D), w2=_t(BF16, E, D, H), counts=_t(I32, E))
    forward = dict(rows, x=_t(BF16, a, D), y=_t(BF16, a, 2 * H), z=_t(BF16, a, H), out=_t(BF16, a, D))
    backward = dict(rows, dout=_t(BF16, a, D), y=_t(BF16, a, 2 * H), dy=_t(BF16, a, 2 * H), z=_t(BF16, a, H),
                    out=_t(BF16, a, D))
    codes = dict({k: v for k, v in backward.items() if k != "y"}, codes=_t(torch.float8_e4m3fn, a, 2 * H),
                 exponents=_t(U8, a, 2))
    space = _t(U8, mb.moe_orthogonalize_workspace_size(2, 200, 160))
    one = dict(g=_t(F32, 2, 200, 160), out=_t(BF16, 2, 200, 160), workspace=space)
    two = dict(w=_t(BF16, 2, 200, 160), grad=_t(BF16, 2, 200, 160), momentum=_t(F32, 2, 200, 160), lr_scale=_t(F32, 1),
               workspace=space)
    return dict(gated=(mb.moe_gated_mlp, forward), gated_grad=(mb.moe_gated_mlp_backward, backward),
                gated_grad_of_codes=(lambda codes, exponents, **s: mb.moe_gated_mlp_backward(
                    y=mb.Checkpoint(codes, exponents, 2), **s), codes),
                orthogonal=(mb.moe_orthogonalize, one),
                update=(lambda **s: mb.moe_muon_update(lr=0.1, **s), two))


@pytest.mark.parametrize("name", ["gated", "gated_grad", "gated_grad_of_codes", "orthogonal", "update"])
def test_each_tensor_of_another_device_is_refused(mb, monkeypatch, name):  # noqa: F811
    """Whichever argument lies on another device than the current one: its pointer does not reach a kernel."""
    world = World(monkeypatch, mb)
    elsewhere = type("Elsewhere", (type(_t(F32, 1)),), {"get_device": lambda self: 1})
    call, args = _device_cases(mb)[name]
    call(**args)
    assert len(world.launched) == 1
    for which, t in args.items():
        with pytest.raises(ValueError, match="device"):
            call(**dict(args, **{which: t.as_subclass(elsewhere)}))
        assert len(world.launched) == 1, which


def _leaves(c, steps: int, margin: float) -> bool:
    """Whether the iteration carries a singular value of [0, 1] past the documented limits: on a fine grid of each
    step's whole range, whose top is moved by the margin."""
    top = 1.0
    for _ in range(steps):
        s = torch.linspace(0, top, 4001, dtype=torch.float64)
        p = (c[1] + c[2] * s * s) * s * s
        top = float(((c[0] + p) * s).abs().max()) * (1 + margin)
        if float(p.abs().max()) * (1 + margin) >= 32 or top >= 4:
            return True
    return False


def _accepted(mb, c, steps):  # noqa: F811
    st = mb.library().moe_orthogonalize(None, 0, 0, 0, 0, 8, 8, steps, (ctypes.c_float * 3)(*c), 1e-7, 1.0, None, None, 0,
                                        None)
    assert st in (mb.MOE_OK, mb.MOE_ERR_INVALID)
    return st == mb.MOE_OK


def test_coefficients_that_leave_the_range_somewhere_are_refused(mb):  # noqa: F811
    f32 = lambda *c: tuple(torch.tensor(c, dtype=F32).double().tolist())
    # just past 3 s - 4 s^3 / R^2, which takes [0, R] onto itself: what is near R / 2 leaves [0, R], by 1e-7, and
    # each further step multiplies that by 9
    for c in ((3.000000238418579, -0.9427371025085449, 0.0), (3.000000238418579, -1.4062495231628418, 0.0),
              (3.000000476837158, -1.4391438961029053, 0.0)):
        assert f32(*c) == c and _leaves(c, 16, 0.0)
        assert not _accepted(mb, c, 16) and _accepted(mb, c, 4)
    always = [ref.COEFFICIENTS, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (3.0, -4.0, 0.0), (1.0, 0.0, 0.0), (0.0, 0.0, 0.0),
              (0.0, 0.0, 3.99), (15 / 8, -10 / 8, 3 / 8)]
    for c in always[:-2] + always[-1:]:
        assert all(_accepted(mb, c, steps) for steps in range(1, 17)), c
    assert _accepted(mb, always[-2], 1) and not _accepted(mb, always[-2], 2)
    g = torch.Generator().manual_seed(0)
    size = torch.tensor([5.0, 12.0, 10.0])
    seen = set()
    for _ in range(400):
        c = f32(*((2 * torch.rand(3, generator=g) - 1) * size).tolist())
        for steps in (1, 2, 3, 5, 16):
            inside, outside = not _leaves(c, steps, 1e-4), _leaves(c, steps, 0.0)
            if inside or outside:
                assert _accepted(mb, c, steps) == inside, (c, steps)
                seen.add((steps, inside))
    assert len(seen) == 10


def test_rows_whose_tiles_pass_31_bits_are_refused(mb):  # noqa: F811
    """The kernels round an expert's rows up to tiles in 32 bits, (rows + tiles - 1) / tiles, with at most 2^23 tiles."""
    inv, uns = mb.MOE_ERR_INVALID, mb.MOE_ERR_UNSUPPORTED
    limit = 2 ** 31 - 1 - 2 ** 24
    for a, want in ((2 ** 31 - 1, uns), (limit + 1, uns), (limit, inv)):      # (inv: no x)
        assert mb.library().moe_gated_mlp(None, FAKE, FAKE, FAKE, 1, a, 16, 16, 0, None, FAKE, FAKE, None) == want
        assert mb.library().moe_gated_mlp_backward(None, FAKE, None, FAKE, FAKE, FAKE, 1, a, 16, 16, 0, FAKE, None, FAKE,
                                                   None) == want


@pytest.mark.parametrize("shape", [(2 ** 32 + 8, 1), (8, 2 ** 32 + 8), (2 ** 32 + 1, 4, 4)])
def test_matrices_of_sizes_past_32_bits_are_refused(mb, monkeypatch, shape):  # noqa: F811
    """A size that a C int cannot hold is refused, not cut to its low bits."""
    world = World(monkeypatch, mb)
    kind = type(_t(F32, 1))
    g = torch.empty(shape, dtype=BF16, device="meta").as_subclass(kind)
    m = torch.empty(shape, dtype=F32, device="meta").as_subclass(kind)
    with pytest.raises(ValueError):
        mb.moe_orthogonalize(g, out=g)
    with pytest.raises(ValueError):
        mb.moe_muon_update(g, g, m, lr=0.1)
    assert not world.launched
