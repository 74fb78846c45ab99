"""Arguments of the training wrappers that would be read as something else, or past their end, by the
library: refused before any call of it.  The library is a fake, so this runs without a GPU."""
import pytest
import torch

from tests.test_streams import BF16, F32, I32, U8, World, _t, mb  # noqa: F401  (mb: a fixture)

CPU = torch.empty(1 << 22, dtype=U8)


def _wrappers(mb):
    """name -> (a call with keywords, the name of its row count, whether it takes a workspace)."""
    x, gamma, stat, rows = _t(BF16, 8, 64), _t(F32, 64), _t(F32, 8), _t(BF16, 16, 64)
    scores = _t(F32, 4096, 64)
    one = mb.Checkpoint(_t(torch.float8_e4m3fn, 16, 64), _t(U8, 16, 1))
    two = mb.Checkpoint(_t(torch.float8_e4m3fn, 16, 64), _t(U8, 16, 2), 2)
    n, r = "num_valid_tokens", "valid_rows"
    return dict(
        norm=(lambda **k: mb.moe_layer_norm(x, gamma, **k), n, False),
        norm_grad=(lambda **k: mb.moe_layer_norm_backward(x, x, gamma, stat, stat, **k), n, True),
        balance=(lambda **k: mb.moe_balance_loss(scores, 2, **k), n, True),
        balance_grad=(lambda **k: mb.moe_balance_loss_backward(scores, _t(I32, 64), 2, **k), n, False),
        pack=(lambda **k: mb.moe_checkpoint_pack(rows, **k), r, False),
        unpack=(lambda **k: mb.moe_checkpoint_unpack(one, **k), r, False),
        silu=(lambda **k: mb.moe_silu_mul_checkpoint(rows, **k), r, False),
        silu_grad=(lambda **k: mb.moe_silu_mul_backward(two, _t(BF16, 16, 32), **k), r, False),
        weight_grad=(lambda **k: mb.moe_grouped_weight_grad(rows, one, _t(I32, 16), **k), None, True))


NAMES = ["norm", "norm_grad", "balance", "balance_grad", "pack", "unpack", "silu", "silu_grad", "weight_grad"]


@pytest.mark.parametrize("name", [n for n in NAMES if n != "weight_grad"])
def test_an_empty_row_count_is_refused(mb, monkeypatch, name):  # noqa: F811
    """Its pointer is null, which the library reads as: all rows."""
    call, count, _ = _wrappers(mb)[name]
    world = World(monkeypatch, mb)
    with pytest.raises(ValueError):
        call(**{count: _t(I32, 0)})
    assert not world.launched
    call(**{count: _t(I32, 1)})
    assert len(world.launched) == 1


def test_an_empty_dloss_is_refused(mb, monkeypatch):  # noqa: F811
    call, _, _ = _wrappers(mb)["balance_grad"]
    world = World(monkeypatch, mb)
    with pytest.raises(ValueError):
        call(dloss=_t(F32, 0))
    assert not world.launched


@pytest.mark.parametrize("name", ["norm_grad", "balance", "weight_grad"])
def test_a_workspace_is_device_memory(mb, monkeypatch, name):  # noqa: F811
    call, _, _ = _wrappers(mb)[name]
    world = World(monkeypatch, mb)
    with pytest.raises(TypeError):
        call(workspace=CPU)                                             # on the host
    with pytest.raises(ValueError):
        call(workspace=_t(U8, 1).expand(1 << 22))                       # one byte, many times
    assert not world.launched
    seen = []
    monkeypatch.setattr(mb, "_lib", type("Lib", (), {"__getattr__": lambda self, f: lambda *a: seen.append(a) or 0})())
    call(workspace=_t(F32, 1 << 20))
    assert seen[0][-2] == 1 << 22                                       # its bytes, whatever its type


def test_a_checkpoint_that_is_read_has_to_be_one(mb, monkeypatch):  # noqa: F811
    world = World(monkeypatch, mb)
    for wrong in (None, _t(BF16, 16, 64)):
        with pytest.raises(TypeError):
            mb.moe_silu_mul_backward(wrong, _t(BF16, 16, 32))
        with pytest.raises(TypeError):
            mb.moe_checkpoint_unpack(wrong)
    assert not world.launched
