"""One row, or one column, whose stride PyTorch is free to set to anything: a row that is the transpose
of a column has the stride 1, and is as dense as any other."""
import pytest
import torch

from tests.helpers import bits

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _mb():
    from moe_token_routing_index_gb300 import binding

    return binding


def _row(W, dtype=BF16):
    """(a [1, W] row with the stride 1, the same values with the stride W)."""
    column = torch.randn(W, 1, device="cuda").to(dtype)
    row = column.t()
    assert row.shape == (1, W) and row.stride() == (1, 1)
    return row, column.flatten().clone().view(1, W)


def _same(got, want):
    got, want = ([r] if isinstance(r, torch.Tensor) else r for r in (got, want))
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert (bits(a) == bits(b)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [5120, 640, 77])
def test_layer_norm_of_a_transposed_column(D, dtype):
    mb = _mb()
    x, dense = _row(D, dtype)
    gamma, dy = torch.rand(D, device="cuda"), torch.randn(1, D, device="cuda").to(dtype)
    want = mb.moe_layer_norm(dense, gamma)
    _same(mb.moe_layer_norm(x, gamma), want)
    _same(mb.moe_layer_norm_backward(dy, x, gamma, *want[1:]), mb.moe_layer_norm_backward(dy, dense, gamma, *want[1:]))
    assert mb.device_error() == 0


def test_checkpoints_and_silu_mul_of_a_transposed_column():
    mb = _mb()
    x, dense = _row(416)
    parts = lambda ck: [ck.codes, ck.exponents]
    _same(parts(mb.moe_checkpoint_pack(x)), parts(mb.moe_checkpoint_pack(dense)))
    for H in (None, 192):
        if H is None:
            _same(mb.moe_silu_mul(x), mb.moe_silu_mul(dense))
            _same(mb.moe_silu_mul_quant(x), mb.moe_silu_mul_quant(dense))
        (z, ck), (wz, wck) = mb.moe_silu_mul_checkpoint(x, H), mb.moe_silu_mul_checkpoint(dense, H)
        _same([z] + parts(ck), [wz] + parts(wck))
    assert mb.device_error() == 0


def test_layer_norm_of_one_column_of_many():
    mb = _mb()
    wide = torch.randn(9, 12, device="cuda")
    x = wide[:, ::3][:, :1]
    assert x.stride() == (12, 3)
    gamma = torch.rand(1, device="cuda")
    _same(mb.moe_layer_norm(x, gamma), mb.moe_layer_norm(x.contiguous(), gamma))
    assert mb.device_error() == 0
