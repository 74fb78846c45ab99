"""Host-side refusals of the training operators' entry points (they return before any CUDA call)."""
import ctypes

import pytest

from moe_token_routing_index_gb300 import build as mbuild

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def mb():
    mbuild.build()
    from moe_token_routing_index_gb300 import binding

    return binding


def _call(fn, args, change):
    a = dict(args)
    a.update(change)
    return fn(*a.values())


def _sweep(mb, fn, args, refusals):
    for change, want in refusals:
        assert _call(fn, args, change) == want, change


def test_layer_norm_refusals(mb):
    inv, uns = mb.MOE_ERR_INVALID, mb.MOE_ERR_UNSUPPORTED
    nan, inf = float("nan"), float("inf")
    fwd = dict(x=FAKE, ldx=64, T=4, D=64, dtype=0, gamma=FAKE, beta=None, wdtype=0, eps=1e-5, valid=None, y=FAKE,
               mean=None, rstd=None, stream=None)
    _sweep(mb, mb.library().moe_layer_norm, fwd, [
        (dict(x=None), inv), (dict(gamma=None), inv), (dict(y=None), inv), (dict(ldx=63), inv), (dict(T=-1), inv),
        (dict(D=-1), inv), (dict(dtype=2), inv), (dict(wdtype=7), inv), (dict(eps=-1.0), inv), (dict(eps=nan), inv),
        (dict(eps=inf), inv), (dict(D=16385, ldx=16385), uns), (dict(x=ODD), uns), (dict(y=ODD), uns),
        (dict(gamma=ODD), uns), (dict(beta=ODD), uns), (dict(T=0, x=None), mb.MOE_OK)])
    n = ctypes.c_size_t(0)
    size = mb.library().moe_layer_norm_backward_workspace_size
    assert size(-1, 64, ctypes.byref(n)) == inv and size(4, 64, None) == inv
    assert size(4, 16385, ctypes.byref(n)) == uns
    assert size(4096, 5120, ctypes.byref(n)) == mb.MOE_OK
    need = n.value
    bwd = dict(dy=FAKE, x=FAKE, ldx=5120, T=4096, D=5120, dtype=0, gamma=FAKE, wdtype=1, mean=FAKE, rstd=FAKE,
               valid=None, res=None, dx=FAKE, dgamma=FAKE, dbeta=None, ws=FAKE, nws=need, stream=None)
    _sweep(mb, mb.library().moe_layer_norm_backward, bwd, [
        (dict(dy=None), inv), (dict(mean=None), inv), (dict(rstd=None), inv), (dict(dx=None), inv),
        (dict(dgamma=None), inv), (dict(gamma=None), inv), (dict(dtype=2), inv), (dict(ldx=5119), inv),
        (dict(res=ODD), uns), (dict(dy=ODD), uns)])
    if need:
        _sweep(mb, mb.library().moe_layer_norm_backward, bwd, [
            (dict(nws=need - 1), mb.MOE_ERR_WORKSPACE), (dict(ws=None), inv), (dict(ws=ODD), inv)])


def test_balance_loss_refusals(mb):
    inv, uns = mb.MOE_ERR_INVALID, mb.MOE_ERR_UNSUPPORTED
    n = ctypes.c_size_t(0)
    size = mb.library().moe_balance_loss_workspace_size
    assert size(-1, 8, ctypes.byref(n)) == inv and size(4, 0, ctypes.byref(n)) == inv
    assert size(4, 1025, ctypes.byref(n)) == uns and size(4096, 64, ctypes.byref(n)) == mb.MOE_OK
    need = n.value
    fwd = dict(scores=FAKE, dtype=0, st=64, se=1, T=4096, E=64, k=2, kind=0, coef=0.1, valid=None, cin=None, cout=FAKE,
               mean=FAKE, loss=FAKE, ws=FAKE, nws=need, stream=None)
    common = [(dict(scores=None), inv), (dict(st=-1), inv), (dict(se=-1), inv), (dict(T=-1), inv), (dict(E=0), inv),
              (dict(k=0), inv), (dict(k=65), inv), (dict(kind=3), inv), (dict(kind=-1), inv), (dict(dtype=2), inv),
              (dict(coef=float("nan")), inv), (dict(coef=float("inf")), inv), (dict(E=1025), uns),
              (dict(scores=ODD), uns), (dict(T=2**30, k=4), inv)]
    _sweep(mb, mb.library().moe_balance_loss, fwd, common + [
        (dict(cout=None), inv), (dict(mean=None), inv), (dict(loss=None), inv), (dict(ws=None), inv),
        (dict(ws=ODD), inv), (dict(nws=need - 1), mb.MOE_ERR_WORKSPACE)])
    bwd = dict(scores=FAKE, dtype=0, st=64, se=1, T=4096, E=64, k=2, kind=0, coef=0.1, valid=None, counts=FAKE,
               dloss=None, ds=FAKE, acc=0, stream=None)
    _sweep(mb, mb.library().moe_balance_loss_backward, bwd, common + [
        (dict(counts=None), inv), (dict(ds=None), inv), (dict(ds=ODD), uns), (dict(T=0, scores=None), mb.MOE_OK)])


def test_checkpoint_refusals(mb):
    inv, uns, ok = mb.MOE_ERR_INVALID, mb.MOE_ERR_UNSUPPORTED, mb.MOE_OK
    off8 = ctypes.c_void_p(0x1008)
    pack = dict(x=FAKE, ld=64, a=4, W=64, valid=None, codes=FAKE, exps=FAKE, stream=None)
    _sweep(mb, mb.library().moe_checkpoint_pack, pack, [
        (dict(x=None), inv), (dict(codes=None), inv), (dict(exps=None), inv), (dict(ld=56), inv), (dict(a=-1), inv),
        (dict(W=-16), inv), (dict(W=24, ld=24), uns), (dict(ld=68), uns), (dict(x=off8), uns), (dict(codes=off8), uns),
        (dict(a=0, x=None), ok), (dict(W=0, x=None), ok)])
    unpack = dict(codes=FAKE, exps=FAKE, a=4, W=64, valid=None, x=FAKE, stream=None)
    _sweep(mb, mb.library().moe_checkpoint_unpack, unpack, [
        (dict(x=None), inv), (dict(codes=None), inv), (dict(exps=None), inv), (dict(W=40), uns), (dict(x=off8), uns)])
    silu = dict(x0=FAKE, x1=FAKE, ld=128, a=4, H=64, valid=None, z=FAKE, codes=FAKE, exps=FAKE, stream=None)
    _sweep(mb, mb.library().moe_silu_mul_checkpoint, silu, [
        (dict(x0=None), inv), (dict(x1=None), inv), (dict(z=None), inv), (dict(ld=48), inv), (dict(ld=130), uns),
        (dict(H=72), uns), (dict(x1=off8), uns), (dict(z=off8), uns), (dict(a=0, z=None), ok)])
    back = dict(codes=FAKE, exps=FAKE, dz=FAKE, a=4, H=64, valid=None, dy=FAKE, z=None, stream=None)
    _sweep(mb, mb.library().moe_silu_mul_backward, back, [
        (dict(codes=None), inv), (dict(dz=None), inv), (dict(dy=None), inv), (dict(H=8), uns), (dict(z=off8), uns),
        (dict(dz=off8), uns), (dict(a=-2), inv)])


def test_weight_grad_refusals(mb):
    inv, uns, ok = mb.MOE_ERR_INVALID, mb.MOE_ERR_UNSUPPORTED, mb.MOE_OK
    n = ctypes.c_size_t(0)
    size = mb.library().moe_grouped_weight_grad_workspace_size
    assert size(0, 64, 64, 64, 0, ctypes.byref(n)) == inv and size(4, 64, 64, 64, 1, ctypes.byref(n)) == inv
    assert size(4, 64, 72, 64, 0, ctypes.byref(n)) == uns and size(1025, 64, 64, 64, 0, ctypes.byref(n)) == uns
    assert size(4, 64, 64, 64, mb.MOE_DTYPE_E4M3, ctypes.byref(n)) == ok and n.value > 0
    packed = n.value
    args = dict(dy=FAKE, x=FAKE, exps=None, counts=FAKE, E=4, a=64, N=64, K=64, dw=FAKE, dtype=0, acc=0, ws=FAKE,
                nws=1 << 20, stream=None)
    _sweep(mb, mb.library().moe_grouped_weight_grad, args, [
        (dict(dy=None), inv), (dict(x=None), inv), (dict(counts=None), inv), (dict(dw=None), inv), (dict(E=0), inv),
        (dict(a=-1), inv), (dict(dtype=2), inv), (dict(acc=1), inv), (dict(N=24), uns), (dict(K=8), uns),
        (dict(E=1025), uns), (dict(dy=ctypes.c_void_p(0x1008)), uns), (dict(dw=ctypes.c_void_p(0x1008)), uns),
        (dict(exps=FAKE, nws=packed - 1), mb.MOE_ERR_WORKSPACE), (dict(exps=FAKE, ws=None), inv),
        (dict(exps=FAKE, ws=ctypes.c_void_p(0x1010)), inv), (dict(N=0, dw=None), ok)])
