"""Calls on a stream that is not the current one: their memory is their own while they run."""
import pytest
import torch

from tests import train_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
WAIT = 20_000_000        # clock cycles that a stream is held, about 10 ms


def _mb():
    from moe_token_routing_index_gb300 import binding

    return binding


def _calls(mb):
    """Calls whose workspaces hold what their results are made of, with those workspaces' sizes."""
    g = ref.gen(0)
    r = lambda *shape: torch.randn(*shape, generator=g).cuda()
    x, dy, gamma = r(1500, 1024).to(BF16), r(1500, 1024).to(BF16), r(1024)
    _, mean, rstd = mb.moe_layer_norm(x, gamma)
    logits = r(20000, 64)
    d, v = r(6000, 256).to(BF16), r(6000, 128).to(BF16)
    counts = torch.tensor([3500, 2500], dtype=torch.int32, device="cuda")
    ck = mb.moe_checkpoint_pack(v)
    route = torch.sigmoid(r(4096, 64)).to(BF16)
    return dict(
        norm=(lambda **s: mb.moe_layer_norm_backward(dy, x, gamma, mean, rstd, **s),
              mb.moe_layer_norm_backward_workspace_size(1500, 1024)),
        balance=(lambda **s: mb.moe_balance_loss(logits, 4, kind=mb.MOE_BALANCE_SOFTMAX, **s),
                 mb.moe_balance_loss_workspace_size(20000, 64)),
        weight_grad=(lambda **s: (mb.moe_grouped_weight_grad(d, ck, counts, dtype=F32, **s),),
                     mb.moe_grouped_weight_grad_workspace_size(2, 6000, 256, 128, mb.MOE_DTYPE_E4M3)),
        route=(lambda **s: tuple(mb.moe_route(route, 2, **s).values())[:4], mb.moe_route_workspace_size(4096, 64, 2)))


@pytest.mark.parametrize("name", ["norm", "balance", "weight_grad", "route"])
def test_memory_of_a_call_on_another_stream(name):
    mb = _mb()
    call, size = _calls(mb)[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # what the current stream allocates while the call has yet to run is not the call's workspace
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    got = call(stream=side)
    filled = [torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda") for n in (size, size, size // 2, 2 * size)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    del got, filled
    # and the call does not write what the current stream has yet to read
    held = [torch.full((max(n, 1),), 7, dtype=torch.uint8, device="cuda") for n in (size, size, size)]
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    copies = [t.clone() for t in held]
    del held
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies), name
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    assert mb.device_error() == 0
