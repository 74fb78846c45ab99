"""Which stream's memory a call takes when it is given a stream: the library and CUDA are fakes, so this
runs without a GPU.

The caching allocator reuses a block in the order of the stream it was allocated on.  A call on
another stream whose workspace came from the current one would share it with whatever the current
stream runs next, and write it while what the current stream ran before still reads it."""
import pytest
import torch

from moe_token_routing_index_gb300 import build as mbuild

BF16, F8, I32, F32, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32, torch.uint8


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Tensor(torch.Tensor):
    """A CPU tensor that passes for a CUDA one and notes the streams it is recorded on."""

    is_cuda = True

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream]


class World:
    def __init__(self, monkeypatch, mb):
        self.main, self.side = Stream(0x10), Stream(0x20)
        self.current, self.allocated, self.launched = [self.main], [], []
        world = self

        class On:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                world.current.append(self.stream)

            def __exit__(self, *_):
                world.current.pop()

        def allocating(make):
            def allocate(*shape, **kw):
                t = make(*shape, **kw).as_subclass(Tensor)
                world.allocated.append((t, world.current[-1]))
                return t
            return allocate

        class Library:
            def __getattr__(self, name):
                if name.endswith("_size"):
                    return getattr(mb_lib, name)
                return lambda *args: world.launched.append((name, args[-1])) or mb.MOE_OK

        mb_lib = mb.library()
        monkeypatch.setattr(mb, "_lib", Library())
        monkeypatch.setattr(mb, "_raw_stream", lambda device: world.current[-1].cuda_stream)
        monkeypatch.setattr(mb, "_current_device", lambda: 0)
        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: world.current[-1])
        monkeypatch.setattr(torch, "empty", allocating(torch.empty))
        monkeypatch.setattr(torch, "zeros", allocating(torch.zeros))


@pytest.fixture(scope="module")
def mb():
    mbuild.build()
    from moe_token_routing_index_gb300 import binding

    return binding


def _t(dtype, *shape):
    return torch.ones(shape).to(dtype).as_subclass(Tensor)


def _calls(mb):
    """name -> a call of each wrapper that launches kernels and allocates."""
    T, D, E, k, a = 8, 64, 16, 2, 16
    x, w, i32 = _t(BF16, T, D), _t(BF16, E, D), lambda n: _t(I32, n)
    rows, scores = _t(BF16, a, D), _t(BF16, T, E)
    w13, w2 = _t(BF16, E, 64, D), _t(BF16, E, D, 32)
    gamma, stat = _t(F32, D), _t(F32, T)
    one = mb.Checkpoint(_t(F8, a, D), _t(U8, a, 1))
    two = mb.Checkpoint(_t(F8, a, 64), _t(U8, a, 2), 2)
    return dict(
        moe_router_scores=lambda **s: mb.moe_router_scores(x, w, **s),
        moe_router_route=lambda **s: mb.moe_router_route(x, w, k, with_weights=True, **s),
        moe_route=lambda **s: mb.moe_route(scores, k, with_weights=True, **s),
        moe_gather_scale=lambda **s: mb.moe_gather_scale(x, i32(a), i32(a), scores, **s),
        moe_gather_scale_quant=lambda **s: mb.moe_gather_scale_quant(x, i32(a), i32(a), scores, **s),
        moe_quantize_rows=lambda **s: mb.moe_quantize_rows(_t(F32, E, D), **s),
        moe_pack_weights=lambda **s: mb.moe_pack_weights(w13, **s),
        moe_grouped_gemm=lambda **s: mb.moe_grouped_gemm(rows, w13, i32(E), **s),
        moe_grouped_gemm_quant=lambda **s: mb.moe_grouped_gemm(rows, w13, i32(E),
                                                               epilogue=mb.MOE_EPILOGUE_SILU_MUL_QUANT, **s),
        moe_grouped_gemm_fp8_rowwise=lambda **s: mb.moe_grouped_gemm_fp8_rowwise(
            _t(F8, a, D), _t(F8, E, 64, D), i32(E), _t(F32, a), _t(F32, E, 64), **s),
        moe_expert_mlp=lambda **s: mb.moe_expert_mlp(rows, w13, w2, i32(E), **s),
        moe_silu_mul=lambda **s: mb.moe_silu_mul(rows, **s),
        moe_silu_mul_quant=lambda **s: mb.moe_silu_mul_quant(rows, **s),
        moe_topk_finalize=lambda **s: mb.moe_topk_finalize(rows, _t(F32, T, k), _t(I32, T, k), **s),
        moe_dense_gemm=lambda **s: mb.moe_dense_gemm(x, w, **s),
        moe_layer_norm=lambda **s: mb.moe_layer_norm(x, gamma, **s),
        moe_layer_norm_backward=lambda **s: mb.moe_layer_norm_backward(x, x, gamma, stat, stat, **s),
        moe_balance_loss=lambda **s: mb.moe_balance_loss(_t(F32, 4096, 64), k, **s),
        moe_balance_loss_backward=lambda **s: mb.moe_balance_loss_backward(scores, i32(E), k, **s),
        moe_checkpoint_pack=lambda **s: mb.moe_checkpoint_pack(rows, **s),
        moe_checkpoint_unpack=lambda **s: mb.moe_checkpoint_unpack(one, **s),
        moe_silu_mul_checkpoint=lambda **s: mb.moe_silu_mul_checkpoint(rows, **s),
        moe_silu_mul_backward=lambda **s: mb.moe_silu_mul_backward(two, _t(BF16, a, 32), **s),
        moe_grouped_weight_grad=lambda **s: mb.moe_grouped_weight_grad(rows, one, i32(E), **s))


def _tensors(mb, result):
    """Every tensor of a call's result."""
    if isinstance(result, torch.Tensor):
        return [result]
    if isinstance(result, mb.Checkpoint):
        return [result.codes, result.exponents]
    if isinstance(result, mb.PackedWeights):
        return [result.data]
    if isinstance(result, dict):
        result = list(result.values())
    return [t for r in result for t in _tensors(mb, r)] if isinstance(result, (tuple, list)) else []


NAMES = """moe_router_scores moe_router_route moe_route moe_gather_scale moe_gather_scale_quant moe_quantize_rows
moe_pack_weights moe_grouped_gemm moe_grouped_gemm_quant moe_grouped_gemm_fp8_rowwise moe_expert_mlp moe_silu_mul
moe_silu_mul_quant moe_topk_finalize moe_dense_gemm moe_layer_norm moe_layer_norm_backward moe_balance_loss
moe_balance_loss_backward moe_checkpoint_pack moe_checkpoint_unpack moe_silu_mul_checkpoint moe_silu_mul_backward
moe_grouped_weight_grad""".split()


@pytest.mark.parametrize("name", NAMES)
def test_a_call_takes_its_memory_from_the_stream_it_runs_on(mb, monkeypatch, name):
    calls = _calls(mb)
    assert sorted(calls) == sorted(NAMES)
    world = World(monkeypatch, mb)
    result = calls[name](stream=world.side)
    assert [s for _, s in world.launched] == [world.side.cuda_stream]
    assert {s.cuda_stream for _, s in world.allocated} == {world.side.cuda_stream}
    assert world.current == [world.main]
    # and what the caller gets of it may not go back while the caller's stream uses it
    made = {id(t) for t, _ in world.allocated}
    got = [t for t in _tensors(mb, result) if id(t) in made]
    assert got and all(world.main in getattr(t, "recorded", []) for t in got)


@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_the_current_stream_takes_its_memory(mb, monkeypatch, name):
    calls = _calls(mb)
    world = World(monkeypatch, mb)
    calls[name]()
    calls[name](stream=world.main)
    assert [s for _, s in world.launched] == [world.main.cuda_stream] * 2
    assert {s.cuda_stream for _, s in world.allocated} == {world.main.cuda_stream}
    assert not any(hasattr(t, "recorded") for t, _ in world.allocated)
