"""ctypes binding of libmoe_gb300 (include/moe.h, include/moe_train.h), with the same entry-point names.

Argument marshalling only: tensors become device pointers and sizes, the
stream given (else PyTorch's current one) becomes the cudaStream_t, and a
non-zero status raises MoEError.  Output tensors may be passed in (pre-allocated,
e.g. to keep rows past the valid count untouched) or are allocated here with
torch.empty, on the stream that the call runs on.  A caller who gives another
stream orders it after what writes the inputs, and keeps them while it runs.
Every computation runs in the library's CUDA kernels; loading fails loudly if
the library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import re
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libmoe_gb300.so"
HEADER = _PKG.parent / "include" / "moe.h"
TRAIN_HEADER = HEADER.with_name("moe_train.h")

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_WORKSPACE = 0, -1, -2, -3, -4
MOE_DTYPE_BF16, MOE_DTYPE_F32, MOE_DTYPE_E4M3 = 0, 1, 2
MOE_EPILOGUE_NONE, MOE_EPILOGUE_SILU_MUL, MOE_EPILOGUE_SILU_MUL_QUANT = 0, 1, 2
MOE_GEMM_CTA_PAIRS = 0x100
MOE_WEIGHTS_PACKED = 0x200
MOE_BALANCE_SCORES, MOE_BALANCE_SOFTMAX, MOE_BALANCE_SIGMOID = 0, 1, 2
MOE_CHECKPOINT_BLOCK = 128
MOE_ACT_SILU, MOE_ACT_GELU = 0, 1
MOE_DEVERR_BAD_INDEX, MOE_DEVERR_BAD_COUNT, MOE_DEVERR_TIMEOUT = 1, 2, 4


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: int = 0):
        self.status = status
        msg = f"{fn} failed: {_lib.moe_status_string(status).decode()} ({status})"
        if status == MOE_ERR_CUDA:
            msg += f", cudaError {cuda_error}"
        super().__init__(msg)


def _load() -> ctypes.CDLL:
    if not LIB_PATH.exists():
        raise ImportError(f"{LIB_PATH.name} is not built: run `python -m moe_token_routing_index_gb300.build` "
                          "(the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(str(LIB_PATH))
    P, I, L, S, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint)
    F = ctypes.c_float
    sigs = {
        "moe_status_string": ([I], ctypes.c_char_p),
        "moe_last_cuda_error": ([], I),
        "moe_device_error": ([U, P], I),
        "moe_router_workspace_size": ([I, I, I, ctypes.POINTER(S)], I),
        "moe_router_scores": ([P, I, I, P, I, P, P, P, S, P], I),
        "moe_router_route_workspace_size": ([I, I, I, I, ctypes.POINTER(S)], I),
        "moe_router_route": ([P, I, I, P, I, I, P, P, P, P, P, P, P, P, P, S, P], I),
        "moe_dense_gemm": ([P, I, I, P, I, P, P, I, P], I),
        "moe_selftest_bounded_wait": ([I, L, P], I),
        "moe_route_workspace_size": ([I, I, I, ctypes.POINTER(S)], I),
        "moe_route": ([P, I, L, L, I, I, I, P, P, P, P, P, P, P, P, S, P], I),
        "moe_route_no_alloc": ([P, I, L, L, I, I, I, P, P, P, P, P, P, P], I),
        "moe_gather_scale": ([P, I, I, P, P, I, P, I, L, L, I, P, P, I, P, P], I),
        "moe_gather_scale_quant": ([P, I, I, P, P, I, P, I, L, L, I, P, P, I, P, P, P, P], I),
        "moe_quantize_rows": ([P, L, I, P, P, P, P], I),
        "moe_grouped_gemm": ([P, P, P, I, I, I, I, P, I, P, I, I, P, P, P, P], I),
        "moe_expert_mlp_workspace_size": ([I, ctypes.POINTER(S)], I),
        "moe_scatter_add_padded": ([P, P, P, I, P, P, I, I, I, I, I, P], I),
        "moe_topk_finalize": ([P, L, I, P, I, P, I, I, P, P, P, P], I),
        "moe_expert_mlp": ([P, P, P, P, I, I, I, I, P, P, P, I, I, P, S, I, P], I),
        "moe_pack_weights_size": ([I, I, I, I, ctypes.POINTER(S)], I),
        "moe_pack_weights": ([P, I, I, I, I, P, P], I),
        "moe_grouped_gemm_fp8_rowwise": ([P, P, P, P, P, I, I, I, I, P, I, P, I, I, P, P, P, P], I),
        "moe_silu_mul": ([P, P, L, I, I, P, P, P], I),
        "moe_silu_mul_quant": ([P, P, L, I, I, P, P, P, P, P], I),
        "moe_scatter_add": ([P, P, P, P, I, I, I, I, P, I, P], I),
        "moe_layer_norm": ([P, L, I, I, I, P, P, I, F, P, P, P, P, P], I),
        "moe_layer_norm_backward_workspace_size": ([I, I, ctypes.POINTER(S)], I),
        "moe_layer_norm_backward": ([P, P, L, I, I, I, P, I, P, P, P, P, P, P, P, P, S, P], I),
        "moe_balance_loss_workspace_size": ([I, I, ctypes.POINTER(S)], I),
        "moe_balance_loss": ([P, I, L, L, I, I, I, I, F, P, P, P, P, P, P, S, P], I),
        "moe_balance_loss_backward": ([P, I, L, L, I, I, I, I, F, P, P, P, P, I, P], I),
        "moe_checkpoint_pack": ([P, L, I, I, P, P, P, P], I),
        "moe_checkpoint_unpack": ([P, P, I, I, P, P, P], I),
        "moe_silu_mul_checkpoint": ([P, P, L, I, I, P, P, P, P, P], I),
        "moe_silu_mul_backward": ([P, P, P, I, I, P, P, P, P], I),
        "moe_grouped_weight_grad_workspace_size": ([I, I, I, I, I, ctypes.POINTER(S)], I),
        "moe_grouped_weight_grad": ([P, P, P, P, I, I, I, I, P, I, I, P, S, P], I),
        "moe_gated_mlp": ([P, P, P, P, I, I, I, I, I, P, P, P, P], I),
        "moe_gated_mlp_backward": ([P, P, P, P, P, P, I, I, I, I, I, P, P, P, P], I),
        "moe_orthogonalize_workspace_size": ([I, I, I, ctypes.POINTER(S)], I),
        "moe_orthogonalize": ([P, I, L, L, I, I, I, I, P, F, F, P, P, S, P], I),
        "moe_muon_update": ([P, I, P, I, P, I, I, I, F, I, F, P, F, I, P, F, P, S, P], I),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    return lib


_lib = _load()


def header_symbols() -> list[str]:
    """Names of the functions include/moe.h and include/moe_train.h declare."""
    text = HEADER.read_text() + TRAIN_HEADER.read_text()
    return sorted(set(re.findall(r"^(?:int|const char\*)\s+(moe_\w+)\s*\(", text, flags=re.M)))


def library() -> ctypes.CDLL:
    return _lib


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status, _lib.moe_last_cuda_error() if status == MOE_ERR_CUDA else 0)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it, which costs a call 2.6 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_current_device())


def _call_on(fn, args: dict):
    """A wrapper's call with its arguments (its locals() on entry), on the stream among them.

    What the call allocates comes from that stream's memory: the caching allocator reuses a block
    in the order of the stream it was allocated on, so a workspace of the current stream's would be
    written while that stream still reads what lay there, and handed out again under the kernel.
    The caller's stream is recorded on the results, which are used there."""
    stream = args.pop("stream")
    if stream.cuda_stream == _stream():
        return fn(**args)
    caller = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        result = fn(**args)
    _record(result, caller)
    return result


def _record(result, stream):
    if isinstance(result, torch.Tensor):
        result.record_stream(stream)
    elif isinstance(result, Checkpoint):
        _record((result.codes, result.exponents), stream)
    elif isinstance(result, PackedWeights):
        _record(result.data, stream)
    elif isinstance(result, dict):
        _record(tuple(result.values()), stream)
    elif isinstance(result, tuple):
        for r in result:
            _record(r, stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MOE_DTYPE_BF16
    if t.dtype == torch.float32:
        return MOE_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t: torch.Tensor, dtype, name: str, contiguous: bool = True):
    """dtype, device and layout checks of a matrix argument: the C ABI reads it as a
    dense row-major array (contiguous=False: only the last dimension must be dense; the
    row stride of a single row, which PyTorch may set to any number, is then not passed on)."""
    if t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not contiguous and t.dim() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be dense along its last dimension")


def device_error(stream=None) -> int:
    """Read and clear the device-side error bits (synchronises the stream)."""
    bits = ctypes.c_uint(0)
    _check("moe_device_error", _lib.moe_device_error(ctypes.byref(bits), _stream(stream)))
    return bits.value


# ------------------------------------------------------------------ routing

def moe_router_workspace_size(T: int, D: int, E: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_router_workspace_size", _lib.moe_router_workspace_size(T, D, E, ctypes.byref(n)))
    return n.value


def moe_router_scores(x: torch.Tensor, w_router: torch.Tensor, num_valid_tokens: torch.Tensor | None = None, *,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """scores[T, E] = bf16(sigmoid(bf16(x @ w_router.T))) for x[T, D] and w_router[E, D] (bf16)."""
    if stream is not None:
        return _call_on(moe_router_scores, locals())
    T, D = x.shape
    E = w_router.shape[0]
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router")
    if num_valid_tokens is not None:
        _need(num_valid_tokens, torch.int32, "num_valid_tokens")
    if out is None:
        out = torch.empty(T, E, dtype=torch.bfloat16, device=x.device)
    _need(out, out.dtype, "out")
    ws_bytes = moe_router_workspace_size(T, D, E)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=x.device)
    st = _lib.moe_router_scores(_ptr(x), T, D, _ptr(w_router), E, _ptr(num_valid_tokens), _ptr(out),
                                _ptr(workspace), workspace.numel(), _stream())
    _check("moe_router_scores", st)
    return out


def moe_router_route_workspace_size(T: int, D: int, E: int, top_k: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_router_route_workspace_size", _lib.moe_router_route_workspace_size(T, D, E, top_k, ctypes.byref(n)))
    return n.value


def moe_router_route(x: torch.Tensor, w_router: torch.Tensor, top_k: int, num_valid_tokens=None, *,
                     scores: torch.Tensor | None = None, with_weights: bool = False, out: dict | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Router scores and routing in two kernels (the top-k selection in the router's
    epilogue).  Returns (scores[T, E] bf16, the dict of moe_route)."""
    if stream is not None:
        return _call_on(moe_router_route, locals())
    T, D = x.shape
    E = w_router.shape[0]
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router")
    if num_valid_tokens is not None:
        _need(num_valid_tokens, torch.int32, "num_valid_tokens")
    if scores is None:
        scores = torch.empty(T, E, dtype=torch.bfloat16, device=x.device)
    _need(scores, torch.bfloat16, "scores")
    dev = x.device
    o = dict(out or {})
    i32 = dict(dtype=torch.int32, device=dev)
    o.setdefault("counts", torch.empty(E + 1, **i32))
    o.setdefault("expert_offsets", torch.empty(E + 1, **i32))
    o.setdefault("expert_indices", torch.empty(T * top_k, **i32))
    o.setdefault("token_indices", torch.empty(T * top_k, **i32))
    o.setdefault("inv_rows", torch.empty(T * top_k, **i32))
    if with_weights:
        o.setdefault("topk_weights", torch.empty(T * top_k, dtype=torch.float32, device=dev))
    else:
        o["topk_weights"] = None
    ws_bytes = moe_router_route_workspace_size(T, D, E, top_k)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    st = _lib.moe_router_route(_ptr(x), T, D, _ptr(w_router), E, top_k, _ptr(num_valid_tokens), _ptr(scores),
                               _ptr(o["counts"]), _ptr(o["expert_offsets"]), _ptr(o["expert_indices"]),
                               _ptr(o["token_indices"]), _ptr(o["inv_rows"]), _ptr(o["topk_weights"]),
                               _ptr(workspace), workspace.numel(), _stream())
    _check("moe_router_route", st)
    return scores, o


def moe_route_workspace_size(T: int, E: int, top_k: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_route_workspace_size", _lib.moe_route_workspace_size(T, E, top_k, ctypes.byref(n)))
    return n.value


def moe_route(scores: torch.Tensor, top_k: int, num_valid_tokens: torch.Tensor | None = None, *,
              with_inv: bool = True, with_weights: bool = False, out: dict | None = None,
              workspace: torch.Tensor | None = None, stream=None):
    """Route scores[T, E]; returns dict(counts, expert_offsets, expert_indices,
    token_indices, inv_rows) of int32 device tensors (index arrays of T * top_k),
    plus topk_weights (fp32 [T * top_k], in inv_rows order) when with_weights."""
    if stream is not None:
        return _call_on(moe_route, locals())
    T, E = scores.shape
    dev = scores.device
    o = dict(out or {})
    i32 = dict(dtype=torch.int32, device=dev)
    o.setdefault("counts", torch.empty(E + 1, **i32))
    o.setdefault("expert_offsets", torch.empty(E + 1, **i32))
    o.setdefault("expert_indices", torch.empty(T * top_k, **i32))
    o.setdefault("token_indices", torch.empty(T * top_k, **i32))
    if with_inv:
        o.setdefault("inv_rows", torch.empty(T * top_k, **i32))
    else:
        o["inv_rows"] = None
    if with_weights:
        o.setdefault("topk_weights", torch.empty(T * top_k, dtype=torch.float32, device=dev))
    else:
        o["topk_weights"] = None
    ws_bytes = moe_route_workspace_size(T, E, top_k)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    if num_valid_tokens is not None:
        _need(num_valid_tokens, torch.int32, "num_valid_tokens")
    st = _lib.moe_route(_ptr(scores), _dtype_code(scores), scores.stride(0), scores.stride(1), T, E, top_k,
                        _ptr(num_valid_tokens), _ptr(o["counts"]), _ptr(o["expert_offsets"]),
                        _ptr(o["expert_indices"]), _ptr(o["token_indices"]), _ptr(o["inv_rows"]),
                        _ptr(o["topk_weights"]), _ptr(workspace), workspace.numel(), _stream())
    _check("moe_route", st)
    return o


def _scores_args(scores):
    """(pointer, dtype code, stride_t, stride_e, E) of a score tensor; None = unit scores."""
    if scores is None:
        return None, MOE_DTYPE_BF16, 0, 0, 1
    return _ptr(scores), _dtype_code(scores), scores.stride(0), scores.stride(1), scores.shape[1]


# ------------------------------------------------------------------- gather

def moe_gather_scale(x, token_indices, expert_indices, scores, valid_token_count=None, *, inv_rows=None,
                     top_k: int = 1, out=None, stream=None):
    if stream is not None:
        return _call_on(moe_gather_scale, locals())
    T, D = x.shape
    a = token_indices.shape[0]
    _need(x, torch.bfloat16, "x")
    if out is None:
        out = torch.empty(a, D, dtype=x.dtype, device=x.device)
    _need(out, out.dtype, "out")
    st = _lib.moe_gather_scale(_ptr(x), T, D, _ptr(token_indices), _ptr(expert_indices), a, *_scores_args(scores),
                               _ptr(valid_token_count), _ptr(inv_rows), top_k, _ptr(out), _stream())
    _check("moe_gather_scale", st)
    return out


def moe_gather_scale_quant(x, token_indices, expert_indices, scores, scale_ub=None, valid_token_count=None, *,
                           inv_rows=None, top_k: int = 1, out=None, out_scale=None, stream=None):
    if stream is not None:
        return _call_on(moe_gather_scale_quant, locals())
    T, D = x.shape
    a = token_indices.shape[0]
    _need(x, torch.bfloat16, "x")
    if out is None:
        out = torch.empty(a, D, dtype=torch.float8_e4m3fn, device=x.device)
    _need(out, out.dtype, "out")
    if out_scale is None:
        out_scale = torch.empty(a, dtype=torch.float32, device=x.device)
    _need(out_scale, out_scale.dtype, "out_scale")
    st = _lib.moe_gather_scale_quant(_ptr(x), T, D, _ptr(token_indices), _ptr(expert_indices), a,
                                     *_scores_args(scores),
                                     _ptr(valid_token_count), _ptr(inv_rows), top_k, _ptr(scale_ub), _ptr(out),
                                     _ptr(out_scale), _stream())
    _check("moe_gather_scale_quant", st)
    return out, out_scale


def moe_quantize_rows(w: torch.Tensor, scale_ub=None, *, out=None, out_scale=None, stream=None):
    """Per-row FP8 quantisation over the last dim of an fp32 tensor."""
    if stream is not None:
        return _call_on(moe_quantize_rows, locals())
    _need(w, torch.float32, "w")
    cols = w.shape[-1]
    rows = w.numel() // cols if cols else 0
    if out is None:
        out = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
    _need(out, out.dtype, "out")
    if out_scale is None:
        out_scale = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
    _need(out_scale, out_scale.dtype, "out_scale")
    st = _lib.moe_quantize_rows(_ptr(w), rows, cols, _ptr(scale_ub), _ptr(out), _ptr(out_scale), _stream())
    _check("moe_quantize_rows", st)
    return out, out_scale


# ------------------------------------------------------------- grouped GEMM

def _scatter_args(scatter_indices, out, accumulate):
    if scatter_indices is None:
        return None, 0, 0
    if out is None:
        raise ValueError("the fused combine writes into a caller-provided out[T, N]")
    return scatter_indices, out.shape[0], int(accumulate)


class PackedWeights:
    """Weights [E, N, K] (bf16 or e4m3) in the tile-packed layout of moe_pack_weights:
    `data` holds the packed bytes on the device; `shape` and `dtype` are the logical
    ones.  Accepted wherever the grouped GEMMs and moe_expert_mlp take weights."""

    def __init__(self, data: torch.Tensor, shape, dtype):
        self.data, self.shape, self.dtype = data, tuple(shape), dtype

    @property
    def device(self):
        return self.data.device


def moe_pack_weights_size(E: int, N: int, K: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_pack_weights_size", _lib.moe_pack_weights_size(E, N, K, dtype, ctypes.byref(n)))
    return n.value


def moe_pack_weights(w: torch.Tensor, stream=None) -> PackedWeights:
    """Tile-packed copy of w [E, N, K] bf16 or e4m3 (every 128-row x 128-byte box contiguous)."""
    if stream is not None:
        return _call_on(moe_pack_weights, locals())
    E, N, K = w.shape
    if w.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError(f"w must be bf16 or e4m3, got {w.dtype}")
    _need(w, w.dtype, "w")
    dt = MOE_DTYPE_E4M3 if w.dtype == torch.float8_e4m3fn else MOE_DTYPE_BF16
    data = torch.empty(moe_pack_weights_size(E, N, K, dt), dtype=torch.uint8, device=w.device)
    _check("moe_pack_weights", _lib.moe_pack_weights(_ptr(w), E, N, K, dt, _ptr(data), _stream()))
    return PackedWeights(data, (E, N, K), w.dtype)


def _weights_arg(w, dtype, name: str, flags: int):
    """Pointer and flags of a weights argument: a row-major [E, N, K] tensor or PackedWeights."""
    if isinstance(w, PackedWeights):
        if w.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got packed {w.dtype}")
        if not w.data.is_cuda:
            raise TypeError(f"{name} must be on a CUDA device")
        return _ptr(w.data), flags | MOE_WEIGHTS_PACKED
    _need(w, dtype, name)
    return _ptr(w), flags


def _gemm_outputs(x, N, epilogue, out, z_out, z_scale):
    """The bf16 output (y, or z for the SiLU epilogues) and, with SILU_MUL_QUANT,
    the e4m3 z and its row scales; allocated when not given."""
    a_max = x.shape[0]
    kind = epilogue & 0xFF
    n_out = N // 2 if kind in (MOE_EPILOGUE_SILU_MUL, MOE_EPILOGUE_SILU_MUL_QUANT) else N
    if out is None:
        out = torch.empty(a_max, n_out, dtype=torch.bfloat16, device=x.device)
    _need(out, out.dtype, "out")
    if kind != MOE_EPILOGUE_SILU_MUL_QUANT:
        return out, None, None
    if z_out is None:
        z_out = torch.empty(a_max, n_out, dtype=torch.float8_e4m3fn, device=x.device)
    _need(z_out, torch.float8_e4m3fn, "z_out")
    if z_scale is None:
        z_scale = torch.empty(a_max, dtype=torch.float32, device=x.device)
    _need(z_scale, torch.float32, "z_scale")
    return out, z_out, z_scale


def moe_grouped_gemm(x, w, counts, *, epilogue: int = MOE_EPILOGUE_NONE, out=None, scatter_indices=None,
                     accumulate: bool = True, scale_ub=None, z_out=None, z_scale=None, stream=None):
    """x[a_max, K] bf16, w[E, N, K] bf16, counts[>= E] int32 -> y[a_max, N or N/2].
    With scatter_indices (top_k = 1), routed row r lands in out[scatter_indices[r]].
    With MOE_EPILOGUE_SILU_MUL_QUANT, out receives the bf16 z and the call returns
    (z_out e4m3 [a_max, N/2], z_scale fp32 [a_max]) instead."""
    if stream is not None:
        return _call_on(moe_grouped_gemm, locals())
    a_max, K = x.shape
    E, N, K2 = w.shape
    assert K == K2
    _need(x, torch.bfloat16, "x")
    w_ptr, epilogue = _weights_arg(w, torch.bfloat16, "w", epilogue)
    si, t_out, acc = _scatter_args(scatter_indices, out, accumulate)
    out, z_out, z_scale = _gemm_outputs(x, N, epilogue, out, z_out, z_scale)
    st = _lib.moe_grouped_gemm(_ptr(x), w_ptr, _ptr(counts), E, a_max, N, K, _ptr(out), epilogue, _ptr(si),
                               t_out, acc, _ptr(scale_ub), _ptr(z_out), _ptr(z_scale), _stream())
    _check("moe_grouped_gemm", st)
    return out if z_out is None else (z_out, z_scale)


def moe_grouped_gemm_fp8_rowwise(x, w, counts, x_scale, w_scale, *, epilogue: int = MOE_EPILOGUE_NONE, out=None,
                                 scatter_indices=None, accumulate: bool = True, scale_ub=None, z_out=None,
                                 z_scale=None, stream=None):
    """As moe_grouped_gemm on e4m3 x[a_max, K] and w[E, N, K] with fp32 row scales
    x_scale[a_max] and w_scale[E, N]."""
    if stream is not None:
        return _call_on(moe_grouped_gemm_fp8_rowwise, locals())
    a_max, K = x.shape
    E, N, K2 = w.shape
    assert K == K2
    _need(x, torch.float8_e4m3fn, "x")
    w_ptr, epilogue = _weights_arg(w, torch.float8_e4m3fn, "w", epilogue)
    si, t_out, acc = _scatter_args(scatter_indices, out, accumulate)
    out, z_out, z_scale = _gemm_outputs(x, N, epilogue, out, z_out, z_scale)
    st = _lib.moe_grouped_gemm_fp8_rowwise(_ptr(x), w_ptr, _ptr(counts), _ptr(x_scale), _ptr(w_scale), E, a_max,
                                           N, K, _ptr(out), epilogue, _ptr(si), t_out, acc, _ptr(scale_ub),
                                           _ptr(z_out), _ptr(z_scale), _stream())
    _check("moe_grouped_gemm_fp8_rowwise", st)
    return out if z_out is None else (z_out, z_scale)


def moe_expert_mlp_workspace_size(E: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_expert_mlp_workspace_size", _lib.moe_expert_mlp_workspace_size(E, ctypes.byref(n)))
    return n.value


def moe_expert_mlp(x, w13, w2, counts, *, z=None, out=None, scatter_indices=None, accumulate: bool = True,
                   workspace=None, stream=None):
    """Both bf16 grouped GEMMs in one launch: z = silu_mul(x w13^T), out = z w2^T per expert
    (with scatter_indices, top_k = 1: row r lands in out[scatter_indices[r]])."""
    if stream is not None:
        return _call_on(moe_expert_mlp, locals())
    a_max, D = x.shape
    E, n2, D2 = w13.shape
    H = n2 // 2
    assert D == D2 and tuple(w2.shape) == (E, D, H)
    _need(x, torch.bfloat16, "x")
    if isinstance(w13, PackedWeights) != isinstance(w2, PackedWeights):
        raise TypeError("w13 and w2 must both be packed or both be row-major")
    w13_ptr, flags = _weights_arg(w13, torch.bfloat16, "w13", 0)
    w2_ptr, _ = _weights_arg(w2, torch.bfloat16, "w2", 0)
    if z is None:
        z = torch.empty(a_max, H, dtype=torch.bfloat16, device=x.device)
    _need(z, z.dtype, "z")
    si, t_out, acc = _scatter_args(scatter_indices, out, accumulate)
    if out is None:
        out = torch.empty(a_max, D, dtype=torch.bfloat16, device=x.device)
    _need(out, out.dtype, "out")
    if workspace is None:   # zero on first use; each call leaves it zero
        workspace = torch.zeros(moe_expert_mlp_workspace_size(E), dtype=torch.uint8, device=x.device)
    st = _lib.moe_expert_mlp(_ptr(x), w13_ptr, w2_ptr, _ptr(counts), E, a_max, D, H, _ptr(z), _ptr(out),
                             _ptr(si), t_out, acc, _ptr(workspace), workspace.numel(), flags, _stream())
    _check("moe_expert_mlp", st)
    return out


# ----------------------------------------------------------------- silu_mul

def moe_silu_mul(y, H: int | None = None, valid_rows=None, *, out=None, stream=None):
    """y[a, 2H] bf16 -> z[a, H] = silu(y[:, :H]) * y[:, H:]."""
    if stream is not None:
        return _call_on(moe_silu_mul, locals())
    a, n2 = y.shape
    H = n2 // 2 if H is None else H
    _need(y, torch.bfloat16, "y", contiguous=False)
    if out is None:
        out = torch.empty(a, H, dtype=torch.bfloat16, device=y.device)
    _need(out, out.dtype, "out")
    x1 = ctypes.c_void_p(y.data_ptr() + H * y.element_size())
    st = _lib.moe_silu_mul(_ptr(y), x1, y.stride(0) if a > 1 else 2 * H, a, H, _ptr(valid_rows), _ptr(out), _stream())
    _check("moe_silu_mul", st)
    return out


def moe_silu_mul_quant(y, H: int | None = None, scale_ub=None, valid_rows=None, *, out=None, out_scale=None,
                       stream=None):
    if stream is not None:
        return _call_on(moe_silu_mul_quant, locals())
    a, n2 = y.shape
    H = n2 // 2 if H is None else H
    _need(y, torch.bfloat16, "y", contiguous=False)
    if out is None:
        out = torch.empty(a, H, dtype=torch.float8_e4m3fn, device=y.device)
    _need(out, out.dtype, "out")
    if out_scale is None:
        out_scale = torch.empty(a, dtype=torch.float32, device=y.device)
    _need(out_scale, out_scale.dtype, "out_scale")
    x1 = ctypes.c_void_p(y.data_ptr() + H * y.element_size())
    st = _lib.moe_silu_mul_quant(_ptr(y), x1, y.stride(0) if a > 1 else 2 * H, a, H, _ptr(valid_rows), _ptr(scale_ub),
                                 _ptr(out), _ptr(out_scale), _stream())
    _check("moe_silu_mul_quant", st)
    return out, out_scale


# -------------------------------------------------------------- scatter-add

def moe_scatter_add(out, rows, token_indices, inv_rows=None, top_k: int = 1, valid_token_count=None, *,
                    accumulate: bool = True, stream=None):
    """out[T, D] += rows[a, D] by token, in place (deterministic); with
    accumulate=False the routed sum overwrites the valid tokens of out."""
    T, D = out.shape
    a = rows.shape[0]
    _need(out, torch.bfloat16, "out")
    _need(rows, torch.bfloat16, "rows")
    st = _lib.moe_scatter_add(_ptr(out), _ptr(rows), _ptr(token_indices), _ptr(inv_rows), top_k, a, T, D,
                              _ptr(valid_token_count), int(accumulate), _stream(stream))
    _check("moe_scatter_add", st)
    return out


def moe_scatter_add_padded(out, rows, token_counts, token_indices, inv_rows=None, top_k: int = 1, *,
                           accumulate: bool = True, stream=None):
    """scatter_add_padded_tokens on one GPU: the first sum(token_counts) rows of
    rows[T_K, D] (by-expert order) are added into out[T, D] by token."""
    T, D = out.shape
    T_K = rows.shape[0]
    E = token_counts.shape[0]
    _need(out, torch.bfloat16, "out")
    _need(rows, torch.bfloat16, "rows")
    _need(token_counts, torch.int32, "token_counts")
    st = _lib.moe_scatter_add_padded(_ptr(out), _ptr(rows), _ptr(token_counts), E, _ptr(token_indices),
                                     _ptr(inv_rows), top_k, T_K, T, D, int(accumulate), _stream(stream))
    _check("moe_scatter_add_padded", st)
    return out


def moe_topk_finalize(rows, expert_weights, expanded_idx_to_permuted_idx, shared_output=None,
                      valid_token_count=None, *, out=None, stream=None):
    """out[M, D] = bf16(sum_j w[t, j] * rows[idx[t, j]]) (-0 -> +0), plus the shared
    output (one more rounding); rows[n, D] bf16, weights fp32 or bf16 [M, k], idx int32 [M, k]."""
    if stream is not None:
        return _call_on(moe_topk_finalize, locals())
    n_rows, D = rows.shape
    M, k = expanded_idx_to_permuted_idx.shape
    _need(rows, torch.bfloat16, "rows")
    _need(expanded_idx_to_permuted_idx, torch.int32, "expanded_idx_to_permuted_idx")
    if shared_output is not None:
        _need(shared_output, torch.bfloat16, "shared_output")
    if out is None:
        out = torch.empty(M, D, dtype=torch.bfloat16, device=rows.device)
    _need(out, out.dtype, "out")
    st = _lib.moe_topk_finalize(_ptr(rows), n_rows, D, _ptr(expert_weights), _dtype_code(expert_weights),
                                _ptr(expanded_idx_to_permuted_idx), M, k, _ptr(valid_token_count),
                                _ptr(shared_output), _ptr(out), _stream())
    _check("moe_topk_finalize", st)
    return out


def moe_dense_gemm(x, w, valid_rows=None, *, epilogue: int = MOE_EPILOGUE_NONE, out=None, stream=None):
    """y = x[M, K] @ w[N, K]^T (bf16, split-K over a cluster); with the SiLU*mul
    epilogue y[M, N/2] = silu_mul of the two halves."""
    if stream is not None:
        return _call_on(moe_dense_gemm, locals())
    M, K = x.shape
    N, K2 = w.shape
    assert K == K2
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    if valid_rows is not None:
        _need(valid_rows, torch.int32, "valid_rows")
    n_out = N // 2 if epilogue == MOE_EPILOGUE_SILU_MUL else N
    if out is None:
        out = torch.empty(M, n_out, dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out")
    st = _lib.moe_dense_gemm(_ptr(x), M, K, _ptr(w), N, _ptr(valid_rows), _ptr(out), epilogue, _stream())
    _check("moe_dense_gemm", st)
    return out


# ----------------------------------------------------------------- layer norm

def _no_value(name: str):
    raise ValueError(f"{name} must hold a value")


def _valid_arg(valid, name: str, dtype=torch.int32):
    """The pointer of a scalar on the device, or none.  (An empty tensor's is null, which would be read as none.)"""
    if valid is None:
        return None
    _need(valid, dtype, name)
    return valid.data_ptr() or _no_value(name)


def _workspace_bytes(workspace) -> int:
    """The size of a caller's workspace, which must be device memory."""
    if not workspace.is_cuda:
        raise TypeError("the workspace must be a CUDA tensor")
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _output(t, shape, dtype, device, name: str) -> torch.Tensor:
    """A caller's output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t
    _need(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {shape}, got {tuple(t.shape)}")
    return t


def _norm_inputs(x, gamma, beta=None) -> int:
    """Checks x [T, D] (rows of any stride) and the weights [D]; returns D."""
    if x.dim() != 2:
        raise ValueError(f"x must be [T, D], got {tuple(x.shape)}")
    _need(x, x.dtype, "x", contiguous=False)
    D = x.shape[1]
    _output(gamma, (D,), gamma.dtype, None, "gamma")
    if beta is not None:
        _output(beta, (D,), gamma.dtype, None, "beta")
    return D


def moe_layer_norm(x, gamma, beta=None, num_valid_tokens=None, *, eps: float = 1e-5, out=None, mean=None, rstd=None,
                   stream=None):
    """Layer norm of x[T, D] (bf16 or fp32, rows of any stride) with gamma, beta [D]: returns
    (y, mean, rstd), mean and rstd [T] in fp32 for the backward pass."""
    if stream is not None:
        return _call_on(moe_layer_norm, locals())
    D = _norm_inputs(x, gamma, beta)
    T, dev = x.shape[0], x.device
    out = _output(out, (T, D), x.dtype, dev, "out")
    mean = _output(mean, (T,), torch.float32, dev, "mean")
    rstd = _output(rstd, (T,), torch.float32, dev, "rstd")
    st = _lib.moe_layer_norm(_ptr(x), x.stride(0) if T > 1 else D, T, D, _dtype_code(x), _ptr(gamma), _ptr(beta),
                             _dtype_code(gamma), eps, _valid_arg(num_valid_tokens, "num_valid_tokens"), _ptr(out),
                             _ptr(mean), _ptr(rstd), _stream())
    _check("moe_layer_norm", st)
    return out, mean, rstd


@functools.lru_cache(maxsize=1024)
def moe_layer_norm_backward_workspace_size(T: int, D: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_layer_norm_backward_workspace_size",
           _lib.moe_layer_norm_backward_workspace_size(T, D, ctypes.byref(n)))
    return n.value


def moe_layer_norm_backward(dy, x, gamma, mean, rstd, num_valid_tokens=None, *, residual_grad=None, out=None,
                            dgamma=None, dbeta=None, with_beta: bool = True, workspace=None, stream=None):
    """The gradient of moe_layer_norm: returns (dx [T, D], dgamma [D], dbeta [D]), the last two in
    fp32 (dbeta None without with_beta).  residual_grad [T, D] is added to dx before its rounding."""
    if stream is not None:
        return _call_on(moe_layer_norm_backward, locals())
    D = _norm_inputs(x, gamma)
    T, dt, dev = x.shape[0], x.dtype, x.device
    _output(dy, (T, D), dt, None, "dy")
    _output(mean, (T,), torch.float32, None, "mean")
    _output(rstd, (T,), torch.float32, None, "rstd")
    if residual_grad is not None:
        _output(residual_grad, (T, D), dt, None, "residual_grad")
    out = _output(out, (T, D), dt, dev, "out")
    dgamma = _output(dgamma, (D,), torch.float32, dev, "dgamma")
    dbeta = _output(dbeta, (D,), torch.float32, dev, "dbeta") if with_beta else None
    if workspace is None:
        ws_bytes = moe_layer_norm_backward_workspace_size(T, D)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    else:
        ws_bytes = _workspace_bytes(workspace)
    st = _lib.moe_layer_norm_backward(_ptr(dy), _ptr(x), x.stride(0) if T > 1 else D, T, D, _dtype_code(x), _ptr(gamma),
                                      _dtype_code(gamma), _ptr(mean), _ptr(rstd),
                                      _valid_arg(num_valid_tokens, "num_valid_tokens"), _ptr(residual_grad),
                                      _ptr(out), _ptr(dgamma), _ptr(dbeta), _ptr(workspace), ws_bytes, _stream())
    _check("moe_layer_norm_backward", st)
    return out, dgamma, dbeta


# --------------------------------------------------------------- balance loss

@functools.lru_cache(maxsize=1024)
def moe_balance_loss_workspace_size(T: int, E: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_balance_loss_workspace_size", _lib.moe_balance_loss_workspace_size(T, E, ctypes.byref(n)))
    return n.value


def _balance_inputs(scores, counts):
    if scores.dim() != 2:
        raise ValueError(f"scores must be [T, E], got {tuple(scores.shape)}")
    if not scores.is_cuda:
        raise TypeError("scores must be a CUDA tensor")
    if counts is not None:
        _need(counts, torch.int32, "counts")
        if counts.numel() < scores.shape[1]:
            raise ValueError("counts must hold a count for each expert")
    return scores.shape


def moe_balance_loss(scores, top_k: int, num_valid_tokens=None, *, kind: int = MOE_BALANCE_SCORES,
                     coefficient: float = 1.0, counts=None, workspace=None, stream=None):
    """Load-balance loss of a top_k router from its output scores[T, E] (bf16 or fp32, any strides):
    returns (loss [1] fp32, counts [E + 1] int32, mean_probs [E] fp32).  counts: those of moe_route for
    the same tokens, when there are some (returned as they are); else the selection is made here."""
    if stream is not None:
        return _call_on(moe_balance_loss, locals())
    T, E = _balance_inputs(scores, counts)
    dev = scores.device
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    mean_probs = torch.empty(E, dtype=torch.float32, device=dev)
    made = torch.empty(E + 1, dtype=torch.int32, device=dev) if counts is None else None
    if workspace is not None:
        ws_bytes = _workspace_bytes(workspace)
    elif ws_bytes := moe_balance_loss_workspace_size(T, E):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = _lib.moe_balance_loss(_ptr(scores), _dtype_code(scores), scores.stride(0), scores.stride(1), T, E, top_k,
                               kind, coefficient, _valid_arg(num_valid_tokens, "num_valid_tokens"), _ptr(counts),
                               _ptr(made), _ptr(mean_probs), _ptr(loss), _ptr(workspace), ws_bytes, _stream())
    _check("moe_balance_loss", st)
    return loss, made if counts is None else counts, mean_probs


def moe_balance_loss_backward(scores, counts, top_k: int, num_valid_tokens=None, *, kind: int = MOE_BALANCE_SCORES,
                              coefficient: float = 1.0, dloss=None, out=None, accumulate: bool = False, stream=None):
    """The gradient of moe_balance_loss with respect to scores (same dtype, [T, E]); dloss: fp32 [1] on the
    device (None: 1).  With accumulate it is added to out."""
    if stream is not None:
        return _call_on(moe_balance_loss_backward, locals())
    T, E = _balance_inputs(scores, counts)
    if accumulate and out is None:
        raise ValueError("accumulate adds to a caller-provided out[T, E]")
    out = _output(out, (T, E), scores.dtype, scores.device, "out")
    st = _lib.moe_balance_loss_backward(_ptr(scores), _dtype_code(scores), scores.stride(0), scores.stride(1), T, E,
                                        top_k, kind, coefficient, _valid_arg(num_valid_tokens, "num_valid_tokens"),
                                        _ptr(counts), _valid_arg(dloss, "dloss", torch.float32), _ptr(out),
                                        int(accumulate), _stream())
    _check("moe_balance_loss_backward", st)
    return out


# ----------------------------------------------------------- 8-bit checkpoints

class Checkpoint:
    """bf16 rows kept in 8 bits: `codes` [a, W] float8_e4m3fn and `exponents` uint8, one per 128 columns of
    a row (of a row's half when halves = 2, as moe_silu_mul_checkpoint writes them)."""

    def __init__(self, codes: torch.Tensor, exponents: torch.Tensor, halves: int = 1):
        if codes.dim() != 2 or halves not in (1, 2) or codes.shape[1] % halves:
            raise ValueError(f"codes [a, W] in {halves} halves, got {tuple(codes.shape)}")
        a, W = codes.shape
        blocks = halves * -(-(W // halves) // MOE_CHECKPOINT_BLOCK)
        _need(codes, torch.float8_e4m3fn, "codes")
        _need(exponents, torch.uint8, "exponents")
        if tuple(exponents.shape) != (a, blocks):
            raise ValueError(f"exponents must have the shape {(a, blocks)}, got {tuple(exponents.shape)}")
        self.codes, self.exponents, self.halves = codes, exponents, halves

    @classmethod
    def empty(cls, a: int, W: int, device, halves: int = 1) -> "Checkpoint":
        blocks = halves * -(-(W // halves) // MOE_CHECKPOINT_BLOCK)
        return cls(torch.empty(a, W, dtype=torch.float8_e4m3fn, device=device),
                   torch.empty(a, blocks, dtype=torch.uint8, device=device), halves)

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device


def _checkpoint_arg(ck, a: int, W: int, halves: int) -> Checkpoint:
    """A checkpoint to be read, or a caller's to be written, checked."""
    if not isinstance(ck, Checkpoint):
        raise TypeError(f"a Checkpoint is needed, got {type(ck).__name__}")
    if tuple(ck.shape) != (a, W) or ck.halves != halves:
        raise ValueError(f"the checkpoint must hold [{a}, {W}] in {halves} half or halves, "
                         f"got {tuple(ck.shape)} in {ck.halves}")
    return ck


def moe_checkpoint_pack(x, valid_rows=None, *, checkpoint=None, stream=None) -> Checkpoint:
    """bf16 rows x[a, W] (any row stride) as an 8-bit checkpoint."""
    if stream is not None:
        return _call_on(moe_checkpoint_pack, locals())
    a, W = x.shape
    _need(x, torch.bfloat16, "x", contiguous=False)
    ck = Checkpoint.empty(a, W, x.device) if checkpoint is None else _checkpoint_arg(checkpoint, a, W, 1)
    st = _lib.moe_checkpoint_pack(_ptr(x), x.stride(0) if a > 1 else W, a, W, _valid_arg(valid_rows, "valid_rows"),
                                  _ptr(ck.codes), _ptr(ck.exponents), _stream())
    _check("moe_checkpoint_pack", st)
    return ck


def moe_checkpoint_unpack(checkpoint: Checkpoint, valid_rows=None, *, out=None, stream=None):
    """The bf16 rows [a, W] that a checkpoint (of one half) holds, exactly."""
    if stream is not None:
        return _call_on(moe_checkpoint_unpack, locals())
    if not isinstance(checkpoint, Checkpoint):
        raise TypeError(f"a Checkpoint is needed, got {type(checkpoint).__name__}")
    a, W = checkpoint.shape
    if checkpoint.halves != 1:
        raise ValueError("a checkpoint in two halves is read by moe_silu_mul_backward")
    out = _output(out, (a, W), torch.bfloat16, checkpoint.device, "out")
    st = _lib.moe_checkpoint_unpack(_ptr(checkpoint.codes), _ptr(checkpoint.exponents), a, W,
                                    _valid_arg(valid_rows, "valid_rows"), _ptr(out), _stream())
    _check("moe_checkpoint_unpack", st)
    return out


def moe_silu_mul_checkpoint(y, H: int | None = None, valid_rows=None, *, out=None, checkpoint=None, stream=None):
    """moe_silu_mul of y[a, 2H] (bf16, any row stride) that keeps y in 8 bits: returns (z [a, H], Checkpoint)."""
    if stream is not None:
        return _call_on(moe_silu_mul_checkpoint, locals())
    a, n2 = y.shape
    H = n2 // 2 if H is None else H
    if 2 * H > n2:
        raise ValueError(f"y must hold two halves of {H} columns, got {n2}")
    _need(y, torch.bfloat16, "y", contiguous=False)
    out = _output(out, (a, H), torch.bfloat16, y.device, "out")
    ck = Checkpoint.empty(a, 2 * H, y.device, 2) if checkpoint is None else _checkpoint_arg(checkpoint, a, 2 * H, 2)
    x1 = ctypes.c_void_p(y.data_ptr() + H * y.element_size())
    st = _lib.moe_silu_mul_checkpoint(_ptr(y), x1, y.stride(0) if a > 1 else 2 * H, a, H,
                                      _valid_arg(valid_rows, "valid_rows"), _ptr(out), _ptr(ck.codes),
                                      _ptr(ck.exponents), _stream())
    _check("moe_silu_mul_checkpoint", st)
    return out, ck


def moe_silu_mul_backward(checkpoint: Checkpoint, dz, valid_rows=None, *, out=None, z=None, with_z: bool = True,
                          stream=None):
    """The gradient of silu_mul at a checkpoint's values: returns (dy [a, 2H], z [a, H]), z computed again from
    them for the gradient of w2 (None without with_z)."""
    if stream is not None:
        return _call_on(moe_silu_mul_backward, locals())
    a, H = dz.shape
    _need(dz, torch.bfloat16, "dz")
    ck = _checkpoint_arg(checkpoint, a, 2 * H, 2)
    out = _output(out, (a, 2 * H), torch.bfloat16, dz.device, "out")
    z = _output(z, (a, H), torch.bfloat16, dz.device, "z") if with_z else None
    st = _lib.moe_silu_mul_backward(_ptr(ck.codes), _ptr(ck.exponents), _ptr(dz), a, H,
                                    _valid_arg(valid_rows, "valid_rows"), _ptr(out), _ptr(z), _stream())
    _check("moe_silu_mul_backward", st)
    return out, z


# --------------------------------------------------------------- weight gradient

@functools.lru_cache(maxsize=1024)
def moe_grouped_weight_grad_workspace_size(E: int, a_max: int, N: int, K: int, x_dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_grouped_weight_grad_workspace_size",
           _lib.moe_grouped_weight_grad_workspace_size(E, a_max, N, K, x_dtype, ctypes.byref(n)))
    return n.value


def moe_grouped_weight_grad(dy, x, counts, *, E: int | None = None, out=None, dtype=torch.bfloat16,
                            accumulate: bool = False, workspace=None, stream=None):
    """dw[e] = dy_e^T x_e over the rows of each expert: dy[a, N] bf16, x[a, K] bf16 or a Checkpoint,
    counts[>= E] int32 (E: len(counts), or out's) -> dw[E, N, K] bf16 or fp32.  accumulate adds to an fp32 out."""
    if stream is not None:
        return _call_on(moe_grouped_weight_grad, locals())
    a_max, N = dy.shape
    _need(dy, torch.bfloat16, "dy")
    _need(counts, torch.int32, "counts")
    packed = isinstance(x, Checkpoint)
    if packed:
        if x.halves != 1:
            raise ValueError("x must be a checkpoint of one half")
        x_ptr, exps, code = _ptr(x.codes), _ptr(x.exponents), MOE_DTYPE_E4M3
    else:
        _need(x, torch.bfloat16, "x")
        x_ptr, exps, code = _ptr(x), None, MOE_DTYPE_BF16
    if len(x.shape) != 2 or x.shape[0] != a_max:
        raise ValueError(f"x must hold {a_max} rows, got {tuple(x.shape)}")
    K = x.shape[1]
    if E is None:
        E = counts.shape[0] if out is None else out.shape[0]
    if counts.shape[0] < E:
        raise ValueError(f"counts must hold {E} experts' rows, got {counts.shape[0]}")
    if accumulate and out is None:
        raise ValueError("accumulate adds to a caller-provided out[E, N, K]")
    out = _output(out, (E, N, K), dtype if out is None else out.dtype, dy.device, "out")
    if workspace is not None:
        ws_bytes = _workspace_bytes(workspace)
    elif ws_bytes := moe_grouped_weight_grad_workspace_size(E, a_max, N, K, code):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dy.device)
    st = _lib.moe_grouped_weight_grad(_ptr(dy), x_ptr, exps, _ptr(counts), E, a_max, N, K, _ptr(out),
                                      _dtype_code(out), int(accumulate), _ptr(workspace),
                                      ws_bytes, _stream())
    _check("moe_grouped_weight_grad", st)
    return out


# -------------------------------------------------- gated feed-forward block

def _on_current(*tensors):
    """The kernels run on the current device: tensors of another one are refused (None: not given)."""
    current = _current_device()
    for t in tensors:
        if t is not None and (d := t.get_device()) >= 0 and d != current:
            raise ValueError(f"a tensor on device {d} while device {current} is the current one")


def _gated_weights(w13, w2, counts):
    """Checks w13 [E, 2H, D], w2 [E, D, H] and counts [>= E]; returns E, D, H."""
    if w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("w13 must be [E, 2H, D] and w2 [E, D, H]")
    E, n2, D = w13.shape
    H = n2 // 2
    if n2 % 2 or w2.shape != (E, D, H):
        raise ValueError(f"w13 [E, 2H, D] and w2 [E, D, H] must fit together, got {tuple(w13.shape)} and "
                         f"{tuple(w2.shape)}")
    _need(w13, torch.bfloat16, "w13")
    _need(w2, torch.bfloat16, "w2")
    _need(counts, torch.int32, "counts")
    if counts.dim() != 1 or counts.shape[0] < E:
        raise ValueError(f"counts must hold {E} experts' rows, got {tuple(counts.shape)}")
    return E, D, H


def _gated_rows(t, D: int, name: str) -> int:
    _need(t, torch.bfloat16, name)
    if t.dim() != 2 or t.shape[1] != D:
        raise ValueError(f"{name} must be [rows, {D}], got {tuple(t.shape)}")
    return t.shape[0]


def moe_gated_mlp(x, w13, w2, counts, *, activation: int = MOE_ACT_SILU, keep: bool = True, y=None, z=None, out=None,
                  stream=None):
    """The experts' gated block: z = act(y0) * y1 with y = x w13_e^T, out = z w2_e^T, for x[a, D], w13[E, 2H, D],
    w2[E, D, H] (bf16) and counts[>= E] int32.  Returns (out [a, D], y [a, 2H]), y being what the gradient
    takes (None with keep=False).  Rows past the counts' sum are not written."""
    if stream is not None:
        return _call_on(moe_gated_mlp, locals())
    E, D, H = _gated_weights(w13, w2, counts)
    a, dev = _gated_rows(x, D, "x"), x.device
    y = _output(y, (a, 2 * H), torch.bfloat16, dev, "y") if keep else None
    z = _output(z, (a, H), torch.bfloat16, dev, "z")
    out = _output(out, (a, D), torch.bfloat16, dev, "out")
    _on_current(x, w13, w2, counts, y, z, out)
    st = _lib.moe_gated_mlp(_ptr(x), _ptr(w13), _ptr(w2), _ptr(counts), E, a, D, H, activation, _ptr(y), _ptr(z),
                            _ptr(out), _stream())
    _check("moe_gated_mlp", st)
    return out, y


def moe_gated_mlp_backward(dout, y, w13, w2, counts, *, activation: int = MOE_ACT_SILU, with_z: bool = True, out=None,
                           dy=None, z=None, stream=None):
    """The gradient of moe_gated_mlp's data path for dout[a, D] and the kept y (bf16 [a, 2H], or a Checkpoint in two
    halves): returns (dx [a, D], dy [a, 2H], z [a, H]).  The weights' gradients are moe_grouped_weight_grad(dy, x,
    counts) and moe_grouped_weight_grad(dout, z, counts); z is None without with_z."""
    if stream is not None:
        return _call_on(moe_gated_mlp_backward, locals())
    E, D, H = _gated_weights(w13, w2, counts)
    a, dev = _gated_rows(dout, D, "dout"), dout.device
    if isinstance(y, Checkpoint):
        ck = _checkpoint_arg(y, a, 2 * H, 2)
        y, exponents = ck.codes, ck.exponents
    else:
        _output(y, (a, 2 * H), torch.bfloat16, None, "y")
        exponents = None
    dy = _output(dy, (a, 2 * H), torch.bfloat16, dev, "dy")
    z = _output(z, (a, H), torch.bfloat16, dev, "z") if with_z else None
    out = _output(out, (a, D), torch.bfloat16, dev, "out")
    _on_current(dout, y, exponents, w13, w2, counts, dy, z, out)
    st = _lib.moe_gated_mlp_backward(_ptr(dout), _ptr(y), _ptr(exponents), _ptr(w13), _ptr(w2), _ptr(counts), E, a, D, H,
                                     activation, _ptr(dy), _ptr(z), _ptr(out), _stream())
    _check("moe_gated_mlp_backward", st)
    return out, dy, z


# --------------------------------------------------- orthogonalised updates

MOE_ORTHOGONALIZE_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


@functools.lru_cache(maxsize=1024)
def moe_orthogonalize_workspace_size(B: int, N: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_orthogonalize_workspace_size", _lib.moe_orthogonalize_workspace_size(B, N, K, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=64)
def _coefficients(c: tuple):
    if len(c) != 3:
        raise ValueError(f"coefficients must be three numbers, got {len(c)}")
    return (ctypes.c_float * 3)(*c)


def _matrices(t, name: str):
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [N, K] or [B, N, K], got {tuple(t.shape)}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if max(t.shape) > 0x7fffffff:  # (ctypes would pass the low bits)
        raise ValueError(f"{name} has a size past 31 bits: {tuple(t.shape)}")
    return t.shape if t.dim() == 3 else (1, *t.shape)


def _ortho_workspace(workspace, B: int, N: int, K: int, device):
    if workspace is not None:
        return workspace, _workspace_bytes(workspace)
    n = moe_orthogonalize_workspace_size(B, N, K)
    return torch.empty(n, dtype=torch.uint8, device=device), n


def moe_orthogonalize(g, *, steps: int = 5, coefficients=MOE_ORTHOGONALIZE_COEFFICIENTS, eps: float = 1e-7,
                      scale: float = 1.0, out=None, workspace=None, stream=None):
    """scale times the matrices g [N, K] or [B, N, K] (bf16 or fp32, rows and matrices of any stride) after `steps`
    Newton-Schulz products X = a X + (b A + c A A) X, A = X X^T, from X = g / (|g| + eps); bf16, of g's shape."""
    if stream is not None:
        return _call_on(moe_orthogonalize, locals())
    B, N, K = _matrices(g, "g")
    _need(g, g.dtype, "g", contiguous=False)
    dt = _dtype_code(g)
    out = _output(out, tuple(g.shape), torch.bfloat16, g.device, "out")
    workspace, ws_bytes = _ortho_workspace(workspace, B, N, K, g.device)
    _on_current(g, out, workspace)
    st = _lib.moe_orthogonalize(_ptr(g), dt, g.stride(0) if B > 1 else 0, g.stride(-2) if N > 1 else 0, B, N, K,
                                steps, _coefficients(tuple(map(float, coefficients))), eps, scale, _ptr(out), _ptr(workspace),
                                ws_bytes, _stream())
    _check("moe_orthogonalize", st)
    return out


def moe_muon_update(w, grad, momentum, *, lr: float, mu: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
                    lr_scale=None, steps: int = 5, coefficients=MOE_ORTHOGONALIZE_COEFFICIENTS, eps: float = 1e-7,
                    workspace=None, stream=None):
    """One update, in place, of the weights w [N, K] or [B, N, K] (bf16 or fp32) by their orthogonalised momentum:
    momentum (fp32) = mu * momentum + grad, u = grad + mu * momentum (nesterov) or momentum,
    w = (1 - r * weight_decay) * w - r * orthogonalized(u), r = lr * lr_scale (fp32 [1] on the device, None: 1).
    Returns w."""
    if stream is not None:
        return _call_on(moe_muon_update, locals())
    B, N, K = _matrices(w, "w")
    _need(w, w.dtype, "w")
    _output(grad, w.shape, grad.dtype, None, "grad")
    _output(momentum, w.shape, torch.float32, None, "momentum")
    wt, gt = _dtype_code(w), _dtype_code(grad)
    workspace, ws_bytes = _ortho_workspace(workspace, B, N, K, w.device)
    _on_current(w, grad, momentum, lr_scale, workspace)
    st = _lib.moe_muon_update(_ptr(w), wt, _ptr(grad), gt, _ptr(momentum), B, N, K, mu, int(nesterov), lr,
                              _valid_arg(lr_scale, "lr_scale", torch.float32), weight_decay, steps,
                              _coefficients(tuple(map(float, coefficients))), eps, _ptr(workspace), ws_bytes, _stream())
    _check("moe_muon_update", st)
    return w


def moe_selftest_bounded_wait(which: int, limit_ns: int = 20_000_000, stream=None) -> int:
    """Run a bounded device wait that never succeeds (0: mbarrier, 1: grid barrier);
    returns the device error bits afterwards (MOE_DEVERR_TIMEOUT expected)."""
    _check("moe_selftest_bounded_wait", _lib.moe_selftest_bounded_wait(which, limit_ns, _stream(stream)))
    return device_error(stream)
