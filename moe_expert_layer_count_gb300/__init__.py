"""Fused Mixture-of-Experts layer hot path for GB300 (sm_103a).

A thin Python binding over the C ABI of ``include/moe_gb300.h`` (``libmoe_gb300.so``):
the functions below carry the C entry points' names and only marshal arguments
(torch tensors -> device pointers, sizes, the current CUDA stream). Every step of the
layer runs in the library's CUDA kernels; there is no fallback of any kind. If the
library is missing or was not built, importing the binding's functions raises.

The layer (vLLM PRs #20903, #20725, #20392): count_expert_num_tokens ->
ep_scatter with 1x128 FP8 quantisation -> block-scaled FP8 grouped GEMM (w13) ->
SiLU-and-mul requantisation -> grouped GEMM (w2) -> ep_gather with the top-k
weight-and-reduce, under a chunking loop that sizes the workspace per chunk.

Beside it, the operators of one training step of a pre-norm MoE block with 16-bit expert
weights, each with its gradient: moe_layer_norm, moe_router_topk, moe_grouped_matmul, and
moe_clip_grad_norm over the gradients (``train.py`` runs them together under autograd).
"""
from __future__ import annotations

import ctypes
import os
from array import array
from operator import attrgetter
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_OK = 0
MOE_QUANT_NONE, MOE_QUANT_FP8_1X128 = 0, 1
MOE_EPI_BF16, MOE_EPI_F32, MOE_EPI_SILU_MUL_QUANT = 0, 1, 2
MOE_DT_F32, MOE_DT_BF16, MOE_DT_F16 = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
_DTYPES = {torch.float32: MOE_DT_F32, torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}

_lib = None


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        _declare(L)
        _lib = L
    return _lib


_p, _i64, _int, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_f = ctypes.c_float

SIGNATURES = {
    "moe_status_string": ([_int], ctypes.c_char_p),
    "moe_kernel_launch_count": ([], ctypes.c_uint64),
    "moe_device_error": ([_int], _int),
    "moe_rp_cap": ([_i64, _int, _int], _i64),
    "moe_scatter_workspace_size": ([_i64, _int, _int], _sz),
    "moe_workspace_size": ([_i64, _int, _int, _int, _int], _sz),
    "moe_count_expert_tokens": ([_p, _i64, _int, _p, _int, _int, _p, _p, _p], _int),
    "moe_count_expert_tokens_i64": ([_p, _i64, _int, _p, _int, _int, _p, _p, _p], _int),
    "moe_scatter": ([_p, _i64, _int, _p, _p, _int, _p, _int, _int, _p, _int, _p, _int, _int, _p, _p, _p, _p,
                     _i64, _p, _sz, _p], _int),
    "moe_scatter_i64": ([_p, _i64, _int, _p, _p, _int, _p, _int, _int, _p, _int, _p, _int, _int, _p, _p, _p, _p,
                         _i64, _p, _sz, _p], _int),
    "moe_scatter_noalloc": ([_p, _i64, _int, _p, _p, _int, _p, _int, _int, _p, _int, _int, _p, _p, _p, _p, _i64,
                             _p], _int),
    "moe_scatter_noalloc_i64": ([_p, _i64, _int, _p, _p, _int, _p, _int, _int, _p, _int, _int, _p, _p, _p, _p,
                                 _i64, _p], _int),
    "moe_grouped_gemm_fp8": ([_p, _p, _p, _p, _p, _p, _int, _i64, _int, _int, _int, _p, _p, _p], _int),
    "moe_silu_mul_quant": ([_p, _p, _int, _i64, _int, _p, _p, _p], _int),
    "moe_gather_weight_reduce": ([_p, _p, _p, _i64, _int, _int, _int, _p, _p], _int),
    "moe_forward_chunked": ([_p, _p, _p, _p, _p, _p, _p, _p, _int, _int, _i64, _int, _int, _int, _i64, _int,
                             _p, _p, _sz, _p, _p], _int),
    "moe_forward_chunked_i64": ([_p, _p, _p, _p, _p, _p, _p, _p, _int, _int, _i64, _int, _int, _int, _i64, _int,
                                 _p, _p, _sz, _p, _p], _int),
    "moe_host_workspace_size": ([_i64, _int, _int, _int, _int, _i64], _sz),
    "moe_ep_combine": ([_p, _int, _i64, _int, _p, _p], _int),
    "moe_forward_host": ([_p, _p, _p, _p, _p, _p, _p, _p, _int, _int, _i64, _int, _int, _int, _i64, _int,
                          _p, _p, _sz, _p, _p, _p], _int),
    "moe_forward_host_i64": ([_p, _p, _p, _p, _p, _p, _p, _p, _int, _int, _i64, _int, _int, _int, _i64, _int,
                              _p, _p, _sz, _p, _p, _p], _int),
    "moe_host_wait": ([_p], _int),
    "moe_layer_norm": ([_p, _i64, _int, _int, _p, _p, _int, _f, _p, _p, _p, _p], _int),
    "moe_layer_norm_workspace_size": ([_i64, _int], _sz),
    "moe_layer_norm_backward": ([_p, _p, _i64, _int, _int, _p, _int, _p, _p, _p, _p, _p, _p, _sz, _p], _int),
    "moe_router_topk": ([_p, _i64, _int, _int, _int, _int, _p, _int, _f, _p, _p, _p], _int),
    "moe_router_topk_i64": ([_p, _i64, _int, _int, _int, _int, _p, _int, _f, _p, _p, _p], _int),
    "moe_router_topk_backward": ([_p, _i64, _int, _int, _p, _int, _int, _int, _f, _p, _p, _p], _int),
    "moe_router_topk_backward_i64": ([_p, _i64, _int, _int, _p, _int, _int, _int, _f, _p, _p, _p], _int),
    "moe_grouped_matmul": ([_p, _i64, _p, _int, _int, _int, _p, _p, _int, _int, _p, _p], _int),
    "moe_grouped_matmul_dgrad": ([_p, _i64, _p, _int, _int, _int, _p, _p, _int, _int, _p, _p], _int),
    "moe_grouped_matmul_wgrad": ([_p, _p, _i64, _int, _int, _int, _p, _p, _int, _int, _p, _p, _sz, _p], _int),
    "moe_grouped_matmul_wgrad_workspace_size": ([_i64, _int, _int, _int], _sz),
    "moe_grad_norm_workspace_size": ([_p, _int], _sz),
    "moe_grad_norm": ([_p, _p, _p, _int, _p, _p, _sz, _p], _int),
    "moe_clip_grad_norm": ([_p, _p, _p, _int, _f, _p, _p, _p, _sz, _p], _int),
}


def _declare(L):
    for name, (args, res) in SIGNATURES.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    return ctypes.c_void_p(_raw_stream(stream))


# The handle of the current device's current stream without a torch.cuda.Stream object around
# it (2.9 us a call).
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _current_raw is None:
        return torch.cuda.current_stream().cuda_stream
    return _current_raw(torch.cuda.current_device())


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status)


def _dt(t, dtype, name):
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")


def _ids_entry(name: str, topk_ids) -> str:
    """The C entry point for the ids' dtype: `name` for int32, `name`_i64 for int64."""
    if topk_ids.dtype == torch.int32:
        return name
    if topk_ids.dtype == torch.int64:
        return name + "_i64"
    raise TypeError(f"topk_ids: expected torch.int32 or torch.int64, got {topk_ids.dtype}")


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def moe_kernel_launch_count() -> int:
    return int(lib().moe_kernel_launch_count())


def moe_device_error(clear: bool = False) -> int:
    """The library's device error word (0 = fine); synchronises the device."""
    return int(lib().moe_device_error(int(bool(clear))))


def moe_rp_cap(chunk_M: int, topk: int, local_num_experts: int) -> int:
    return int(lib().moe_rp_cap(chunk_M, topk, local_num_experts))


def moe_scatter_workspace_size(M: int, topk: int, local_num_experts: int) -> int:
    return int(lib().moe_scatter_workspace_size(M, topk, local_num_experts))


def moe_workspace_size(chunk_M: int, K: int, N: int, topk: int, local_num_experts: int) -> int:
    return int(lib().moe_workspace_size(chunk_M, K, N, topk, local_num_experts))


# ------------------------------------------------------------------- entry points
def moe_count_expert_tokens(topk_ids, E, local_num_experts, expert_map=None, expert_num_tokens=None,
                            err_count=None, stream=None):
    """Tokens per local expert: int32 [local_num_experts]. topk_ids is int32 or int64."""
    fn = _ids_entry("moe_count_expert_tokens", topk_ids)
    _dt(expert_map, torch.int32, "expert_map")
    M, topk = topk_ids.shape
    if expert_num_tokens is None:
        expert_num_tokens = torch.empty(local_num_experts, dtype=torch.int32, device=topk_ids.device)
    _check(fn, getattr(lib(), fn)(
        _ptr(topk_ids), M, topk, _ptr(expert_map), E, local_num_experts, _ptr(expert_num_tokens),
        _ptr(err_count), _stream(stream)))
    return expert_num_tokens


def moe_scatter(hidden_states, topk_ids, topk_weights, E, local_num_experts, expert_num_tokens,
                expert_map=None, apply_router_weight_on_input=False, quant=MOE_QUANT_FP8_1X128,
                rp_cap=None, a_out=None, a_scale=None, expert_offsets=None, src2dst=None,
                workspace=None, count_here=False, err_count=None, stream=None):
    """Permute rows into expert-contiguous, 128-aligned blocks (+ FP8 1x128 quant).
    With count_here, expert_num_tokens is an output (the count step fused into the
    scatter). topk_ids is int32 or int64. Returns (a_out, a_scale, expert_offsets, src2dst)."""
    _dt(hidden_states, torch.bfloat16, "hidden_states")
    fn = _ids_entry("moe_scatter", topk_ids)
    _dt(topk_weights, torch.float32, "topk_weights")
    M, K = hidden_states.shape
    topk = topk_ids.shape[1]
    El = local_num_experts
    dev = hidden_states.device
    cap = moe_rp_cap(M, topk, El) if rp_cap is None else rp_cap
    if a_out is None:
        a_out = torch.empty(cap, K, dtype=torch.uint8 if quant else torch.bfloat16, device=dev)
    if a_scale is None and quant:
        a_scale = torch.empty(cap, K // 128, dtype=torch.float32, device=dev)
    if expert_offsets is None:
        expert_offsets = torch.empty(El + 1, dtype=torch.int32, device=dev)
    if src2dst is None:
        src2dst = torch.empty(M, topk, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(moe_scatter_workspace_size(M, topk, El), dtype=torch.uint8, device=dev)
    _check(fn, getattr(lib(), fn)(
        _ptr(hidden_states), M, K, _ptr(topk_ids), _ptr(topk_weights), topk, _ptr(expert_map), E, El,
        _ptr(expert_num_tokens), int(bool(count_here)), _ptr(err_count), int(bool(apply_router_weight_on_input)),
        quant, _ptr(a_out), _ptr(a_scale), _ptr(expert_offsets), _ptr(src2dst), cap, _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return a_out, a_scale, expert_offsets, src2dst


def moe_scatter_noalloc(hidden_states, topk_ids, topk_weights, E, local_num_experts, expert_num_tokens,
                        a_out, a_scale, expert_offsets, src2dst, expert_map=None,
                        apply_router_weight_on_input=False, quant=MOE_QUANT_FP8_1X128, rp_cap=None, stream=None):
    """moe_scatter for callers that cannot allocate: every output buffer is the caller's,
    and the scratch is a fixed array inside the library (see the C header for its limit
    and for the rule that calls must not overlap on the GPU). topk_ids is int32 or int64.
    Returns the outputs."""
    _dt(hidden_states, torch.bfloat16, "hidden_states")
    fn = _ids_entry("moe_scatter_noalloc", topk_ids)
    M, K = hidden_states.shape
    topk = topk_ids.shape[1]
    cap = a_out.shape[0] if rp_cap is None else rp_cap
    _check(fn, getattr(lib(), fn)(
        _ptr(hidden_states), M, K, _ptr(topk_ids), _ptr(topk_weights), topk, _ptr(expert_map), E,
        local_num_experts, _ptr(expert_num_tokens), int(bool(apply_router_weight_on_input)), quant,
        _ptr(a_out), _ptr(a_scale), _ptr(expert_offsets), _ptr(src2dst), cap, _stream(stream)))
    return a_out, a_scale, expert_offsets, src2dst


def moe_grouped_gemm_fp8(a, a_scale, w, w_scale, expert_offsets, epilogue=MOE_EPI_BF16, out=None,
                         out_scale=None, stream=None, expert_num_tokens=None):
    """Block-scaled FP8 grouped GEMM over the permuted rows (see the C header). With
    expert_num_tokens, 32-row groups of padding rows are neither computed nor written."""
    _dt(a, torch.uint8, "a")
    _dt(w, torch.uint8, "w")
    rp_cap, k_in = a.shape
    El, n_out, _ = w.shape
    dev = a.device
    if out is None:
        if epilogue == MOE_EPI_SILU_MUL_QUANT:
            out = torch.empty(rp_cap, n_out // 2, dtype=torch.uint8, device=dev)
        else:
            out = torch.empty(rp_cap, n_out, device=dev,
                              dtype=torch.float32 if epilogue == MOE_EPI_F32 else torch.bfloat16)
    if out_scale is None and epilogue == MOE_EPI_SILU_MUL_QUANT:
        out_scale = torch.empty(rp_cap, n_out // 256, dtype=torch.float32, device=dev)
    _check("moe_grouped_gemm_fp8", lib().moe_grouped_gemm_fp8(
        _ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(expert_offsets), _ptr(expert_num_tokens), El, rp_cap,
        n_out, k_in,
        epilogue, _ptr(out), _ptr(out_scale), _stream(stream)))
    return (out, out_scale) if epilogue == MOE_EPI_SILU_MUL_QUANT else out


def moe_silu_mul_quant(c1, expert_offsets, h=None, h_scale=None, stream=None):
    """h = silu(gate) * up, requantised 1x128 to FP8. Returns (h, h_scale)."""
    _dt(c1, torch.float32, "c1")
    rp_cap, N2 = c1.shape
    N = N2 // 2
    El = expert_offsets.numel() - 1
    if h is None:
        h = torch.empty(rp_cap, N, dtype=torch.uint8, device=c1.device)
    if h_scale is None:
        h_scale = torch.empty(rp_cap, N // 128, dtype=torch.float32, device=c1.device)
    _check("moe_silu_mul_quant", lib().moe_silu_mul_quant(
        _ptr(c1), _ptr(expert_offsets), El, rp_cap, N, _ptr(h), _ptr(h_scale), _stream(stream)))
    return h, h_scale


def moe_gather_weight_reduce(y, src2dst, topk_weights, apply_router_weight_on_input=False, out=None,
                             stream=None):
    """Unpermute + top-k weight-and-reduce: bf16 [M, K]."""
    _dt(y, torch.bfloat16, "y")
    M, topk = src2dst.shape
    K = y.shape[1]
    if out is None:
        out = torch.empty(M, K, dtype=torch.bfloat16, device=y.device)
    _check("moe_gather_weight_reduce", lib().moe_gather_weight_reduce(
        _ptr(y), _ptr(src2dst), _ptr(topk_weights), M, topk, K, int(bool(apply_router_weight_on_input)),
        _ptr(out), _stream(stream)))
    return out


def moe_forward_chunked(hidden_states, topk_ids, topk_weights, w13, w13_scale, w2, w2_scale, E,
                        expert_map=None, chunk_size=None, apply_router_weight_on_input=False, out=None,
                        workspace=None, err_count=None, stream=None):
    """The whole MoE layer under the chunking loop: bf16 [M, K]. topk_ids is int32 or int64."""
    _dt(hidden_states, torch.bfloat16, "hidden_states")
    fn = _ids_entry("moe_forward_chunked", topk_ids)
    _dt(topk_weights, torch.float32, "topk_weights")
    M, K = hidden_states.shape
    El, N2, _ = w13.shape
    topk = topk_ids.shape[1]
    chunk = M if chunk_size is None else int(chunk_size)
    if out is None:
        out = torch.empty(M, K, dtype=torch.bfloat16, device=hidden_states.device)
    if workspace is None:
        workspace = torch.empty(max(1, moe_workspace_size(max(1, min(chunk, M)), K, N2 // 2, topk, El)),
                                dtype=torch.uint8, device=hidden_states.device)
    _check(fn, getattr(lib(), fn)(
        _ptr(hidden_states), _ptr(topk_ids), _ptr(topk_weights), _ptr(w13), _ptr(w13_scale), _ptr(w2),
        _ptr(w2_scale), _ptr(expert_map), E, El, M, K, N2 // 2, topk, max(1, chunk),
        int(bool(apply_router_weight_on_input)), _ptr(out), _ptr(workspace), workspace.numel(),
        _ptr(err_count), _stream(stream)))
    return out


def _hptr(t: torch.Tensor):
    """Address of a page-locked, contiguous host tensor."""
    if t.is_cuda:
        raise ValueError("expected a host tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if not t.is_pinned():
        raise ValueError("expected a pinned (page-locked) host tensor")
    return ctypes.c_void_p(t.data_ptr())


def _event(done):
    if done is None:
        return None
    if done.cuda_event == 0:  # torch creates the CUDA event lazily, on its first record
        done.record()
    return ctypes.c_void_p(done.cuda_event)


def moe_host_workspace_size(M: int, K: int, N: int, topk: int, local_num_experts: int, chunk_size: int) -> int:
    return int(lib().moe_host_workspace_size(M, K, N, topk, local_num_experts, chunk_size))


def moe_forward_host(hidden_states, topk_ids, topk_weights, w13, w13_scale, w2, w2_scale, E, expert_map=None,
                     chunk_size=None, apply_router_weight_on_input=False, out=None, workspace=None, err_count=None,
                     stream=None, done=None):
    """The layer with the batch in pinned HOST memory (hidden_states, topk_ids,
    topk_weights and out are pinned CPU tensors); asynchronous: `out` holds the result
    once the torch.cuda.Event `done` has completed, or once the stream has passed a later
    moe_host_wait(). topk_ids is int32 or int64."""
    _dt(hidden_states, torch.bfloat16, "hidden_states")
    fn = _ids_entry("moe_forward_host", topk_ids)
    _dt(topk_weights, torch.float32, "topk_weights")
    M, K = hidden_states.shape
    El, N2, _ = w13.shape
    topk = topk_ids.shape[1]
    chunk = M if chunk_size is None else int(chunk_size)
    if out is None:
        out = torch.empty(M, K, dtype=torch.bfloat16).pin_memory()
    if workspace is None:
        workspace = torch.empty(max(1, moe_host_workspace_size(max(1, M), K, N2 // 2, topk, El, max(1, chunk))),
                                dtype=torch.uint8, device=w13.device)
    _check(fn, getattr(lib(), fn)(
        _hptr(hidden_states), _hptr(topk_ids), _hptr(topk_weights), _ptr(w13), _ptr(w13_scale), _ptr(w2),
        _ptr(w2_scale), _ptr(expert_map), E, El, M, K, N2 // 2, topk, max(1, chunk),
        int(bool(apply_router_weight_on_input)), _hptr(out), _ptr(workspace), workspace.numel(),
        _ptr(err_count), _stream(stream), _event(done)))
    return out


def moe_host_wait(stream=None):
    """Orders `stream` after every output copy moe_forward_host has enqueued so far."""
    _check("moe_host_wait", lib().moe_host_wait(_stream(stream)))


def moe_ep_combine(partials, out=None, stream=None):
    """Sum of the ranks' partial layer outputs (bf16 [M, K] CUDA tensors, in rank order):
    fp32 accumulation in ascending rank order, one rounding to bf16."""
    if not partials:
        raise ValueError("moe_ep_combine: no partial outputs")
    for p in partials:
        _dt(p, torch.bfloat16, "partials")
    M, K = partials[0].shape
    if any(tuple(p.shape) != (M, K) for p in partials):
        raise ValueError("moe_ep_combine: partial outputs of different shapes")
    if out is None:
        out = torch.empty(M, K, dtype=torch.bfloat16, device=partials[0].device)
    arr = (ctypes.c_void_p * len(partials))(*[_ptr(p).value for p in partials])
    _check("moe_ep_combine", lib().moe_ep_combine(arr, len(partials), M, K, _ptr(out), _stream(stream)))
    return out


# ------------------------------------------------------ training step of an MoE block
def _dtype_code(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected torch.float32, torch.bfloat16 or torch.float16, got {t.dtype}")
    return code


def _addr(t: Optional[torch.Tensor]):
    """The device address of a contiguous CUDA tensor (None for None)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _same(t, shape, dtype, name):
    """Checks an output buffer or a second operand against the shape and type it has to have."""
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory for a call on `stream` (None: the current one), from that stream's own pool: no
    work of another stream that is still under way has it in use."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def moe_layer_norm(x, weight, bias=None, eps=1e-5, out=None, mean=None, rstd=None, stream=None):
    """Layer norm over the last dimension of x [M, K] (bf16, fp16 or fp32); weight and bias
    [K] in x's type or fp32. Returns (y, mean, rstd), the statistics in fp32 [M]."""
    dt = _dtype_code(x, "x")
    pdt = _dtype_code(weight, "weight")
    M, K = x.shape
    _same(weight, (K,), weight.dtype, "weight")
    _same(bias, (K,), weight.dtype, "bias")
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    if mean is None:
        mean = _empty(M, torch.float32, x.device, stream)
    if rstd is None:
        rstd = _empty(M, torch.float32, x.device, stream)
    _same(out, (M, K), x.dtype, "out")
    _same(mean, (M,), torch.float32, "mean")
    _same(rstd, (M,), torch.float32, "rstd")
    _check("moe_layer_norm", lib().moe_layer_norm(
        _addr(x), M, K, dt, _addr(weight), _addr(bias), pdt, eps, _addr(out), _addr(mean), _addr(rstd), _raw_stream(stream)))
    return out, mean, rstd


def moe_layer_norm_workspace_size(M: int, K: int) -> int:
    return int(lib().moe_layer_norm_workspace_size(M, K))


def moe_layer_norm_backward(dy, x, weight, mean, rstd, dx=None, d_weight=None, d_bias=None, workspace=None,
                            stream=None, has_bias=True):
    """Gradients of moe_layer_norm from its inputs and statistics: (dx, d_weight, d_bias). d_bias is None for
    a norm without a bias (has_bias false)."""
    dt = _dtype_code(x, "x")
    pdt = _dtype_code(weight, "weight")
    M, K = x.shape
    _same(dy, (M, K), x.dtype, "dy")
    _same(weight, (K,), weight.dtype, "weight")
    _same(mean, (M,), torch.float32, "mean")
    _same(rstd, (M,), torch.float32, "rstd")
    if dx is None:
        dx = _empty(x.shape, x.dtype, x.device, stream)
    if d_weight is None:
        d_weight = _empty(weight.shape, weight.dtype, weight.device, stream)
    if not has_bias and d_bias is not None:
        raise ValueError("d_bias: given for a norm without a bias")
    if d_bias is None and has_bias:
        d_bias = _empty(weight.shape, weight.dtype, weight.device, stream)
    _same(dx, (M, K), x.dtype, "dx")
    _same(d_weight, (K,), weight.dtype, "d_weight")
    _same(d_bias, (K,), weight.dtype, "d_bias")
    if workspace is None:
        workspace = _empty(moe_layer_norm_workspace_size(M, K), torch.uint8, x.device, stream)
    _check("moe_layer_norm_backward", lib().moe_layer_norm_backward(
        _addr(dy), _addr(x), M, K, dt, _addr(weight), pdt, _addr(mean), _addr(rstd), _addr(dx), _addr(d_weight),
        _addr(d_bias), _addr(workspace), workspace.numel(), _raw_stream(stream)))
    return dx, d_weight, d_bias


def moe_router_topk(logits, topk, scoring=MOE_SCORE_SOFTMAX, renormalize=True, scale=1.0, bias=None,
                    topk_weights=None, topk_ids=None, stream=None):
    """The topk experts of every token and their weights from logits [M, E] (bf16, fp16 or
    fp32): (topk_weights fp32 [M, topk], topk_ids int32, or int64 if such a buffer is
    given). Ties go to the lowest expert; a slot without an available expert is -1."""
    dt = _dtype_code(logits, "logits")
    M, E = logits.shape
    _same(bias, (E,), torch.float32, "bias")
    if topk_weights is None:
        topk_weights = _empty((M, topk), torch.float32, logits.device, stream)
    if topk_ids is None:
        topk_ids = _empty((M, topk), torch.int32, logits.device, stream)
    fn = _ids_entry("moe_router_topk", topk_ids)
    _same(topk_weights, (M, topk), torch.float32, "topk_weights")
    _same(topk_ids, (M, topk), topk_ids.dtype, "topk_ids")
    _check(fn, getattr(lib(), fn)(
        _addr(logits), M, E, dt, topk, scoring, _addr(bias), int(bool(renormalize)), scale, _addr(topk_weights),
        _addr(topk_ids), _raw_stream(stream)))
    return topk_weights, topk_ids


def moe_router_topk_backward(logits, topk_ids, d_topk_weights, scoring=MOE_SCORE_SOFTMAX, renormalize=True,
                             scale=1.0, d_logits=None, stream=None):
    """Gradient of the router's weights with respect to its logits: [M, E] of their type."""
    dt = _dtype_code(logits, "logits")
    M, E = logits.shape
    fn = _ids_entry("moe_router_topk_backward", topk_ids)
    topk = topk_ids.shape[1]
    _same(topk_ids, (M, topk), topk_ids.dtype, "topk_ids")
    _same(d_topk_weights, (M, topk), torch.float32, "d_topk_weights")
    if d_logits is None:
        d_logits = _empty(logits.shape, logits.dtype, logits.device, stream)
    _same(d_logits, (M, E), logits.dtype, "d_logits")
    _check(fn, getattr(lib(), fn)(
        _addr(logits), M, E, dt, _addr(topk_ids), topk, scoring, int(bool(renormalize)), scale, _addr(d_topk_weights),
        _addr(d_logits), _raw_stream(stream)))
    return d_logits


def moe_grouped_matmul_wgrad_workspace_size(R: int, local_num_experts: int, n_out: int, k_in: int) -> int:
    return int(lib().moe_grouped_matmul_wgrad_workspace_size(R, local_num_experts, n_out, k_in))


def _grouped(fn, a, b, shape, dims, expert_offsets, expert_num_tokens, out, out_dtype, stream, workspace=None):
    """The three grouped products: operands a and b, the result's shape, (El, n_out, k_in)."""
    dt = _dtype_code(a, "rows")
    _same(b, b.shape, a.dtype, "second operand")
    El, N, K = dims
    _same(expert_offsets, (El + 1,), torch.int32, "expert_offsets")
    _same(expert_num_tokens, (El,), torch.int32, "expert_num_tokens")
    if out is None:
        out = _empty(shape, a.dtype if out_dtype is None else out_dtype, a.device, stream)
    _same(out, shape, out.dtype if out_dtype is None else out_dtype, "out")
    odt = _dtype_code(out, "out")
    off, cnt = _addr(expert_offsets), _addr(expert_num_tokens)
    if fn == "moe_grouped_matmul_wgrad":
        if workspace is None:
            need = moe_grouped_matmul_wgrad_workspace_size(a.shape[0], El, N, K)
            if need:
                workspace = _empty(need, torch.uint8, a.device, stream)
        st = lib().moe_grouped_matmul_wgrad(_addr(a), _addr(b), a.shape[0], El, N, K, off, cnt, dt, odt, _addr(out),
                                            _addr(workspace), 0 if workspace is None else workspace.numel(),
                                            _raw_stream(stream))
    else:
        st = getattr(lib(), fn)(_addr(a), a.shape[0], _addr(b), El, N, K, off, cnt, dt, odt, _addr(out), _raw_stream(stream))
    _check(fn, st)
    return out


def moe_grouped_matmul(x, w, expert_offsets, expert_num_tokens=None, out=None, out_dtype=None, stream=None):
    """out[r] = w[l] @ x[r] for the rows r of every group l: x [R, k_in] and w [El, n_out,
    k_in] in bf16 or fp16, out [R, n_out] in their type or fp32. Group l has the rows
    [expert_offsets[l], expert_offsets[l + 1]), or the first expert_num_tokens[l] from
    expert_offsets[l]; rows of no group are not written."""
    El, N, K = w.shape
    R = x.shape[0]
    _same(x, (R, K), w.dtype, "x")
    return _grouped("moe_grouped_matmul", x, w, (R, N), (El, N, K), expert_offsets, expert_num_tokens, out, out_dtype,
                    stream)


def moe_grouped_matmul_dgrad(dy, w, expert_offsets, expert_num_tokens=None, out=None, out_dtype=None, stream=None):
    """Gradient of moe_grouped_matmul's rows: w[l].T @ dy[r], [R, k_in]."""
    El, N, K = w.shape
    R = dy.shape[0]
    _same(dy, (R, N), w.dtype, "dy")
    return _grouped("moe_grouped_matmul_dgrad", dy, w, (R, K), (El, N, K), expert_offsets, expert_num_tokens, out,
                    out_dtype, stream)


def moe_grouped_matmul_wgrad(dy, x, expert_offsets, expert_num_tokens=None, out=None, out_dtype=None, stream=None,
                             workspace=None):
    """Gradient of moe_grouped_matmul's weights: sum over group l's rows of the outer
    products dy[r] x[r], [El, n_out, k_in]; zeros for a group without rows."""
    El = expert_offsets.shape[0] - 1
    R, N = dy.shape
    K = x.shape[1]
    _same(x, (R, K), dy.dtype, "x")
    return _grouped("moe_grouped_matmul_wgrad", dy, x, (El, N, K), (El, N, K), expert_offsets, expert_num_tokens, out,
                    out_dtype, stream, workspace)


_dtype_of, _is_cuda = attrgetter("dtype"), attrgetter("is_cuda")


def _addresses(tensors) -> array:
    """The device addresses of a list of contiguous CUDA tensors."""
    if not all(map(_is_cuda, tensors)):
        raise ValueError("expected CUDA tensors")
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        raise ValueError("expected contiguous tensors")
    return array("Q", map(torch.Tensor.data_ptr, tensors))


def moe_grad_norm_workspace_size(numels) -> int:
    n = len(numels)
    return int(lib().moe_grad_norm_workspace_size((ctypes.c_int64 * n)(*numels), n))


def moe_grad_norm(tensors, norm=None, workspace=None, stream=None):
    """2-norm of all values of a list of tensors (bf16, fp16, fp32 mixed), as fp32 [1]."""
    return _norm_call("moe_grad_norm", tensors, None, None, norm, workspace, stream)


def moe_clip_grad_norm(tensors, max_norm, out=None, norm=None, workspace=None, stream=None):
    """Scales the tensors by max_norm / norm where their common 2-norm exceeds max_norm, in
    place or into the tensors `out`; with an infinite or NaN norm they keep their values.
    Returns the norm before clipping, fp32 [1]."""
    return _norm_call("moe_clip_grad_norm", tensors, float(max_norm), out, norm, workspace, stream)


def _norm_call(fn, tensors, max_norm, out, norm, workspace, stream):
    tensors = list(tensors)
    n = len(tensors)
    if n == 0 and norm is None:
        raise ValueError(f"{fn}: no tensors, and no norm buffer to say where the norm goes")
    dtypes = list(map(_dtype_of, tensors))
    try:
        types = array("i", map(_DTYPES.__getitem__, dtypes))
    except KeyError as e:
        raise TypeError(f"{fn}: expected torch.float32, torch.bfloat16 or torch.float16, got {e.args[0]}") from None
    lens = array("q", map(torch.Tensor.numel, tensors))
    ptrs = _addresses(tensors)
    dev = tensors[0].device if n else norm.device
    if norm is None:
        norm = _empty(1, torch.float32, dev, stream)
    _same(norm, (1,), torch.float32, "norm")
    lens_at = lens.buffer_info()[0]
    if workspace is None:
        workspace = _empty(int(lib().moe_grad_norm_workspace_size(lens_at, n)), torch.uint8, dev, stream)
    ptrs_at, types_at = ptrs.buffer_info()[0], types.buffer_info()[0]
    if max_norm is None:
        st = lib().moe_grad_norm(ptrs_at, lens_at, types_at, n, _addr(norm), _addr(workspace), workspace.numel(),
                                 _raw_stream(stream))
    else:
        outs = None
        if out is not None:
            out = list(out)
            if array("q", map(torch.Tensor.numel, out)) != lens or list(map(_dtype_of, out)) != dtypes:
                raise ValueError(f"{fn}: outputs of other lengths or types than the tensors")
            outs = _addresses(out)
        st = lib().moe_clip_grad_norm(ptrs_at, lens_at, types_at, n, max_norm, outs.buffer_info()[0] if outs else None,
                                      _addr(norm), _addr(workspace), workspace.numel(), _raw_stream(stream))
    _check(fn, st)
    return norm
