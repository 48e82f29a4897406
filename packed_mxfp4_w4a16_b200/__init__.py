"""Packed-MXFP4 W4A16 top-4 MoE expert FFN for NVIDIA B200 (sm_100a).

Python binding of the C-ABI library ``libmoe_mxfp4.so`` (declared in
``include/moe_mxfp4.h``). The functions below carry the C names and only
marshal arguments: torch tensors give device pointers, the current torch
stream gives the CUDA stream, every step of the computation runs in the
library's kernels. There is no CPU fallback: if the library is missing or the
device is not sm_100, the calls raise.

``MoELayer``, ``DenseFFN`` and ``MoEStack`` bundle the calls with their buffers:
a single MoE layer (route + experts + combine), a dense feed-forward layer
(gated block + down projection, with a low-rank adapter per request), and a
stack of layers (weightless RMSNorm, route, experts, combine with residual add,
per layer; dense layers where the model has them) captured in one CUDA
graph per decode step.
"""
from __future__ import annotations

import ctypes as C
import functools

import torch

from ._lib import MoEError, check, library_path, load

__all__ = [
    "MoEError", "MoELayer", "DenseFFN", "MoEStack", "library_path", "load",
    "moe_create", "moe_destroy", "moe_load_packed", "moe_load_packed_nvfp4", "moe_load_packed_sym8",
    "moe_load_expert_table",
    "moe_workspace_bytes", "moe_set_workspace", "moe_route", "moe_route_ex",
    "moe_forward", "moe_forward_ex", "moe_layer_ex", "moe_get_intermediates", "moe_get_status", "moe_get_status_stream",
    "moe_bytes_per_expert", "moe_set_tuning", "moe_device_check", "moe_debug_dequant",
    "moe_forward_noalloc", "moe_forward_noalloc_status", "moe_stack_create", "moe_stack_destroy", "moe_stack_workspace_bytes",
    "moe_stack_set_workspace", "moe_stack_decode", "moe_stack_get_status",
    "moe_stack_set_spin_limit", "moe_stack_set_trace", "STACK_TRACE_SLOTS",
    "ROUTE_RMSNORM", "ROUTE_SIGMOID", "FWD_KEEP_INTERMEDIATES", "FWD_FORCE_DECODE", "FWD_FORCE_GROUPED",
    "FWD_PHASE_GATEUP", "FWD_PHASE_DOWN", "FWD_FORCE_TCGEN05", "FWD_FORCE_MMA",
    "FUSION_NONE", "FUSION_ROUTER", "FUSION_LAYER", "moe_set_fusion",
    "DEVICE_BAD_EXPERT_ID",
    "moe_gated_ffn", "moe_gated_ffn_backward_workspace_bytes", "moe_gated_ffn_backward",
    "moe_adapter_proj_workspace_bytes", "moe_adapter_proj", "moe_adapter_proj_plan", "moe_dense_status",
    "moe_dense_set_spin_limit",
    "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH", "FFN_RMSNORM", "DEVICE_BAD_ADAPTER_ID",
]

ROUTE_RMSNORM = 0x1
ROUTE_SIGMOID = 0x2
FWD_KEEP_INTERMEDIATES = 0x1
FWD_FORCE_DECODE = 0x2
FWD_FORCE_GROUPED = 0x4
FWD_PHASE_GATEUP = 0x8
FWD_PHASE_DOWN = 0x10
FWD_FORCE_TCGEN05 = 0x20
FWD_FORCE_MMA = 0x40
FUSION_NONE, FUSION_ROUTER, FUSION_LAYER = 0, 1, 2
DEVICE_BAD_EXPERT_ID = 0x1
DEVICE_TIMEOUT = 0x2
DEVICE_BAD_ADAPTER_ID = 0x4
ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2
FFN_RMSNORM = 0x1


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _s(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _need(t, dtype, name, ndim=None):
    if t is None:
        return
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise MoEError(name, -1)
    if ndim is not None and t.dim() != ndim:
        raise MoEError(name, -1)


# ------------------------------------------------------------ C-ABI names

def moe_create(E: int, H: int, I: int, top_k: int) -> int:
    h = C.c_void_p()
    check("moe_create", load().moe_create(E, H, I, top_k, C.byref(h)))
    return h.value


def moe_destroy(h: int) -> None:
    check("moe_destroy", load().moe_destroy(C.c_void_p(h)))


def moe_load_packed(h: int, codes: torch.Tensor, scales: torch.Tensor) -> None:
    _need(codes, torch.uint8, "moe_load_packed")
    _need(scales, torch.uint8, "moe_load_packed")
    check("moe_load_packed", load().moe_load_packed(C.c_void_p(h), _p(codes), _p(scales)))


def moe_load_packed_nvfp4(h: int, codes: torch.Tensor, scales: torch.Tensor,
                          gscales: torch.Tensor) -> None:
    """NVFP4 experts: codes uint8 [E, 3*I*H/2], E4M3 scales uint8
    [E, 3*I*H/16], multipliers float32 [E, 2] (gate/up, down)."""
    _need(codes, torch.uint8, "moe_load_packed_nvfp4")
    _need(scales, torch.uint8, "moe_load_packed_nvfp4")
    _need(gscales, torch.float32, "moe_load_packed_nvfp4")
    check("moe_load_packed_nvfp4",
          load().moe_load_packed_nvfp4(C.c_void_p(h), _p(codes), _p(scales), _p(gscales)))


def moe_load_packed_sym8(h: int, codes: torch.Tensor, scales: torch.Tensor) -> None:
    """sym8 experts: codes int8 [E, 3*I*H] (one byte per weight), scales
    binary16 words [E, 3*I*H/32] (a float16 or int16/uint16 tensor of the bit
    patterns)."""
    _need(codes, torch.int8, "moe_load_packed_sym8")
    if (scales.dtype not in (torch.float16, torch.int16, torch.uint16) or not scales.is_cuda
            or not scales.is_contiguous()):
        raise MoEError("moe_load_packed_sym8", -1)
    check("moe_load_packed_sym8",
          load().moe_load_packed_sym8(C.c_void_p(h), _p(codes), _p(scales)))


def moe_load_expert_table(h: int, codes_ptrs, scales_ptrs) -> None:
    """codes_ptrs / scales_ptrs: sequences of 3*E device addresses (ints)."""
    n = len(codes_ptrs)
    ca = (C.c_void_p * n)(*codes_ptrs)
    sa = (C.c_void_p * n)(*scales_ptrs)
    check("moe_load_expert_table", load().moe_load_expert_table(C.c_void_p(h), ca, sa))


def moe_workspace_bytes(h: int, max_tokens: int) -> int:
    n = C.c_size_t()
    check("moe_workspace_bytes", load().moe_workspace_bytes(C.c_void_p(h), max_tokens, C.byref(n)))
    return n.value


def moe_set_workspace(h: int, ws: torch.Tensor, max_tokens: int) -> None:
    _need(ws, torch.uint8, "moe_set_workspace")
    check("moe_set_workspace",
          load().moe_set_workspace(C.c_void_p(h), _p(ws), ws.numel(), max_tokens))


def moe_route(h, x, router_w, router_bias, topk_ids, topk_w, stream=None) -> None:
    moe_route_ex(h, x, router_w, router_bias, 0, None, None, topk_ids, topk_w, stream)


def moe_route_ex(h, x, router_w, router_bias, flags, x_norm, logits, topk_ids, topk_w,
                 stream=None) -> None:
    _need(x, torch.bfloat16, "moe_route", 2)
    _need(router_w, torch.bfloat16, "moe_route", 2)
    _need(router_bias, torch.float32, "moe_route")
    _need(x_norm, torch.bfloat16, "moe_route")
    _need(logits, torch.float32, "moe_route")
    _need(topk_ids, torch.int32, "moe_route")
    _need(topk_w, torch.float32, "moe_route")
    check("moe_route", load().moe_route_ex(
        C.c_void_p(h), _p(x), x.shape[0], _p(router_w), _p(router_bias), flags, _p(x_norm),
        _p(logits), _p(topk_ids), _p(topk_w), _s(stream)))


def moe_forward(h, x, topk_ids, topk_w, y, stream=None) -> None:
    moe_forward_ex(h, x, topk_ids, topk_w, None, y, 0, stream)


def moe_forward_ex(h, x, topk_ids, topk_w, residual, y, flags, stream=None) -> None:
    _need(x, torch.bfloat16, "moe_forward", 2)
    _need(topk_ids, torch.int32, "moe_forward")
    _need(topk_w, torch.float32, "moe_forward")
    _need(residual, torch.bfloat16, "moe_forward")
    _need(y, torch.bfloat16, "moe_forward")
    check("moe_forward", load().moe_forward_ex(
        C.c_void_p(h), _p(x), x.shape[0], _p(topk_ids), _p(topk_w), _p(residual), _p(y),
        flags, _s(stream)))


def moe_layer_ex(h, x, router_w, router_bias, route_flags, x_norm, logits, topk_ids, topk_w,
                 residual, y, fwd_flags, stream=None) -> None:
    _need(x, torch.bfloat16, "moe_layer_ex", 2)
    _need(router_w, torch.bfloat16, "moe_layer_ex", 2)
    _need(router_bias, torch.float32, "moe_layer_ex")
    _need(x_norm, torch.bfloat16, "moe_layer_ex")
    _need(logits, torch.float32, "moe_layer_ex")
    _need(topk_ids, torch.int32, "moe_layer_ex")
    _need(topk_w, torch.float32, "moe_layer_ex")
    _need(residual, torch.bfloat16, "moe_layer_ex")
    _need(y, torch.bfloat16, "moe_layer_ex")
    check("moe_layer_ex", load().moe_layer_ex(
        C.c_void_p(h), _p(x), x.shape[0], _p(router_w), _p(router_bias), route_flags,
        _p(x_norm), _p(logits), _p(topk_ids), _p(topk_w), _p(residual), _p(y), fwd_flags,
        _s(stream)))


def moe_get_intermediates(h: int):
    """Device addresses (h_ptr, o_ptr) of the intermediates of the last forward
    run with FWD_KEEP_INTERMEDIATES."""
    hp, op = C.c_void_p(), C.c_void_p()
    check("moe_get_intermediates",
          load().moe_get_intermediates(C.c_void_p(h), C.byref(hp), C.byref(op)))
    return hp.value, op.value


def moe_get_status(h: int) -> int:
    v = C.c_uint()
    check("moe_get_status", load().moe_get_status(C.c_void_p(h), C.byref(v)))
    return v.value


def moe_get_status_stream(h: int, stream=None) -> int:
    """Device status of the handle's work on `stream` (torch stream or None:
    the current stream), cleared; waits for that stream only."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    v = C.c_uint()
    check("moe_get_status_stream",
          load().moe_get_status_stream(C.c_void_p(h), C.c_void_p(s.cuda_stream), C.byref(v)))
    return v.value


def moe_bytes_per_expert(h: int) -> int:
    n = C.c_size_t()
    check("moe_bytes_per_expert", load().moe_bytes_per_expert(C.c_void_p(h), C.byref(n)))
    return n.value


def moe_set_tuning(h: int, use_pdl: bool, prefetch_down: bool) -> None:
    check("moe_set_tuning", load().moe_set_tuning(C.c_void_p(h), int(use_pdl), int(prefetch_down)))


def moe_set_fusion(h: int, mode: int) -> None:
    check("moe_set_fusion", load().moe_set_fusion(C.c_void_p(h), int(mode)))


def moe_device_check() -> None:
    check("moe_device_check", load().moe_device_check())


def moe_debug_dequant(codes, scales, n, out, stream=None) -> None:
    _need(codes, torch.uint8, "moe_debug_dequant")
    _need(scales, torch.uint8, "moe_debug_dequant")
    _need(out, torch.float32, "moe_debug_dequant")
    check("moe_debug_dequant", load().moe_debug_dequant(_p(codes), _p(scales), n, _p(out), _s(stream)))


def _noalloc_args_ok(E, H, I, top_k, codes, scales, x, topk_ids, topk_w, residual, y,
                     device=None):
    """Shape, dtype, layout and device checks of moe_forward_noalloc's tensors
    (the C call takes bare pointers and cannot check sizes).  Raises MoEError
    (MOE_ERR_ARG) on a mismatch.  `device`: the device every tensor must be on
    (default: the current CUDA device)."""
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    device = torch.device(device)

    def need(t, dtype, numel, what):
        ok = (t is not None and t.dtype == dtype and t.is_contiguous() and t.numel() == numel
              and t.device == device)
        if not ok:
            raise MoEError(f"moe_forward_noalloc ({what})", -1)

    if x is None or x.dim() != 2 or x.shape[1] != H:
        raise MoEError("moe_forward_noalloc (x shape)", -1)
    T = x.shape[0]
    need(codes, torch.uint8, E * 3 * I * H // 2, "codes")
    need(scales, torch.uint8, E * 3 * I * H // 32, "scales")
    need(x, torch.bfloat16, T * H, "x")
    need(topk_ids, torch.int32, T * top_k, "topk_ids")
    need(topk_w, torch.float32, T * top_k, "topk_w")
    need(y, torch.bfloat16, T * H, "y")
    if residual is not None:
        need(residual, torch.bfloat16, T * H, "residual")
    return T


def moe_forward_noalloc(E, H, I, top_k, codes, scales, x, topk_ids, topk_w, residual, y,
                        stream=None) -> None:
    """Expert FFN + combine for callers that may not allocate device memory:
    no handle, no workspace; scratch lives in a fixed device array inside the
    library (see include/moe_mxfp4.h for its limits and its sharing rules).
    Every tensor is checked against E, H, I, top_k and T = x.shape[0] and must
    be on the current device."""
    T = _noalloc_args_ok(E, H, I, top_k, codes, scales, x, topk_ids, topk_w, residual, y)
    check("moe_forward_noalloc", load().moe_forward_noalloc(
        E, H, I, top_k, _p(codes), _p(scales), _p(x), T, _p(topk_ids), _p(topk_w),
        _p(residual), _p(y), _s(stream)))


def moe_forward_noalloc_status(stream=None) -> int:
    """Status bits of moe_forward_noalloc on the current device since the
    last read (synchronises `stream`), cleared."""
    v = C.c_uint()
    check("moe_forward_noalloc_status", load().moe_forward_noalloc_status(_s(stream), C.byref(v)))
    return v.value


def moe_stack_create(handles, router_ws, router_bs=None) -> int:
    """A decode stack over layer handles (ints); router_ws / router_bs:
    sequences of device tensors (BF16 [E, H]; FP32 [E] or None)."""
    n = len(handles)
    for t in router_ws:
        _need(t, torch.bfloat16, "moe_stack_create", 2)
    ha = (C.c_void_p * n)(*handles)
    wa = (C.c_void_p * n)(*[t.data_ptr() for t in router_ws])
    ba = None
    if router_bs is not None and any(b is not None for b in router_bs):
        for t in router_bs:
            _need(t, torch.float32, "moe_stack_create")
        ba = (C.c_void_p * n)(*[None if b is None else b.data_ptr() for b in router_bs])
    out = C.c_void_p()
    check("moe_stack_create", load().moe_stack_create(ha, n, wa, ba, C.byref(out)))
    return out.value


def moe_stack_destroy(s: int) -> None:
    check("moe_stack_destroy", load().moe_stack_destroy(C.c_void_p(s)))


def moe_stack_workspace_bytes(s: int) -> int:
    n = C.c_size_t()
    check("moe_stack_workspace_bytes", load().moe_stack_workspace_bytes(C.c_void_p(s), C.byref(n)))
    return n.value


def moe_stack_set_workspace(s: int, ws: torch.Tensor) -> None:
    _need(ws, torch.uint8, "moe_stack_set_workspace")
    check("moe_stack_set_workspace", load().moe_stack_set_workspace(C.c_void_p(s), _p(ws), ws.numel()))


def moe_stack_decode(s, r, r_hist=None, xn_hist=None, logits=None, topk_ids=None, topk_w=None,
                     stream=None) -> None:
    _need(r, torch.bfloat16, "moe_stack_decode")
    _need(r_hist, torch.bfloat16, "moe_stack_decode")
    _need(xn_hist, torch.bfloat16, "moe_stack_decode")
    _need(logits, torch.float32, "moe_stack_decode")
    _need(topk_ids, torch.int32, "moe_stack_decode")
    _need(topk_w, torch.float32, "moe_stack_decode")
    check("moe_stack_decode", load().moe_stack_decode(
        C.c_void_p(s), _p(r), _p(r_hist), _p(xn_hist), _p(logits), _p(topk_ids), _p(topk_w),
        _s(stream)))


def moe_stack_get_status(s: int, stream=None) -> int:
    v = C.c_uint()
    check("moe_stack_get_status", load().moe_stack_get_status(C.c_void_p(s), _s(stream), C.byref(v)))
    return v.value


STACK_TRACE_SLOTS = 16


def moe_stack_set_trace(s: int, trace) -> None:
    """trace: device int64 tensor of n_layers * SMs * STACK_TRACE_SLOTS
    elements (phase time stamps of every later decode), or None."""
    if trace is None:
        check("moe_stack_set_trace", load().moe_stack_set_trace(C.c_void_p(s), None, 0))
        return
    _need(trace, torch.int64, "moe_stack_set_trace")
    check("moe_stack_set_trace",
          load().moe_stack_set_trace(C.c_void_p(s), _p(trace), trace.numel() * 8))


def moe_stack_set_spin_limit(s: int, polls: int) -> None:
    check("moe_stack_set_spin_limit", load().moe_stack_set_spin_limit(C.c_void_p(s), int(polls)))


# ------------------------------------------- dense feed-forward layers
# A call at small sizes is a few microseconds on the GPU, so the checks below
# are written to cost little.

_BF16 = torch.bfloat16
_MOST = 2 ** 31 - 1  # larger integers would reach the C calls cut to 32 bits


def _in_range(name, *values):
    if max(values) > _MOST or min(values) < -_MOST:
        raise MoEError(name, -1)


def _is(t, dtype, shape):
    """t is a contiguous tensor of this dtype and shape (the C calls take bare
    pointers and cannot check sizes; they refuse host memory and other
    devices)."""
    return t is not None and t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _other(stream, like):
    """Whether `stream` is given and not the current one of the device of
    `like`.  What a call allocates must then belong to `stream`: the allocator
    hands memory of the current stream out again while that stream's last work
    on it is still to come, and kernels on `stream` would not wait for it."""
    return stream is not None and like.is_cuda and stream != torch.cuda.current_stream(like.device)


def _new(like, shape, stream):
    """A new BF16 output beside `like`, written on `stream`; the current stream
    may read it too (ordered behind the call)."""
    if _other(stream, like):
        current = torch.cuda.current_stream(like.device)
        with torch.cuda.stream(stream):
            t = like.new_empty(shape)
        t.record_stream(current)
        return t
    return torch.empty_like(like) if like.shape == shape else like.new_empty(shape)


def _workspace(ws, need, like, name, stream):
    if ws is None:
        if _other(stream, like):
            with torch.cuda.stream(stream):
                return like.new_empty(need, dtype=torch.uint8)
        return like.new_empty(need, dtype=torch.uint8)
    if ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise MoEError(f"{name} (workspace)", -1)
    return ws


def _raw_stream(stream, like):
    """cudaStream_t of `stream`, or of the current stream of the device of
    `like` (the C calls refuse memory of any but the current device)."""
    if stream is not None:
        return stream.cuda_stream
    if not like.is_cuda:
        return None
    return torch._C._cuda_getCurrentRawStream(like.get_device())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _gated_shapes(x, w_gate, w_up, name):
    try:
        (T, H), (I, K) = x.shape, w_gate.shape
        ok = (H == K and w_up.shape == w_gate.shape and x.dtype is _BF16 and w_gate.dtype is _BF16
              and w_up.dtype is _BF16 and x.is_contiguous() and w_gate.is_contiguous()
              and w_up.is_contiguous() and T <= _MOST and H <= _MOST and I <= _MOST)
    except (AttributeError, ValueError):  # None, or not two dimensions
        ok = False
    if not ok:
        raise MoEError(f"{name} (x [T, H], w_gate and w_up [I, H]: BF16, contiguous)", -1)
    return T, H, I


def moe_gated_ffn(x, w_gate, w_up, act=ACT_SILU, h=None, flags=0, x_norm=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T): x BF16 [T, H], w_gate and w_up BF16
    [I, H]; returns h BF16 [T, I] (a new tensor when h is None). With
    FFN_RMSNORM x is a residual stream and x_norm [T, H] receives the
    normalised input."""
    T, H, I = _gated_shapes(x, w_gate, w_up, "moe_gated_ffn")
    if h is None:
        h = _new(x, (T, I), stream)
    elif not _is(h, _BF16, (T, I)):
        raise MoEError("moe_gated_ffn (h)", -1)
    if x_norm is not None and not _is(x_norm, _BF16, (T, H)):
        raise MoEError("moe_gated_ffn (x_norm)", -1)
    check("moe_gated_ffn", load().moe_gated_ffn(
        x.data_ptr(), T, H, I, w_gate.data_ptr(), w_up.data_ptr(), act, flags, _ptr(x_norm),
        h.data_ptr(), _raw_stream(stream, x)))
    return h


@functools.lru_cache(maxsize=4096)
def moe_gated_ffn_backward_workspace_bytes(T: int, H: int, I: int) -> int:
    n = C.c_size_t()
    _in_range("moe_gated_ffn_backward_workspace_bytes", T, H, I)
    check("moe_gated_ffn_backward_workspace_bytes",
          load().moe_gated_ffn_backward_workspace_bytes(T, H, I, C.byref(n)))
    return n.value


def moe_gated_ffn_backward(x, w_gate, w_up, dh, act=ACT_SILU, dx=None, dw_gate=None, dw_up=None,
                           need_dx=True, need_dw=True, workspace=None, stream=None):
    """Gradients of moe_gated_ffn for dh = dL/dh BF16 [T, I]: returns (dx
    [T, H], dw_gate [I, H], dw_up [I, H]), BF16; None for those not needed.
    Outputs and workspace (uint8) that are not given are new tensors."""
    name = "moe_gated_ffn_backward"
    T, H, I = _gated_shapes(x, w_gate, w_up, name)
    if not _is(dh, _BF16, (T, I)):
        raise MoEError(f"{name} (dh)", -1)
    if (not need_dx and dx is not None) or (not need_dw and (dw_gate is not None or dw_up is not None)):
        raise MoEError(f"{name} (an output that is not needed)", -1)
    if need_dx:
        if dx is None:
            dx = _new(x, (T, H), stream)
        elif not _is(dx, _BF16, (T, H)):
            raise MoEError(f"{name} (dx)", -1)
    if need_dw:
        if dw_gate is None:
            dw_gate = _new(w_gate, (I, H), stream)
        if dw_up is None:
            dw_up = _new(w_up, (I, H), stream)
        if not (_is(dw_gate, _BF16, (I, H)) and _is(dw_up, _BF16, (I, H))):
            raise MoEError(f"{name} (dw_gate or dw_up)", -1)
    workspace = _workspace(workspace, moe_gated_ffn_backward_workspace_bytes(T, H, I), x, name,
                           stream)
    check(name, load().moe_gated_ffn_backward(
        x.data_ptr(), T, H, I, w_gate.data_ptr(), w_up.data_ptr(), act, dh.data_ptr(), _ptr(dx),
        _ptr(dw_gate), _ptr(dw_up), workspace.data_ptr(), workspace.numel(), _raw_stream(stream, x)))
    return dx, dw_gate, dw_up


@functools.lru_cache(maxsize=4096)
def moe_adapter_proj_workspace_bytes(T: int, K: int, N: int, n_adapters: int, rank: int) -> int:
    n = C.c_size_t()
    _in_range("moe_adapter_proj_workspace_bytes", T, K, N, n_adapters, rank)
    check("moe_adapter_proj_workspace_bytes",
          load().moe_adapter_proj_workspace_bytes(T, K, N, n_adapters, rank, C.byref(n)))
    return n.value


def moe_adapter_proj(x, w, lora_a=None, lora_b=None, lora_scale=None, adapter_ids=None,
                     residual=None, y=None, workspace=None, stream=None):
    """y[t] = w x[t] + lora_scale[a] lora_b[a] (lora_a[a] x[t]) (+ residual[t])
    with a = adapter_ids[t] (-1: none): x BF16 [T, K], w BF16 [N, K], lora_a
    BF16 [n, rank, K], lora_b BF16 [n, N, rank], lora_scale FP32 [n],
    adapter_ids int32 [T]. All four adapter arguments None: the plain
    projection. residual may be y. Returns y BF16 [T, N]."""
    name = "moe_adapter_proj"
    try:
        (T, K), (N, L) = x.shape, w.shape
        ok = (K == L and x.dtype is _BF16 and w.dtype is _BF16 and x.is_contiguous()
              and w.is_contiguous() and T <= _MOST and K <= _MOST and N <= _MOST)
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        raise MoEError(f"{name} (x [T, K], w [N, K]: BF16, contiguous)", -1)
    n = rank = need = 0
    pa = pb = ps = pi = pw = None
    if lora_a is not None:
        try:
            n, rank, L = lora_a.shape
            ok = (n > 0 and L == K and lora_b.shape == (n, N, rank) and lora_scale.shape == (n,)
                  and adapter_ids.shape == (T,) and lora_a.dtype is _BF16 and lora_b.dtype is _BF16
                  and lora_scale.dtype is torch.float32 and adapter_ids.dtype is torch.int32
                  and lora_a.is_contiguous() and lora_b.is_contiguous()
                  and lora_scale.is_contiguous() and adapter_ids.is_contiguous())
        except (AttributeError, ValueError):
            ok = False
        if not ok:
            raise MoEError(f"{name} (lora_a [n, rank, K], lora_b [n, N, rank] BF16, lora_scale [n] "
                           "FP32, adapter_ids [T] int32, contiguous)", -1)
        pa, pb, ps, pi = (lora_a.data_ptr(), lora_b.data_ptr(), lora_scale.data_ptr(),
                          adapter_ids.data_ptr())
        workspace = _workspace(workspace, moe_adapter_proj_workspace_bytes(T, K, N, n, rank), x,
                               name, stream)
        need, pw = workspace.numel(), workspace.data_ptr()
    elif lora_b is not None or lora_scale is not None or adapter_ids is not None:
        raise MoEError(f"{name} (adapters)", -1)
    if residual is not None and not _is(residual, _BF16, (T, N)):
        raise MoEError(f"{name} (residual)", -1)
    if y is None:
        y = _new(x if residual is None else residual, (T, N), stream)
    elif not _is(y, _BF16, (T, N)):
        raise MoEError(f"{name} (y)", -1)
    check(name, load().moe_adapter_proj(
        x.data_ptr(), T, K, N, w.data_ptr(), _ptr(residual), n, rank, pa, pb, ps, pi, y.data_ptr(),
        pw, need, _raw_stream(stream, x)))
    return y


def moe_adapter_proj_plan(T, K, N, n_adapters=0, rank=0, num_sms=0, cluster_ctas=None) -> dict:
    """Which kernels a moe_adapter_proj call of these sizes launches, on the
    current device or on one of ``num_sms`` SMs that runs ``cluster_ctas`` =
    (CTAs at once in clusters of 2, of 4, of 8)."""
    _in_range("moe_adapter_proj_plan", T, K, N, n_adapters, rank, num_sms, *(cluster_ctas or ()))
    plan = (C.c_int * 6)()
    ctas = None if cluster_ctas is None else (C.c_int * 3)(*cluster_ctas)
    check("moe_adapter_proj_plan", load().moe_adapter_proj_plan(T, K, N, n_adapters, rank, num_sms, ctas, plan))
    return {"products": ("streamed", "single", "pairs")[plan[0]], "splits": plan[1],
            "inner": ("none", "loads", "named", "every")[plan[2]], "inner_splits": plan[3],
            "direct": bool(plan[4]), "groups": plan[5]}


def moe_dense_status(stream=None) -> int:
    """Status bits of the dense calls on the current device since the last
    read (synchronises `stream`), cleared. The word is one for all streams and
    layers of the GPU: whoever reads first gets the bits."""
    v = C.c_uint()
    check("moe_dense_status", load().moe_dense_status(_s(stream), C.byref(v)))
    return v.value


def moe_dense_set_spin_limit(polls: int) -> None:
    """Polls of each bounded wait of later dense calls (default 2^22)."""
    _in_range("moe_dense_set_spin_limit", polls)
    check("moe_dense_set_spin_limit", load().moe_dense_set_spin_limit(polls))


# ------------------------------------------------------------- bundles

class MoELayer:
    """One MoE layer bound to packed weights already on the device.

    codes uint8 [E, 3*I*H/2] and scales uint8 [E, 3*I*H/32] (layout of
    include/moe_mxfp4.h) are read in place; the layer keeps references to
    them. ``router_w`` BF16 [E, H], ``router_b`` FP32 [E] or None.  With
    ``gscales`` (float32 [E, 2]) the experts are NVFP4: scales are then E4M3
    bytes [E, 3*I*H/16].  With int8 ``codes`` [E, 3*I*H] the experts are
    sym8: scales are then binary16 words [E, 3*I*H/32].
    """

    def __init__(self, E, H, I, top_k, codes, scales, router_w=None, router_b=None,
                 max_tokens=4, workspace=None, gscales=None):
        moe_device_check()
        self.E, self.H, self.I, self.k = E, H, I, top_k
        self.codes, self.scales, self.gscales = codes, scales, gscales
        self.router_w, self.router_b = router_w, router_b
        self.max_tokens = max_tokens
        self.handle = moe_create(E, H, I, top_k)
        try:
            if codes.dtype == torch.int8:
                moe_load_packed_sym8(self.handle, codes, scales)
            elif gscales is None:
                moe_load_packed(self.handle, codes, scales)
            else:
                moe_load_packed_nvfp4(self.handle, codes, scales, gscales)
            need = moe_workspace_bytes(self.handle, max_tokens)
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=codes.device)
            self.workspace = workspace
            moe_set_workspace(self.handle, workspace, max_tokens)
        except Exception:
            moe_destroy(self.handle)
            self.handle = None
            raise

    def close(self):
        if getattr(self, "handle", None):
            moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def route(self, x, ids=None, w=None, logits=None, x_norm=None, rmsnorm=False, sigmoid=False,
              stream=None):
        T = x.shape[0]
        dev = x.device
        ids = ids if ids is not None else torch.empty(T, self.k, dtype=torch.int32, device=dev)
        w = w if w is not None else torch.empty(T, self.k, dtype=torch.float32, device=dev)
        flags = (ROUTE_RMSNORM if rmsnorm else 0) | (ROUTE_SIGMOID if sigmoid else 0)
        if rmsnorm and x_norm is None:
            x_norm = torch.empty_like(x)
        moe_route_ex(self.handle, x, self.router_w, self.router_b, flags,
                     x_norm if rmsnorm else None, logits, ids, w, stream)
        return (ids, w, x_norm) if rmsnorm else (ids, w)

    def forward(self, x, ids, w, y=None, residual=None, flags=0, stream=None):
        y = y if y is not None else torch.empty_like(x)
        moe_forward_ex(self.handle, x, ids, w, residual, y, flags, stream)
        return y

    def __call__(self, x, stream=None):
        ids, w = self.route(x, stream=stream)
        return self.forward(x, ids, w, stream=stream)

    def intermediates(self, T):
        """Views (h [T,k,I], o [T,k,H], BF16) into the workspace of the last
        forward run with FWD_KEEP_INTERMEDIATES."""
        hp, op = moe_get_intermediates(self.handle)
        base = self.workspace.data_ptr()
        hv = self.workspace[hp - base: hp - base + T * self.k * self.I * 2]
        ov = self.workspace[op - base: op - base + T * self.k * self.H * 2]
        return (hv.view(torch.bfloat16).view(T, self.k, self.I),
                ov.view(torch.bfloat16).view(T, self.k, self.H))

    def status(self, stream=None) -> int:
        """Device status bits (cleared).  With a stream: waits for that stream
        only; without: for the whole device."""
        if stream is not None:
            return moe_get_status_stream(self.handle, stream)
        return moe_get_status(self.handle)


class DenseFFN:
    """A dense feed-forward layer bound to BF16 weights already on the device:
    h = act(x w_gate^T) * (x w_up^T), y = h w_down^T (+ the adapter of each
    token's request) (+ residual).  w_gate, w_up [I, H], w_down [H, I];
    ``lora``: None or (lora_a BF16 [n, rank, I], lora_b BF16 [n, H, rank],
    lora_scale FP32 [n]), adapters of the down projection.

    The layer keeps the buffers of up to ``max_tokens`` tokens (h, the
    normalised input, the adapters' workspace), so its calls must be ordered
    on the GPU; captured in a CUDA graph they stay valid as long as the layer.
    Making a layer waits for the current stream."""

    def __init__(self, w_gate, w_up, w_down, act=ACT_SILU, lora=None, max_tokens=4):
        moe_device_check()
        _gated_shapes(w_gate, w_gate, w_up, "DenseFFN")
        self.I, self.H = w_gate.shape
        if not _is(w_down, _BF16, (self.H, self.I)):
            raise MoEError("DenseFFN (w_down)", -1)
        self.w_gate, self.w_up, self.w_down, self.act, self.lora = w_gate, w_up, w_down, act, lora
        self.max_tokens = max_tokens
        self.h = w_gate.new_empty(max_tokens, self.I)
        self.x_norm = w_gate.new_empty(max_tokens, self.H)
        need = 0
        if lora is not None:
            n, rank = lora[0].shape[:2]
            need = max(moe_adapter_proj_workspace_bytes(t, self.I, self.H, n, rank)
                       for t in {max_tokens, min(max_tokens, 8)})
        self.workspace = w_gate.new_empty(need, dtype=torch.uint8)
        # the buffers may be used on any stream, so the current one must be done
        # with what it had in their place (nothing may be asked of it in a capture)
        if w_gate.is_cuda and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(w_gate.device).synchronize()

    def forward(self, x, adapter_ids=None, residual=None, y=None, rmsnorm=False, stream=None):
        """y [T, H] for x [T, H], T <= max_tokens.  rmsnorm: x is a residual
        stream, the layer runs on its RMSNorm.  adapter_ids int32 [T] (-1:
        none); None: no adapters.  A layer without adapters does not look at
        them.  residual may be y."""
        T = x.shape[0]
        if T > self.max_tokens:
            raise MoEError("DenseFFN.forward", -5)
        moe_gated_ffn(x, self.w_gate, self.w_up, self.act, self.h[:T],
                      FFN_RMSNORM if rmsnorm else 0, self.x_norm[:T] if rmsnorm else None, stream)
        if self.lora is None or adapter_ids is None:
            return moe_adapter_proj(self.h[:T], self.w_down, residual=residual, y=y, stream=stream)
        return moe_adapter_proj(self.h[:T], self.w_down, *self.lora, adapter_ids, residual=residual,
                                y=y, workspace=self.workspace, stream=stream)

    def __call__(self, x, adapter_ids=None, stream=None):
        return self.forward(x, adapter_ids, stream=stream)

    def gated_backward(self, x, dh, stream=None):
        """(dx, dw_gate, dw_up) of the gated block for dh = dL/dh [T, I] (any
        T; a workspace of its own per call)."""
        return moe_gated_ffn_backward(x, self.w_gate, self.w_up, dh, self.act, stream=stream)

    def status(self, stream=None) -> int:
        """Status bits of the dense calls on the current device (cleared)."""
        return moe_dense_status(stream)

    def close(self):
        pass


class MoEStack:
    """A stack of MoE layers run as one decode step on a residual stream r:
    per layer xn = RMSNorm(r) (weightless, eps 1e-6), route(xn), experts,
    r = BF16(r + combine).  ``step()`` replays one CUDA graph of all layers.
    Layers share one workspace (they run in order on one stream).
    ``layers_weights``: per layer (codes, scales, router_w, router_b), or
    with a fifth item, the NVFP4 multipliers [E, 2] (see MoELayer); or a
    DenseFFN of the same H and max_tokens >= T: r = BF16(r + FFN(RMSNorm(r))),
    with the adapters that ``adapter_ids`` (int32 [T], -1 at first) names.

    ``persistent``: run all MoE layers as one launch (moe_stack_decode);
    None = when the shape allows it (T = 1, MXFP4 layers, shapes of
    moe_stack_create, dense layers only ahead of the MoE layers), False = one
    layer at a time (moe_layer_ex), True = required."""

    def __init__(self, layers_weights, E, H, I, top_k, T=1, device="cuda", persistent=None):
        moe_device_check()
        self.E, self.H, self.I, self.k, self.T = E, H, I, top_k, T
        self.layers = []
        ws = None
        for lw in layers_weights:
            if isinstance(lw, DenseFFN):
                if lw.H != H or lw.max_tokens < T:
                    raise MoEError("MoEStack (dense layer)", -1)
                self.layers.append(lw)
                continue
            codes, scales, router_w, router_b = lw[:4]
            gscales = lw[4] if len(lw) > 4 else None
            L = MoELayer(E, H, I, top_k, codes, scales, router_w, router_b, max_tokens=T,
                         workspace=ws, gscales=gscales)
            ws = L.workspace
            self.layers.append(L)
        dev = torch.device(device)
        n = len(self.layers)
        self.moe_layers = [L for L in self.layers if isinstance(L, MoELayer)]
        # dense layers ahead of all MoE layers, and whether there are others
        self.lead = next((l for l, L in enumerate(self.layers) if isinstance(L, MoELayer)), n)
        mixed = self.lead + len(self.moe_layers) != n
        self.adapter_ids = torch.full((T,), -1, dtype=torch.int32, device=dev)
        self.r = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)
        self.xn = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)
        self.ids = torch.zeros(n, T, top_k, dtype=torch.int32, device=dev)
        self.w = torch.zeros(n, T, top_k, dtype=torch.float32, device=dev)
        self.graph = None
        self.stream = torch.cuda.Stream(device=dev)
        # one launch for the whole step (moe_stack_*) when the shape allows it
        self.stack = None
        self.stack_ws = None
        if persistent is not False and T == 1 and self.moe_layers and not mixed:
            try:
                self.stack = moe_stack_create([L.handle for L in self.moe_layers],
                                              [L.router_w for L in self.moe_layers],
                                              [L.router_b for L in self.moe_layers])
                self.stack_ws = torch.empty(moe_stack_workspace_bytes(self.stack),
                                            dtype=torch.uint8, device=dev)
                moe_stack_set_workspace(self.stack, self.stack_ws)
            except MoEError:
                if self.stack is not None:
                    moe_stack_destroy(self.stack)
                self.stack = None
                if persistent:
                    raise
        elif persistent:
            raise MoEError("moe_stack_create", -1)

    def set_tuning(self, use_pdl=True, prefetch_down=True):
        for L in self.moe_layers:
            moe_set_tuning(L.handle, use_pdl, prefetch_down)

    def set_fusion(self, mode):
        """Launch structure of every layer (FUSION_NONE / _ROUTER / _LAYER)."""
        for L in self.moe_layers:
            moe_set_fusion(L.handle, mode)

    def enqueue(self, stream=None):
        """Enqueue one decode step (all layers) on `stream`."""
        if self.stack is not None:
            for L in self.layers[:self.lead]:
                self._enqueue_dense(L, stream)
            moe_stack_decode(self.stack, self.r, topk_ids=self.ids[self.lead:],
                             topk_w=self.w[self.lead:], stream=stream)
        else:
            self.enqueue_layers(stream)

    def _enqueue_dense(self, L, stream):
        L.forward(self.r, self.adapter_ids, residual=self.r, y=self.r, rmsnorm=True, stream=stream)

    def enqueue_layers(self, stream=None):
        """The same step as one moe_layer_ex call per MoE layer."""
        for l, L in enumerate(self.layers):
            if isinstance(L, DenseFFN):
                self._enqueue_dense(L, stream)
                continue
            moe_layer_ex(L.handle, self.r, L.router_w, L.router_b, ROUTE_RMSNORM, self.xn, None,
                         self.ids[l], self.w[l], self.r, self.r, 0, stream)

    def status(self, stream=None) -> int:
        """Device status bits of the stack kernel, of every layer handle and,
        with dense layers, of the dense calls (synchronises), cleared."""
        st = 0
        if self.stack is not None:
            st |= moe_stack_get_status(self.stack, stream)
        for L in self.moe_layers:
            st |= L.status()
        if len(self.moe_layers) != len(self.layers):
            st |= moe_dense_status(stream)
        return st

    def capture(self):
        """Capture one decode step into a CUDA graph (warm-up run first)."""
        s = self.stream
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            saved = self.r.clone()
            self.enqueue(s)
            self.r.copy_(saved)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            self.enqueue(s)
        self.graph = g
        return g

    def step(self):
        """One decode step: replay the captured graph (captures on first use)."""
        if self.graph is None:
            self.capture()
        self.graph.replay()

    def decode_host(self, x_host, y_host):
        """Decode the tokens of x_host one step each (T rows per step) from
        host memory: per step, copy its input into the residual stream,
        replay the captured step, copy the residual stream back into y_host.
        Returns after the last copy has landed.  Pinned buffers make the
        copies asynchronous."""
        if self.graph is None:
            self.capture()
        T = self.T
        for i in range(x_host.shape[0] // T):
            self.r.copy_(x_host[i * T:(i + 1) * T], non_blocking=True)
            self.graph.replay()
            y_host[i * T:(i + 1) * T].copy_(self.r, non_blocking=True)
        torch.cuda.current_stream().synchronize()
        return y_host

    def close(self):
        self.graph = None
        if getattr(self, "stack", None) is not None:
            moe_stack_destroy(self.stack)
            self.stack = None
        for L in self.layers:
            L.close()
