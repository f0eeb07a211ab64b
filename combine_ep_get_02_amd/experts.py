"""Thin Python binding of the second part of libep.so (the C ABI in include/ep_experts.h): the
router, the experts' products in E4M3 and the combine of grouped rows.

As in ``ep``, the functions carry the C names and marshal arguments: torch tensors become raw
device pointers, the stream defaults to torch's current stream, and a non-OK status becomes an
``EpError``.  Before that each tensor is checked for what the library cannot see: its device, its
type and that it is contiguous and large enough (``ValueError``).  There is no fallback path.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from combine_ep_get_02_amd import ep
from combine_ep_get_02_amd.ep import _check, _stream

EP_DEV_BAD_LOGIT = 32
EP_LOGITS_F32, EP_LOGITS_BF16 = 0, 1
EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
SCALE_BLOCK = 128

EXPORTED = ("ep_route", "ep_route_backward", "ep_expert_gemm_fp8", "ep_expert_gemm_swiglu_fp8", "ep_combine_grouped",
            "ep_combine_grouped_backward")


class ep_router_t(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("groups_kept", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("weight_scale", ctypes.c_float)]


_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64
_S = ctypes.POINTER(ep.ep_shape_t)
_R = ctypes.POINTER(ep_router_t)
_lib: ctypes.CDLL | None = None


def load() -> ctypes.CDLL:
    """libep.so with the argument types of this part's calls set (as ``ep.load``, no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    lib = ep.load()
    lib.ep_route.argtypes = [_S, _R, _P, _I, _L, _P, _P, _P, _P, _P, _P]
    lib.ep_route_backward.argtypes = [_S, _R, _P, _I, _L, _P, _P, _P, _L, _P, _P]
    lib.ep_expert_gemm_fp8.argtypes = [_I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _P, _P]
    lib.ep_expert_gemm_swiglu_fp8.argtypes = [_I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P]
    lib.ep_combine_grouped.argtypes = [_S, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P]
    lib.ep_combine_grouped_backward.argtypes = [_S] + [_P] * 8 + [_I, _I, _P, _P, _P, _P]
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


_ONE_BYTE = (torch.uint8, torch.float8_e4m3fn)
_BF16, _F32, _I32, _I64 = (torch.bfloat16,), (torch.float32,), (torch.int32,), (torch.int64,)
_MASK = (torch.uint8, torch.bool)
_LOGITS = {torch.float32: EP_LOGITS_F32, torch.bfloat16: EP_LOGITS_BF16}


# what every call asks for: small calls cost the host more than they cost the GPU
_initialized, _current_device, _current_stream = (torch.cuda.is_initialized, torch._C._cuda_getDevice,
                                                  torch._C._cuda_getCurrentRawStream)


def _device() -> int:
    """The current GPU; none before the first use of one, when no tensor can be on it."""
    return _current_device() if _initialized() else -2


def _raw_stream(stream, device) -> int | None:
    # the handle alone: building torch's stream object costs as much as the rest of a small call
    if stream is None and device >= 0:
        return _current_stream(device)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != device:
        raise ValueError(f"stream: on GPU {stream.device_index}, not on the current one")
    return _stream(stream)


def _at(name, t, count, dtypes, device) -> int | None:
    """Address of a tensor of at least `count` elements of one of `dtypes` on `device`, without gaps."""
    if t is None and count <= 0:
        return None
    if t is None or t.get_device() != device or t.dtype not in dtypes or not t.is_contiguous() or t.numel() < count:
        _refuse(name, t, f"{count} contiguous elements of {dtypes}")
    return t.data_ptr()


def _at_or_null(name, t, count, dtypes, device) -> int | None:
    return None if t is None else _at(name, t, count, dtypes, device)


def _refuse(name, t, wanted) -> None:
    got = "None" if t is None else f"{tuple(t.shape)} {t.dtype} strides {t.stride()} on {t.device}"
    raise ValueError(f"{name}: {got}, but {wanted} on the current GPU needed")


def _logit_rows(name, t, tokens, experts, device, dtype=None) -> int:
    """The stride between rows of a [tokens][experts] tensor whose rows may lie apart."""
    if t is None:
        _refuse(name, t, f"[{tokens}][{experts}] of {dtype or 'float32 or bfloat16'}")
    if t.shape == (tokens, experts) and t.is_contiguous() and t.get_device() == device and t.dtype in _LOGITS and \
            (dtype is None or t.dtype == dtype):
        return experts
    rows, columns = t.shape if t.dim() == 2 else (-1, -1)
    apart, along = t.stride() if t.dim() == 2 else (0, 0)
    if t.get_device() != device or t.dtype not in _LOGITS or (dtype is not None and t.dtype != dtype) or \
            rows < tokens or columns < experts or (columns > 1 and along != 1) or (rows > 1 and apart < experts):
        _refuse(name, t, f"[{tokens}][{experts}] of {dtype or 'float32 or bfloat16'}, rows without gaps,")
    return max(apart, experts)


def make_router(score, num_groups=1, groups_kept=1, group_best=1, renormalize=True, weight_scale=1.0) -> ep_router_t:
    return ep_router_t(score, num_groups, groups_kept, group_best, int(bool(renormalize)), weight_scale)


def ep_route(shape, router, logits, bias, token_mask, topk_idx, topk_weights, dev_status=None, stream=None) -> None:
    T, K, E, at = shape.num_tokens, shape.num_topk, shape.num_experts, _device()
    stride = _logit_rows("logits", logits, T, E, at)
    _check(load().ep_route(
        ctypes.byref(shape), ctypes.byref(router), logits.data_ptr(), _LOGITS[logits.dtype], stride,
        _at_or_null("bias", bias, E, _F32, at), _at_or_null("token_mask", token_mask, T, _MASK, at),
        _at("topk_idx", topk_idx, T * K, _I64, at), _at("topk_weights", topk_weights, T * K, _F32, at),
        _at_or_null("dev_status", dev_status, 1, _I32, at), _raw_stream(stream, at)), "ep_route")


def ep_route_backward(shape, router, logits, topk_idx, grad_weights, grad_logits, dev_status=None,
                      stream=None) -> None:
    T, K, E, at = shape.num_tokens, shape.num_topk, shape.num_experts, _device()
    stride = _logit_rows("logits", logits, T, E, at)
    grad_stride = _logit_rows("grad_logits", grad_logits, T, E, at, logits.dtype)
    _check(load().ep_route_backward(
        ctypes.byref(shape), ctypes.byref(router), logits.data_ptr(), _LOGITS[logits.dtype], stride,
        _at("topk_idx", topk_idx, T * K, _I64, at), _at("grad_weights", grad_weights, T * K, _F32, at),
        grad_logits.data_ptr(), grad_stride, _at_or_null("dev_status", dev_status, 1, _I32, at),
        _raw_stream(stream, at)), "ep_route_backward")


def _product_arguments(num_experts, n, weight_rows, k, x, x_scales, w, w_scales, expert_rows, num_rows, at):
    blocks = k // SCALE_BLOCK
    return (num_experts, n, k, _at("x", x, num_rows * k, _ONE_BYTE, at),
            _at("x_scales", x_scales, num_rows * blocks, _F32, at),
            _at("w", w, num_experts * weight_rows * k, _ONE_BYTE, at),
            _at("w_scales", w_scales, num_experts * -(-weight_rows // SCALE_BLOCK) * blocks, _F32, at),
            _at_or_null("expert_rows", expert_rows, num_experts, _I32, at), num_rows)


def ep_expert_gemm_fp8(num_experts, n, k, x, x_scales, w, w_scales, expert_rows, num_rows, out, dev_status=None,
                       stream=None) -> None:
    at = _device()
    _check(load().ep_expert_gemm_fp8(
        *_product_arguments(num_experts, n, n, k, x, x_scales, w, w_scales, expert_rows, num_rows, at),
        _at("out", out, num_rows * n, _BF16, at), _at_or_null("dev_status", dev_status, 1, _I32, at),
        _raw_stream(stream, at)), "ep_expert_gemm_fp8")


def ep_expert_gemm_swiglu_fp8(num_experts, n, k, x, x_scales, w, w_scales, expert_rows, num_rows, out, out_scales,
                              dev_status=None, stream=None) -> None:
    at = _device()
    _check(load().ep_expert_gemm_swiglu_fp8(
        *_product_arguments(num_experts, n, 2 * n, k, x, x_scales, w, w_scales, expert_rows, num_rows, at),
        _at("out", out, num_rows * n, _ONE_BYTE, at),
        _at("out_scales", out_scales, num_rows * (n // SCALE_BLOCK), _F32, at),
        _at_or_null("dev_status", dev_status, 1, _I32, at), _raw_stream(stream, at)), "ep_expert_gemm_swiglu_fp8")


def _combine_arguments(shape, y, topk_idx, topk_weights, send_slot, slot_pos, num_recv_rows, num_grouped_rows, at):
    T, K = shape.num_tokens, shape.num_topk
    return (_at("y", y, num_grouped_rows * shape.hidden if T > 0 else 0, _BF16, at),
            _at("topk_idx", topk_idx, T * K, _I64, at), _at("topk_weights", topk_weights, T * K, _F32, at),
            _at("send_slot", send_slot, T * shape.num_ranks, _I32, at),
            _at("slot_pos", slot_pos, num_recv_rows * K, _I32, at))


def ep_combine_grouped(shape, y, topk_idx, topk_weights, send_slot, slot_pos, num_recv_rows, num_grouped_rows,
                       combined_x, dev_status=None, stream=None) -> None:
    at = _device()
    _check(load().ep_combine_grouped(
        ctypes.byref(shape),
        *_combine_arguments(shape, y, topk_idx, topk_weights, send_slot, slot_pos, num_recv_rows, num_grouped_rows,
                            at), num_recv_rows, num_grouped_rows,
        _at("combined_x", combined_x, shape.num_tokens * shape.hidden, _BF16, at),
        _at_or_null("dev_status", dev_status, 1, _I32, at), _raw_stream(stream, at)), "ep_combine_grouped")


def ep_combine_grouped_backward(shape, grad_combined, y, topk_idx, topk_weights, send_slot, slot_pos, grouped_row,
                                num_grouped, num_recv_rows, num_grouped_rows, grad_y, grad_topk_weights,
                                dev_status=None, stream=None) -> None:
    T, H, at = shape.num_tokens, shape.hidden, _device()
    _check(load().ep_combine_grouped_backward(
        ctypes.byref(shape), _at("grad_combined", grad_combined, T * H, _BF16, at),
        *_combine_arguments(shape, y, topk_idx, topk_weights, send_slot, slot_pos, num_recv_rows, num_grouped_rows,
                            at), _at("grouped_row", grouped_row, num_grouped_rows, _I32, at),
        _at("num_grouped", num_grouped, 1 if num_grouped_rows > 0 else 0, _I32, at), num_recv_rows,
        num_grouped_rows, _at("grad_y", grad_y, num_grouped_rows * H, _BF16, at),
        _at("grad_topk_weights", grad_topk_weights, T * shape.num_topk, _F32, at),
        _at_or_null("dev_status", dev_status, 1, _I32, at), _raw_stream(stream, at)), "ep_combine_grouped_backward")


# ----------------------------------------------------------------------------- an expert layer
@dataclass
class ExpertBuffers:
    """What a layer's pass needs beside ``ep.Buffers``, for `capacity` grouped rows."""
    capacity: int
    inner: int
    topk_idx: torch.Tensor      # [t][k] the router's choice
    topk_weights: torch.Tensor  # [t][k]
    x8: torch.Tensor            # [t][h] E4M3 codes of x
    x_scales: torch.Tensor      # [t][h / 128]
    grouped_x: torch.Tensor     # [cap][h] E4M3 codes, grouped by expert
    grouped_scales: torch.Tensor
    grouped_row: torch.Tensor   # [cap]
    grouped_w: torch.Tensor     # [cap]
    slot_pos: torch.Tensor      # [b.capacity][k]
    num_grouped: torch.Tensor   # [1]
    act: torch.Tensor           # [cap][inner] E4M3 codes of silu(gate) * up
    act_scales: torch.Tensor    # [cap][inner / 128]
    y: torch.Tensor             # [cap][h] expert outputs


def allocate_experts(b: ep.Buffers, inner: int, capacity: int, device="cuda") -> ExpertBuffers:
    """inner: width of the experts' hidden layer; capacity: grouped rows, normally the sum of
    b.recv_per_expert, at most t * k + E * (expert_alignment - 1)."""
    T, H, K = b.shape.num_tokens, b.shape.hidden, b.shape.num_topk
    cap = max(int(capacity), 0)
    i32 = dict(dtype=torch.int32, device=device)
    u8 = dict(dtype=torch.uint8, device=device)
    f32 = dict(dtype=torch.float32, device=device)
    return ExpertBuffers(
        capacity=cap, inner=int(inner), topk_idx=torch.empty((T, K), dtype=torch.int64, device=device),
        topk_weights=torch.empty((T, K), **f32), x8=torch.empty((T, H), **u8),
        x_scales=torch.empty((T, H // SCALE_BLOCK), **f32), grouped_x=torch.empty((cap, H), **u8),
        grouped_scales=torch.empty((cap, H // SCALE_BLOCK), **f32), grouped_row=torch.empty(cap, **i32),
        grouped_w=torch.empty(cap, **f32), slot_pos=torch.empty((b.capacity, K), **i32),
        num_grouped=torch.empty(1, **i32), act=torch.empty((cap, inner), **u8),
        act_scales=torch.empty((cap, inner // SCALE_BLOCK), **f32),
        y=torch.empty((cap, H), dtype=torch.bfloat16, device=device))


def run_route(b: ep.Buffers, e: ExpertBuffers, router, logits, bias=None, token_mask=None, stream=None) -> None:
    ep_route(b.shape, router, logits, bias, token_mask, e.topk_idx, e.topk_weights, b.dev_status, stream)


def run_experts(b: ep.Buffers, e: ExpertBuffers, x, w_in, w_in_scales, w_out, w_out_scales, stream=None) -> None:
    """A layer's pass from e.topk_idx and e.topk_weights on: layout and notify, x quantised and
    dispatched into the grouped layout, both products, and the weighted sum into b.combined_x.
    x [t][h] bf16; w_in [E][2 inner][h] (gate rows, then up rows) and w_out [E][h][inner] E4M3
    codes with their block scales.  b.shape.hidden and inner are multiples of 128."""
    s = b.shape
    H, S, E = s.hidden, s.hidden // SCALE_BLOCK, s.num_experts
    ep.run_layout_notify(b, e.topk_idx, stream=stream)
    ep.ep_quantize_fp8(x, s.num_tokens, H, S, e.x8, e.x_scales, stream)
    ep.ep_dispatch_grouped(s, e.x8, 1, e.x_scales, S, e.topk_idx, e.topk_weights, b.in_rank, b.gbl, b.recv_gbl,
                           b.recv_per_expert, b.workspace, b.capacity, b.recv_w, b.recv_idx, b.src_info, b.send_slot,
                           e.capacity, e.grouped_x, e.grouped_scales, e.grouped_row, e.grouped_w, e.slot_pos,
                           e.num_grouped, b.dev_status, stream)
    ep_expert_gemm_swiglu_fp8(E, e.inner, H, e.grouped_x, e.grouped_scales, w_in, w_in_scales, b.recv_per_expert,
                              e.capacity, e.act, e.act_scales, b.dev_status, stream)
    ep_expert_gemm_fp8(E, H, e.inner, e.act, e.act_scales, w_out, w_out_scales, b.recv_per_expert, e.capacity, e.y,
                       b.dev_status, stream)
    run_combine_grouped(b, e, stream=stream)


def run_combine_grouped(b: ep.Buffers, e: ExpertBuffers, y=None, stream=None) -> None:
    ep_combine_grouped(b.shape, e.y if y is None else y, e.topk_idx, e.topk_weights, b.send_slot, e.slot_pos,
                       b.capacity, e.capacity, b.combined_x, b.dev_status, stream)


def run_combine_grouped_backward(b: ep.Buffers, e: ExpertBuffers, grad_combined, grad_y, grad_topk_weights,
                                 stream=None) -> None:
    ep_combine_grouped_backward(b.shape, grad_combined, e.y, e.topk_idx, e.topk_weights, b.send_slot, e.slot_pos,
                                e.grouped_row, e.num_grouped, b.capacity, e.capacity, grad_y, grad_topk_weights,
                                b.dev_status, stream)
