"""MI355X (gfx950) MoE routing layout, dispatch copy and combine, and the
operators of the expert layer around them (norm, activation, the experts'
products with 4-bit, 8-bit and bf16 weights).

A thin ctypes binding of the C ABI declared in ``include/ep.h``,
``include/ep_layer.h`` and ``include/ep_expert.h`` and built into ``libep.so`` next to this file (``python -m combine_ep_layout_08_amd.build``).
Every step of the computation runs in the library's HIP kernels; this module
only marshals arguments.  PyTorch supplies device memory and the current
stream.  There is no fallback: without the built library, every entry point
raises.

Low-level functions carry the C names (``ep_layout``, ``ep_dispatch``, ...)
and take raw pointers.  :class:`Handle` wraps them for torch tensors.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch  # noqa: F401  (loaded first so libep.so binds torch's HIP runtime)

__all__ = [
    "EP_OK", "EP_ERR_NULL", "EP_ERR_SHAPE", "EP_ERR_DTYPE", "EP_ERR_UNSUPPORTED",
    "EP_ERR_MISALIGNED", "EP_ERR_WORKSPACE", "EP_ERR_NOT_LAID_OUT", "EP_ERR_CAPACITY",
    "EP_ERR_INVALID_ID", "EP_ERR_HIP", "EP_ERR_TIMEOUT", "EP_BF16", "EP_FP8_E4M3", "EP_F32", "EP_I32",
    "EP_I64", "EpError", "ep_handle", "lib", "Handle", "BoundCall", "ep_capacity_bound",
    "ep_workspace_bytes", "ep_handle_init", "ep_layout", "ep_layout_noalloc", "ep_layout_dispatch",
    "ep_handle_read_counts",
    "ep_handle_import", "ep_dispatch", "ep_combine", "ep_status_str", "ep_handle_sizeof",
    "ep_time_next_call", "time_next_call", "ep_combine_backward", "ep_dispatch_backward",
    "ep_dispatch_rank", "ep_dispatch_rank_quant", "ep_combine_rank", "ep_tma_aligned_rows",
    "ep_sf_packs",
    "ep_quantize_fp8", "ep_dispatch_quant", "EP_SF_F32", "EP_SF_UE8M0", "quantize_fp8",
    "EP_W4_INT4", "EP_W4_MXFP4", "W4Weights", "ep_add_rmsnorm", "ep_add_rmsnorm_backward",
    "ep_add_rmsnorm_backward_workspace", "ep_w4_code_bytes", "ep_w4_scale_bytes", "ep_w4_pack",
    "ep_expert_w4", "ep_swiglu", "ep_swiglu_backward", "add_rmsnorm", "bind_add_rmsnorm",
    "add_rmsnorm_backward", "pack_w4",
    "ep_quantize_i8", "ep_quantize_i8_rows", "ep_expert_i8", "ep_expert_ffn",
    "ep_expert_ffn_backward", "ep_expert_ffn_backward_workspace", "quantize_i8",
    "bind_quantize_i8", "bind_expert_i8", "bind_expert_ffn",
]

LIB_PATH = os.environ.get("EP_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libep.so")

(EP_OK, EP_ERR_NULL, EP_ERR_SHAPE, EP_ERR_DTYPE, EP_ERR_UNSUPPORTED, EP_ERR_MISALIGNED,
 EP_ERR_WORKSPACE, EP_ERR_NOT_LAID_OUT, EP_ERR_CAPACITY, EP_ERR_INVALID_ID,
 EP_ERR_HIP, EP_ERR_TIMEOUT) = range(12)
EP_BF16, EP_FP8_E4M3, EP_F32, EP_I32, EP_I64 = range(5)
EP_DISPATCH_ZERO_PADDING, EP_DISPATCH_STREAMING = 1, 2
EP_SF_F32, EP_SF_UE8M0 = 0, 1
EP_W4_INT4, EP_W4_MXFP4 = 0, 1
_SF_FORMATS = {"f32": EP_SF_F32, "ue8m0": EP_SF_UE8M0}
EP_ERRBIT_CAPACITY = 1
EP_ERRBIT_INVALID_ID = 2
EP_ERRBIT_SCAN_TIMEOUT = 4
# Indices into the handle's device scalars (Handle.scalars), as in ep.h.
EP_SCALAR_NUM_RECV_TOKENS, EP_SCALAR_ERROR_BITS, EP_SCALAR_INVALID_COUNT = 0, 1, 2
EP_SCALAR_NUM_EXPANDED = 5


class ep_handle(ctypes.Structure):
    """Mirror of ``struct ep_handle`` (checked against ep_handle_sizeof)."""
    _fields_ = [
        ("max_tokens", ctypes.c_int32),
        ("num_tokens", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("expert_alignment", ctypes.c_int32),
        ("laid_out", ctypes.c_int32),
        ("capacity", ctypes.c_int64),
        ("counts", ctypes.c_void_p),
        ("psum", ctypes.c_void_p),
        ("dst_slot", ctypes.c_void_p),
        ("src_meta", ctypes.c_void_p),
        ("scalars", ctypes.c_void_p),
        ("tile_status", ctypes.c_void_p),
        ("topk_idx", ctypes.c_void_p),
        ("topk_idx_dtype", ctypes.c_int32),
        ("status_tiles", ctypes.c_int32),
        ("recv_row", ctypes.c_void_p),
        ("recv_src", ctypes.c_void_p),
    ]


class EpError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {ep_status_str(status)}" if what else ep_status_str(status))


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_HP = ctypes.POINTER(ep_handle)

_SIGNATURES = {
    "ep_handle_sizeof": (ctypes.c_size_t, []),
    "ep_capacity_bound": (_I64, [_I32, _I32, _I32, _I32]),
    "ep_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32, _I32, _I64]),
    "ep_handle_init": (ctypes.c_int, [_HP, _I32, _I32, _I32, _I32, _I64, _P, ctypes.c_size_t, _P]),
    "ep_layout": (ctypes.c_int, [_HP, _P, ctypes.c_int, _I32, _P, _P]),
    "ep_layout_noalloc": (ctypes.c_int, [_HP, _P, ctypes.c_int, _I32, _P, _P]),
    "ep_handle_read_counts": (ctypes.c_int, [_HP, _P, _P, _P, _P, _P, _P, _P]),
    "ep_handle_import": (ctypes.c_int, [_HP, _P, ctypes.c_int, _I32, _P, _P, _P, _P, _I32, _P]),
    "ep_dispatch": (ctypes.c_int, [_HP, _P, ctypes.c_int, _I32, _P, _I64, _I64, _I32, _P, _P,
                                   _P, _I64, _I64, _P, _I32, _P]),
    "ep_layout_dispatch": (ctypes.c_int, [_HP, _P, ctypes.c_int, _I32, _P,
                                          _P, ctypes.c_int, _I32, _P, _I64, _I64, _I32, _P, _P,
                                          _P, _I64, _I64, _P, _I32, _P]),
    "ep_tma_aligned_rows": (_I64, [_I64]),
    "ep_sf_packs": (_I32, [_I32, ctypes.c_int]),
    "ep_quantize_fp8": (ctypes.c_int, [_P, _I32, _I32, ctypes.c_int, _P, _P, _I64, _I64, _P]),
    "ep_dispatch_quant": (ctypes.c_int, [_HP, _P, _I32, ctypes.c_int, _P, _P, _P, _I64, _I64,
                                         _P, _I32, _P]),
    "ep_combine": (ctypes.c_int, [_HP, _P, ctypes.c_int, _I32, _P, _P, _P, _P, _P, _P]),
    "ep_dispatch_rank": (ctypes.c_int, [_HP, _P, ctypes.c_int, _I32, _P, _I64, _I64, _I32, _P,
                                        _P, _P, _I64, _I64, _P, _P, _P]),
    "ep_dispatch_rank_quant": (ctypes.c_int, [_HP, _P, _I32, ctypes.c_int, _P, _P, _P, _I64,
                                              _I64, _P, _P, _P]),
    "ep_combine_rank": (ctypes.c_int, [_HP, _P, _I32, _P, _P, _P, _P]),
    "ep_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "ep_time_next_call": (ctypes.c_int, [_P, _P]),
    "ep_combine_backward": (ctypes.c_int, [_HP, _P, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "ep_dispatch_backward": (ctypes.c_int, [_HP, _P, _I32, _P, _P, _P, _P]),
    # ep_layer.h
    "ep_add_rmsnorm": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, ctypes.c_float, _I32, _I32, _P, _P,
                                      ctypes.c_int, _P, _P, _I64, _I64, _P, _P]),
    "ep_add_rmsnorm_backward_workspace": (ctypes.c_size_t, [_I32, _I32]),
    "ep_add_rmsnorm_backward": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, _P, _P, _I32, _I32, _P,
                                               _P, _P, ctypes.c_size_t, _P]),
    "ep_w4_code_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "ep_w4_scale_bytes": (ctypes.c_size_t, [_I32, _I32, _I32, ctypes.c_int, _I32]),
    "ep_w4_pack": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, ctypes.c_int, _I32, _P, _P, _P]),
    "ep_expert_w4": (ctypes.c_int, [_HP, _P, ctypes.c_int, _I32, _I32, _P, ctypes.c_int, _I64,
                                    _I64, _P, _P, ctypes.c_int, _I32, _I32, _P, _P]),
    "ep_swiglu": (ctypes.c_int, [_HP, _P, _I32, _P, ctypes.c_int, _P, ctypes.c_int, _P, _I64, _I64,
                                 _P, ctypes.c_int, _P, _I64, _I64, _P]),
    "ep_swiglu_backward": (ctypes.c_int, [_HP, _P, _I32, _P, _P, ctypes.c_int, ctypes.c_int, _P,
                                          _I64, _I64, _P, _P, _P, _P]),
    # ep_expert.h
    "ep_quantize_i8": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P]),
    "ep_quantize_i8_rows": (ctypes.c_int, [_HP, _P, _I32, _P, _P, _P]),
    "ep_expert_i8": (ctypes.c_int, [_HP, _P, _P, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _P]),
    "ep_expert_ffn": (ctypes.c_int, [_HP, _P, _I32, _I32, _P, _P, _I32, _P, _P, _P, _P, _P]),
    "ep_expert_ffn_backward_workspace": (ctypes.c_size_t, [_HP, _I32]),
    "ep_expert_ffn_backward": (ctypes.c_int, [_HP, _P, _P, _I32, _I32, _P, _P, _I32, _P, _P, _P,
                                              _I32, _P, _P, ctypes.c_int, _P, _P, _P, _P,
                                              ctypes.c_size_t, _P]),
}

_lib = None


def lib():
    """The loaded ``libep.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m combine_ep_layout_08_amd.build` (there is no fallback path)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        if handle.ep_handle_sizeof() != ctypes.sizeof(ep_handle):
            raise RuntimeError("ep_handle layout mismatch between libep.so and the binding")
        _lib = handle
    return _lib


# ---------------------------------------------------------------- C-named calls

def ep_handle_sizeof() -> int:
    return int(lib().ep_handle_sizeof())


def ep_capacity_bound(num_tokens: int, num_topk: int, num_experts: int,
                      expert_alignment: int) -> int:
    return int(lib().ep_capacity_bound(num_tokens, num_topk, num_experts, expert_alignment))


def ep_workspace_bytes(max_tokens: int, num_topk: int, num_experts: int,
                       expert_alignment: int, capacity: int) -> int:
    return int(lib().ep_workspace_bytes(max_tokens, num_topk, num_experts,
                                        expert_alignment, capacity))


def ep_handle_init(h: ep_handle, max_tokens, num_topk, num_experts, expert_alignment,
                   capacity, workspace_ptr, ws_bytes, stream) -> int:
    return lib().ep_handle_init(ctypes.byref(h), max_tokens, num_topk, num_experts,
                                expert_alignment, capacity, workspace_ptr, ws_bytes, stream)


def ep_layout(h: ep_handle, topk_idx_ptr, idx_dtype, num_tokens, stats_ptr, stream) -> int:
    return lib().ep_layout(ctypes.byref(h), topk_idx_ptr, idx_dtype, num_tokens, stats_ptr,
                           stream)


def ep_layout_noalloc(h: ep_handle, topk_idx_ptr, idx_dtype, num_tokens, stats_ptr,
                      stream) -> int:
    return lib().ep_layout_noalloc(ctypes.byref(h), topk_idx_ptr, idx_dtype, num_tokens,
                                   stats_ptr, stream)


def ep_handle_read_counts(h: ep_handle, counts_ptr, psum_ptr, num_expanded_ptr,
                          num_recv_ptr, error_bits_ptr, invalid_ptr, stream) -> int:
    return lib().ep_handle_read_counts(ctypes.byref(h), counts_ptr, psum_ptr,
                                       num_expanded_ptr, num_recv_ptr, error_bits_ptr,
                                       invalid_ptr, stream)


def ep_handle_import(h: ep_handle, topk_idx_ptr, idx_dtype, num_tokens, counts_ptr, psum_ptr,
                     dst_ptr, src_meta_ptr, num_recv_tokens, stream) -> int:
    return lib().ep_handle_import(ctypes.byref(h), topk_idx_ptr, idx_dtype, num_tokens,
                                  counts_ptr, psum_ptr, dst_ptr, src_meta_ptr,
                                  num_recv_tokens, stream)


def ep_dispatch(h: ep_handle, x_ptr, x_dtype, hidden, sf_ptr, sf_ts, sf_hs, num_sf_packs,
                w_ptr, out_x_ptr, out_sf_ptr, out_ts, out_hs, out_w_ptr, flags,
                stream) -> int:
    return lib().ep_dispatch(ctypes.byref(h), x_ptr, x_dtype, hidden, sf_ptr, sf_ts, sf_hs,
                             num_sf_packs, w_ptr, out_x_ptr, out_sf_ptr, out_ts, out_hs,
                             out_w_ptr, flags, stream)


def ep_tma_aligned_rows(rows: int) -> int:
    return int(lib().ep_tma_aligned_rows(rows))


def ep_sf_packs(hidden: int, fmt: int) -> int:
    return int(lib().ep_sf_packs(hidden, fmt))


def ep_quantize_fp8(x_ptr, num_tokens, hidden, fmt, out_q_ptr, out_sf_ptr, out_ts, out_hs,
                    stream) -> int:
    return lib().ep_quantize_fp8(x_ptr, num_tokens, hidden, fmt, out_q_ptr, out_sf_ptr, out_ts,
                                 out_hs, stream)


def ep_dispatch_quant(h: ep_handle, x_ptr, hidden, fmt, w_ptr, out_x_ptr, out_sf_ptr, out_ts,
                      out_hs, out_w_ptr, zero_padding, stream) -> int:
    return lib().ep_dispatch_quant(ctypes.byref(h), x_ptr, hidden, fmt, w_ptr, out_x_ptr,
                                   out_sf_ptr, out_ts, out_hs, out_w_ptr, zero_padding, stream)


def ep_combine(h: ep_handle, y_ptr, y_dtype, hidden, w_ptr, bias_ptr, bias0_ptr, bias1_ptr,
               out_ptr, stream) -> int:
    return lib().ep_combine(ctypes.byref(h), y_ptr, y_dtype, hidden, w_ptr, bias_ptr, bias0_ptr,
                            bias1_ptr, out_ptr, stream)


def ep_dispatch_rank(h: ep_handle, x_ptr, x_dtype, hidden, sf_ptr, sf_ts, sf_hs,
                     num_sf_packs, w_ptr, out_x_ptr, out_sf_ptr, out_ts, out_hs, out_idx_ptr,
                     out_w_ptr, stream) -> int:
    return lib().ep_dispatch_rank(ctypes.byref(h), x_ptr, x_dtype, hidden, sf_ptr, sf_ts, sf_hs,
                                  num_sf_packs, w_ptr, out_x_ptr, out_sf_ptr, out_ts, out_hs,
                                  out_idx_ptr, out_w_ptr, stream)


def ep_dispatch_rank_quant(h: ep_handle, x_ptr, hidden, fmt, w_ptr, out_x_ptr, out_sf_ptr,
                           out_ts, out_hs, out_idx_ptr, out_w_ptr, stream) -> int:
    return lib().ep_dispatch_rank_quant(ctypes.byref(h), x_ptr, hidden, fmt, w_ptr, out_x_ptr,
                                        out_sf_ptr, out_ts, out_hs, out_idx_ptr, out_w_ptr,
                                        stream)


def ep_combine_rank(h: ep_handle, x_ptr, hidden, bias0_ptr, bias1_ptr, out_ptr, stream) -> int:
    return lib().ep_combine_rank(ctypes.byref(h), x_ptr, hidden, bias0_ptr, bias1_ptr, out_ptr,
                                 stream)


def ep_combine_backward(h: ep_handle, grad_out_ptr, hidden, w_ptr, y_ptr, bias_ptr, grad_y_ptr,
                        grad_w_ptr, grad_bias_ptr, stream) -> int:
    return lib().ep_combine_backward(ctypes.byref(h), grad_out_ptr, hidden, w_ptr, y_ptr,
                                     bias_ptr, grad_y_ptr, grad_w_ptr, grad_bias_ptr, stream)


def ep_dispatch_backward(h: ep_handle, grad_out_x_ptr, hidden, grad_out_w_ptr, grad_x_ptr,
                         grad_w_ptr, stream) -> int:
    return lib().ep_dispatch_backward(ctypes.byref(h), grad_out_x_ptr, hidden, grad_out_w_ptr,
                                      grad_x_ptr, grad_w_ptr, stream)


def ep_add_rmsnorm(x_ptr, residual_ptr, weight_ptr, weight_dtype, eps, num_tokens, hidden,
                   out_z_ptr, out_y_ptr, fmt, out_q_ptr, out_sf_ptr, out_ts, out_hs, out_rstd_ptr,
                   stream) -> int:
    return lib().ep_add_rmsnorm(x_ptr, residual_ptr, weight_ptr, weight_dtype, eps, num_tokens,
                                hidden, out_z_ptr, out_y_ptr, fmt, out_q_ptr, out_sf_ptr, out_ts,
                                out_hs, out_rstd_ptr, stream)


def ep_add_rmsnorm_backward_workspace(num_tokens: int, hidden: int) -> int:
    return int(lib().ep_add_rmsnorm_backward_workspace(num_tokens, hidden))


def ep_add_rmsnorm_backward(grad_y_ptr, z_ptr, weight_ptr, weight_dtype, rstd_ptr, grad_z_ptr,
                            num_tokens, hidden, grad_x_ptr, grad_weight_ptr, workspace_ptr,
                            ws_bytes, stream) -> int:
    return lib().ep_add_rmsnorm_backward(grad_y_ptr, z_ptr, weight_ptr, weight_dtype, rstd_ptr,
                                         grad_z_ptr, num_tokens, hidden, grad_x_ptr,
                                         grad_weight_ptr, workspace_ptr, ws_bytes, stream)


def ep_w4_code_bytes(num_experts: int, n: int, k: int) -> int:
    return int(lib().ep_w4_code_bytes(num_experts, n, k))


def ep_w4_scale_bytes(num_experts: int, n: int, k: int, fmt: int, group: int) -> int:
    return int(lib().ep_w4_scale_bytes(num_experts, n, k, fmt, group))


def ep_w4_pack(codes_ptr, scales_ptr, num_experts, n, k, fmt, group, out_codes_ptr,
               out_scales_ptr, stream) -> int:
    return lib().ep_w4_pack(codes_ptr, scales_ptr, num_experts, n, k, fmt, group, out_codes_ptr,
                            out_scales_ptr, stream)


def ep_expert_w4(h: ep_handle, x_ptr, x_dtype, token_rows, k, sf_ptr, sf_fmt, sf_ts, sf_hs,
                 codes_ptr, scales_ptr, fmt, group, n, out_ptr, stream) -> int:
    return lib().ep_expert_w4(ctypes.byref(h), x_ptr, x_dtype, token_rows, k, sf_ptr, sf_fmt,
                              sf_ts, sf_hs, codes_ptr, scales_ptr, fmt, group, n, out_ptr, stream)


def ep_swiglu(h: ep_handle, gate_up_ptr, inter, row_weights_ptr, h_dtype, out_h_ptr, fmt,
              out_sf_ptr, out_ts, out_hs, saved_ptr, saved_fmt, saved_sf_ptr, saved_ts, saved_hs,
              stream) -> int:
    return lib().ep_swiglu(ctypes.byref(h), gate_up_ptr, inter, row_weights_ptr, h_dtype,
                           out_h_ptr, fmt, out_sf_ptr, out_ts, out_hs, saved_ptr, saved_fmt,
                           saved_sf_ptr, saved_ts, saved_hs, stream)


def ep_swiglu_backward(h: ep_handle, grad_h_ptr, inter, row_weights_ptr, saved_ptr, saved_dtype,
                       saved_fmt, saved_sf_ptr, saved_ts, saved_hs, grad_gate_up_ptr,
                       grad_row_weights_ptr, out_h_ptr, stream) -> int:
    return lib().ep_swiglu_backward(ctypes.byref(h), grad_h_ptr, inter, row_weights_ptr,
                                    saved_ptr, saved_dtype, saved_fmt, saved_sf_ptr, saved_ts,
                                    saved_hs, grad_gate_up_ptr, grad_row_weights_ptr, out_h_ptr,
                                    stream)


def ep_quantize_i8(x_ptr, num_rows, channels, out_q_ptr, out_scale_ptr, stream) -> int:
    return lib().ep_quantize_i8(x_ptr, num_rows, channels, out_q_ptr, out_scale_ptr, stream)


def ep_quantize_i8_rows(h: ep_handle, x_ptr, channels, out_q_ptr, out_scale_ptr, stream) -> int:
    return lib().ep_quantize_i8_rows(ctypes.byref(h), x_ptr, channels, out_q_ptr, out_scale_ptr,
                                     stream)


def ep_expert_i8(h: ep_handle, x_ptr, x_scale_ptr, token_rows, k, w_ptr, w_scale_ptr, n, gated,
                 row_weights_ptr, out_ptr, stream) -> int:
    return lib().ep_expert_i8(ctypes.byref(h), x_ptr, x_scale_ptr, token_rows, k, w_ptr,
                              w_scale_ptr, n, gated, row_weights_ptr, out_ptr, stream)


def ep_expert_ffn(h: ep_handle, x_ptr, token_rows, hidden, w13_ptr, w2_ptr, inter,
                  row_weights_ptr, out_h_ptr, saved_ptr, out_y_ptr, stream) -> int:
    return lib().ep_expert_ffn(ctypes.byref(h), x_ptr, token_rows, hidden, w13_ptr, w2_ptr, inter,
                               row_weights_ptr, out_h_ptr, saved_ptr, out_y_ptr, stream)


def ep_expert_ffn_backward_workspace(h: ep_handle, inter: int) -> int:
    return int(lib().ep_expert_ffn_backward_workspace(ctypes.byref(h), inter))


def ep_expert_ffn_backward(h: ep_handle, grad_y_ptr, x_ptr, token_rows, hidden, w13_ptr, w2_ptr,
                           inter, row_weights_ptr, saved_ptr, rows_h_ptr, remake_h,
                           grad_gate_up_ptr, grad_x_ptr, grad_dtype, grad_w13_ptr, grad_w2_ptr,
                           grad_row_weights_ptr, workspace_ptr, ws_bytes, stream) -> int:
    return lib().ep_expert_ffn_backward(ctypes.byref(h), grad_y_ptr, x_ptr, token_rows, hidden,
                                        w13_ptr, w2_ptr, inter, row_weights_ptr, saved_ptr,
                                        rows_h_ptr, remake_h, grad_gate_up_ptr, grad_x_ptr,
                                        grad_dtype, grad_w13_ptr, grad_w2_ptr,
                                        grad_row_weights_ptr, workspace_ptr, ws_bytes, stream)


def ep_status_str(status: int) -> str:
    return lib().ep_status_str(status).decode()


def ep_time_next_call(start_event, stop_event) -> int:
    """Attach raw HIP events (handles) to the next layout/dispatch/combine."""
    return lib().ep_time_next_call(start_event, stop_event)


def time_next_call(start: "torch.cuda.Event", stop: "torch.cuda.Event") -> None:
    """Stamp two torch events with the first kernel start and last kernel end
    of the next layout/dispatch/combine call on this thread."""
    for e in (start, stop):
        if e.cuda_event == 0:           # torch creates events lazily on first record
            e.record()
    _check(ep_time_next_call(start.cuda_event, stop.cuda_event), "ep_time_next_call")


# ---------------------------------------------------------------- torch wrapper

def _stream() -> int:
    """Raw handle of the current device's current stream: the value of
    torch.cuda.current_stream().cuda_stream, read without building a Stream
    object (0.3 us instead of 2.8 us per call on MI355X)."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check(status: int, what: str):
    if status != EP_OK:
        raise EpError(status, what)


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dev_strided(t: torch.Tensor, name: str):
    """Scale tensors may have any non-negative strides (the kernels take them)."""
    _need(t.is_cuda, f"{name} must be a device tensor")
    _need(t.dim() == 2 and min(t.stride()) >= 0, f"{name} must be a 2-D strided view")


class BoundCall:
    """One entry point with its arguments validated and marshalled once.

    Calling it enqueues the same call on the current stream (read at every
    call) and returns what the direct method returns.  It keeps the tensors it
    was bound to alive, and the handle whose workspace the call reads: their
    contents may change between calls (new routing, new payloads), their storage
    and shapes may not.  A direct method spends
    about 5-6 us of host time per call on validation and marshalling, a bound
    call about 3 us (the C entry point and the launch), which lets small
    batches run at the GPU's pace.

    Dispatch and combine calls are bound for the handle's token count at bind
    time (their tensors were checked against it) and refuse to run once a
    later layout has changed it, as the direct methods would."""
    __slots__ = ("_fn", "_args", "_what", "_result", "_keep", "_h", "_tokens")

    def __init__(self, fn, args, what, result, keep, h=None):
        # converted once: 0.3 us less per call
        types = getattr(fn, "argtypes", None)
        if types:
            args = tuple(a if a is None or not isinstance(a, (int, float)) else t(a)
                         for a, t in zip(args, types))
        self._fn, self._args, self._what = fn, args, what
        self._result, self._keep = result, keep
        self._h = h
        self._tokens = None if h is None else h.num_tokens

    def __call__(self):
        if self._h is not None and self._h.num_tokens != self._tokens:
            raise ValueError(f"{self._what}: bound for {self._tokens} tokens, but the handle's "
                             f"layout now has {self._h.num_tokens}")
        status = self._fn(*self._args, _stream())
        if status != EP_OK:
            raise EpError(status, self._what)
        return self._result


_SF_DTYPES = (torch.float32, torch.int32)


def _scale_packs(sf, T, H, rows, out_sf, col_major, device):
    """Check FP8 scale packs and allocate their output.  sf: fp32 [T, H/128]
    (one scale per 128 channels) or int32 [T, P] (P packs of four UE8M0
    exponent bytes), any strides.  Returns (packs, sf strides, out_sf, out
    strides); a column-major out_sf has token stride 1 and pack stride
    ep_tma_aligned_rows(rows)."""
    _need(sf is not None, "FP8 dispatch needs scale factors")
    _dev_strided(sf, "sf")
    _need(sf.dtype in _SF_DTYPES and sf.dim() == 2 and sf.shape[0] == T,
          "sf must be fp32 [T, H/128] or int32 packs [T, P]")
    packs = sf.shape[1]
    _need(sf.dtype == torch.int32 or packs == H // 128, "fp32 sf must be [T, H/128]")
    if out_sf is None:
        if col_major:
            store = torch.empty((packs, ep_tma_aligned_rows(rows)), dtype=sf.dtype, device=device)
            out_sf = store[:, :rows].t()
        else:
            out_sf = torch.empty((rows, packs), dtype=sf.dtype, device=device)
    _dev_strided(out_sf, "out_sf")
    _need(out_sf.dtype == sf.dtype and tuple(out_sf.shape) == (rows, packs),
          f"out_sf must be [{rows}, {packs}] of sf's dtype")
    return packs, sf.stride(), out_sf, out_sf.stride()


def _sf_format(scale_format) -> int:
    fmt = _SF_FORMATS.get(scale_format, scale_format)
    _need(fmt in (EP_SF_F32, EP_SF_UE8M0), "scale_format must be 'f32' or 'ue8m0'")
    return fmt


def _quant_sf_out(out_sf, rows, packs, fmt, col_major, device):
    dt = torch.float32 if fmt == EP_SF_F32 else torch.int32
    if out_sf is None:
        if col_major:
            out_sf = torch.empty((packs, ep_tma_aligned_rows(rows)), dtype=dt,
                                 device=device)[:, :rows].t()
        else:
            out_sf = torch.empty((rows, packs), dtype=dt, device=device)
    _dev_strided(out_sf, "out_sf")
    _need(out_sf.dtype == dt and tuple(out_sf.shape) == (rows, packs),
          f"out_sf must be [{rows}, {packs}] {dt}")
    return out_sf


def quantize_fp8(x: torch.Tensor, scale_format="f32", out_q=None, out_sf=None,
                 col_major_sf: bool = False):
    """bf16 [T, H] -> (E4M3FN codes uint8 [T, H], scales): fp32 [T, H/128]
    for 'f32', int32 packs [T, ceil(H/512)] of UE8M0 exponents for 'ue8m0'."""
    _dev(x, "x")
    _need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be bf16 [T, H]")
    T, H = x.shape
    fmt = _sf_format(scale_format)
    packs = ep_sf_packs(H, fmt)
    _need(packs > 0, "hidden must be a positive multiple of 128")
    if out_q is None:
        out_q = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    _dev(out_q, "out_q")
    _need(out_q.dtype in (torch.uint8, torch.float8_e4m3fn) and tuple(out_q.shape) == (T, H),
          "out_q must be FP8 codes [T, H]")
    out_sf = _quant_sf_out(out_sf, T, packs, fmt, col_major_sf, x.device)
    ts, hs = out_sf.stride()
    _check(ep_quantize_fp8(_ptr(x), T, H, fmt, _ptr(out_q), _ptr(out_sf), ts, hs, _stream()),
           "ep_quantize_fp8")
    return out_q, out_sf


def _buffer(t, name, shape, want, device, dtype=torch.bfloat16):
    """``t``, checked, or a new tensor where none is given and one is wanted."""
    if t is None and want:
        return torch.empty(shape, dtype=dtype, device=device)
    if t is not None:
        _rows_of(t, name, shape, dtype)
    return t


def _i8_rows(x, rows, what, out_q, out_scale):
    """Check bf16 rows and the buffers of their int8 codes and scales, or make these."""
    _dev(x, "x")
    _need(x.dtype == torch.bfloat16 and x.dim() == 2 and (rows is None or x.shape[0] == rows),
          f"x must be bf16 [{what}, C]")
    out_q = _buffer(out_q, "out_q", tuple(x.shape), True, x.device, torch.int8)
    out_scale = _buffer(out_scale, "out_scale", (x.shape[0],), True, x.device, torch.float32)
    return out_q, out_scale


def _quantize_i8_call(x, out_q, out_scale):
    out_q, out_scale = _i8_rows(x, None, "T", out_q, out_scale)
    _here(x, out_q, out_scale)
    args = (_ptr(x), x.shape[0], x.shape[1], _ptr(out_q), _ptr(out_scale))
    return lib().ep_quantize_i8, args, (out_q, out_scale), x


def quantize_i8(x: torch.Tensor, out_q=None, out_scale=None):
    """bf16 [T, C] -> (int8 codes [T, C], fp32 scales [T]): scale = max |row| / 127, codes
    rounded to nearest even.  A row with a NaN or an infinity gets scale NaN and codes 0."""
    fn, args, result, _ = _quantize_i8_call(x, out_q, out_scale)
    _check(fn(*args, _stream()), "ep_quantize_i8")
    return result


def bind_quantize_i8(x: torch.Tensor, out_q=None, out_scale=None,
                     handle: Optional["Handle"] = None) -> "BoundCall":
    """``quantize_i8``, or with a ``handle`` ``Handle.quantize_i8`` of its expert rows, bound to
    these tensors (see BoundCall)."""
    if handle is None:
        fn, args, result, keep = _quantize_i8_call(x, out_q, out_scale)
        return BoundCall(fn, args, "ep_quantize_i8", result, keep)
    fn, args, result, keep = handle._quantize_i8_call(x, out_q, out_scale)
    return BoundCall(fn, args, "ep_quantize_i8_rows", result, (handle, keep), handle.h)


def bind_expert_i8(handle: "Handle", x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor,
                   w_scale: torch.Tensor, gated: bool = False,
                   row_weights: Optional[torch.Tensor] = None, token_rows: bool = False,
                   out: Optional[torch.Tensor] = None) -> "BoundCall":
    """``handle.expert_i8`` bound to these tensors (see BoundCall)."""
    fn, args, out, keep = handle._expert_i8_call(x, x_scale, w, w_scale, gated, row_weights,
                                                 token_rows, out)
    return BoundCall(fn, args, "ep_expert_i8", out, (handle, keep), handle.h)


def bind_expert_ffn(handle: "Handle", x: torch.Tensor, w13: torch.Tensor,
                    w2: Optional[torch.Tensor], row_weights: Optional[torch.Tensor] = None,
                    token_rows: bool = False, want_saved: bool = False, out_h=None, saved=None,
                    out=None) -> "BoundCall":
    """``handle.expert_ffn`` bound to these tensors (see BoundCall)."""
    fn, args, result, keep = handle._expert_ffn_call(x, w13, w2, row_weights, token_rows,
                                                     want_saved, out_h, saved, out)
    return BoundCall(fn, args, "ep_expert_ffn", result, (handle, keep), handle.h)


_CODE_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def _here(*tensors):
    """The calls enqueue on the current device's stream: every tensor must live there."""
    current = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d >= 0 and current is None:
                current = torch.cuda.current_device()
            if d >= 0 and d != current:
                raise ValueError("tensors must be on the current device")


def _rows_of(t, name, shape, dtype):
    """``t`` must be a contiguous device tensor of this shape and type."""
    _dev(t, name)
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}")


def _norm_weight(weight, hidden) -> int:
    _dev(weight, "weight")
    if weight.shape != (hidden,) or weight.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("weight must be bf16 or fp32 [H]")
    return EP_BF16 if weight.dtype == torch.bfloat16 else EP_F32


def _add_rmsnorm_call(x, weight, residual, eps, out_z, out_y, want_y, scale_format, out_q, out_sf,
                      col_major_sf, want_rstd, out_rstd):
    _dev(x, "x")
    _need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be bf16 [T, H]")
    T, H = x.shape
    wdt = _norm_weight(weight, H)
    if residual is not None:
        _rows_of(residual, "residual", x.shape, torch.bfloat16)
        if out_z is None:
            out_z = torch.empty_like(x)
    if out_z is not None:
        _rows_of(out_z, "out_z", x.shape, torch.bfloat16)
    if want_y and out_y is None:
        out_y = torch.empty_like(x)
    if out_y is not None:
        _rows_of(out_y, "out_y", x.shape, torch.bfloat16)
    fmt, ts, hs = EP_SF_F32, 0, 0
    if scale_format is not None:
        fmt = _sf_format(scale_format)
        packs = ep_sf_packs(H, fmt)
        _need(packs > 0, "hidden must be a positive multiple of 128")
        if out_q is None:
            out_q = torch.empty((T, H), dtype=torch.uint8, device=x.device)
        _dev(out_q, "out_q")
        _need(out_q.dtype in _CODE_DTYPES and tuple(out_q.shape) == (T, H),
              "out_q must be FP8 codes [T, H]")
        out_sf = _quant_sf_out(out_sf, T, packs, fmt, col_major_sf, x.device)
        ts, hs = out_sf.stride()
    else:
        _need(out_q is None and out_sf is None, "FP8 rows need a scale_format")
    if want_rstd and out_rstd is None:
        out_rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    if out_rstd is not None:
        _dev(out_rstd, "out_rstd")
        _need(out_rstd.dtype == torch.float32 and tuple(out_rstd.shape) == (T,),
              "out_rstd must be fp32 [T]")
    _here(x, weight, residual, out_z, out_y, out_q, out_sf, out_rstd)
    args = (_ptr(x), _ptr(residual), _ptr(weight), wdt, eps, T, H, _ptr(out_z), _ptr(out_y), fmt,
            _ptr(out_q), _ptr(out_sf), ts, hs, _ptr(out_rstd))
    return (lib().ep_add_rmsnorm, args, (out_y, out_z, out_q, out_sf, out_rstd),
            (x, weight, residual))


def add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                eps: float = 1e-6, out_z=None, out_y=None, want_y: bool = True,
                scale_format=None, out_q=None, out_sf=None, col_major_sf: bool = False,
                want_rstd: bool = False, out_rstd=None):
    """z = x + residual (bf16 [T, H]), its root-mean-square norm times ``weight``
    (bf16 or fp32 [H]).  Returns (y, z, codes, scales, rstd): y bf16 unless
    ``want_y`` is false; z None without a residual (it is x then) unless
    ``out_z`` is given; E4M3 codes and scales of the fp32 y with ``scale_format``
    'f32' or 'ue8m0' (as quantize_fp8 makes them); rstd fp32 [T] for the backward
    pass with ``want_rstd``."""
    fn, args, result, _ = _add_rmsnorm_call(x, weight, residual, eps, out_z, out_y, want_y,
                                            scale_format, out_q, out_sf, col_major_sf, want_rstd,
                                            out_rstd)
    _check(fn(*args, _stream()), "ep_add_rmsnorm")
    return result


def bind_add_rmsnorm(x: torch.Tensor, weight: torch.Tensor,
                     residual: Optional[torch.Tensor] = None, eps: float = 1e-6, out_z=None,
                     out_y=None, want_y: bool = True, scale_format=None, out_q=None, out_sf=None,
                     col_major_sf: bool = False, want_rstd: bool = False,
                     out_rstd=None) -> "BoundCall":
    """``add_rmsnorm`` bound to these tensors (see BoundCall)."""
    fn, args, result, keep = _add_rmsnorm_call(x, weight, residual, eps, out_z, out_y, want_y,
                                               scale_format, out_q, out_sf, col_major_sf,
                                               want_rstd, out_rstd)
    return BoundCall(fn, args, "ep_add_rmsnorm", result, keep)


def add_rmsnorm_backward(grad_y: torch.Tensor, z: torch.Tensor, weight: torch.Tensor,
                         rstd: torch.Tensor, grad_residual: Optional[torch.Tensor] = None,
                         want_grad_x: bool = True, want_grad_weight: bool = True, grad_x=None,
                         grad_weight=None, workspace=None):
    """Gradients of ``add_rmsnorm`` from its z and rstd.  ``grad_residual`` is the
    gradient that reaches z along the residual.  Returns (grad_x bf16 [T, H], of
    x and of the residual alike, or None, grad_weight fp32 [H] or None)."""
    _dev(z, "z")
    _need(z.dtype == torch.bfloat16 and z.dim() == 2, "z must be bf16 [T, H]")
    T, H = z.shape
    _rows_of(grad_y, "grad_y", z.shape, torch.bfloat16)
    wdt = _norm_weight(weight, H)
    _rows_of(rstd, "rstd", (T,), torch.float32)
    if grad_residual is not None:
        _rows_of(grad_residual, "grad_residual", z.shape, torch.bfloat16)
    _here(grad_y, z, weight, rstd, grad_residual, grad_x, grad_weight, workspace)
    if grad_x is not None:
        _rows_of(grad_x, "grad_x", z.shape, torch.bfloat16)
    elif want_grad_x:
        grad_x = torch.empty_like(z)
    if grad_weight is not None:
        _rows_of(grad_weight, "grad_weight", (H,), torch.float32)
    elif want_grad_weight:
        grad_weight = rstd.new_empty(H)
    nbytes = 0
    if grad_weight is not None:
        if workspace is None:
            nbytes = ep_add_rmsnorm_backward_workspace(T, H)
            if nbytes:
                workspace = rstd.new_empty(nbytes // 4)
        else:
            _dev(workspace, "workspace")
            nbytes = workspace.numel() * workspace.element_size()
    _check(lib().ep_add_rmsnorm_backward(
        grad_y.data_ptr(), z.data_ptr(), weight.data_ptr(), wdt, rstd.data_ptr(),
        _ptr(grad_residual), T, H, _ptr(grad_x), _ptr(grad_weight), _ptr(workspace), nbytes,
        _stream()), "ep_add_rmsnorm_backward")
    return grad_x, grad_weight


class W4Weights:
    """The experts' 4-bit weights in the layout of ep_expert_w4: what ``pack_w4``
    makes, or the same bytes from a file."""
    __slots__ = ("codes", "scales", "num_experts", "n", "k", "format", "group")

    def __init__(self, codes, scales, num_experts, n, k, fmt, group):
        # the kernel reads as many bytes as the sizes say
        _dev(codes, "codes")
        _dev(scales, "scales")
        nc, ns = ep_w4_code_bytes(num_experts, n, k), ep_w4_scale_bytes(num_experts, n, k, fmt,
                                                                        group)
        _need(nc > 0 and ns > 0, "invalid sizes of 4-bit weights")
        _need(codes.numel() * codes.element_size() == nc and
              scales.numel() * scales.element_size() == ns,
              f"packed weights of these sizes have {nc} bytes of codes and {ns} of scales")
        _need(codes.device == scales.device, "codes and scales must be on one device")
        self.codes, self.scales = codes, scales
        self.num_experts, self.n, self.k, self.format, self.group = num_experts, n, k, fmt, group


def pack_w4(codes: torch.Tensor, scales: torch.Tensor) -> W4Weights:
    """Lay 4-bit weights out for ``Handle.expert_w4``, once.  codes: uint8
    [E, n, k/2], channel 2j in the low half of byte j.  scales [E, n, k/group]:
    bf16 for codes that stand for code - 8 (group 32, 64 or 128), or uint8 /
    float8_e8m0fnu exponents for E2M1 codes (group 32)."""
    _dev(codes, "codes")
    _dev(scales, "scales")
    _need(codes.dtype == torch.uint8 and codes.dim() == 3, "codes must be uint8 [E, n, k/2]")
    E, n, k = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    _need(scales.dim() == 3 and tuple(scales.shape[:2]) == (E, n) and scales.shape[2] > 0 and
          k % scales.shape[2] == 0, "scales must be [E, n, k/group]")
    group = k // scales.shape[2]
    if scales.dtype == torch.bfloat16:
        fmt = EP_W4_INT4
    else:
        _need(scales.dtype in (torch.uint8, torch.float8_e8m0fnu),
              "scales must be bf16 (int4) or uint8 exponents (mxfp4)")
        fmt = EP_W4_MXFP4
    nc, ns = ep_w4_code_bytes(E, n, k), ep_w4_scale_bytes(E, n, k, fmt, group)
    _need(nc > 0 and ns > 0, "4-bit weights: n % 8 == 0, k % 128 == 0, k <= 32768, E <= 1024, "
          "group 32, 64 or 128 with bf16 scales and 32 with exponents")
    out_codes = torch.empty(nc, dtype=torch.uint8, device=codes.device)
    out_scales = torch.empty(ns, dtype=torch.uint8, device=codes.device)
    _here(codes, scales)
    _check(ep_w4_pack(_ptr(codes), _ptr(scales), E, n, k, fmt, group, _ptr(out_codes),
                      _ptr(out_scales), _stream()), "ep_w4_pack")
    return W4Weights(out_codes, out_scales, E, n, k, fmt, group)


class Handle:
    """Routing state in a torch-allocated workspace, with layout, dispatch and
    combine on torch tensors.  ``capacity`` defaults to the worst-case bound,
    so no count needs to be read back before dispatch."""

    def __init__(self, max_tokens: int, num_topk: int, num_experts: int,
                 expert_alignment: int = 1, capacity: Optional[int] = None,
                 device="cuda"):
        if capacity is None:
            capacity = ep_capacity_bound(max_tokens, num_topk, num_experts, expert_alignment)
            _need(capacity >= 0, "invalid sizes")
        nbytes = ep_workspace_bytes(max_tokens, num_topk, num_experts, expert_alignment,
                                    capacity)
        _need(nbytes > 0, "sizes outside the library's limits")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.h = ep_handle()
        _check(ep_handle_init(self.h, max_tokens, num_topk, num_experts, expert_alignment,
                              capacity, self.workspace.data_ptr(), nbytes, _stream()),
               "ep_handle_init")
        self.capacity = capacity
        self.topk_idx = None      # kept alive: the handle borrows it

    # -- views of the handle's device arrays
    def _view(self, ptr: int, n: int) -> torch.Tensor:
        off = ptr - self.workspace.data_ptr()
        return self.workspace[off:off + 4 * n].view(torch.int32)

    @property
    def num_tokens(self) -> int:
        return self.h.num_tokens

    @property
    def counts(self) -> torch.Tensor:
        return self._view(self.h.counts, self.h.num_experts)

    @property
    def psum(self) -> torch.Tensor:
        return self._view(self.h.psum, self.h.num_experts + 1)

    @property
    def dst_slot(self) -> torch.Tensor:
        return self._view(self.h.dst_slot, self.h.num_tokens * self.h.num_topk).view(
            self.h.num_tokens, self.h.num_topk)

    @property
    def src_meta(self) -> torch.Tensor:
        return self._view(self.h.src_meta, self.capacity)

    @property
    def scalars(self) -> torch.Tensor:
        return self._view(self.h.scalars, 8)

    @property
    def recv_row(self) -> torch.Tensor:
        return self._view(self.h.recv_row, self.h.num_tokens)

    @property
    def recv_src(self) -> torch.Tensor:
        return self._view(self.h.recv_src, self.h.max_tokens)

    def _layout_call(self, topk_idx, cumulative_stats, noalloc=False):
        _dev(topk_idx, "topk_idx")
        _need(topk_idx.dim() == 2 and topk_idx.shape[1] == self.h.num_topk,
              "topk_idx must be [num_tokens, num_topk]")
        _need(topk_idx.dtype in (torch.int64, torch.int32), "topk_idx must be int64 or int32")
        if cumulative_stats is not None:
            _dev(cumulative_stats, "cumulative_stats")
            _need(cumulative_stats.dtype == torch.int32 and
                  cumulative_stats.numel() == self.h.num_experts,
                  "cumulative_stats must be int32 [num_experts]")
        dt = EP_I64 if topk_idx.dtype == torch.int64 else EP_I32
        fn = lib().ep_layout_noalloc if noalloc else lib().ep_layout
        return fn, (ctypes.byref(self.h), _ptr(topk_idx), dt, topk_idx.shape[0],
                    _ptr(cumulative_stats))

    def layout(self, topk_idx: torch.Tensor,
               cumulative_stats: Optional[torch.Tensor] = None) -> "Handle":
        fn, args = self._layout_call(topk_idx, cumulative_stats)
        _check(fn(*args, _stream()), "ep_layout")
        self.topk_idx = topk_idx
        return self

    def layout_noalloc(self, topk_idx: torch.Tensor,
                       cumulative_stats: Optional[torch.Tensor] = None) -> "Handle":
        """``layout`` through ep_layout_noalloc: the scans' scratch is the
        library's static per-device array, not the handle's workspace (calls
        that overlap on one device race)."""
        fn, args = self._layout_call(topk_idx, cumulative_stats, noalloc=True)
        _check(fn(*args, _stream()), "ep_layout_noalloc")
        self.topk_idx = topk_idx
        return self

    def bind_layout(self, topk_idx: torch.Tensor,
                    cumulative_stats: Optional[torch.Tensor] = None) -> BoundCall:
        """``layout`` bound to these tensors (see BoundCall); the handle
        borrows ``topk_idx`` from now on."""
        fn, args = self._layout_call(topk_idx, cumulative_stats)
        self.topk_idx = topk_idx
        return BoundCall(fn, args, "ep_layout", self, (topk_idx, cumulative_stats))

    def _layout_dispatch_call(self, topk_idx, x, sf, topk_weights, zero_padding, out_x, out_sf,
                              out_w, want_weights, col_major_sf, cumulative_stats, streaming):
        lfn, largs = self._layout_call(topk_idx, cumulative_stats)
        _, dargs, result, keep = self._dispatch_call(
            x, sf, topk_weights, zero_padding, out_x, out_sf, out_w, want_weights, col_major_sf,
            num_tokens=topk_idx.shape[0], streaming=streaming)
        # ep_layout_dispatch takes the layout's arguments, then the dispatch's
        # (the handle appears once)
        args = largs + dargs[1:]
        return lib().ep_layout_dispatch, args, result, keep + (topk_idx, cumulative_stats)

    def layout_dispatch(self, topk_idx: torch.Tensor, x: torch.Tensor,
                        sf: Optional[torch.Tensor] = None,
                        topk_weights: Optional[torch.Tensor] = None, zero_padding: bool = False,
                        out_x: Optional[torch.Tensor] = None, out_sf: Optional[torch.Tensor] = None,
                        out_w: Optional[torch.Tensor] = None, want_weights: bool = False,
                        col_major_sf: bool = False,
                        cumulative_stats: Optional[torch.Tensor] = None,
                        streaming: bool = False):
        """``layout`` then ``dispatch`` in one call (ep_layout_dispatch: the
        same outputs, one host-side check of both argument sets).  Returns
        (out_x, out_sf, out_w)."""
        fn, args, result, _ = self._layout_dispatch_call(
            topk_idx, x, sf, topk_weights, zero_padding, out_x, out_sf, out_w, want_weights,
            col_major_sf, cumulative_stats, streaming)
        _check(fn(*args, _stream()), "ep_layout_dispatch")
        self.topk_idx = topk_idx
        return result

    def bind_layout_dispatch(self, topk_idx: torch.Tensor, x: torch.Tensor,
                             sf: Optional[torch.Tensor] = None,
                             topk_weights: Optional[torch.Tensor] = None,
                             zero_padding: bool = False, out_x: Optional[torch.Tensor] = None,
                             out_sf: Optional[torch.Tensor] = None,
                             out_w: Optional[torch.Tensor] = None, want_weights: bool = False,
                             col_major_sf: bool = False,
                             cumulative_stats: Optional[torch.Tensor] = None,
                             streaming: bool = False) -> "BoundCall":
        """``layout_dispatch`` bound to these tensors (see BoundCall)."""
        fn, args, result, keep = self._layout_dispatch_call(
            topk_idx, x, sf, topk_weights, zero_padding, out_x, out_sf, out_w, want_weights,
            col_major_sf, cumulative_stats, streaming)
        self.topk_idx = topk_idx
        # no token-count check: the call lays the batch out itself
        return BoundCall(fn, args, "ep_layout_dispatch", result, (self, keep))

    def import_layout(self, topk_idx: torch.Tensor, counts, psum, dst_slot, src_meta,
                      num_recv_tokens: int) -> "Handle":
        """Install a host-computed layout (numpy int32 arrays)."""
        import numpy as np
        _dev(topk_idx, "topk_idx")
        c = np.ascontiguousarray(counts, np.int32)
        p = np.ascontiguousarray(psum, np.int32)
        d = np.ascontiguousarray(dst_slot, np.int32)
        s = np.ascontiguousarray(src_meta, np.int32)
        dt = EP_I64 if topk_idx.dtype == torch.int64 else EP_I32
        _check(ep_handle_import(self.h, _ptr(topk_idx), dt, topk_idx.shape[0], c.ctypes.data,
                                p.ctypes.data, d.ctypes.data, s.ctypes.data if s.size else None,
                                num_recv_tokens, _stream()), "ep_handle_import")
        self.topk_idx = topk_idx
        return self

    def read_counts(self, check: bool = True) -> dict:
        """Blocking: wait for the stream and read counts, psum and scalars."""
        import numpy as np
        E = self.h.num_experts
        counts = np.zeros(E, np.int32)
        psum = np.zeros(E + 1, np.int32)
        ne = ctypes.c_int64(0)
        nr = ctypes.c_int32(0)
        eb = ctypes.c_uint32(0)
        inv = ctypes.c_int32(0)
        st = ep_handle_read_counts(self.h, counts.ctypes.data, psum.ctypes.data,
                                   ctypes.addressof(ne), ctypes.addressof(nr),
                                   ctypes.addressof(eb), ctypes.addressof(inv), _stream())
        if check and st not in (EP_OK,):
            raise EpError(st, "ep_handle_read_counts")
        return dict(status=st, counts=counts, psum=psum, num_expanded=ne.value,
                    num_recv_tokens=nr.value, error_bits=eb.value, invalid_count=inv.value)

    def dispatch(self, x: torch.Tensor, sf: Optional[torch.Tensor] = None,
                 topk_weights: Optional[torch.Tensor] = None, zero_padding: bool = False,
                 out_x: Optional[torch.Tensor] = None, out_sf: Optional[torch.Tensor] = None,
                 out_w: Optional[torch.Tensor] = None, want_weights: bool = False,
                 col_major_sf: bool = False, streaming: bool = False):
        """x: bf16 [T, H], or FP8 (float8_e4m3fn or uint8 codes) [T, H] with
        scales ``sf``: fp32 [T, H/128] or int32 packs [T, P] (any strides).
        Returns (out_x, out_sf, out_w); outputs are allocated with
        ``capacity`` rows unless given (out_sf column-major, TMA-aligned, when
        ``col_major_sf``).  ``streaming``: non-temporal stores of the rows
        (EP_DISPATCH_STREAMING)."""
        fn, args, result, _ = self._dispatch_call(x, sf, topk_weights, zero_padding, out_x,
                                                  out_sf, out_w, want_weights, col_major_sf,
                                                  streaming=streaming)
        _check(fn(*args, _stream()), "ep_dispatch")
        return result

    def bind_dispatch(self, x: torch.Tensor, sf: Optional[torch.Tensor] = None,
                      topk_weights: Optional[torch.Tensor] = None, zero_padding: bool = False,
                      out_x: Optional[torch.Tensor] = None, out_sf: Optional[torch.Tensor] = None,
                      out_w: Optional[torch.Tensor] = None, want_weights: bool = False,
                      col_major_sf: bool = False, streaming: bool = False) -> BoundCall:
        """``dispatch`` bound to these tensors (see BoundCall); each call
        returns (out_x, out_sf, out_w)."""
        fn, args, result, keep = self._dispatch_call(x, sf, topk_weights, zero_padding, out_x,
                                                      out_sf, out_w, want_weights, col_major_sf,
                                                      streaming=streaming)
        return BoundCall(fn, args, "ep_dispatch", result, (self, keep), self.h)

    def _dispatch_call(self, x, sf, topk_weights, zero_padding, out_x, out_sf, out_w,
                       want_weights, col_major_sf, num_tokens=None, streaming=False):
        T = self.h.num_tokens if num_tokens is None else num_tokens
        _dev(x, "x")
        _need(x.dim() == 2 and x.shape[0] == T, "x must be [num_tokens, hidden]")
        H = x.shape[1]
        fp8 = x.dtype in (torch.float8_e4m3fn, torch.uint8)
        _need(fp8 or x.dtype == torch.bfloat16, "x must be bf16 or FP8 e4m3")
        cap = self.capacity
        if out_x is None:
            out_x = torch.empty((cap, H), dtype=x.dtype, device=x.device)
        _dev(out_x, "out_x")
        _need(out_x.shape == (cap, H) and out_x.dtype == x.dtype, "out_x must be [capacity, H]")
        packs, (sf_ts, sf_hs), (o_ts, o_hs) = 0, (0, 0), (0, 0)
        if fp8:
            packs, (sf_ts, sf_hs), out_sf, (o_ts, o_hs) = _scale_packs(
                sf, T, H, cap, out_sf, col_major_sf, x.device)
        else:
            _need(sf is None and out_sf is None, "scale factors are for FP8 only")
        if topk_weights is not None:
            _dev(topk_weights, "topk_weights")
            _need(topk_weights.dtype == torch.float32 and
                  tuple(topk_weights.shape) == (T, self.h.num_topk),
                  "topk_weights must be fp32 [T, K]")
        if want_weights and out_w is None:
            out_w = torch.empty(cap, dtype=torch.float32, device=x.device)
        if out_w is not None:
            _dev(out_w, "out_w")
            _need(out_w.dtype == torch.float32 and out_w.numel() == cap, "out_w: fp32 [capacity]")
        args = (ctypes.byref(self.h), _ptr(x), EP_FP8_E4M3 if fp8 else EP_BF16, H, _ptr(sf),
                sf_ts, sf_hs, packs, _ptr(topk_weights), _ptr(out_x), _ptr(out_sf), o_ts, o_hs,
                _ptr(out_w), (EP_DISPATCH_ZERO_PADDING if zero_padding else 0) |
                (EP_DISPATCH_STREAMING if streaming else 0))
        return lib().ep_dispatch, args, (out_x, out_sf, out_w), (x, sf, topk_weights)

    def dispatch_quant(self, x: torch.Tensor, scale_format="f32",
                       topk_weights: Optional[torch.Tensor] = None, zero_padding: bool = False,
                       out_x=None, out_sf=None, out_w=None, want_weights: bool = False,
                       col_major_sf: bool = False):
        """Quantise bf16 x [T, H] to FP8 and dispatch in one pass.  Returns
        (codes uint8 [capacity, H], scales [capacity, packs], out_w)."""
        T = self.h.num_tokens
        _dev(x, "x")
        _need(x.dtype == torch.bfloat16 and x.dim() == 2 and x.shape[0] == T,
              "x must be bf16 [num_tokens, H]")
        H = x.shape[1]
        fmt = _sf_format(scale_format)
        packs = ep_sf_packs(H, fmt)
        _need(packs > 0, "hidden must be a positive multiple of 128")
        cap = self.capacity
        if out_x is None:
            out_x = torch.empty((cap, H), dtype=torch.uint8, device=x.device)
        _dev(out_x, "out_x")
        _need(out_x.dtype in (torch.uint8, torch.float8_e4m3fn) and
              tuple(out_x.shape) == (cap, H), "out_x must be FP8 codes [capacity, H]")
        out_sf = _quant_sf_out(out_sf, cap, packs, fmt, col_major_sf, x.device)
        o_ts, o_hs = out_sf.stride()
        if topk_weights is not None:
            _dev(topk_weights, "topk_weights")
            _need(topk_weights.dtype == torch.float32 and
                  tuple(topk_weights.shape) == (T, self.h.num_topk),
                  "topk_weights must be fp32 [T, K]")
        if want_weights and out_w is None:
            out_w = torch.empty(cap, dtype=torch.float32, device=x.device)
        if out_w is not None:
            _dev(out_w, "out_w")
            _need(out_w.dtype == torch.float32 and out_w.numel() == cap, "out_w: fp32 [capacity]")
        _check(ep_dispatch_quant(self.h, _ptr(x), H, fmt, _ptr(topk_weights), _ptr(out_x),
                                 _ptr(out_sf), o_ts, o_hs, _ptr(out_w),
                                 1 if zero_padding else 0, _stream()), "ep_dispatch_quant")
        return out_x, out_sf, out_w

    def combine(self, y: torch.Tensor, topk_weights: Optional[torch.Tensor] = None,
                bias: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None,
                bias_0: Optional[torch.Tensor] = None,
                bias_1: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y: bf16 [capacity, H] expert outputs; returns bf16 [T, H].  bias is
        the per-expert [E, H] bias; bias_0 / bias_1 are per-token [T, H]
        biases added after the reduction."""
        fn, args, out, _ = self._combine_call(y, topk_weights, bias, out, bias_0, bias_1)
        _check(fn(*args, _stream()), "ep_combine")
        return out

    def bind_combine(self, y: torch.Tensor, topk_weights: Optional[torch.Tensor] = None,
                     bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     bias_0: Optional[torch.Tensor] = None,
                     bias_1: Optional[torch.Tensor] = None) -> BoundCall:
        """``combine`` bound to these tensors (see BoundCall); each call
        returns ``out``."""
        fn, args, out, keep = self._combine_call(y, topk_weights, bias, out, bias_0, bias_1)
        return BoundCall(fn, args, "ep_combine", out, (self, keep), self.h)

    def _combine_call(self, y, topk_weights, bias, out, bias_0, bias_1):
        T = self.h.num_tokens
        _dev(y, "y")
        _need(y.dtype == torch.bfloat16, "combine input must be bf16")
        _need(y.dim() == 2 and y.shape[0] == self.capacity, "y must be [capacity, H]")
        H = y.shape[1]
        if topk_weights is not None:
            _dev(topk_weights, "topk_weights")
            _need(topk_weights.dtype == torch.float32 and
                  tuple(topk_weights.shape) == (T, self.h.num_topk),
                  "topk_weights must be fp32 [T, K]")
        if bias is not None:
            _dev(bias, "bias")
            _need(bias.dtype == torch.bfloat16 and tuple(bias.shape) == (self.h.num_experts, H),
                  "bias must be bf16 [E, H]")
        for name, b in (("bias_0", bias_0), ("bias_1", bias_1)):
            if b is not None:
                _dev(b, name)
                _need(b.dtype == torch.bfloat16 and tuple(b.shape) == (T, H),
                      f"{name} must be bf16 [T, H]")
        if out is None:
            out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
        _dev(out, "out")
        _need(tuple(out.shape) == (T, H) and out.dtype == torch.bfloat16, "out must be bf16 [T, H]")
        args = (ctypes.byref(self.h), _ptr(y), EP_BF16, H, _ptr(topk_weights), _ptr(bias),
                _ptr(bias_0), _ptr(bias_1), _ptr(out))
        return lib().ep_combine, args, out, (y, topk_weights, bias, bias_0, bias_1)


    # ------------------------------------------------------------ backward

    def combine_backward(self, grad_out: torch.Tensor, topk_weights=None, y=None, bias=None,
                         grad_y=None, want_grad_y: bool = True, want_grad_weights: bool = False,
                         want_grad_bias: bool = False):
        """Backward of combine.  grad_out: bf16 [T, H].  Returns
        (grad_y bf16 [capacity, H] or None, grad_topk_weights fp32 [T, K] or
        None, grad_bias fp32 [E, H] or None).  Rows of grad_y without a slot
        are left as they were (uninitialised when allocated here)."""
        T, K, E = self.h.num_tokens, self.h.num_topk, self.h.num_experts
        _dev(grad_out, "grad_out")
        _need(grad_out.dtype == torch.bfloat16 and grad_out.dim() == 2 and
              grad_out.shape[0] == T, "grad_out must be bf16 [T, H]")
        H = grad_out.shape[1]
        if topk_weights is not None:
            _dev(topk_weights, "topk_weights")
            _need(topk_weights.dtype == torch.float32 and tuple(topk_weights.shape) == (T, K),
                  "topk_weights must be fp32 [T, K]")
        if y is not None:
            _dev(y, "y")
            _need(y.dtype == torch.bfloat16 and tuple(y.shape) == (self.capacity, H),
                  "y must be bf16 [capacity, H]")
        if bias is not None:
            _dev(bias, "bias")
            _need(bias.dtype == torch.bfloat16 and tuple(bias.shape) == (E, H),
                  "bias must be bf16 [E, H]")
        if want_grad_y and grad_y is None:
            grad_y = torch.empty((self.capacity, H), dtype=torch.bfloat16, device=grad_out.device)
        if grad_y is not None:
            _dev(grad_y, "grad_y")
            _need(grad_y.dtype == torch.bfloat16 and tuple(grad_y.shape) == (self.capacity, H),
                  "grad_y must be bf16 [capacity, H]")
        gw = torch.empty((T, K), dtype=torch.float32, device=grad_out.device) \
            if want_grad_weights else None
        if gw is not None:
            _need(y is not None, "the weight gradient needs y")
        gb = torch.empty((E, H), dtype=torch.float32, device=grad_out.device) \
            if want_grad_bias else None
        _check(ep_combine_backward(self.h, _ptr(grad_out), H, _ptr(topk_weights), _ptr(y),
                                   _ptr(bias), _ptr(grad_y), _ptr(gw), _ptr(gb), _stream()),
               "ep_combine_backward")
        return grad_y, gw, gb

    def dispatch_backward(self, grad_out_x: torch.Tensor, grad_out_w=None,
                          want_grad_weights: bool = False):
        """Backward of dispatch.  grad_out_x: bf16 [capacity, H].  Returns
        (grad_x bf16 [T, H], grad_topk_weights fp32 [T, K] or None)."""
        T, K = self.h.num_tokens, self.h.num_topk
        _dev(grad_out_x, "grad_out_x")
        _need(grad_out_x.dtype == torch.bfloat16 and grad_out_x.dim() == 2 and
              grad_out_x.shape[0] == self.capacity, "grad_out_x must be bf16 [capacity, H]")
        H = grad_out_x.shape[1]
        if grad_out_w is not None:
            _dev(grad_out_w, "grad_out_w")
            _need(grad_out_w.dtype == torch.float32 and grad_out_w.numel() == self.capacity,
                  "grad_out_w must be fp32 [capacity]")
        gx = torch.empty((T, H), dtype=torch.bfloat16, device=grad_out_x.device)
        gw = torch.empty((T, K), dtype=torch.float32, device=grad_out_x.device) \
            if want_grad_weights else None
        _check(ep_dispatch_backward(self.h, _ptr(grad_out_x), H, _ptr(grad_out_w), _ptr(gx),
                                    _ptr(gw), _stream()), "ep_dispatch_backward")
        return gx, gw


    # ------------------------------------------------------------ rank layout

    def dispatch_rank(self, x: torch.Tensor, sf: Optional[torch.Tensor] = None,
                      topk_weights: Optional[torch.Tensor] = None, out_x=None, out_sf=None,
                      out_topk_idx=None, out_topk_weights=None, col_major_sf: bool = False):
        """Rank (non-expanded) dispatch: one row per received token, in token
        order, with [max_tokens] rows allocated; rows past num_recv_tokens are
        not written.  Returns (out_x, out_sf, out_topk_idx, out_topk_weights)."""
        T, K = self.h.num_tokens, self.h.num_topk
        M = self.h.max_tokens
        _dev(x, "x")
        _need(x.dim() == 2 and x.shape[0] == T, "x must be [num_tokens, hidden]")
        H = x.shape[1]
        fp8 = x.dtype in (torch.float8_e4m3fn, torch.uint8)
        _need(fp8 or x.dtype == torch.bfloat16, "x must be bf16 or FP8 e4m3")
        if out_x is None:
            out_x = torch.empty((M, H), dtype=x.dtype, device=x.device)
        _need(tuple(out_x.shape) == (M, H) and out_x.dtype == x.dtype and out_x.is_cuda,
              "out_x must be [max_tokens, H]")
        packs, (sf_ts, sf_hs), (o_ts, o_hs) = 0, (0, 0), (0, 0)
        if fp8:
            packs, (sf_ts, sf_hs), out_sf, (o_ts, o_hs) = _scale_packs(
                sf, T, H, M, out_sf, col_major_sf, x.device)
        else:
            _need(sf is None and out_sf is None, "scale factors are for FP8 only")
        idx_dtype = torch.int64 if self.h.topk_idx_dtype == EP_I64 else torch.int32
        if out_topk_idx is None:
            out_topk_idx = torch.empty((M, K), dtype=idx_dtype, device=x.device)
        _need(out_topk_idx.dtype == idx_dtype and tuple(out_topk_idx.shape) == (M, K),
              "out_topk_idx must be [max_tokens, K] of the layout's id dtype")
        if out_topk_weights is None:
            out_topk_weights = torch.empty((M, K), dtype=torch.float32, device=x.device)
        if topk_weights is not None:
            _dev(topk_weights, "topk_weights")
        _check(ep_dispatch_rank(self.h, _ptr(x), EP_FP8_E4M3 if fp8 else EP_BF16, H, _ptr(sf),
                                sf_ts, sf_hs, packs, _ptr(topk_weights), _ptr(out_x),
                                _ptr(out_sf),
                                o_ts, o_hs, _ptr(out_topk_idx), _ptr(out_topk_weights),
                                _stream()), "ep_dispatch_rank")
        return out_x, out_sf, out_topk_idx, out_topk_weights

    def dispatch_rank_quant(self, x: torch.Tensor, scale_format="f32",
                            topk_weights: Optional[torch.Tensor] = None, out_x=None, out_sf=None,
                            out_topk_idx=None, out_topk_weights=None,
                            col_major_sf: bool = False):
        """Quantise bf16 x [T, H] to FP8 and dispatch into the rank layout in
        one pass.  Returns (codes uint8 [max_tokens, H], scales [max_tokens,
        packs], out_topk_idx, out_topk_weights)."""
        T, K = self.h.num_tokens, self.h.num_topk
        M = self.h.max_tokens
        _dev(x, "x")
        _need(x.dtype == torch.bfloat16 and x.dim() == 2 and x.shape[0] == T,
              "x must be bf16 [num_tokens, H]")
        H = x.shape[1]
        fmt = _sf_format(scale_format)
        packs = ep_sf_packs(H, fmt)
        _need(packs > 0, "hidden must be a positive multiple of 128")
        if out_x is None:
            out_x = torch.empty((M, H), dtype=torch.uint8, device=x.device)
        _dev(out_x, "out_x")
        _need(out_x.dtype in (torch.uint8, torch.float8_e4m3fn) and tuple(out_x.shape) == (M, H),
              "out_x must be FP8 codes [max_tokens, H]")
        out_sf = _quant_sf_out(out_sf, M, packs, fmt, col_major_sf, x.device)
        o_ts, o_hs = out_sf.stride()
        idx_dtype = torch.int64 if self.h.topk_idx_dtype == EP_I64 else torch.int32
        if out_topk_idx is None:
            out_topk_idx = torch.empty((M, K), dtype=idx_dtype, device=x.device)
        _need(out_topk_idx.dtype == idx_dtype and tuple(out_topk_idx.shape) == (M, K),
              "out_topk_idx must be [max_tokens, K] of the layout's id dtype")
        if out_topk_weights is None:
            out_topk_weights = torch.empty((M, K), dtype=torch.float32, device=x.device)
        _need(out_topk_weights.dtype == torch.float32 and tuple(out_topk_weights.shape) == (M, K),
              "out_topk_weights must be fp32 [max_tokens, K]")
        if topk_weights is not None:
            _dev(topk_weights, "topk_weights")
            _need(topk_weights.dtype == torch.float32 and tuple(topk_weights.shape) == (T, K),
                  "topk_weights must be fp32 [T, K]")
        _check(ep_dispatch_rank_quant(self.h, _ptr(x), H, fmt, _ptr(topk_weights), _ptr(out_x),
                                      _ptr(out_sf), o_ts, o_hs, _ptr(out_topk_idx),
                                      _ptr(out_topk_weights), _stream()),
               "ep_dispatch_rank_quant")
        return out_x, out_sf, out_topk_idx, out_topk_weights

    def combine_rank(self, x: torch.Tensor, bias_0=None, bias_1=None, out=None) -> torch.Tensor:
        """x: bf16 [max_tokens, H] rank-layout rows; returns bf16 [T, H]."""
        T, M = self.h.num_tokens, self.h.max_tokens
        _dev(x, "x")
        _need(x.dtype == torch.bfloat16 and x.dim() == 2 and x.shape[0] == M,
              "x must be bf16 [max_tokens, H]")
        H = x.shape[1]
        for name, b in (("bias_0", bias_0), ("bias_1", bias_1)):
            if b is not None:
                _dev(b, name)
                _need(b.dtype == torch.bfloat16 and tuple(b.shape) == (T, H),
                      f"{name} must be bf16 [T, H]")
        if out is None:
            out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        _check(ep_combine_rank(self.h, _ptr(x), H, _ptr(bias_0), _ptr(bias_1), _ptr(out),
                               _stream()), "ep_combine_rank")
        return out

    # ------------------------------------------------------------ expert layer

    def expert_w4(self, x: torch.Tensor, weights: W4Weights, sf: Optional[torch.Tensor] = None,
                  token_rows: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Every expert's rows times its 4-bit weights: bf16 [capacity, n].  x: bf16
        rows or FP8 codes with scales ``sf``, as dispatch writes them
        ([capacity, k]), or with ``token_rows`` the tokens' own rows ([T, k]), which
        needs no dispatch.  Rows without a slot are left as they were."""
        fn, args, out, _ = self._expert_w4_call(x, weights, sf, token_rows, out)
        _check(fn(*args, _stream()), "ep_expert_w4")
        return out

    def bind_expert_w4(self, x: torch.Tensor, weights: W4Weights,
                       sf: Optional[torch.Tensor] = None, token_rows: bool = False,
                       out: Optional[torch.Tensor] = None) -> BoundCall:
        """``expert_w4`` bound to these tensors (see BoundCall)."""
        fn, args, out, keep = self._expert_w4_call(x, weights, sf, token_rows, out)
        return BoundCall(fn, args, "ep_expert_w4", out, (self, keep), self.h)

    def _expert_w4_call(self, x, weights, sf, token_rows, out):
        rows = self.h.num_tokens if token_rows else self.capacity
        _need(weights.num_experts == self.h.num_experts, "weights of another number of experts")
        _dev(x, "x")
        _need(x.dim() == 2 and tuple(x.shape) == (rows, weights.k),
              f"x must be [{rows}, {weights.k}]")
        fp8 = x.dtype in _CODE_DTYPES
        _need(fp8 or x.dtype == torch.bfloat16, "x must be bf16 or FP8 e4m3")
        fmt, ts, hs = EP_SF_F32, 0, 0
        if fp8:
            fmt, ts, hs = self._sf_in(sf, "sf", rows, weights.k)
        else:
            _need(sf is None, "scale factors are for FP8 only")
        if out is None:
            out = torch.empty((self.capacity, weights.n), dtype=torch.bfloat16, device=x.device)
        _rows_of(out, "out", (self.capacity, weights.n), torch.bfloat16)
        _here(x, sf, out, weights.codes, self.workspace)
        args = (ctypes.byref(self.h), _ptr(x), EP_FP8_E4M3 if fp8 else EP_BF16,
                1 if token_rows else 0, weights.k, _ptr(sf), fmt, ts, hs, _ptr(weights.codes),
                _ptr(weights.scales), weights.format, weights.group, weights.n, _ptr(out))
        return lib().ep_expert_w4, args, out, (x, weights, sf)

    @staticmethod
    def _sf_in(sf, name, rows, cols):
        """Format and strides of FP8 rows' scales: fp32 [rows, cols/128] or int32
        packs of UE8M0 exponents."""
        _need(sf is not None, "FP8 rows need scale factors")
        _dev_strided(sf, name)
        _need(sf.dtype in _SF_DTYPES, f"{name} must be fp32 scales or int32 packs")
        fmt = EP_SF_F32 if sf.dtype == torch.float32 else EP_SF_UE8M0
        packs = ep_sf_packs(cols, fmt)
        if packs <= 0 or sf.shape != (rows, packs):
            raise ValueError(f"{name} must be [{rows}, {packs}] for FP8 rows of {cols} channels")
        return (fmt, *sf.stride())

    def _row_weights(self, row_weights):
        if row_weights is not None:
            _dev(row_weights, "row_weights")
            _need(row_weights.dtype == torch.float32 and row_weights.numel() == self.capacity,
                  "row_weights must be fp32 [capacity]")

    def swiglu(self, gate_up: torch.Tensor, row_weights: Optional[torch.Tensor] = None,
               scale_format=None, out=None, out_sf=None, checkpoint=None, saved=None,
               saved_sf=None, col_major_sf: bool = False):
        """silu(gate) * up (* row_weights) of the expert rows gate_up bf16
        [capacity, 2 inter], gate first.  Returns (h, scales, saved, saved_scales): h
        bf16 [capacity, inter], or E4M3 codes with ``scale_format`` 'f32' or 'ue8m0';
        with ``checkpoint`` 'f32' or 'ue8m0', saved holds gate_up in E4M3 for
        ``swiglu_backward``.  Rows without a slot are left as they were."""
        fn, args, result, _ = self._swiglu_call(gate_up, row_weights, scale_format, out, out_sf,
                                                checkpoint, saved, saved_sf, col_major_sf)
        _check(fn(*args, _stream()), "ep_swiglu")
        return result

    def bind_swiglu(self, gate_up: torch.Tensor, row_weights: Optional[torch.Tensor] = None,
                    scale_format=None, out=None, out_sf=None, checkpoint=None, saved=None,
                    saved_sf=None, col_major_sf: bool = False) -> BoundCall:
        """``swiglu`` bound to these tensors (see BoundCall)."""
        fn, args, result, keep = self._swiglu_call(gate_up, row_weights, scale_format, out,
                                                   out_sf, checkpoint, saved, saved_sf,
                                                   col_major_sf)
        return BoundCall(fn, args, "ep_swiglu", result, (self, keep), self.h)

    def _swiglu_call(self, gate_up, row_weights, scale_format, out, out_sf, checkpoint, saved,
                     saved_sf, col_major_sf):
        cap, dev = self.capacity, gate_up.device
        _dev(gate_up, "gate_up")
        _need(gate_up.dtype == torch.bfloat16 and gate_up.dim() == 2 and
              gate_up.shape[0] == cap and gate_up.shape[1] % 2 == 0,
              "gate_up must be bf16 [capacity, 2 inter]")
        inter = gate_up.shape[1] // 2
        self._row_weights(row_weights)
        fmt, ts, hs = EP_SF_F32, 0, 0
        if scale_format is None:
            _need(out_sf is None, "FP8 rows need a scale_format")
            if out is None:
                out = torch.empty((cap, inter), dtype=torch.bfloat16, device=dev)
            _rows_of(out, "out", (cap, inter), torch.bfloat16)
        else:
            fmt = _sf_format(scale_format)
            packs = ep_sf_packs(inter, fmt)
            _need(packs > 0, "inter must be a positive multiple of 128")
            if out is None:
                out = torch.empty((cap, inter), dtype=torch.uint8, device=dev)
            _dev(out, "out")
            _need(out.dtype in _CODE_DTYPES and tuple(out.shape) == (cap, inter),
                  f"out must be FP8 codes [{cap}, {inter}]")
            out_sf = _quant_sf_out(out_sf, cap, packs, fmt, col_major_sf, dev)
            ts, hs = out_sf.stride()
        sfmt, sts, shs = EP_SF_F32, 0, 0
        if checkpoint is None:
            _need(saved is None and saved_sf is None, "saved rows need a checkpoint format")
        else:
            sfmt = _sf_format(checkpoint)
            packs = ep_sf_packs(2 * inter, sfmt)
            _need(inter % 128 == 0 and packs > 0, "inter must be a positive multiple of 128")
            if saved is None:
                saved = torch.empty((cap, 2 * inter), dtype=torch.uint8, device=dev)
            _dev(saved, "saved")
            _need(saved.dtype in _CODE_DTYPES and tuple(saved.shape) == (cap, 2 * inter),
                  f"saved must be FP8 codes [{cap}, {2 * inter}]")
            saved_sf = _quant_sf_out(saved_sf, cap, packs, sfmt, False, dev)
            sts, shs = saved_sf.stride()
        _here(gate_up, row_weights, out, out_sf, saved, saved_sf, self.workspace)
        args = (ctypes.byref(self.h), _ptr(gate_up), inter, _ptr(row_weights),
                EP_BF16 if scale_format is None else EP_FP8_E4M3, _ptr(out), fmt, _ptr(out_sf),
                ts, hs, _ptr(saved), sfmt, _ptr(saved_sf), sts, shs)
        return (lib().ep_swiglu, args, (out, out_sf, saved, saved_sf), (gate_up, row_weights))

    def swiglu_backward(self, grad_h: torch.Tensor, saved: torch.Tensor,
                        saved_sf: Optional[torch.Tensor] = None,
                        row_weights: Optional[torch.Tensor] = None, grad_gate_up=None,
                        grad_row_weights=None, want_grad_weights: bool = False, out=None,
                        want_h: bool = False):
        """Gradients of ``swiglu``.  saved: its E4M3 checkpoint with ``saved_sf``, or the
        bf16 gate_up.  Returns (grad_gate_up bf16 [capacity, 2 inter],
        grad_row_weights fp32 [capacity] or None, for ``dispatch_backward``, and with
        ``want_h`` the activation made again from ``saved``, bf16 [capacity, inter],
        or None).  Rows without a slot are left as they were."""
        cap = self.capacity
        _dev(grad_h, "grad_h")
        _need(grad_h.dtype == torch.bfloat16 and grad_h.dim() == 2 and grad_h.shape[0] == cap,
              "grad_h must be bf16 [capacity, inter]")
        inter = grad_h.shape[1]
        _dev(saved, "saved")
        fp8 = saved.dtype in _CODE_DTYPES
        if saved.shape != (cap, 2 * inter) or not (fp8 or saved.dtype == torch.bfloat16):
            raise ValueError(f"saved must be bf16 or FP8 codes [{cap}, {2 * inter}]")
        fmt, ts, hs = EP_SF_F32, 0, 0
        if fp8:
            _need(inter % 128 == 0, "inter must be a positive multiple of 128")
            fmt, ts, hs = self._sf_in(saved_sf, "saved_sf", cap, 2 * inter)
        else:
            _need(saved_sf is None, "scale factors are for FP8 only")
        self._row_weights(row_weights)
        if grad_gate_up is None:
            grad_gate_up = torch.empty((cap, 2 * inter), dtype=torch.bfloat16,
                                       device=grad_h.device)
        _rows_of(grad_gate_up, "grad_gate_up", (cap, 2 * inter), torch.bfloat16)
        if want_grad_weights and grad_row_weights is None:
            grad_row_weights = torch.empty(cap, dtype=torch.float32, device=grad_h.device)
        if grad_row_weights is not None:
            _dev(grad_row_weights, "grad_row_weights")
            _need(grad_row_weights.dtype == torch.float32 and grad_row_weights.numel() == cap,
                  "grad_row_weights must be fp32 [capacity]")
        if want_h and out is None:
            out = torch.empty((cap, inter), dtype=torch.bfloat16, device=grad_h.device)
        if out is not None:
            _rows_of(out, "out", (cap, inter), torch.bfloat16)
        _here(grad_h, saved, saved_sf, row_weights, grad_gate_up, grad_row_weights, out,
              self.workspace)
        _check(ep_swiglu_backward(self.h, _ptr(grad_h), inter, _ptr(row_weights), _ptr(saved),
                                  EP_FP8_E4M3 if fp8 else EP_BF16, fmt, _ptr(saved_sf), ts, hs,
                                  _ptr(grad_gate_up), _ptr(grad_row_weights), _ptr(out),
                                  _stream()), "ep_swiglu_backward")
        return grad_gate_up, grad_row_weights, out

    def quantize_i8(self, x: torch.Tensor, out_q=None, out_scale=None):
        """Expert rows bf16 [capacity, C] as int8 codes [capacity, C] with one fp32 scale a
        row, [capacity] (see ``ep.quantize_i8``).  Rows without a slot are left as they were."""
        fn, args, result, _ = self._quantize_i8_call(x, out_q, out_scale)
        _check(fn(*args, _stream()), "ep_quantize_i8_rows")
        return result

    def _quantize_i8_call(self, x, out_q, out_scale):
        out_q, out_scale = _i8_rows(x, self.capacity, "capacity", out_q, out_scale)
        _here(x, out_q, out_scale, self.workspace)
        args = (ctypes.byref(self.h), _ptr(x), x.shape[1], _ptr(out_q), _ptr(out_scale))
        return lib().ep_quantize_i8_rows, args, (out_q, out_scale), x

    def expert_i8(self, x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor,
                  w_scale: torch.Tensor, gated: bool = False,
                  row_weights: Optional[torch.Tensor] = None, token_rows: bool = False,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Every expert's int8 rows times its int8 weights w [E, n, k], with a scale for each
        row, x_scale fp32 [rows], and each output channel, w_scale fp32 [E, n]: bf16
        [capacity, n].  With ``gated`` w is gate above up, and silu(gate) * up
        (* row_weights) comes out, bf16 [capacity, n/2].  x: [capacity, k] as dispatch
        writes it, or with ``token_rows`` the tokens' own rows [T, k].  Rows without a
        slot are left as they were."""
        fn, args, out, _ = self._expert_i8_call(x, x_scale, w, w_scale, gated, row_weights,
                                                token_rows, out)
        _check(fn(*args, _stream()), "ep_expert_i8")
        return out

    def _expert_i8_call(self, x, x_scale, w, w_scale, gated, row_weights, token_rows, out):
        E, rows = self.h.num_experts, self.h.num_tokens if token_rows else self.capacity
        _dev(w, "w")
        _need(w.dtype == torch.int8 and w.dim() == 3 and w.shape[0] == E,
              f"w must be int8 [{E}, n, k]")
        n, k = w.shape[1:]
        _rows_of(x, "x", (rows, k), torch.int8)
        _rows_of(x_scale, "x_scale", (rows,), torch.float32)
        _rows_of(w_scale, "w_scale", (E, n), torch.float32)
        _need(not gated or n % 2 == 0, "gated weights are gate above up")
        _need(gated or row_weights is None, "row_weights are for gated products")
        self._row_weights(row_weights)
        cols = n // 2 if gated else n
        if out is None:
            out = torch.empty((self.capacity, cols), dtype=torch.bfloat16, device=x.device)
        _rows_of(out, "out", (self.capacity, cols), torch.bfloat16)
        _here(x, x_scale, w, w_scale, row_weights, out, self.workspace)
        args = (ctypes.byref(self.h), _ptr(x), _ptr(x_scale), 1 if token_rows else 0, k, _ptr(w),
                _ptr(w_scale), n, 1 if gated else 0, _ptr(row_weights), _ptr(out))
        return lib().ep_expert_i8, args, out, (x, x_scale, w, w_scale, row_weights)

    def expert_ffn(self, x: torch.Tensor, w13: torch.Tensor, w2: Optional[torch.Tensor],
                   row_weights: Optional[torch.Tensor] = None, token_rows: bool = False,
                   want_saved: bool = False, out_h=None, saved=None, out=None):
        """The experts' gated feed-forward block in bf16: gate and up = w13[e] . x (w13
        [E, 2 inter, H], gate above up), h = silu(gate) * up (* row_weights), y = w2[e] . h
        (w2 [E, H, inter]).  x: [capacity, H] as dispatch writes it, or with ``token_rows`` the
        tokens' own rows [T, H].  Returns (y [capacity, H], h [capacity, inter], saved): with
        ``want_saved`` gate and up [capacity, 2 inter] for ``expert_ffn_backward``.  With w2
        None y is None.  Rows without a slot are left as they were."""
        fn, args, result, _ = self._expert_ffn_call(x, w13, w2, row_weights, token_rows,
                                                    want_saved, out_h, saved, out)
        _check(fn(*args, _stream()), "ep_expert_ffn")
        return result

    def _ffn_sizes(self, w13, w2):
        E = self.h.num_experts
        _dev(w13, "w13")
        _need(w13.dtype == torch.bfloat16 and w13.dim() == 3 and w13.shape[0] == E and
              w13.shape[1] % 2 == 0, f"w13 must be bf16 [{E}, 2 inter, H]")
        inter, H = w13.shape[1] // 2, w13.shape[2]
        if w2 is not None:
            _rows_of(w2, "w2", (E, H, inter), torch.bfloat16)
        return H, inter

    def _expert_ffn_call(self, x, w13, w2, row_weights, token_rows, want_saved, out_h, saved, out):
        cap, dev = self.capacity, x.device
        H, inter = self._ffn_sizes(w13, w2)
        _rows_of(x, "x", (self.h.num_tokens if token_rows else cap, H), torch.bfloat16)
        self._row_weights(row_weights)
        _need(w2 is not None or out is None, "out needs w2")
        out_h = _buffer(out_h, "out_h", (cap, inter), True, dev)
        saved = _buffer(saved, "saved", (cap, 2 * inter), want_saved, dev)
        out = _buffer(out, "out", (cap, H), w2 is not None, dev)
        _here(x, w13, w2, row_weights, out_h, saved, out, self.workspace)
        args = (ctypes.byref(self.h), _ptr(x), 1 if token_rows else 0, H, _ptr(w13), _ptr(w2),
                inter, _ptr(row_weights), _ptr(out_h), _ptr(saved), _ptr(out))
        return lib().ep_expert_ffn, args, (out, out_h, saved), (x, w13, w2, row_weights)

    def expert_ffn_backward(self, grad_y: torch.Tensor, x: Optional[torch.Tensor],
                            w13: torch.Tensor, w2: torch.Tensor, saved: torch.Tensor,
                            h: Optional[torch.Tensor] = None,
                            row_weights: Optional[torch.Tensor] = None, token_rows: bool = False,
                            remake_h: bool = False, grad_gate_up=None, grad_x=None,
                            want_grad_x: bool = True, grad_w13=None, grad_w2=None,
                            want_grad_w: bool = True, grad_dtype: torch.dtype = torch.bfloat16,
                            grad_row_weights=None, want_grad_weights: bool = False,
                            workspace=None):
        """Gradients of ``expert_ffn`` from its ``saved`` gate and up and its ``h`` (which
        ``remake_h`` makes again from ``saved``, into ``h`` if that is given).  Returns (grad_x
        bf16 [capacity, H] for ``dispatch_backward``, grad_w13, grad_w2 in ``grad_dtype``, bf16 or
        fp32 (or that of the tensors given), grad_row_weights fp32 [capacity] with
        ``want_grad_weights``, grad_gate_up bf16 [capacity, 2 inter], which may be ``saved``
        itself); what is not wanted is None.  Rows without a slot are left as they were."""
        cap, dev = self.capacity, grad_y.device
        _need(w2 is not None, "the gradients need w2")
        H, inter = self._ffn_sizes(w13, w2)
        _rows_of(grad_y, "grad_y", (cap, H), torch.bfloat16)
        _rows_of(saved, "saved", (cap, 2 * inter), torch.bfloat16)
        self._row_weights(row_weights)
        given = [g.dtype for g in (grad_w13, grad_w2) if g is not None]
        if given:
            grad_dtype = given[0]
        _need(grad_dtype in (torch.bfloat16, torch.float32), "weight gradients are bf16 or fp32")
        grad_w13 = _buffer(grad_w13, "grad_w13", tuple(w13.shape), want_grad_w, dev, grad_dtype)
        grad_w2 = _buffer(grad_w2, "grad_w2", tuple(w2.shape), want_grad_w, dev, grad_dtype)
        grad_x = _buffer(grad_x, "grad_x", (cap, H), want_grad_x, dev)
        grad_gate_up = _buffer(grad_gate_up, "grad_gate_up", (cap, 2 * inter), True, dev)
        grad_row_weights = _buffer(grad_row_weights, "grad_row_weights", (cap,),
                                   want_grad_weights, dev, torch.float32)
        h = _buffer(h, "h", (cap, inter), remake_h, dev)
        _need(h is not None or grad_w2 is None, "the gradient of w2 needs h")
        if x is not None:
            _rows_of(x, "x", (self.h.num_tokens if token_rows else cap, H), torch.bfloat16)
        _need(x is not None or grad_w13 is None, "the gradient of w13 needs x")
        nbytes = 0
        if grad_row_weights is not None:
            nbytes = ep_expert_ffn_backward_workspace(self.h, inter)
            if workspace is None:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            _dev(workspace, "workspace")
            _need(workspace.numel() * workspace.element_size() >= nbytes,
                  f"workspace must have {nbytes} bytes")
        else:
            workspace = None
        _here(grad_y, x, w13, w2, saved, h, row_weights, grad_gate_up, grad_x, grad_w13, grad_w2,
              grad_row_weights, workspace, self.workspace)
        _check(ep_expert_ffn_backward(
            self.h, _ptr(grad_y), _ptr(x), 1 if token_rows else 0, H, _ptr(w13), _ptr(w2), inter,
            _ptr(row_weights), _ptr(saved), _ptr(h), 1 if remake_h else 0, _ptr(grad_gate_up),
            _ptr(grad_x), EP_F32 if grad_dtype == torch.float32 else EP_BF16, _ptr(grad_w13),
            _ptr(grad_w2), _ptr(grad_row_weights), _ptr(workspace), nbytes, _stream()),
            "ep_expert_ffn_backward")
        return grad_x, grad_w13, grad_w2, grad_row_weights, grad_gate_up
