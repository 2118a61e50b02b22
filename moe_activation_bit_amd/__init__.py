"""Python binding of the MI355X fused SwiGLU + top-k weight + FP8/FP4 cast,
the stand-alone cast, the top-k gating and the weighted top-k reduce, and of
the operators of an MoE layer around them (RMS norm with FP8 output, routing,
the experts' products with 4-bit weights; grouped products, their gradients and
SwiGLU's from 8-bit checkpoints).

Argument marshalling only: every function here forwards to the C ABI in
``include/tk.h``, ``include/tk_layer.h`` and ``include/tk_expert.h`` (library
``libtk.so`` built from ``csrc/*.hip``) under the same name, through the small CPython extension ``_tkpy`` (``csrc/tk_py.c``,
a fraction of a microsecond per call where ctypes took a few).  All
arithmetic runs in the library's HIP kernels; there is no CPU fallback, and
calling a function whose library or extension is missing raises.

Tensor arguments may be torch tensors (their ``data_ptr()`` is passed) or raw
device addresses as ints; ``None`` is a null pointer.  ``stream`` defaults to
torch's current stream on the current device.
"""
from __future__ import annotations

import ctypes
import enum
import os
from typing import Any, Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtk.so")

__all__ = [
    "TkStatus", "TK_SCALE_FP32", "TK_SCALE_UE8M0", "TK_SCALE_FP32_COLMAJOR", "TK_SCALE_UE8M0_COLMAJOR",
    "TK_SCALE_UE8M0_PACKED", "TK_DTYPE_BF16", "TK_DTYPE_FP32", "TK_DTYPE_FP8", "TK_SCORE_SIGMOID", "TK_SCORE_SOFTMAX",
    "TK_RMSNORM_PARTS", "LIB_PATH", "load_library", "load_extension",
    "tk_init", "tk_swiglu_cast_fp8", "tk_swiglu_cast_fp4", "tk_swiglu_forward", "tk_cast_fp8", "tk_cast_fp4",
    "tk_topk_gate", "tk_moe_reduce", "tk_status_str", "tk_rmsnorm_cast_fp8", "tk_rmsnorm_backward", "tk_route",
    "tk_route_backward", "tk_expert_gemv_fp4", "TK_DTYPE_FP4", "tk_expert_gemm", "tk_expert_gemm_dgrad",
    "tk_expert_gemm_wgrad", "tk_swiglu_checkpoint_fp8", "tk_swiglu_backward",
]

TK_SCALE_FP32 = 0
TK_SCALE_UE8M0 = 1
TK_SCALE_FP32_COLMAJOR = 2
TK_SCALE_UE8M0_COLMAJOR = 3
TK_SCALE_UE8M0_PACKED = 4
TK_DTYPE_BF16 = 0
TK_DTYPE_FP32 = 1
TK_DTYPE_FP8 = 2
TK_DTYPE_FP4 = 3
TK_SCORE_SIGMOID = 0
TK_SCORE_SOFTMAX = 1
TK_RMSNORM_PARTS = 256


class TkStatus(enum.IntEnum):
    TK_OK = 0
    TK_ERR_INVALID_ARG = 1
    TK_ERR_UNSUPPORTED = 2
    TK_ERR_HIP = 3


_lib: Optional[ctypes.CDLL] = None

# the exported symbols and their C signatures, as declared in include/tk.h, include/tk_layer.h
# and include/tk_expert.h
_CAST_ARGS = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
              ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
              ctypes.c_void_p]
SIGNATURES = {
    "tk_init": (ctypes.c_int, [ctypes.c_int]),
    "tk_swiglu_cast_fp8": (ctypes.c_int, _CAST_ARGS),
    "tk_swiglu_cast_fp4": (ctypes.c_int, _CAST_ARGS),
    "tk_swiglu_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_cast_fp8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                   ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_cast_fp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                   ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_topk_gate": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_moe_reduce": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_float, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                     ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_topk_to_pos": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "tk_rmsnorm_cast_fp8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_int64, ctypes.c_float, ctypes.c_int64,
                                           ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_rmsnorm_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_route": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_route_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_expert_gemv_fp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                          ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                          ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                          ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_expert_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.c_void_p]),
    "tk_expert_gemm_dgrad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                            ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_expert_gemm_wgrad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                            ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                            ctypes.c_void_p, ctypes.c_void_p]),
    "tk_swiglu_checkpoint_fp8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tk_swiglu_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p]),
}


def load_library() -> ctypes.CDLL:
    """Load libtk.so (fails loudly when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build the HIP library first (__graft_entry__.build())")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


EXT_NAME = "_tkpy"  # the CPython extension that marshals arguments to libtk.so (csrc/tk_py.c)
_ext = None
_STATUS = tuple(TkStatus(i) for i in range(len(TkStatus)))


def _current_stream() -> int:
    import torch
    if torch.cuda.is_initialized():
        try:  # the handle alone: making torch's stream object around it takes 2.9 us of a small launch's 7
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:  # a torch without these two, which are not of its public interface
            pass
    return int(torch.cuda.current_stream().cuda_stream)


def load_extension():
    """Import the argument-marshalling extension (fails loudly when it has not
    been built); its default stream is torch's current stream."""
    global _ext
    if _ext is None:
        load_library()
        import importlib
        try:
            mod = importlib.import_module(f"{__name__}.{EXT_NAME}")
        except ImportError as e:
            raise RuntimeError(f"{EXT_NAME} is missing: build the package first (__graft_entry__.build())") from e
        mod._set_stream_getter(_current_stream)
        _ext = mod
    return _ext


# Pointer arguments: a torch tensor (its data_ptr()), an int address or None.
# stream: None (torch's current stream), an int handle or a torch stream.


def tk_init(device: int) -> TkStatus:
    return _STATUS[(_ext or load_extension()).tk_init(int(device))]


def tk_swiglu_cast_fp8(x, topk_weight, n, hidden, group_size, clamp_limit, scale_fmt, codes, scales,
                       clamped_count=None, stream=None) -> TkStatus:
    """See tk_swiglu_cast_fp8 in include/tk.h."""
    return _STATUS[(_ext or load_extension()).tk_swiglu_cast_fp8(
        x, topk_weight, n, hidden, group_size, clamp_limit, scale_fmt, codes, scales, clamped_count, stream)]


def tk_swiglu_cast_fp4(x, topk_weight, n, hidden, group_size, clamp_limit, scale_fmt, codes, scales,
                       clamped_count=None, stream=None) -> TkStatus:
    """See tk_swiglu_cast_fp4 in include/tk.h."""
    return _STATUS[(_ext or load_extension()).tk_swiglu_cast_fp4(
        x, topk_weight, n, hidden, group_size, clamp_limit, scale_fmt, codes, scales, clamped_count, stream)]


def tk_swiglu_forward(x, topk_weight, n, hidden, clamp_limit, y, clamped_count=None,
                      stream=None) -> TkStatus:
    """See tk_swiglu_forward in include/tk.h."""
    return _STATUS[(_ext or load_extension()).tk_swiglu_forward(x, topk_weight, n, hidden, clamp_limit, y,
                                                                  clamped_count, stream)]


def tk_cast_fp8(x, in_dtype, n, hidden, group_size, scale_fmt, codes, scales, stream=None) -> TkStatus:
    """See tk_cast_fp8 in include/tk.h."""
    return _STATUS[(_ext or load_extension()).tk_cast_fp8(x, in_dtype, n, hidden, group_size, scale_fmt, codes,
                                                            scales, stream)]


def tk_cast_fp4(x, in_dtype, n, hidden, group_size, scale_fmt, codes, scales, stream=None) -> TkStatus:
    """See tk_cast_fp4 in include/tk.h."""
    return _STATUS[(_ext or load_extension()).tk_cast_fp4(x, in_dtype, n, hidden, group_size, scale_fmt, codes,
                                                            scales, stream)]


def tk_topk_gate(scores, tokens, experts, k, n_group, topk_group, normalise, topk_idx, topk_weight,
                 stream=None) -> TkStatus:
    """See tk_topk_gate in include/tk.h."""
    return _STATUS[(_ext or load_extension()).tk_topk_gate(scores, tokens, experts, k, n_group, topk_group,
                                                             normalise, topk_idx, topk_weight, stream)]


def tk_moe_reduce(x, row_scale, pos, topk_weight, global_scale, tokens, k, hidden, n_rows, out_dtype, out,
                  stream=None) -> TkStatus:
    """See tk_moe_reduce in include/tk.h."""
    return _STATUS[(_ext or load_extension()).tk_moe_reduce(x, row_scale, pos, topk_weight, global_scale, tokens,
                                                              k, hidden, n_rows, out_dtype, out, stream)]


def tk_topk_to_pos(topk_idx, tokens, k, experts, pos, expert_offsets, stream=None) -> TkStatus:
    """See tk_topk_to_pos in include/tk.h."""
    return _STATUS[(_ext or load_extension()).tk_topk_to_pos(topk_idx, tokens, k, experts, pos, expert_offsets,
                                                               stream)]


def tk_rmsnorm_cast_fp8(x, residual, in_dtype, weight, n, hidden, eps, group_size, scale_fmt, residual_out, y, rstd,
                        codes, scales, stream=None) -> TkStatus:
    """See tk_rmsnorm_cast_fp8 in include/tk_layer.h."""
    return _STATUS[(_ext or load_extension()).tk_rmsnorm_cast_fp8(
        x, residual, in_dtype, weight, n, hidden, eps, group_size, scale_fmt, residual_out, y, rstd, codes, scales,
        stream)]


def tk_rmsnorm_backward(dy, h, in_dtype, weight, rstd, dresidual, n, hidden, dx, dweight, workspace,
                        stream=None) -> TkStatus:
    """See tk_rmsnorm_backward in include/tk_layer.h."""
    return _STATUS[(_ext or load_extension()).tk_rmsnorm_backward(dy, h, in_dtype, weight, rstd, dresidual, n, hidden,
                                                                  dx, dweight, workspace, stream)]


def tk_route(logits, in_dtype, bias, tokens, experts, k, n_group, topk_group, scoring, normalise, scale, topk_idx,
             topk_weight, stream=None) -> TkStatus:
    """See tk_route in include/tk_layer.h."""
    return _STATUS[(_ext or load_extension()).tk_route(logits, in_dtype, bias, tokens, experts, k, n_group, topk_group,
                                                       scoring, normalise, scale, topk_idx, topk_weight, stream)]


def tk_route_backward(dweight, topk_idx, logits, in_dtype, tokens, experts, k, scoring, normalise, scale, dlogits,
                      stream=None) -> TkStatus:
    """See tk_route_backward in include/tk_layer.h."""
    return _STATUS[(_ext or load_extension()).tk_route_backward(dweight, topk_idx, logits, in_dtype, tokens, experts, k,
                                                                scoring, normalise, scale, dlogits, stream)]


def tk_expert_gemv_fp4(x, x_scales, x_dtype, x_scale_fmt, x_group, topk_idx, tokens, k, x_slots, codes, scales,
                       scale_fmt, group_size, experts, out_features, in_features, out_dtype, out,
                       stream=None) -> TkStatus:
    """See tk_expert_gemv_fp4 in include/tk_layer.h."""
    return _STATUS[(_ext or load_extension()).tk_expert_gemv_fp4(
        x, x_scales, x_dtype, x_scale_fmt, x_group, topk_idx, tokens, k, x_slots, codes, scales, scale_fmt, group_size,
        experts, out_features, in_features, out_dtype, out, stream)]


def tk_expert_gemm(x, x_scales, x_dtype, x_scale_fmt, x_group, x_rows, row_index, expert_offsets, n_rows, w, w_scales,
                   w_dtype, w_scale_fmt, w_group, experts, out_features, in_features, out_dtype, out,
                   stream=None) -> TkStatus:
    """See tk_expert_gemm in include/tk_expert.h."""
    return _STATUS[(_ext or load_extension()).tk_expert_gemm(
        x, x_scales, x_dtype, x_scale_fmt, x_group, x_rows, row_index, expert_offsets, n_rows, w, w_scales, w_dtype,
        w_scale_fmt, w_group, experts, out_features, in_features, out_dtype, out, stream)]


def tk_expert_gemm_dgrad(dy, dy_rows, row_index, expert_offsets, n_rows, w, experts, out_features, in_features,
                         out_dtype, dx, stream=None) -> TkStatus:
    """See tk_expert_gemm_dgrad in include/tk_expert.h."""
    return _STATUS[(_ext or load_extension()).tk_expert_gemm_dgrad(
        dy, dy_rows, row_index, expert_offsets, n_rows, w, experts, out_features, in_features, out_dtype, dx, stream)]


def tk_expert_gemm_wgrad(dy, dy_rows, dy_index, x, x_scales, x_dtype, x_group, x_rows, x_index, expert_offsets, n_rows,
                         experts, out_features, in_features, accumulate, out_dtype, dw, stream=None) -> TkStatus:
    """See tk_expert_gemm_wgrad in include/tk_expert.h."""
    return _STATUS[(_ext or load_extension()).tk_expert_gemm_wgrad(
        dy, dy_rows, dy_index, x, x_scales, x_dtype, x_group, x_rows, x_index, expert_offsets, n_rows, experts,
        out_features, in_features, accumulate, out_dtype, dw, stream)]


def tk_swiglu_checkpoint_fp8(x, topk_weight, n, hidden, group_size, clamp_limit, scale_fmt, codes, scales, x_codes,
                             x_scales, stream=None) -> TkStatus:
    """See tk_swiglu_checkpoint_fp8 in include/tk_expert.h."""
    return _STATUS[(_ext or load_extension()).tk_swiglu_checkpoint_fp8(
        x, topk_weight, n, hidden, group_size, clamp_limit, scale_fmt, codes, scales, x_codes, x_scales, stream)]


def tk_swiglu_backward(dy, h, h_scales, h_dtype, scale_fmt, group_size, topk_weight, n, hidden, clamp_limit, dh,
                       dweight, y, stream=None) -> TkStatus:
    """See tk_swiglu_backward in include/tk_expert.h."""
    return _STATUS[(_ext or load_extension()).tk_swiglu_backward(
        dy, h, h_scales, h_dtype, scale_fmt, group_size, topk_weight, n, hidden, clamp_limit, dh, dweight, y, stream)]


def tk_status_str(status: int) -> str:
    return (_ext or load_extension()).tk_status_str(int(status))
