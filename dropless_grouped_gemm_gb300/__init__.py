"""GB300-native dropless MoE expert MLP: Python binding of libmoe.

Argument marshalling only: every step of the path runs in libmoe's CUDA
kernels (``csrc/``).  PyTorch supplies device memory and the current CUDA
stream.  There is no CPU fallback: if ``libmoe.so`` is missing or a call
fails, an exception is raised.

Functions mirror the C ABI in ``include/moe.h``:

    route_offsets      -> moe_route_offsets
    permute            -> moe_permute (moe_permute_tokens with row_of_pair)
    unpermute          -> moe_unpermute
    grouped_mlp_fwd    -> moe_grouped_mlp_fwd
    grouped_mlp_bwd    -> moe_grouped_mlp_bwd
    router_loss        -> moe_router_loss (and router_loss_bwd)
    router_select      -> moe_router_select (and router_select_bwd)
    grouped_linear     -> moe_grouped_linear (and grouped_linear_bwd)
    fp4_quantize       -> moe_fp4_quantize (and fp4_tensor_scale, fp4_permute,
                          fp4_quantize_weights, fp4_dequantize)
    fp4_linear         -> moe_fp4_linear (and fp4_linear_bwd)
    checkpoint_pack    -> moe_checkpoint_pack (and checkpoint_unpack,
                          permute_checkpoint, grouped_mlp_fwd_ckpt,
                          grouped_mlp_bwd_routed_ckpt)
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "ACT", "FLAG_SAVE_H", "DEV_BAD_EXPERT", "DEV_OVERFLOW", "DEV_TIMEOUT", "DEV_BAD_OFFSETS",
    "lib", "lib_path", "version", "last_launch_count", "route_workspace_size", "workspace_size",
    "route_offsets",
    "router_topk",
    "permute", "unpermute", "grouped_mlp_fwd", "grouped_mlp_bwd", "MoeError",
    "FLAG_MXFP8", "MxFwd", "mx_quantize_weights", "mx_quantize", "mx_buffers",
    "MxBwd", "mx_quantize_weights_rowwise", "mx_quantize_tiled", "mx_bwd_workspace_size", "grouped_mlp_bwd_mx",
    "grouped_mlp_bwd_routed", "router_grad_rows", "mx_quantize_weights2", "FLAG_ACCUMULATE_DW",
    "grouped_gemm", "activation", "activation_bwd", "grouped_mlp_fwd_gather",
    "grouped_mlp_bwd_routed_gather", "route_logits", "FLAG_MX_SEPARATE_DH_QUANT",
    "mx_bwd_workspace_layout", "set_pair_mma",
    "LINEAR_ACT", "router_loss", "router_loss_bwd", "router_loss_workspace_size", "grouped_linear",
    "grouped_linear_bwd", "grouped_linear_bwd_workspace_size", "grouped_linear_plan", "checkpoint_pack",
    "checkpoint_unpack", "permute_checkpoint", "grouped_mlp_fwd_ckpt",
    "grouped_mlp_bwd_routed_ckpt",
    "SCORE", "router_select", "router_select_bwd",
    "FP4", "fp4_scale_bytes", "fp4_tensor_scale", "fp4_quantize", "fp4_permute",
    "fp4_quantize_weights", "fp4_dequantize", "fp4_linear", "fp4_linear_plan", "fp4_linear_bwd",
    "fp4_linear_bwd_workspace_size",
]

ACT = {"swiglu": 0, "geglu": 1, "srelu": 2}
LINEAR_ACT = {**ACT, "none": 3, "relu": 4, "silu": 5, "gelu": 6}
SCORE = {"softmax": 0, "sigmoid": 1}
FP4 = {"nvfp4": 0, "mxfp4": 1}
FLAG_SAVE_H = 1
FLAG_MXFP8 = 2
FLAG_ACCUMULATE_DW = 4
FLAG_MX_SEPARATE_DH_QUANT = 8
DEV_BAD_EXPERT, DEV_OVERFLOW, DEV_TIMEOUT, DEV_BAD_OFFSETS = 1, 2, 4, 8
_RC = {-1: "MOE_E_NULL", -2: "MOE_E_ALIGN", -3: "MOE_E_SIZE", -4: "MOE_E_ARG",
       -5: "MOE_E_CUDA", -6: "MOE_E_WORKSPACE"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


class MoeError(RuntimeError):
    pass


class MxFwd(ctypes.Structure):
    """moe_mx_fwd: MXFP8 buffers of the forward (device pointers)."""
    _fields_ = [("w2_q", ctypes.c_void_p), ("w2_s", ctypes.c_void_p), ("a_q", ctypes.c_void_p),
                ("a_s", ctypes.c_void_p), ("a_qT", ctypes.c_void_p), ("a_sT", ctypes.c_void_p),
                ("y_q", ctypes.c_void_p), ("y_s", ctypes.c_void_p)]


class MxBwd(ctypes.Structure):
    """moe_mx_bwd: MXFP8 operands and workspace of the backward (device pointers)."""
    _fields_ = [("a_qT", ctypes.c_void_p), ("a_sT", ctypes.c_void_p), ("w2_q", ctypes.c_void_p),
                ("w2_s", ctypes.c_void_p), ("w1_q", ctypes.c_void_p), ("w1_s", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t),
                ("dx_q", ctypes.c_void_p), ("dx_s", ctypes.c_void_p)]


def lib_path() -> str:
    return os.path.join(_HERE, "libmoe.so")


def lib():
    """The loaded libmoe (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        p = lib_path()
        if not os.path.exists(p):
            raise MoeError(f"{p} is missing: build it with dropless_grouped_gemm_gb300.build.build()")
        L = ctypes.CDLL(p)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_version.restype = ctypes.c_char_p
        L.moe_version.argtypes = []
        L.moe_last_launch_count.restype = i32
        L.moe_last_launch_count.argtypes = []
        L.moe_router_topk.restype = i32
        L.moe_router_topk.argtypes = [vp, i32, i32, i32, vp, vp, vp]
        L.moe_route_logits.restype = i32
        L.moe_route_logits.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                       sz, vp, vp]
        L.moe_route_workspace_size.restype = sz
        L.moe_route_workspace_size.argtypes = [i32, i32, i32]
        L.moe_route_offsets.restype = i32
        L.moe_route_offsets.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz,
                                        vp, vp]
        L.moe_permute.restype = i32
        L.moe_permute.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp]
        L.moe_permute_tokens.restype = i32
        L.moe_permute_tokens.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
        L.moe_unpermute.restype = i32
        L.moe_unpermute.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
        L.moe_grouped_mlp_fwd.restype = i32
        L.moe_grouped_mlp_fwd.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, i32, i32, vp, vp, vp,
                                          vp, vp, vp, vp]
        L.moe_mx_quantize_weights.restype = i32
        L.moe_mx_quantize_weights.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
        L.moe_mx_quantize.restype = i32
        L.moe_mx_quantize.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp]
        L.moe_set_launch_events.restype = i32
        L.moe_set_launch_events.argtypes = [vp, i32]
        L.moe_launch_events_used.restype = i32
        L.moe_launch_events_used.argtypes = []
        L.moe_grouped_mlp_bwd.restype = i32
        L.moe_grouped_mlp_bwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, i32, i32,
                                          vp, vp, vp, vp, vp, vp, vp]
        L.moe_mx_quantize_weights2.restype = i32
        L.moe_mx_quantize_weights2.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp]
        L.moe_mx_quantize_tiled.restype = i32
        L.moe_mx_quantize_tiled.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp]
        L.moe_mx_quantize_weights_rowwise.restype = i32
        L.moe_mx_quantize_weights_rowwise.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp]
        L.moe_mx_bwd_workspace_size.restype = sz
        L.moe_mx_bwd_workspace_size.argtypes = [i32, i32, i32, i32]
        L.moe_set_pair_mma.restype = i32
        L.moe_set_pair_mma.argtypes = [i32]
        L.moe_mx_bwd_workspace_layout.restype = sz
        L.moe_mx_bwd_workspace_layout.argtypes = [i32, i32, i32, i32, vp]
        L.moe_workspace_size.restype = sz
        L.moe_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32]
        L.moe_grouped_mlp_bwd_mx.restype = i32
        L.moe_grouped_mlp_bwd_mx.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp,
                                             vp, vp, vp, vp, vp]
        L.moe_grouped_mlp_bwd_routed.restype = i32
        L.moe_grouped_mlp_bwd_routed.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp,
                                                 vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_grouped_mlp_fwd_gather.restype = i32
        L.moe_grouped_mlp_fwd_gather.argtypes = [vp, i32, i32, vp, vp, i32, i32, i32, i32, vp, vp,
                                                 i32, i32, vp, vp, vp, vp, vp, vp]
        L.moe_grouped_mlp_bwd_routed_gather.restype = i32
        L.moe_grouped_mlp_bwd_routed_gather.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, i32, i32,
                                                        i32, i32, vp, vp, i32, i32, vp, vp, vp, vp,
                                                        vp, vp, vp, vp, vp]
        L.moe_grouped_gemm.restype = i32
        L.moe_grouped_gemm.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, vp]
        L.moe_activation.restype = i32
        L.moe_activation.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp]
        L.moe_activation_bwd.restype = i32
        L.moe_activation_bwd.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp]
        L.moe_router_grad_rows.restype = i32
        L.moe_router_grad_rows.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp]
        L.moe_router_loss_workspace_size.restype = sz
        L.moe_router_loss_workspace_size.argtypes = [i32, i32, i32]
        L.moe_router_loss.restype = i32
        L.moe_router_loss.argtypes = [vp, i32, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp,
                                      sz, vp, vp]
        L.moe_router_loss_bwd.restype = i32
        L.moe_router_loss_bwd.argtypes = [vp, i32, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp,
                                          vp, vp, vp, i32, vp]
        f32 = ctypes.c_float
        L.moe_router_select.restype = i32
        L.moe_router_select.argtypes = [vp, i32, i32, i32, i32, i32, vp, i32, i32, i32, i32, f32,
                                        vp, vp, vp]
        L.moe_router_select_bwd.restype = i32
        L.moe_router_select_bwd.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, f32,
                                            i32, vp, i32, vp]
        i64 = ctypes.c_longlong
        L.moe_fp4_scale_bytes.restype = sz
        L.moe_fp4_scale_bytes.argtypes = [i64, i32, i32, i32]
        L.moe_fp4_tensor_scale.restype = i32
        L.moe_fp4_tensor_scale.argtypes = [vp, i32, i64, vp, vp]
        L.moe_fp4_tensor_scale_rows.restype = i32
        L.moe_fp4_tensor_scale_rows.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp]
        L.moe_fp4_quantize.restype = i32
        L.moe_fp4_quantize.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp]
        L.moe_fp4_permute.restype = i32
        L.moe_fp4_permute.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp,
                                      vp]
        L.moe_fp4_quantize_weights.restype = i32
        L.moe_fp4_quantize_weights.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        L.moe_fp4_dequantize.restype = i32
        L.moe_fp4_dequantize.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, i32, vp, i32, vp, vp]
        L.moe_fp4_linear.restype = i32
        L.moe_fp4_linear.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, i32,
                                     vp, vp, vp, i32, vp, vp, vp, vp]
        L.moe_fp4_linear_plan.restype = i32
        L.moe_fp4_linear_plan.argtypes = [i32, i32, i32, i32, i32, vp]
        L.moe_fp4_linear_bwd_workspace_size.restype = sz
        L.moe_fp4_linear_bwd_workspace_size.argtypes = [i32, i32, i32, i32]
        L.moe_fp4_linear_bwd.restype = i32
        L.moe_fp4_linear_bwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, i32, i32,
                                         i32, i32, vp, vp, vp, vp, vp, sz, vp, vp]
        L.moe_grouped_linear.restype = i32
        L.moe_grouped_linear.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, vp, i32, vp, vp, vp,
                                         i32, vp, vp]
        L.moe_grouped_linear_plan.restype = i32
        L.moe_grouped_linear_plan.argtypes = [i32, i32, i32, i32, i32, i32, vp]
        L.moe_grouped_linear_bwd_workspace_size.restype = sz
        L.moe_grouped_linear_bwd_workspace_size.argtypes = [i32, i32, i32]
        L.moe_grouped_linear_bwd.restype = i32
        L.moe_grouped_linear_bwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, i32, i32,
                                             vp, vp, vp, vp, vp, sz, vp, vp]
        L.moe_checkpoint_pack.restype = i32
        L.moe_checkpoint_pack.argtypes = [vp, i32, i32, vp, vp, vp]
        L.moe_checkpoint_unpack.restype = i32
        L.moe_checkpoint_unpack.argtypes = [vp, vp, i32, i32, vp, vp]
        L.moe_permute_checkpoint.restype = i32
        L.moe_permute_checkpoint.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
        L.moe_grouped_mlp_fwd_ckpt.restype = i32
        L.moe_grouped_mlp_fwd_ckpt.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, i32, vp, vp, vp,
                                               vp, vp, vp]
        L.moe_grouped_mlp_bwd_routed_ckpt.restype = i32
        L.moe_grouped_mlp_bwd_routed_ckpt.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32,
                                                      i32, vp, vp, i32, i32, vp, vp, vp, vp, vp,
                                                      vp, vp, vp]
        L.moe_selftest_bounded_wait.restype = i32
        L.moe_selftest_bounded_wait.argtypes = [i32, vp, vp, vp]
        _LIB = L
    return _LIB


def version() -> str:
    return lib().moe_version().decode()


def last_launch_count() -> int:
    return int(lib().moe_last_launch_count())


def _check(rc: int, what: str):
    if rc != 0:
        raise MoeError(f"{what} failed: {_RC.get(rc, rc)}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _current_stream() -> int:
    """Handle of the current stream of the current device.  (The raw getter
    takes 0.1 us where building a Stream object takes 3.)"""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return torch.cuda.current_stream().cuda_stream
    return raw(torch.cuda.current_device())


def _stream(stream=None):
    return _current_stream() if stream is None else stream.cuda_stream


def _need(t, dtype, name, ndim=None):
    if t is None:
        return
    if not t.is_cuda:
        raise MoeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise MoeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise MoeError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise MoeError(f"{name} must have {ndim} dims")


# Fresh error words: zeroed 64 at a time, each handed out once, per device and
# stream (their zeroing is ordered before the calls on that stream).  A zeroed
# tensor of its own costs a call 10 us and a launch.
_ERR_WORDS: dict = {}


def _err_word(err, device, stream=None):
    if err is None:
        if stream is not None and stream.cuda_stream != _current_stream():
            with torch.cuda.stream(stream):     # zeroed in the call's own order
                return _err_word(None, device)
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(1, dtype=torch.int32, device=device)
        key = (device.index, _current_stream())
        try:
            return _ERR_WORDS[key].pop()
        except (KeyError, IndexError):
            words = _ERR_WORDS.setdefault(key, [])
            with torch.inference_mode(False):   # ordinary tensors: later calls get them too
                words.extend(torch.zeros(64, dtype=torch.int32, device=device).split(1))
            return words.pop()
    _need(err, torch.int32, "err")
    return err


# What a call makes for itself comes from the memory of the stream that it runs
# on: a block that the current stream has freed, with work on it still queued
# there, is no block that another stream may write.

def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """An output of a call on ``stream``.  The caller reads it on the current
    stream, so it is kept from reuse until that stream too is past its end."""
    if stream is None or stream.cuda_stream == _current_stream():
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _workspace(given, nbytes: int, device, stream=None) -> torch.Tensor:
    """The caller's workspace (any type; the library checks its size), or a new one."""
    if given is None:
        return _scratch(nbytes, device, stream)
    if not given.is_cuda or not given.is_contiguous():
        raise MoeError("workspace must be a contiguous CUDA tensor")
    return given


def _scratch(nbytes: int, device, stream=None) -> torch.Tensor:
    """Workspace of a call on ``stream`` alone."""
    if stream is None or stream.cuda_stream == _current_stream():
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def router_topk(logits: torch.Tensor, k: int, stream=None):
    """Top-k experts per token and their softmax weights (moe_router_topk).
    Returns (topk_idx int32 [T, k], probs float32 [T, k])."""
    _need(logits, torch.float32, "logits", 2)
    T, E = logits.shape
    idx = _empty((T, k), torch.int32, logits.device, stream)
    probs = _empty((T, k), torch.float32, logits.device, stream)
    rc = lib().moe_router_topk(_ptr(logits), T, E, k, _ptr(idx), _ptr(probs), _stream(stream))
    _check(rc, "moe_router_topk")
    return idx, probs


def route_workspace_size(T: int, k: int, E: int) -> int:
    return int(lib().moe_route_workspace_size(T, k, E))


def workspace_size(T: int, k: int, E: int, M_cap: int, d: int, n: int, act: str = "swiglu",
                   mxfp8: bool = False) -> int:
    """Device scratch for one layer's calls (moe_workspace_size): the routing
    layout's and, with ``mxfp8``, the MXFP8 backward's, one buffer for both."""
    return int(lib().moe_workspace_size(T, k, E, M_cap, d, n, ACT[act],
                                        FLAG_MXFP8 if mxfp8 else 0))


def route_offsets(topk_idx: torch.Tensor, E: int, align: int = 1, M_cap: int | None = None,
                  err: torch.Tensor | None = None, out: dict | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Routing layout on the device (see moe_route_offsets).  Returns a dict
    of device tensors: counts, offsets, row_of_pair, pair_of_row, true_total,
    err."""
    _need(topk_idx, torch.int32, "topk_idx", 2)
    T, k = topk_idx.shape
    if M_cap is None:
        M_cap = T * k + E * (align - 1)
    dev = topk_idx.device
    o = out if out is not None else {
        "counts": _empty(E, torch.int32, dev, stream),
        "offsets": _empty(E + 1, torch.int32, dev, stream),
        "row_of_pair": _empty(T * k, torch.int32, dev, stream),
        "pair_of_row": _empty(M_cap, torch.int32, dev, stream),
        "true_total": _empty(1, torch.int32, dev, stream),
    }
    o["err"] = _err_word(err if err is not None else o.get("err"), dev, stream)
    ws_bytes = route_workspace_size(T, k, E)
    workspace = _workspace(workspace, ws_bytes, dev, stream)
    rc = lib().moe_route_offsets(_ptr(topk_idx), T, k, E, align, M_cap, _ptr(o["counts"]),
                                 _ptr(o["offsets"]), _ptr(o["row_of_pair"]), _ptr(o["pair_of_row"]),
                                 _ptr(o["true_total"]), _ptr(workspace), workspace.numel(),
                                 _ptr(o["err"]), _stream(stream))
    _check(rc, "moe_route_offsets")
    return o


def route_logits(logits: torch.Tensor, k: int, align: int = 1, M_cap: int | None = None,
                 err: torch.Tensor | None = None, out: dict | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> dict:
    """The router fused into the routing layout (see moe_route_logits):
    from logits [T, E] float32 to the dict of route_offsets plus topk_idx
    [T, k] and probs [T, k]."""
    _need(logits, torch.float32, "logits", 2)
    T, E = logits.shape
    if M_cap is None:
        M_cap = T * k + E * (align - 1)
    dev = logits.device
    o = out if out is not None else {
        "topk_idx": _empty((T, k), torch.int32, dev, stream),
        "probs": _empty((T, k), torch.float32, dev, stream),
        "counts": _empty(E, torch.int32, dev, stream),
        "offsets": _empty(E + 1, torch.int32, dev, stream),
        "row_of_pair": _empty(T * k, torch.int32, dev, stream),
        "pair_of_row": _empty(M_cap, torch.int32, dev, stream),
        "true_total": _empty(1, torch.int32, dev, stream),
    }
    o["err"] = _err_word(err if err is not None else o.get("err"), dev, stream)
    ws_bytes = route_workspace_size(T, k, E)
    workspace = _workspace(workspace, ws_bytes, dev, stream)
    rc = lib().moe_route_logits(_ptr(logits), T, E, k, align, M_cap, _ptr(o["topk_idx"]),
                                _ptr(o["probs"]), _ptr(o["counts"]), _ptr(o["offsets"]),
                                _ptr(o["row_of_pair"]), _ptr(o["pair_of_row"]),
                                _ptr(o["true_total"]), _ptr(workspace), workspace.numel(),
                                _ptr(o["err"]), _stream(stream))
    _check(rc, "moe_route_logits")
    return o


def permute(src: torch.Tensor, pair_of_row: torch.Tensor, k: int, scale: torch.Tensor | None = None,
            out: torch.Tensor | None = None, stream=None,
            row_of_pair: torch.Tensor | None = None) -> torch.Tensor:
    """Expert-major gather (see moe_permute).  With ``row_of_pair`` (the
    routing layout's inverse map) the copy runs in token order
    (moe_permute_tokens), reading each token row once."""
    _need(src, torch.bfloat16, "src", 2)
    _need(pair_of_row, torch.int32, "pair_of_row")
    _need(row_of_pair, torch.int32, "row_of_pair")
    _need(scale, torch.float32, "scale")
    T, d = src.shape
    M_cap = pair_of_row.numel()
    if out is None:
        out = _empty((M_cap, d), torch.bfloat16, src.device, stream)
    _need(out, torch.bfloat16, "out", 2)
    if row_of_pair is not None:
        if row_of_pair.numel() != T * k:
            raise MoeError("row_of_pair must hold T*k entries")
        rc = lib().moe_permute_tokens(_ptr(src), _ptr(scale), _ptr(row_of_pair), _ptr(pair_of_row),
                                      T, k, d, M_cap, _ptr(out), _stream(stream))
        _check(rc, "moe_permute_tokens")
        return out
    rc = lib().moe_permute(_ptr(src), _ptr(scale), _ptr(pair_of_row), T, k, d, M_cap, _ptr(out),
                           _stream(stream))
    _check(rc, "moe_permute")
    return out


def unpermute(src: torch.Tensor, row_of_pair: torch.Tensor, T: int, k: int,
              probs: torch.Tensor | None = None, out: torch.Tensor | None = None,
              dO: torch.Tensor | None = None, dprobs: torch.Tensor | None = None,
              combine: bool = True, stream=None):
    """Combine and/or router-score gradient (see moe_unpermute).  Returns
    (out, dprobs); either may be None."""
    _need(src, torch.bfloat16, "src", 2)
    _need(row_of_pair, torch.int32, "row_of_pair")
    _need(probs, torch.float32, "probs")
    _need(dO, torch.bfloat16, "dO")
    d = src.shape[1]
    if combine and out is None:
        out = _empty((T, d), torch.bfloat16, src.device, stream)
    if not combine:
        out = None
    if dO is not None and dprobs is None:
        dprobs = _empty((T, k), torch.float32, src.device, stream)
    _need(out, torch.bfloat16, "out")
    _need(dprobs, torch.float32, "dprobs")
    rc = lib().moe_unpermute(_ptr(src), _ptr(probs), _ptr(row_of_pair), T, k, d, src.shape[0],
                             _ptr(out),
                             _ptr(dO), _ptr(dprobs), _stream(stream))
    _check(rc, "moe_unpermute")
    return out, dprobs


def grouped_mlp_fwd(x_perm: torch.Tensor, offsets: torch.Tensor, W1: torch.Tensor,
                    W2: torch.Tensor, act: str = "swiglu", save_h: bool = False,
                    h_saved: torch.Tensor | None = None, a: torch.Tensor | None = None,
                    y_perm: torch.Tensor | None = None, err: torch.Tensor | None = None,
                    mx: dict | None = None, amax: torch.Tensor | None = None, stream=None):
    """Grouped expert MLP forward (see moe_grouped_mlp_fwd).  With ``mx`` (a
    dict of uint8 device tensors w2_q, w2_s, a_q, a_s and optionally a_qT,
    a_sT; see ``mx_buffers``) the MXFP8 path runs.  ``amax`` (a float32
    device tensor of one element) is raised to max |A|.  Returns
    (h_saved or None, a, y_perm, err)."""
    if amax is not None:
        _need(amax, torch.float32, "amax")
    _need(x_perm, torch.bfloat16, "x_perm", 2)
    _need(offsets, torch.int32, "offsets", 1)
    _need(W1, torch.bfloat16, "W1", 3)
    _need(W2, torch.bfloat16, "W2", 3)
    M_cap, d = x_perm.shape
    E, n, d2 = W2.shape
    n1 = n if act == "srelu" else 2 * n
    if d2 != d or tuple(W1.shape) != (E, d, n1) or offsets.numel() != E + 1:
        raise MoeError("inconsistent shapes")
    dev = x_perm.device
    if save_h and h_saved is None:
        h_saved = _empty((M_cap, n1), torch.bfloat16, dev, stream)
    if a is None:
        a = _empty((M_cap, n), torch.bfloat16, dev, stream)
    if y_perm is None:
        y_perm = _empty((M_cap, d), torch.bfloat16, dev, stream)
    err = _err_word(err, dev, stream)
    flags = FLAG_SAVE_H if save_h else 0
    mxs = None
    if mx is not None:
        names = ("w2_q", "w2_s", "a_q", "a_s", "a_qT", "a_sT", "y_q", "y_s")
        for k_ in names:
            _need(mx.get(k_), torch.uint8, k_)
        mxs = MxFwd(*[(mx[k_].data_ptr() if mx.get(k_) is not None else None) for k_ in names])
        flags |= FLAG_MXFP8
    rc = lib().moe_grouped_mlp_fwd(_ptr(x_perm), _ptr(offsets), E, M_cap, d, n, _ptr(W1), _ptr(W2),
                                   ACT[act], flags, _ptr(h_saved) if save_h else None, _ptr(a),
                                   _ptr(y_perm), ctypes.byref(mxs) if mxs is not None else None,
                                   _ptr(amax), _ptr(err), _stream(stream))
    _check(rc, "moe_grouped_mlp_fwd")
    return (h_saved if save_h else None), a, y_perm, err


def grouped_mlp_fwd_gather(x: torch.Tensor, pair_of_row: torch.Tensor, k: int,
                           offsets: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                           act: str = "swiglu", save_h: bool = False, h_saved=None, a=None,
                           y_perm=None, err=None, amax=None, stream=None):
    """Grouped expert MLP forward reading the token rows of x [T, d] through
    the routing map (moe_grouped_mlp_fwd_gather): no permuted copy of x.
    Returns (h_saved or None, a, y_perm, err) like ``grouped_mlp_fwd``."""
    if amax is not None:
        _need(amax, torch.float32, "amax")
    _need(x, torch.bfloat16, "x", 2)
    _need(pair_of_row, torch.int32, "pair_of_row", 1)
    _need(offsets, torch.int32, "offsets", 1)
    _need(W1, torch.bfloat16, "W1", 3)
    _need(W2, torch.bfloat16, "W2", 3)
    T, d = x.shape
    M_cap = pair_of_row.numel()
    E, n, d2 = W2.shape
    n1 = n if act == "srelu" else 2 * n
    if d2 != d or tuple(W1.shape) != (E, d, n1) or offsets.numel() != E + 1:
        raise MoeError("inconsistent shapes")
    dev = x.device
    if save_h and h_saved is None:
        h_saved = _empty((M_cap, n1), torch.bfloat16, dev, stream)
    if a is None:
        a = _empty((M_cap, n), torch.bfloat16, dev, stream)
    if y_perm is None:
        y_perm = _empty((M_cap, d), torch.bfloat16, dev, stream)
    err = _err_word(err, dev, stream)
    if T == 0:      # the library reads nothing of x then, but needs an address
        x = _empty((1, d), torch.bfloat16, dev, stream)
    rc = lib().moe_grouped_mlp_fwd_gather(
        _ptr(x), T, k, _ptr(pair_of_row), _ptr(offsets), E, M_cap, d, n, _ptr(W1), _ptr(W2),
        ACT[act], FLAG_SAVE_H if save_h else 0, _ptr(h_saved) if save_h else None, _ptr(a),
        _ptr(y_perm), _ptr(amax), _ptr(err), _stream(stream))
    _check(rc, "moe_grouped_mlp_fwd_gather")
    return (h_saved if save_h else None), a, y_perm, err


def _bwd_flags(accumulate_dw: bool, dW1, dW2) -> int:
    if not accumulate_dw:
        return 0
    if dW1 is None or dW2 is None:
        raise ValueError("accumulate_dw needs the dW1 and dW2 to accumulate into")
    return FLAG_ACCUMULATE_DW


def grouped_mlp_bwd(x_perm, h_saved, a, dy_perm, offsets, W1, W2, act: str = "swiglu",
                    dh=None, dx_perm=None, dW1=None, dW2=None, err=None, amax=None, stream=None,
                    accumulate_dw: bool = False):
    """Grouped expert MLP backward (see moe_grouped_mlp_bwd).  Returns
    (dh, dx_perm, dW1, dW2, err).  accumulate_dw: add this step's weight
    gradients to the given dW1, dW2 (MOE_FLAG_ACCUMULATE_DW)."""
    flags = _bwd_flags(accumulate_dw, dW1, dW2)
    for t, nm in ((x_perm, "x_perm"), (h_saved, "h_saved"), (a, "a"), (dy_perm, "dy_perm"),
                  (W1, "W1"), (W2, "W2")):
        _need(t, torch.bfloat16, nm)
    _need(offsets, torch.int32, "offsets", 1)
    M_cap, d = x_perm.shape
    E, n, _ = W2.shape
    n1 = n if act == "srelu" else 2 * n
    dev = x_perm.device
    if dh is None:
        dh = _empty((M_cap, n1), torch.bfloat16, dev, stream)
    if dx_perm is None:
        dx_perm = _empty((M_cap, d), torch.bfloat16, dev, stream)
    if dW1 is None:
        dW1 = _empty((E, d, n1), torch.bfloat16, dev, stream)
    if dW2 is None:
        dW2 = _empty((E, n, d), torch.bfloat16, dev, stream)
    err = _err_word(err, dev, stream)
    rc = lib().moe_grouped_mlp_bwd(_ptr(x_perm), _ptr(h_saved), _ptr(a), _ptr(dy_perm),
                                   _ptr(offsets), E, M_cap, d, n, _ptr(W1), _ptr(W2), ACT[act], flags,
                                   _ptr(dh), _ptr(dx_perm), _ptr(dW1), _ptr(dW2), _ptr(amax),
                                   _ptr(err), _stream(stream))
    _check(rc, "moe_grouped_mlp_bwd")
    return dh, dx_perm, dW1, dW2, err


def mx_buffers(E: int, n: int, d: int, M_cap: int, device, transposed: bool = True,
               quantize_y: bool = False) -> dict:
    """Allocate the uint8 buffers of moe_mx_fwd (sizes as moe.h states)."""
    u8 = torch.uint8
    b = {"w2_q": torch.empty((E, n, d), dtype=u8, device=device),
         "w2_s": torch.empty(E * (n // 32) * d, dtype=u8, device=device),
         "a_q": torch.empty((M_cap, n), dtype=u8, device=device),
         "a_s": torch.empty((M_cap // 32) * (n // 128) * 512, dtype=u8, device=device)}
    if transposed:
        b["a_qT"] = torch.empty((n, M_cap), dtype=u8, device=device)
        b["a_sT"] = torch.empty((n, M_cap // 32), dtype=u8, device=device)
    if quantize_y:
        b["y_q"] = torch.empty((M_cap, d), dtype=u8, device=device)
        b["y_s"] = torch.empty((M_cap, d // 32), dtype=u8, device=device)
    return b


def _offsets_arg(offsets, E):
    if offsets is None:
        return None
    _need(offsets, torch.int32, "offsets", 1)
    if offsets.numel() != E + 1:
        raise ValueError(f"offsets has {offsets.numel()} entries, want E+1 = {E + 1}")
    return offsets


def mx_quantize_weights(W2: torch.Tensor, w2_q: torch.Tensor | None = None,
                        w2_s: torch.Tensor | None = None, stream=None, offsets=None):
    """MXFP8 codes and MMA-tiled scales of W2 [E, n, d] (moe_mx_quantize_weights).
    With the routing ``offsets``, experts without rows are skipped (left as
    they were in w2_q / w2_s)."""
    _need(W2, torch.bfloat16, "W2", 3)
    E, n, d = W2.shape
    offsets = _offsets_arg(offsets, E)
    if w2_q is None:
        w2_q = _empty((E, n, d), torch.uint8, W2.device, stream)
    if w2_s is None:
        w2_s = _empty(E * (n // 32) * d, torch.uint8, W2.device, stream)
    _need(w2_q, torch.uint8, "w2_q")
    _need(w2_s, torch.uint8, "w2_s")
    rc = lib().moe_mx_quantize_weights(_ptr(W2), E, n, d, _ptr(offsets), _ptr(w2_q), _ptr(w2_s),
                                       _stream(stream))
    _check(rc, "moe_mx_quantize_weights")
    return w2_q, w2_s


def mx_quantize(src: torch.Tensor, offsets: torch.Tensor, transposed: bool = True,
                err: torch.Tensor | None = None, stream=None):
    """Group-aware MXFP8 quantisation (moe_mx_quantize).  Returns
    (q, s, qT, sT, err); qT/sT are None unless ``transposed``."""
    _need(src, torch.bfloat16, "src", 2)
    _need(offsets, torch.int32, "offsets", 1)
    rows, cols = src.shape
    dev = src.device
    q = _empty((rows, cols), torch.uint8, dev, stream)
    s = _empty((rows, cols // 32), torch.uint8, dev, stream)
    qT = _empty((cols, rows), torch.uint8, dev, stream) if transposed else None
    sT = _empty((cols, rows // 32), torch.uint8, dev, stream) if transposed else None
    err = _err_word(err, dev, stream)
    rc = lib().moe_mx_quantize(_ptr(src), rows, cols, _ptr(offsets), offsets.numel() - 1, _ptr(q),
                               _ptr(s), _ptr(qT), _ptr(sT), _ptr(err), _stream(stream))
    _check(rc, "moe_mx_quantize")
    return q, s, qT, sT, err


def mx_quantize_tiled(src: torch.Tensor, offsets: torch.Tensor, rowwise: bool = True,
                      transposed: bool = True, err: torch.Tensor | None = None, stream=None):
    """Group-aware MXFP8 quantisation with the scales in the block-scaled
    GEMM's layouts (moe_mx_quantize_tiled).  Returns (q, s, qT, sT, err);
    q/s are None unless ``rowwise``, qT/sT None unless ``transposed``; s and
    sT are rows*cols/8 bytes each."""
    _need(src, torch.bfloat16, "src", 2)
    _need(offsets, torch.int32, "offsets", 1)
    if not (rowwise or transposed):
        raise ValueError("at least one copy")
    rows, cols = src.shape
    dev = src.device
    u8 = torch.uint8
    q = _empty((rows, cols), u8, dev, stream) if rowwise else None
    s = _empty(rows * cols // 8, u8, dev, stream) if rowwise else None
    qT = _empty((cols, rows), u8, dev, stream) if transposed else None
    sT = _empty(rows * cols // 8, u8, dev, stream) if transposed else None
    err = _err_word(err, dev, stream)
    rc = lib().moe_mx_quantize_tiled(_ptr(src), rows, cols, _ptr(offsets), offsets.numel() - 1,
                                     _ptr(q), _ptr(s), _ptr(qT), _ptr(sT), _ptr(err),
                                     _stream(stream))
    _check(rc, "moe_mx_quantize_tiled")
    return q, s, qT, sT, err


def mx_quantize_weights_rowwise(W: torch.Tensor, q: torch.Tensor | None = None,
                                s: torch.Tensor | None = None, stream=None, offsets=None):
    """MXFP8 codes of a weight with blocks along its last axis and scales in
    weight tiles (moe_mx_quantize_weights_rowwise); W is [E, R, K] or [R, K].
    With the routing ``offsets`` (W then [E, R, K]), experts without rows
    are skipped (left as they were in q / s)."""
    _need(W, torch.bfloat16, "W")
    K = W.shape[-1]
    rows = W.numel() // K
    E = W.shape[0] if offsets is not None else 0
    if offsets is not None and W.dim() != 3:
        raise ValueError("offsets needs W as [E, R, K]")
    offsets = _offsets_arg(offsets, E) if offsets is not None else None
    if q is None:
        q = _empty(tuple(W.shape), torch.uint8, W.device, stream)
    if s is None:
        s = _empty(rows * K // 32, torch.uint8, W.device, stream)
    _need(q, torch.uint8, "q")
    _need(s, torch.uint8, "s")
    rc = lib().moe_mx_quantize_weights_rowwise(_ptr(W), rows, K, _ptr(offsets), E, _ptr(q), _ptr(s),
                                               _stream(stream))
    _check(rc, "moe_mx_quantize_weights_rowwise")
    return q, s


def mx_bwd_workspace_size(M_cap: int, d: int, n: int, act: str = "swiglu") -> int:
    return int(lib().moe_mx_bwd_workspace_size(M_cap, d, n, ACT[act]))


PAIR_NEVER, PAIR_AUTO, PAIR_ALWAYS = 0, 1, 2


def set_pair_mma(mode: int) -> int:
    """moe_set_pair_mma: 0 never, 1 automatic (default), 2 always pair the
    two CTAs of a cluster with 2-SM MMAs; returns the previous mode."""
    rc = int(lib().moe_set_pair_mma(int(mode)))
    _check(rc if rc < 0 else 0, "moe_set_pair_mma")
    return rc


MX_BWD_SECTIONS = ("dy_q", "dy_s", "dy_qT", "dy_sT", "x_qT", "x_sT", "a_sT", "dh_q", "dh_s",
                   "dh_qT", "dh_sT")


def mx_bwd_workspace_layout(M_cap: int, d: int, n: int, act: str = "swiglu") -> dict:
    """Byte offsets of the MXFP8 backward's quantised operands inside its
    workspace (moe_mx_bwd_workspace_layout), by section name, plus "bytes"."""
    offs = (ctypes.c_size_t * len(MX_BWD_SECTIONS))()
    total = int(lib().moe_mx_bwd_workspace_layout(M_cap, d, n, ACT[act], offs))
    if total == 0:
        raise MoeError("moe_mx_bwd_workspace_layout: invalid sizes")
    out = {nm: int(offs[i]) for i, nm in enumerate(MX_BWD_SECTIONS)}
    out["bytes"] = total
    return out


def grouped_mlp_bwd_mx(x_perm, h_saved, dy_perm, offsets, mx: dict, act: str = "swiglu",
                       dh=None, dx_perm=None, dW1=None, dW2=None, err=None, workspace=None,
                       stream=None, accumulate_dw: bool = False, separate_dh_quant: bool = False):
    """MXFP8 grouped expert MLP backward (moe_grouped_mlp_bwd_mx).  ``mx``
    holds uint8 tensors a_qT, a_sT (the forward's transposed copy), w2_q, w2_s
    (W2 with blocks along d) and w1_q, w1_s (W1 with blocks along n1).
    Returns (dh, dx_perm, dW1, dW2, err).  accumulate_dw as in
    grouped_mlp_bwd; separate_dh_quant selects the unfused control (dH
    quantised in its own pass, MOE_FLAG_MX_SEPARATE_DH_QUANT)."""
    flags = _bwd_flags(accumulate_dw, dW1, dW2)
    if separate_dh_quant:
        flags |= FLAG_MX_SEPARATE_DH_QUANT
    for t, nm in ((x_perm, "x_perm"), (h_saved, "h_saved"), (dy_perm, "dy_perm")):
        _need(t, torch.bfloat16, nm)
    _need(offsets, torch.int32, "offsets", 1)
    for k_ in ("a_qT", "a_sT", "w2_q", "w2_s", "w1_q", "w1_s"):
        _need(mx.get(k_), torch.uint8, k_)
    M_cap, d = x_perm.shape
    E = offsets.numel() - 1
    n = mx["a_qT"].shape[0]
    n1 = h_saved.shape[1]
    dev = x_perm.device
    if dh is None:
        dh = _empty((M_cap, n1), torch.bfloat16, dev, stream)
    if dx_perm is None:
        dx_perm = _empty((M_cap, d), torch.bfloat16, dev, stream)
    if dW1 is None:
        dW1 = _empty((E, d, n1), torch.bfloat16, dev, stream)
    if dW2 is None:
        dW2 = _empty((E, n, d), torch.bfloat16, dev, stream)
    err = _err_word(err, dev, stream)
    need = mx_bwd_workspace_size(M_cap, d, n, act)
    if workspace is None:
        workspace = _scratch(need, dev, stream)
    _need(workspace, torch.uint8, "workspace")
    for k_ in ("dx_q", "dx_s"):
        _need(mx.get(k_), torch.uint8, k_)
    st = MxBwd(mx["a_qT"].data_ptr(), mx["a_sT"].data_ptr(), mx["w2_q"].data_ptr(),
               mx["w2_s"].data_ptr(), mx["w1_q"].data_ptr(), mx["w1_s"].data_ptr(),
               workspace.data_ptr(), workspace.numel(),
               mx["dx_q"].data_ptr() if mx.get("dx_q") is not None else None,
               mx["dx_s"].data_ptr() if mx.get("dx_s") is not None else None)
    rc = lib().moe_grouped_mlp_bwd_mx(_ptr(x_perm), _ptr(h_saved), _ptr(dy_perm), _ptr(offsets),
                                      E, M_cap, d, n, ACT[act], flags, ctypes.byref(st), _ptr(dh),
                                      _ptr(dx_perm), _ptr(dW1), _ptr(dW2), _ptr(err),
                                      _stream(stream))
    _check(rc, "moe_grouped_mlp_bwd_mx")
    return dh, dx_perm, dW1, dW2, err


def grouped_mlp_bwd_routed(x_perm, h_saved, do_perm, pair_of_row, probs, offsets, W1, W2,
                           act: str = "swiglu", dh=None, a_scaled=None, ds_part=None,
                           dx_perm=None, dW1=None, dW2=None, err=None, amax=None, stream=None,
                           accumulate_dw: bool = False):
    """Backward with the router gradient inside the expert MLP
    (moe_grouped_mlp_bwd_routed).  do_perm is the gathered dO without the
    router probability.  Returns (dh, a_scaled, ds_part, dx_perm, dW1, dW2,
    err).  accumulate_dw as in grouped_mlp_bwd."""
    flags = _bwd_flags(accumulate_dw, dW1, dW2)
    for t, nm in ((x_perm, "x_perm"), (h_saved, "h_saved"), (do_perm, "do_perm"), (W1, "W1"),
                  (W2, "W2")):
        _need(t, torch.bfloat16, nm)
    _need(pair_of_row, torch.int32, "pair_of_row", 1)
    _need(probs, torch.float32, "probs")
    _need(offsets, torch.int32, "offsets", 1)
    M_cap, d = x_perm.shape
    E, n, _ = W2.shape
    n1 = n if act == "srelu" else 2 * n
    dev = x_perm.device
    bf = torch.bfloat16
    if dh is None:
        dh = _empty((M_cap, n1), bf, dev, stream)
    if a_scaled is None:
        a_scaled = _empty((M_cap, n), bf, dev, stream)
    if ds_part is None:
        ds_part = _empty((M_cap, (n + 127) // 128), torch.float32, dev, stream)
    if dx_perm is None:
        dx_perm = _empty((M_cap, d), bf, dev, stream)
    if dW1 is None:
        dW1 = _empty((E, d, n1), bf, dev, stream)
    if dW2 is None:
        dW2 = _empty((E, n, d), bf, dev, stream)
    err = _err_word(err, dev, stream)
    rc = lib().moe_grouped_mlp_bwd_routed(
        _ptr(x_perm), _ptr(h_saved), _ptr(do_perm), _ptr(pair_of_row), _ptr(probs), _ptr(offsets),
        E, M_cap, d, n, _ptr(W1), _ptr(W2), ACT[act], flags, _ptr(dh), _ptr(a_scaled), _ptr(ds_part),
        _ptr(dx_perm), _ptr(dW1), _ptr(dW2), _ptr(amax), _ptr(err), _stream(stream))
    _check(rc, "moe_grouped_mlp_bwd_routed")
    return dh, a_scaled, ds_part, dx_perm, dW1, dW2, err


def grouped_mlp_bwd_routed_gather(x, dO, pair_of_row, k: int, h_saved, probs, offsets, W1, W2,
                                  act: str = "swiglu", dh=None, a_scaled=None, ds_part=None,
                                  dx_perm=None, dW1=None, dW2=None, err=None, amax=None,
                                  stream=None, accumulate_dw: bool = False):
    """Routed backward reading x [T, d] and dO [T, d] through the routing map
    (moe_grouped_mlp_bwd_routed_gather): no permuted copies.  Returns (dh,
    a_scaled, ds_part, dx_perm, dW1, dW2, err) like
    ``grouped_mlp_bwd_routed``."""
    flags = _bwd_flags(accumulate_dw, dW1, dW2)
    for t, nm in ((x, "x"), (dO, "dO"), (h_saved, "h_saved"), (W1, "W1"), (W2, "W2")):
        _need(t, torch.bfloat16, nm)
    _need(pair_of_row, torch.int32, "pair_of_row", 1)
    _need(probs, torch.float32, "probs")
    _need(offsets, torch.int32, "offsets", 1)
    T, d = x.shape
    M_cap = pair_of_row.numel()
    E, n, _ = W2.shape
    n1 = n if act == "srelu" else 2 * n
    dev = x.device
    bf = torch.bfloat16
    if dh is None:
        dh = _empty((M_cap, n1), bf, dev, stream)
    if a_scaled is None:
        a_scaled = _empty((M_cap, n), bf, dev, stream)
    if ds_part is None:
        ds_part = _empty((M_cap, (n + 127) // 128), torch.float32, dev, stream)
    if dx_perm is None:
        dx_perm = _empty((M_cap, d), bf, dev, stream)
    if dW1 is None:
        dW1 = _empty((E, d, n1), bf, dev, stream)
    if dW2 is None:
        dW2 = _empty((E, n, d), bf, dev, stream)
    err = _err_word(err, dev, stream)
    if T == 0:      # nothing of x or dO is read then, but the maps need addresses
        x = dO = _empty((1, d), bf, dev, stream)
    rc = lib().moe_grouped_mlp_bwd_routed_gather(
        _ptr(x), _ptr(dO), T, k, _ptr(h_saved), _ptr(pair_of_row), _ptr(probs), _ptr(offsets), E,
        M_cap, d, n, _ptr(W1), _ptr(W2), ACT[act], flags, _ptr(dh), _ptr(a_scaled), _ptr(ds_part),
        _ptr(dx_perm), _ptr(dW1), _ptr(dW2), _ptr(amax), _ptr(err), _stream(stream))
    _check(rc, "moe_grouped_mlp_bwd_routed_gather")
    return dh, a_scaled, ds_part, dx_perm, dW1, dW2, err


def router_grad_rows(ds_part, row_of_pair, T: int, k: int, dprobs=None, stream=None):
    """dprobs [T, k] from the routed backward's partials (moe_router_grad_rows)."""
    _need(ds_part, torch.float32, "ds_part", 2)
    _need(row_of_pair, torch.int32, "row_of_pair", 1)
    M_cap, n_parts = ds_part.shape
    if dprobs is None:
        dprobs = _empty((T, k), torch.float32, ds_part.device, stream)
    rc = lib().moe_router_grad_rows(_ptr(ds_part), n_parts, _ptr(row_of_pair), T, k, M_cap,
                                    _ptr(dprobs), _stream(stream))
    _check(rc, "moe_router_grad_rows")
    return dprobs


def mx_quantize_weights2(W2: torch.Tensor, w2_q=None, w2_s=None, w2_q_rows=None, w2_s_rows=None,
                         stream=None, offsets=None):
    """Both MXFP8 copies of W2 [E, n, d] from one read (moe_mx_quantize_weights2):
    blocks along n (w2_q, w2_s; forward FC2) and along d (w2_q_rows,
    w2_s_rows; backward FC2-dgrad).  Returns the four tensors.  With the
    routing ``offsets``, experts without rows are skipped."""
    _need(W2, torch.bfloat16, "W2", 3)
    E, n, d = W2.shape
    offsets = _offsets_arg(offsets, E)
    u8 = torch.uint8
    dev = W2.device
    if w2_q is None:
        w2_q = _empty((E, n, d), u8, dev, stream)
    if w2_s is None:
        w2_s = _empty(E * (n // 32) * d, u8, dev, stream)
    if w2_q_rows is None:
        w2_q_rows = _empty((E, n, d), u8, dev, stream)
    if w2_s_rows is None:
        w2_s_rows = _empty(E * n * d // 32, u8, dev, stream)
    for t, nm in ((w2_q, "w2_q"), (w2_s, "w2_s"), (w2_q_rows, "w2_q_rows"), (w2_s_rows, "w2_s_rows")):
        _need(t, u8, nm)
    rc = lib().moe_mx_quantize_weights2(_ptr(W2), E, n, d, _ptr(offsets), _ptr(w2_q), _ptr(w2_s),
                                        _ptr(w2_q_rows), _ptr(w2_s_rows), _stream(stream))
    _check(rc, "moe_mx_quantize_weights2")
    return w2_q, w2_s, w2_q_rows, w2_s_rows


# ----------------------------------------------------------------- unfused pieces

def grouped_gemm(a, offsets, B, b_layout: str = "kn", out=None, err=None, stream=None):
    """Plain grouped GEMM (moe_grouped_gemm): out_e = a_e B_e with B [E, K, N]
    ("kn"), or B stored [E, N, K] and out_e = a_e B_e^T ("nk").  Returns
    (out, err)."""
    _need(a, torch.bfloat16, "a", 2)
    _need(B, torch.bfloat16, "B", 3)
    _need(offsets, torch.int32, "offsets", 1)
    layout = {"kn": 0, "nk": 1}[b_layout]
    M_cap, K = a.shape
    E = B.shape[0]
    N = B.shape[2] if layout == 0 else B.shape[1]
    if out is None:
        out = _empty((M_cap, N), torch.bfloat16, a.device, stream)
    err = _err_word(err, a.device, stream)
    rc = lib().moe_grouped_gemm(_ptr(a), _ptr(offsets), E, M_cap, K, N, _ptr(B), layout, _ptr(out),
                                _ptr(err), _stream(stream))
    _check(rc, "moe_grouped_gemm")
    return out, err


def activation(h, offsets, act: str = "swiglu", a=None, stream=None):
    """A = act(H) as its own memory pass (moe_activation)."""
    _need(h, torch.bfloat16, "h", 2)
    _need(offsets, torch.int32, "offsets", 1)
    M_cap, n1 = h.shape
    n = n1 if act == "srelu" else n1 // 2
    if a is None:
        a = _empty((M_cap, n), torch.bfloat16, h.device, stream)
    rc = lib().moe_activation(_ptr(h), _ptr(offsets), offsets.numel() - 1, M_cap, n, ACT[act],
                              _ptr(a), _stream(stream))
    _check(rc, "moe_activation")
    return a


def activation_bwd(h, da, offsets, act: str = "swiglu", dh=None, stream=None):
    """dH = act'(H; dA) as its own memory pass (moe_activation_bwd)."""
    _need(h, torch.bfloat16, "h", 2)
    _need(da, torch.bfloat16, "da", 2)
    _need(offsets, torch.int32, "offsets", 1)
    M_cap, n = da.shape
    if dh is None:
        dh = _empty(h.shape, h.dtype, h.device, stream)
    rc = lib().moe_activation_bwd(_ptr(h), _ptr(da), _ptr(offsets), offsets.numel() - 1, M_cap, n,
                                  ACT[act], _ptr(dh), _stream(stream))
    _check(rc, "moe_activation_bwd")
    return dh


# ----------------------------------------------------------------- router losses

_TYPE = {torch.float32: 0, torch.bfloat16: 1}


def _float_type(t, name):
    if t not in _TYPE:
        raise MoeError(f"{name} must be torch.float32 or torch.bfloat16, got {t}")
    return _TYPE[t]


def _same_shape(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise MoeError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def router_loss_workspace_size(T: int, E: int, S: int = 1) -> int:
    return int(lib().moe_router_loss_workspace_size(T, E, S))


def _router_args(logits, topk_idx, seg_offsets, token_mask):
    lt = _float_type(logits.dtype, "logits")
    _need(logits, logits.dtype, "logits", 2)
    _need(topk_idx, torch.int32, "topk_idx", 2)
    _need(seg_offsets, torch.int32, "seg_offsets", 1)
    _need(token_mask, torch.uint8, "token_mask", 1)
    T, E = logits.shape
    if topk_idx.shape[0] != T or (token_mask is not None and token_mask.numel() != T):
        raise MoeError("logits, topk_idx and token_mask must have the same number of tokens")
    S = 1 if seg_offsets is None else seg_offsets.numel() - 1
    return lt, T, E, topk_idx.shape[1], S


def router_loss(logits: torch.Tensor, topk_idx: torch.Tensor, seg_offsets=None, token_mask=None,
                err=None, out: dict | None = None, workspace=None, stream=None) -> dict:
    """The router's load-balance and z losses with the per-expert counts
    (moe_router_loss).  logits [T, E] float32 or bf16, topk_idx [T, k] int32,
    seg_offsets [S+1] int32 (None: one sequence), token_mask [T] uint8 (None:
    every token).  Returns a dict of device tensors: loss [2] (balance, z),
    counts [S, E], lse [T], n_valid [S], err."""
    lt, T, E, k, S = _router_args(logits, topk_idx, seg_offsets, token_mask)
    dev = logits.device
    o = out if out is not None else {
        "loss": _empty(2, torch.float32, dev, stream),
        "counts": _empty((S, E), torch.int32, dev, stream),
        "lse": _empty(T, torch.float32, dev, stream),
        "n_valid": _empty(S, torch.int32, dev, stream),
    }
    if out is not None:
        for nm, ty, shape in (("loss", torch.float32, (2,)), ("counts", torch.int32, (S, E)),
                              ("lse", torch.float32, (T,)), ("n_valid", torch.int32, (S,))):
            if o.get(nm) is None:
                raise MoeError(f"out needs {nm}")
            _need(o[nm], ty, nm)
            _same_shape(o[nm], shape, nm)
    o["err"] = _err_word(err if err is not None else o.get("err"), dev, stream)
    workspace = _workspace(workspace, router_loss_workspace_size(T, E, S), dev, stream)
    rc = lib().moe_router_loss(_ptr(logits), lt, _ptr(topk_idx), T, E, k, _ptr(seg_offsets), S,
                               _ptr(token_mask), _ptr(o["loss"]), _ptr(o["counts"]),
                               _ptr(o["lse"]), _ptr(o["n_valid"]), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(o["err"]),
                               _stream(stream))
    _check(rc, "moe_router_loss")
    return o


def router_loss_bwd(logits: torch.Tensor, topk_idx: torch.Tensor, fwd: dict, dloss: torch.Tensor,
                    probs=None, dprobs=None, seg_offsets=None, token_mask=None, dtype=None,
                    dlogits=None, stream=None) -> torch.Tensor:
    """Gradient of the logits (moe_router_loss_bwd): of dloss [2] times the
    two losses and, with the router's probs and their gradient dprobs
    [T, k], of the softmax over the selected logits.  fwd: the dict that
    ``router_loss`` returned; dtype: of dlogits (float32, or bf16 for the
    gate's weight gradient)."""
    lt, T, E, k, S = _router_args(logits, topk_idx, seg_offsets, token_mask)
    if dlogits is None:
        ot = _float_type(dtype or torch.float32, "dlogits")
        dlogits = _empty((T, E), dtype or torch.float32, logits.device, stream)
    else:
        ot = _float_type(dlogits.dtype, "dlogits")
        _need(dlogits, dlogits.dtype, "dlogits", 2)
        _same_shape(dlogits, (T, E), "dlogits")
    for t, ty, nm, shape in ((dloss, torch.float32, "dloss", (2,)),
                             (probs, torch.float32, "probs", (T, k)),
                             (dprobs, torch.float32, "dprobs", (T, k)),
                             (fwd["lse"], torch.float32, "lse", (T,)),
                             (fwd["counts"], torch.int32, "counts", (S, E)),
                             (fwd["n_valid"], torch.int32, "n_valid", (S,))):
        _need(t, ty, nm)
        _same_shape(t, shape, nm)
    rc = lib().moe_router_loss_bwd(_ptr(logits), lt, _ptr(topk_idx), T, E, k, _ptr(seg_offsets), S,
                                   _ptr(token_mask), _ptr(fwd["lse"]), _ptr(fwd["counts"]),
                                   _ptr(fwd["n_valid"]), _ptr(dloss), _ptr(probs), _ptr(dprobs),
                                   _ptr(dlogits), ot, _stream(stream))
    _check(rc, "moe_router_loss_bwd")
    return dlogits


# ----------------------------------------------------------------- choice by scores

def _select_args(logits, score):
    lt = _float_type(logits.dtype, "logits")
    _need(logits, logits.dtype, "logits", 2)
    if score not in SCORE:
        raise MoeError(f"score must be one of {sorted(SCORE)}, got {score!r}")
    return lt, logits.shape[0], logits.shape[1]


def router_select(logits: torch.Tensor, k: int, score: str = "softmax", bias=None, groups: int = 1,
                  top_groups: int | None = None, group_best: int = 1, renorm: bool = True,
                  scale: float = 1.0, topk_idx=None, probs=None, stream=None):
    """The router's choice by scores (moe_router_select): "softmax" over all
    experts or "sigmoid"; ``bias`` [E] float32 moves the choice alone; of
    ``groups`` groups of experts the ``top_groups`` (None: all) best by the
    sum of their ``group_best`` largest scores stay; the weights are
    renormalised over the k chosen (``renorm``) and multiplied by ``scale``.
    Returns (topk_idx int32 [T, k], probs float32 [T, k])."""
    lt, T, E = _select_args(logits, score)
    _need(bias, torch.float32, "bias", 1)
    _same_shape(bias, (E,), "bias")
    _buffers((topk_idx, torch.int32, "topk_idx", (T, k)), (probs, torch.float32, "probs", (T, k)))
    if topk_idx is None:
        topk_idx = _empty((T, k), torch.int32, logits.device, stream)
    if probs is None:
        probs = _empty((T, k), torch.float32, logits.device, stream)
    rc = lib().moe_router_select(_ptr(logits), lt, T, E, k, SCORE[score], _ptr(bias), groups,
                                 groups if top_groups is None else top_groups, group_best,
                                 int(bool(renorm)), scale, _ptr(topk_idx), _ptr(probs),
                                 _stream(stream))
    _check(rc, "moe_router_select")
    return topk_idx, probs


def router_select_bwd(logits: torch.Tensor, topk_idx: torch.Tensor, probs: torch.Tensor,
                      dprobs: torch.Tensor, score: str = "softmax", renorm: bool = True,
                      scale: float = 1.0, dlogits=None, dtype=None, accumulate: bool = False,
                      stream=None) -> torch.Tensor:
    """Gradient of the logits from the weights' gradient dprobs [T, k]
    (moe_router_select_bwd).  dtype: of dlogits (float32, or bf16);
    accumulate adds to the given dlogits (``router_loss_bwd``'s, say)."""
    lt, T, E = _select_args(logits, score)
    _need(topk_idx, torch.int32, "topk_idx", 2)
    k = topk_idx.shape[1]
    if accumulate and dlogits is None:
        raise ValueError("accumulate needs the dlogits to accumulate into")
    _buffers((topk_idx, torch.int32, "topk_idx", (T, k)), (probs, torch.float32, "probs", (T, k)),
             (dprobs, torch.float32, "dprobs", (T, k)))
    if probs is None or dprobs is None:
        raise MoeError("probs and dprobs are needed")
    if dlogits is None:
        ot = _float_type(dtype or torch.float32, "dlogits")
        dlogits = _empty((T, E), dtype or torch.float32, logits.device, stream)
    else:
        ot = _float_type(dlogits.dtype, "dlogits")
        _need(dlogits, dlogits.dtype, "dlogits", 2)
        _same_shape(dlogits, (T, E), "dlogits")
    rc = lib().moe_router_select_bwd(_ptr(logits), lt, _ptr(topk_idx), _ptr(probs), _ptr(dprobs),
                                     T, E, k, SCORE[score], int(bool(renorm)), scale,
                                     int(bool(accumulate)), _ptr(dlogits), ot, _stream(stream))
    _check(rc, "moe_router_select_bwd")
    return dlogits


# ----------------------------------------------------------------- linear

def _linear_args(a, offsets, B, act, b_layout):
    _need(a, torch.bfloat16, "a", 2)
    _need(offsets, torch.int32, "offsets", 1)
    _need(B, torch.bfloat16, "B")
    if act not in LINEAR_ACT:
        raise MoeError(f"act must be one of {sorted(LINEAR_ACT)}, got {act!r}")
    if b_layout not in ("kn", "nk"):
        raise MoeError(f"b_layout must be 'kn' or 'nk', got {b_layout!r}")
    if B.dim() not in (2, 3):
        raise MoeError("B must have 2 or 3 dims")
    layout = 0 if b_layout == "kn" else 1
    E = B.shape[0] if B.dim() == 3 else 1
    K, N = (B.shape[-2], B.shape[-1]) if layout == 0 else (B.shape[-1], B.shape[-2])
    if a.shape[1] != K or (offsets is not None and offsets.numel() != E + 1):
        raise MoeError("inconsistent shapes")
    gated = act in ("swiglu", "geglu")
    return E, a.shape[0], K, N, layout, (N // 2 if gated else N)


def grouped_linear(a: torch.Tensor, offsets, B: torch.Tensor, act: str = "none", bias=None,
                   residual=None, b_layout: str = "kn", save_z: bool = False, out=None, z=None,
                   out_dtype=torch.bfloat16, err=None, stream=None):
    """out = act(a B_e + bias_e) + residual over the experts' rows
    (moe_grouped_linear).  offsets [E+1] int32, or None for a dense product
    (B [K, N], or [1, K, N]; b_layout "nk": B stored [N, K]).  act: "none",
    "relu", "silu", "gelu", "srelu", or the gated "swiglu", "geglu" (columns
    2j gate, 2j+1 up).  bias bf16 [E, N], residual bf16 [M, n_out] (may be
    ``out``).  Returns (out, z, err); z, the bf16 pre-activation that the
    backward reads, is None unless save_z or z is given."""
    E, M_cap, K, N, layout, n_out = _linear_args(a, offsets, B, act, b_layout)
    _need(bias, torch.bfloat16, "bias")
    _need(residual, torch.bfloat16, "residual")
    if bias is not None and bias.numel() != E * N:
        raise MoeError("bias must hold E*N values")
    _same_shape(residual, (M_cap, n_out), "residual")
    if out is None:
        ot = _float_type(out_dtype, "out")
        out = _empty((M_cap, n_out), out_dtype, a.device, stream)
    else:
        ot = _float_type(out.dtype, "out")
        _need(out, out.dtype, "out")
        _same_shape(out, (M_cap, n_out), "out")
    if z is not None:
        _need(z, torch.bfloat16, "z")
        _same_shape(z, (M_cap, N), "z")
    elif save_z:
        z = _empty((M_cap, N), torch.bfloat16, a.device, stream)
    err = _err_word(err, a.device, stream)
    rc = lib().moe_grouped_linear(_ptr(a), _ptr(offsets), E, M_cap, K, N, _ptr(B), layout,
                                  _ptr(bias), LINEAR_ACT[act], _ptr(residual), _ptr(z), _ptr(out),
                                  ot, _ptr(err), _stream(stream))
    _check(rc, "moe_grouped_linear")
    return out, z, err


def grouped_linear_plan(E: int, M_cap: int, K: int, N: int, ragged: bool,
                        out_dtype=torch.bfloat16) -> tuple:
    """Which kernel ``grouped_linear`` runs for these sizes
    (moe_grouped_linear_plan): (tokens of a few-row tile or 0 for the grouped
    GEMM, parts of the reduction, whether two CTAs share a tile)."""
    plan = (ctypes.c_int * 3)()
    rc = lib().moe_grouped_linear_plan(E, M_cap, K, N, int(ragged), _float_type(out_dtype, "out"),
                                       ctypes.byref(plan))
    _check(rc, "moe_grouped_linear_plan")
    return plan[0], plan[1], bool(plan[2])


def grouped_linear_bwd_workspace_size(E: int, M_cap: int, N: int) -> int:
    return int(lib().moe_grouped_linear_bwd_workspace_size(E, M_cap, N))


def grouped_linear_bwd(dout: torch.Tensor, a: torch.Tensor, offsets, B: torch.Tensor,
                       act: str = "none", z=None, bias: bool = False, b_layout: str = "kn",
                       dz=None, da=None, dB=None, dbias=None, accumulate_dw: bool = False,
                       workspace=None, err=None, stream=None):
    """Backward of ``grouped_linear`` (moe_grouped_linear_bwd).  z: the saved
    pre-activation (not needed for act "none"); bias: also the bias gradient.
    Returns (dz, da, dB, dbias, err): dz is dout itself for act "none", dbias
    (float32 [E, N]) None without bias; the residual's gradient is dout.
    accumulate_dw adds to the given dB (and dbias)."""
    E, M_cap, K, N, layout, n_out = _linear_args(a, offsets, B, act, b_layout)
    _need(dout, torch.bfloat16, "dout", 2)
    _same_shape(dout, (M_cap, n_out), "dout")
    _need(z, torch.bfloat16, "z")
    _same_shape(z, (M_cap, N), "z")
    if act != "none" and z is None:
        raise MoeError("act needs the saved pre-activation z")
    bias = bias or dbias is not None
    if accumulate_dw and (dB is None or (bias and dbias is None)):
        raise ValueError("accumulate_dw needs the dB (and dbias) to accumulate into")
    dev = a.device
    for t, ty, nm, shape in ((dz, torch.bfloat16, "dz", (M_cap, N)),
                             (da, torch.bfloat16, "da", (M_cap, K)),
                             (dB, torch.bfloat16, "dB", tuple(B.shape)),
                             (dbias, torch.float32, "dbias", (E, N))):
        _need(t, ty, nm)
        _same_shape(t, shape, nm)
    if act != "none" and dz is None:
        dz = _empty((M_cap, N), torch.bfloat16, dev, stream)
    if da is None:
        da = _empty((M_cap, K), torch.bfloat16, dev, stream)
    if dB is None:
        dB = _empty(B.shape, torch.bfloat16, dev, stream)
    if bias and dbias is None:
        dbias = _empty((E, N), torch.float32, dev, stream)
    if bias:
        workspace = _workspace(workspace, grouped_linear_bwd_workspace_size(E, M_cap, N), dev, stream)
    err = _err_word(err, dev, stream)
    rc = lib().moe_grouped_linear_bwd(
        _ptr(dout), _ptr(z), _ptr(a), _ptr(offsets), E, M_cap, K, N, _ptr(B), layout,
        LINEAR_ACT[act], FLAG_ACCUMULATE_DW if accumulate_dw else 0, _ptr(dz), _ptr(da), _ptr(dB),
        _ptr(dbias), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(err),
        _stream(stream))
    _check(rc, "moe_grouped_linear_bwd")
    return (dout if act == "none" else dz), da, dB, dbias, err


# ----------------------------------------------------------------- 4 bits
# A tensor in 4 bits is a pair (q, s): packed codes and scale bytes (uint8).

def _fp4_format(fmt):
    if fmt not in FP4:
        raise MoeError(f"fmt must be one of {sorted(FP4)}, got {fmt!r}")
    return FP4[fmt]


def fp4_scale_bytes(rows: int, E: int, K: int, fmt: str = "nvfp4") -> int:
    """Bytes of the scales of E experts' ``rows`` rows of K values
    (moe_fp4_scale_bytes, without its check of the sizes)."""
    return (rows // 128 + E) * (K // 64 if _fp4_format(fmt) == 0 else (K + 127) // 128) * 512


def _fp4_t(t, n, fmt, name):
    _need(t, torch.float32, name)
    if t is not None and fmt != "nvfp4":
        raise MoeError(f"{name}: only nvfp4 has a tensor scale")
    if t is not None and t.numel() != n:
        raise MoeError(f"{name} must hold {n} values, got {t.numel()}")


def _fp4_offsets(offsets):
    _need(offsets, torch.int32, "offsets", 1)
    if offsets is not None and offsets.numel() < 2:
        raise MoeError("offsets must hold at least 2 entries")
    return 1 if offsets is None else offsets.numel() - 1


def _fp4_pair(x, name):
    if not isinstance(x, (tuple, list)) or len(x) != 2:
        raise MoeError(f"{name} must be a pair (codes, scales)")
    for t in x:
        if t is None:
            raise MoeError(f"{name} must be a pair (codes, scales)")
        _need(t, torch.uint8, name)
    return x


def _fp4_out(out, q_shape, rows, E, K, fmt, device, stream):
    """The (q, s) to write: the given pair, or a new one."""
    n = fp4_scale_bytes(rows, E, K, fmt)
    if out is None:
        return (_empty(q_shape, torch.uint8, device, stream),
                _empty(n, torch.uint8, device, stream))
    q, s = _fp4_pair(out, "out")
    _same_shape(q, q_shape, "out's codes")
    if s.numel() != n:
        raise MoeError(f"out's scales must hold {n} bytes, got {s.numel()}")
    return q, s


def _fp4_width(K, name):
    if K <= 0 or K % 64:
        raise MoeError(f"{name} must have a multiple of 64 columns, got {K}")


def fp4_tensor_scale(src: torch.Tensor, per_expert: bool = False, t=None, stream=None, offsets=None,
                     err=None):
    """nvfp4's scale of a bf16 tensor (moe_fp4_tensor_scale): float32 [1], or
    with ``per_expert`` [E], one for each src[e]: the smallest power of two t
    with max|v| <= 6 * 448 t.  ``offsets`` [E+1]: of src's [rows, K] the
    experts' rows alone (moe_fp4_tensor_scale_rows); without them all of src
    counts, rows that no call has written too."""
    _need(src, torch.bfloat16, "src", None if offsets is None else 2)
    if offsets is not None and per_expert:
        raise MoeError("offsets and per_expert exclude each other")
    E = src.shape[0] if per_expert else 1
    n = src.numel() // max(E, 1)
    _buffers((t, torch.float32, "t", (E,)))
    if offsets is not None:
        experts = _fp4_offsets(offsets)
        _fp4_width(src.shape[1], "src")
    if t is None:
        t = _empty(E, torch.float32, src.device, stream)
    if offsets is not None:
        err = _err_word(err, src.device, stream)
        rc = lib().moe_fp4_tensor_scale_rows(_ptr(src), _ptr(offsets), experts, *src.shape, _ptr(t),
                                             _ptr(err), _stream(stream))
        _check(rc, "moe_fp4_tensor_scale_rows")
        return t
    rc = lib().moe_fp4_tensor_scale(_ptr(src), E, n, _ptr(t), _stream(stream))
    _check(rc, "moe_fp4_tensor_scale")
    return t


def fp4_quantize(src: torch.Tensor, offsets=None, fmt: str = "nvfp4", scale=None, out=None,
                 err=None, stream=None):
    """Rows [rows, K] bf16 in 4 bits (moe_fp4_quantize): "nvfp4" (``scale``:
    its float32 tensor scale, None: 1) or "mxfp4"; ``offsets`` [E+1] of the
    experts' rows (None: one block of rows).  Returns (q, s): codes [rows,
    K/2] and scales, both uint8."""
    f = _fp4_format(fmt)
    _need(src, torch.bfloat16, "src", 2)
    E = _fp4_offsets(offsets)
    rows, K = src.shape
    _fp4_width(K, "src")
    _fp4_t(scale, 1, fmt, "scale")
    q, s = _fp4_out(out, (rows, K // 2), rows, E, K, fmt, src.device, stream)
    err = _err_word(err, src.device, stream)
    rc = lib().moe_fp4_quantize(_ptr(src), _ptr(offsets), E, rows, K, f, _ptr(scale), _ptr(q),
                                _ptr(s), _ptr(err), _stream(stream))
    _check(rc, "moe_fp4_quantize")
    return q, s


def fp4_permute(src: torch.Tensor, pair_of_row: torch.Tensor, k: int, offsets: torch.Tensor,
                fmt: str = "nvfp4", scale=None, row_of_pair=None, out=None, err=None, stream=None):
    """``permute`` into 4 bits (moe_fp4_permute): token rows [T, K] bf16 to
    expert-major rows, zeros for pad rows; with row_of_pair each token is read
    and quantised once.  Returns (q, s)."""
    f = _fp4_format(fmt)
    _need(src, torch.bfloat16, "src", 2)
    _need(pair_of_row, torch.int32, "pair_of_row", 1)
    _need(row_of_pair, torch.int32, "row_of_pair", 1)
    if offsets is None or pair_of_row is None:
        raise MoeError("the routing layout's offsets and pair_of_row are needed")
    E = _fp4_offsets(offsets)
    T, K = src.shape
    _fp4_width(K, "src")
    _fp4_t(scale, 1, fmt, "scale")
    if row_of_pair is not None and row_of_pair.numel() != T * k:
        raise MoeError("row_of_pair must hold T*k entries")
    M_cap = pair_of_row.numel()
    q, s = _fp4_out(out, (M_cap, K // 2), M_cap, E, K, fmt, src.device, stream)
    err = _err_word(err, src.device, stream)
    rc = lib().moe_fp4_permute(_ptr(src), _ptr(row_of_pair), _ptr(pair_of_row), _ptr(offsets), E, T,
                               k, K, M_cap, f, _ptr(scale), _ptr(q), _ptr(s), _ptr(err),
                               _stream(stream))
    _check(rc, "moe_fp4_permute")
    return q, s


def fp4_quantize_weights(W: torch.Tensor, fmt: str = "nvfp4", along: str = "rows", scale=None,
                         out=None, stream=None):
    """Weights [E, rows, cols] (or [rows, cols]) bf16 in 4 bits
    (moe_fp4_quantize_weights).  along "rows": blocks along rows, for a
    product that contracts them (W [E, K, N] in the forward), codes [E, cols,
    rows/2]; "cols": along cols (its data gradient, or W stored [E, N, K]),
    codes [E, rows, cols/2].  scale float32 [E] or None.  Returns (q, s)."""
    f = _fp4_format(fmt)
    _need(W, torch.bfloat16, "W")
    if along not in ("rows", "cols"):
        raise MoeError(f"along must be 'rows' or 'cols', got {along!r}")
    if W.dim() not in (2, 3):
        raise MoeError("W must have 2 or 3 dims")
    E = W.shape[0] if W.dim() == 3 else 1
    R, C = W.shape[-2:]
    N, K = (C, R) if along == "rows" else (R, C)
    _fp4_width(R, "W's transpose")
    _fp4_width(C, "W")
    _fp4_t(scale, E, fmt, "scale")
    q, s = _fp4_out(out, (E, N, K // 2), E * N, E, K, fmt, W.device, stream)
    rc = lib().moe_fp4_quantize_weights(_ptr(W), E, R, C, 1 if along == "rows" else 0, f,
                                        _ptr(scale), _ptr(q), _ptr(s), _stream(stream))
    _check(rc, "moe_fp4_quantize_weights")
    return q, s


def fp4_dequantize(x, offsets=None, fmt: str = "nvfp4", scale=None, dtype=torch.bfloat16, out=None,
                   err=None, stream=None) -> torch.Tensor:
    """The values of (q, s) (moe_fp4_dequantize), bf16 or float32: rows [rows,
    K] (offsets as they were quantised with, scale [1]) or weights [E, N, K]
    (scale [E]).  Rows outside every expert are not written."""
    f = _fp4_format(fmt)
    q, s = _fp4_pair(x, "x")
    if q.dim() not in (2, 3) or (q.dim() == 3 and offsets is not None):
        raise MoeError("codes must be [rows, K/2], or [E, N, K/2] without offsets")
    E = q.shape[0] if q.dim() == 3 else _fp4_offsets(offsets)
    K = q.shape[-1] * 2
    rows = q.numel() // max(K // 2, 1)
    _fp4_width(K, "x")
    _fp4_t(scale, E if q.dim() == 3 else 1, fmt, "scale")
    if s.numel() != fp4_scale_bytes(rows, E, K, fmt):
        raise MoeError("x's scales do not fit its codes")
    shape = tuple(q.shape[:-1]) + (K,)
    if out is None:
        ot = _float_type(dtype, "out")
        out = _empty(shape, dtype, q.device, stream)
    else:
        ot = _float_type(out.dtype, "out")
        _need(out, out.dtype, "out")
        _same_shape(out, shape, "out")
    err = _err_word(err, q.device, stream)
    rc = lib().moe_fp4_dequantize(_ptr(q), _ptr(s), _ptr(offsets), E, rows, K, f, _ptr(scale),
                                  1 if q.dim() == 3 else 0, _ptr(out), ot, _ptr(err),
                                  _stream(stream))
    _check(rc, "moe_fp4_dequantize")
    return out


def _fp4_linear_args(q, offsets, wq, act):
    if act not in LINEAR_ACT:
        raise MoeError(f"act must be one of {sorted(LINEAR_ACT)}, got {act!r}")
    if q.dim() != 2 or wq.dim() != 3:
        raise MoeError("a's codes must have 2 dims and w's 3")
    E, N, K2 = wq.shape
    if _fp4_offsets(offsets) != E or q.shape[1] != K2:
        raise MoeError("inconsistent shapes")
    gated = act in ("swiglu", "geglu")
    return E, q.shape[0], 2 * K2, N, (N // 2 if gated else N)


def fp4_linear(a, offsets, w, fmt: str = "nvfp4", act: str = "none", bias=None, residual=None,
               save_z: bool = False, out=None, z=None, out_dtype=torch.bfloat16, a_scale=None,
               w_scale=None, out_scale=None, err=None, stream=None):
    """out = act(a w_e^T + bias_e) + residual of operands in 4 bits
    (moe_fp4_linear).  a: (q, s) of ``fp4_quantize`` or ``fp4_permute`` with
    these offsets (None: one expert); w: (q, s) of ``fp4_quantize_weights``,
    codes [E, N, K/2]; a_scale [1], w_scale [E]: the tensor scales they were
    quantised with.  act, bias, residual, z as in ``grouped_linear``.
    out_dtype: bf16, float32, or "fp4": then out is the (q, s) that the next
    product takes (out_scale [1]: its tensor scale, None: 1).  Returns (out,
    z, err)."""
    f = _fp4_format(fmt)
    q, s = _fp4_pair(a, "a")
    wq, ws = _fp4_pair(w, "w")
    E, M_cap, K, N, n_out = _fp4_linear_args(q, offsets, wq, act)
    _fp4_width(K, "a")
    if s.numel() != fp4_scale_bytes(M_cap, E, K, fmt) or ws.numel() != fp4_scale_bytes(E * N, E, K, fmt):
        raise MoeError("scales do not fit their codes")
    _fp4_t(a_scale, 1, fmt, "a_scale")
    _fp4_t(w_scale, E, fmt, "w_scale")
    _need(bias, torch.bfloat16, "bias")
    _need(residual, torch.bfloat16, "residual")
    if bias is not None and bias.numel() != E * N:
        raise MoeError("bias must hold E*N values")
    _same_shape(residual, (M_cap, n_out), "residual")
    out_s = None
    if out_dtype == "fp4" or isinstance(out, (tuple, list)):
        _fp4_t(out_scale, 1, fmt, "out_scale")
        _fp4_width(n_out, "out")
        out, out_s = _fp4_out(out, (M_cap, n_out // 2), M_cap, E, n_out, fmt, q.device, stream)
        ot = 2
    else:
        if out_scale is not None:
            raise MoeError("out_scale is of a 4-bit output")
        if out is None:
            ot = _float_type(out_dtype, "out")
            out = _empty((M_cap, n_out), out_dtype, q.device, stream)
        else:
            ot = _float_type(out.dtype, "out")
            _need(out, out.dtype, "out")
            _same_shape(out, (M_cap, n_out), "out")
    if z is not None:
        _need(z, torch.bfloat16, "z")
        _same_shape(z, (M_cap, N), "z")
    elif save_z:
        z = _empty((M_cap, N), torch.bfloat16, q.device, stream)
    err = _err_word(err, q.device, stream)
    rc = lib().moe_fp4_linear(_ptr(q), _ptr(s), _ptr(a_scale), _ptr(offsets), E, M_cap, K, N,
                              _ptr(wq), _ptr(ws), _ptr(w_scale), f, _ptr(bias), LINEAR_ACT[act],
                              _ptr(residual), _ptr(z), _ptr(out), ot, _ptr(out_s), _ptr(out_scale),
                              _ptr(err), _stream(stream))
    _check(rc, "moe_fp4_linear")
    return (out if out_s is None else (out, out_s)), z, err


def fp4_linear_plan(E: int, M_cap: int, K: int, N: int, ragged: bool) -> tuple:
    """Which kernel ``fp4_linear`` runs for these sizes (moe_fp4_linear_plan):
    (tokens of a few-row tile, or 0 for the 256 x 256 tiles; parts of the
    reduction)."""
    plan = (ctypes.c_int * 2)()
    _check(lib().moe_fp4_linear_plan(E, M_cap, K, N, int(ragged), ctypes.byref(plan)),
           "moe_fp4_linear_plan")
    return plan[0], plan[1]


def fp4_linear_bwd_workspace_size(E: int, M_cap: int, N: int, fmt: str = "nvfp4") -> int:
    return int(lib().moe_fp4_linear_bwd_workspace_size(E, M_cap, N, _fp4_format(fmt)))


def fp4_linear_bwd(dout: torch.Tensor, a: torch.Tensor, offsets, wt, fmt: str = "nvfp4",
                   act: str = "none", z=None, bias: bool = False, w_scale=None,
                   b_layout: str = "kn", dz=None, da=None, dB=None, dbias=None,
                   accumulate_dw: bool = False, workspace=None, err=None, stream=None):
    """Backward of ``fp4_linear`` (moe_fp4_linear_bwd).  a: the bf16 rows [M,
    K] that were quantised; wt: (q, s) of the weights with blocks along N,
    codes [E, K, N/2], w_scale [E] their tensor scales; z: the saved
    pre-activation.  da is the product of dz in 4 bits with wt, dB [E, K, N]
    ("kn") or [E, N, K] ("nk") of the bf16 a and dz.  Returns (dz, da, dB,
    dbias, err) as ``grouped_linear_bwd`` does."""
    f = _fp4_format(fmt)
    wq, ws = _fp4_pair(wt, "wt")
    if wq.dim() != 3:
        raise MoeError("wt's codes must have 3 dims")
    if act not in LINEAR_ACT:
        raise MoeError(f"act must be one of {sorted(LINEAR_ACT)}, got {act!r}")
    if b_layout not in ("kn", "nk"):
        raise MoeError(f"b_layout must be 'kn' or 'nk', got {b_layout!r}")
    E, K, N = wq.shape[0], wq.shape[1], 2 * wq.shape[2]
    _need(a, torch.bfloat16, "a", 2)
    _need(dout, torch.bfloat16, "dout", 2)
    _need(z, torch.bfloat16, "z")
    M_cap = a.shape[0]
    gated = act in ("swiglu", "geglu")
    if _fp4_offsets(offsets) != E or a.shape[1] != K:
        raise MoeError("inconsistent shapes")
    _fp4_width(K, "a")
    _fp4_width(N, "wt")
    if ws.numel() != fp4_scale_bytes(E * K, E, N, fmt):
        raise MoeError("wt's scales do not fit its codes")
    _fp4_t(w_scale, E, fmt, "w_scale")
    _same_shape(dout, (M_cap, N // 2 if gated else N), "dout")
    _same_shape(z, (M_cap, N), "z")
    if act != "none" and z is None:
        raise MoeError("act needs the saved pre-activation z")
    bias = bias or dbias is not None
    if accumulate_dw and (dB is None or (bias and dbias is None)):
        raise ValueError("accumulate_dw needs the dB (and dbias) to accumulate into")
    dev = a.device
    shape = (E, K, N) if b_layout == "kn" else (E, N, K)
    _buffers((dz, torch.bfloat16, "dz", (M_cap, N)), (da, torch.bfloat16, "da", (M_cap, K)),
             (dB, torch.bfloat16, "dB", shape), (dbias, torch.float32, "dbias", (E, N)))
    if act != "none" and dz is None:
        dz = _empty((M_cap, N), torch.bfloat16, dev, stream)
    if da is None:
        da = _empty((M_cap, K), torch.bfloat16, dev, stream)
    if dB is None:
        dB = _empty(shape, torch.bfloat16, dev, stream)
    if bias and dbias is None:
        dbias = _empty((E, N), torch.float32, dev, stream)
    workspace = _workspace(workspace, fp4_linear_bwd_workspace_size(E, M_cap, N, fmt), dev, stream)
    err = _err_word(err, dev, stream)
    rc = lib().moe_fp4_linear_bwd(
        _ptr(dout), _ptr(z), _ptr(a), _ptr(offsets), E, M_cap, K, N, _ptr(wq), _ptr(ws),
        _ptr(w_scale), f, 0 if b_layout == "kn" else 1, LINEAR_ACT[act],
        FLAG_ACCUMULATE_DW if accumulate_dw else 0, _ptr(dz), _ptr(da), _ptr(dB), _ptr(dbias),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream))
    _check(rc, "moe_fp4_linear_bwd")
    return (dout if act == "none" else dz), da, dB, dbias, err


# ----------------------------------------------------------------- 8-bit checkpoints

def checkpoint_pack(src: torch.Tensor, q=None, s=None, stream=None):
    """Rows [rows, cols] bf16 in 8 bits (moe_checkpoint_pack): E4M3 codes q
    [rows, cols] and one E8M0 scale per 32 values of a row, s [rows, cols/32]
    (both uint8).  Returns (q, s)."""
    _need(src, torch.bfloat16, "src", 2)
    rows, cols = src.shape
    for t, nm, shape in ((q, "q", (rows, cols)), (s, "s", (rows, cols // 32))):
        _need(t, torch.uint8, nm)
        _same_shape(t, shape, nm)
    if q is None:
        q = _empty((rows, cols), torch.uint8, src.device, stream)
    if s is None:
        s = _empty((rows, cols // 32), torch.uint8, src.device, stream)
    rc = lib().moe_checkpoint_pack(_ptr(src), rows, cols, _ptr(q), _ptr(s), _stream(stream))
    _check(rc, "moe_checkpoint_pack")
    return q, s


def _ckpt_args(q, s, name):
    _need(q, torch.uint8, name + "_q", 2)
    _need(s, torch.uint8, name + "_s", 2)
    _same_shape(s, (q.shape[0], q.shape[1] // 32), name + "_s")
    return q.shape


def checkpoint_unpack(q: torch.Tensor, s: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """The bf16 values of a checkpoint (moe_checkpoint_unpack), exact."""
    rows, cols = _ckpt_args(q, s, "checkpoint")
    if out is None:
        out = _empty((rows, cols), torch.bfloat16, q.device, stream)
    _need(out, torch.bfloat16, "out", 2)
    _same_shape(out, (rows, cols), "out")
    rc = lib().moe_checkpoint_unpack(_ptr(q), _ptr(s), rows, cols, _ptr(out), _stream(stream))
    _check(rc, "moe_checkpoint_unpack")
    return out


def permute_checkpoint(q: torch.Tensor, s: torch.Tensor, pair_of_row: torch.Tensor, k: int,
                       row_of_pair=None, out=None, stream=None) -> torch.Tensor:
    """``permute`` from packed token rows (moe_permute_checkpoint): expert-major
    bf16 rows, zeros for pad rows; with row_of_pair in token order."""
    T, d = _ckpt_args(q, s, "checkpoint")
    _need(pair_of_row, torch.int32, "pair_of_row", 1)
    _need(row_of_pair, torch.int32, "row_of_pair", 1)
    if row_of_pair is not None and row_of_pair.numel() != T * k:
        raise MoeError("row_of_pair must hold T*k entries")
    M_cap = pair_of_row.numel()
    if out is None:
        out = _empty((M_cap, d), torch.bfloat16, q.device, stream)
    _need(out, torch.bfloat16, "out", 2)
    _same_shape(out, (M_cap, d), "out")
    rc = lib().moe_permute_checkpoint(_ptr(q), _ptr(s), _ptr(row_of_pair), _ptr(pair_of_row), T, k,
                                      d, M_cap, _ptr(out), _stream(stream))
    _check(rc, "moe_permute_checkpoint")
    return out


def _mlp_args(x_perm, offsets, W1, W2, act):
    if act not in ACT:
        raise MoeError(f"act must be one of {sorted(ACT)}, got {act!r}")
    if x_perm.dim() != 2 or W2.dim() != 3:
        raise MoeError("x_perm must have 2 dims and W2 3")
    M_cap, d = x_perm.shape
    E, n, d2 = W2.shape
    n1 = n if act == "srelu" else 2 * n
    if d2 != d or tuple(W1.shape) != (E, d, n1) or offsets.numel() != E + 1:
        raise MoeError("inconsistent shapes")
    return M_cap, d, E, n, n1


def _buffers(*given):
    """Checks (tensor or None, dtype, name, shape) of buffers to write."""
    for t, ty, nm, shape in given:
        _need(t, ty, nm)
        _same_shape(t, shape, nm)


def grouped_mlp_fwd_ckpt(x_perm: torch.Tensor, offsets: torch.Tensor, W1: torch.Tensor,
                         W2: torch.Tensor, act: str = "swiglu", h_q=None, h_s=None, a=None,
                         y_perm=None, err=None, stream=None):
    """Grouped expert MLP forward that keeps H in 8 bits
    (moe_grouped_mlp_fwd_ckpt).  Returns (h_q, h_s, a, y_perm, err); a and
    y_perm are ``grouped_mlp_fwd``'s bit for bit."""
    _need(x_perm, torch.bfloat16, "x_perm", 2)
    _need(offsets, torch.int32, "offsets", 1)
    _need(W1, torch.bfloat16, "W1", 3)
    _need(W2, torch.bfloat16, "W2", 3)
    M_cap, d, E, n, n1 = _mlp_args(x_perm, offsets, W1, W2, act)
    dev = x_perm.device
    if h_q is None:
        h_q = _empty((M_cap, n1), torch.uint8, dev, stream)
    if h_s is None:
        h_s = _empty((M_cap, n1 // 32), torch.uint8, dev, stream)
    if a is None:
        a = _empty((M_cap, n), torch.bfloat16, dev, stream)
    if y_perm is None:
        y_perm = _empty((M_cap, d), torch.bfloat16, dev, stream)
    _ckpt_args(h_q, h_s, "h")
    _same_shape(h_q, (M_cap, n1), "h_q")
    _buffers((a, torch.bfloat16, "a", (M_cap, n)), (y_perm, torch.bfloat16, "y_perm", (M_cap, d)))
    err = _err_word(err, dev, stream)
    rc = lib().moe_grouped_mlp_fwd_ckpt(_ptr(x_perm), _ptr(offsets), E, M_cap, d, n, _ptr(W1),
                                        _ptr(W2), ACT[act], _ptr(h_q), _ptr(h_s), _ptr(a),
                                        _ptr(y_perm), _ptr(err), _stream(stream))
    _check(rc, "moe_grouped_mlp_fwd_ckpt")
    return h_q, h_s, a, y_perm, err


def grouped_mlp_bwd_routed_ckpt(x_perm, h_q, h_s, do_perm, pair_of_row, probs, offsets, W1, W2,
                                act: str = "swiglu", dh=None, a_scaled=None, ds_part=None,
                                dx_perm=None, dW1=None, dW2=None, err=None, stream=None,
                                accumulate_dw: bool = False):
    """Routed backward from the 8-bit H (moe_grouped_mlp_bwd_routed_ckpt).
    Returns (dh, a_scaled, ds_part, dx_perm, dW1, dW2, err) like
    ``grouped_mlp_bwd_routed``."""
    flags = _bwd_flags(accumulate_dw, dW1, dW2)
    for t, nm in ((x_perm, "x_perm"), (do_perm, "do_perm"), (W1, "W1"), (W2, "W2")):
        _need(t, torch.bfloat16, nm)
    _need(pair_of_row, torch.int32, "pair_of_row", 1)
    _need(probs, torch.float32, "probs")
    _need(offsets, torch.int32, "offsets", 1)
    M_cap, d, E, n, n1 = _mlp_args(x_perm, offsets, W1, W2, act)
    _same_shape(do_perm, (M_cap, d), "do_perm")
    _same_shape(pair_of_row, (M_cap,), "pair_of_row")
    _ckpt_args(h_q, h_s, "h")
    _same_shape(h_q, (M_cap, n1), "h_q")
    dev = x_perm.device
    bf = torch.bfloat16
    _buffers((dh, bf, "dh", (M_cap, n1)), (a_scaled, bf, "a_scaled", (M_cap, n)),
             (ds_part, torch.float32, "ds_part", (M_cap, (n + 127) // 128)),
             (dx_perm, bf, "dx_perm", (M_cap, d)), (dW1, bf, "dW1", (E, d, n1)),
             (dW2, bf, "dW2", (E, n, d)))
    if dh is None:
        dh = _empty((M_cap, n1), bf, dev, stream)
    if a_scaled is None:
        a_scaled = _empty((M_cap, n), bf, dev, stream)
    if ds_part is None:
        ds_part = _empty((M_cap, (n + 127) // 128), torch.float32, dev, stream)
    if dx_perm is None:
        dx_perm = _empty((M_cap, d), bf, dev, stream)
    if dW1 is None:
        dW1 = _empty((E, d, n1), bf, dev, stream)
    if dW2 is None:
        dW2 = _empty((E, n, d), bf, dev, stream)
    err = _err_word(err, dev, stream)
    rc = lib().moe_grouped_mlp_bwd_routed_ckpt(
        _ptr(x_perm), _ptr(h_q), _ptr(h_s), _ptr(do_perm), _ptr(pair_of_row), _ptr(probs),
        _ptr(offsets), E, M_cap, d, n, _ptr(W1), _ptr(W2), ACT[act], flags, _ptr(dh),
        _ptr(a_scaled), _ptr(ds_part), _ptr(dx_perm), _ptr(dW1), _ptr(dW2), _ptr(err),
        _stream(stream))
    _check(rc, "moe_grouped_mlp_bwd_routed_ckpt")
    return dh, a_scaled, ds_part, dx_perm, dW1, dW2, err
