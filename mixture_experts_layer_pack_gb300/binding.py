"""Thin ctypes binding of libmoe.so (include/moe.h): same names, argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; PyTorch only
supplies device memory (tensors) and streams. There is no other code path: if
the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

c_int64, c_int32, c_float, c_void_p, c_size_t = (ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                                                 ctypes.c_void_p, ctypes.c_size_t)

MOE_OK = 0
MOE_ERR_ROUTING, MOE_ERR_TIMEOUT = 3, 5    # device-detected errors (moe_device_status)
MOE_ERR_STATE = 6
MOE_W_BF16, MOE_W_MXFP8 = 0, 1
MOE_G_FP32, MOE_G_BF16 = 0, 1
MOE_ACT_FP32, MOE_ACT_BF16 = 0, 1   # activations between the expert GEMMs (include/moe.h, moe_act)
MOE_DECODE_MAX_TOKENS = 64
MOE_DECODE_TABLE_SETS = 64           # sets of per-expert tables that a decoder keeps
MOE_NORM_LAYER, MOE_NORM_RMS = 0, 1
MOE_T_BF16, MOE_T_FP32 = 0, 1       # element types of the norm's and the router's tensors (moe_dtype)
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_B_ROW, MOE_B_COL, MOE_B_SQUARE = 0, 1, 2   # blocks of an 8-bit matrix's scales (moe_block)
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_ROUTING",
                4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_STATE"}
WEIGHT_NAMES = ("shared_gate", "shared_up", "shared_down", "routed_gate", "routed_up", "routed_down")


class moe_config(ctypes.Structure):
    _fields_ = [("max_tokens", c_int64), ("hidden", c_int64), ("num_experts", c_int64), ("topk", c_int64),
                ("inter", c_int64), ("routed_wtype", c_int32), ("swiglu_limit", c_float),
                ("recompute_dispatch", c_int32), ("act_precision", c_int32), ("no_shared_expert", c_int32)]


class moe_wview(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("expert_stride", c_int64), ("row_stride", c_int64), ("scale", c_void_p),
                ("col_data", c_void_p), ("col_scale", c_void_p), ("expert_ptrs", c_void_p)]


class moe_weights(ctypes.Structure):
    _fields_ = [(n, moe_wview) for n in WEIGHT_NAMES] + [("shared_output_gate", c_void_p)]


class moe_main_grads(ctypes.Structure):
    _fields_ = ([(n, c_void_p) for n in WEIGHT_NAMES] + [("strides", (c_int64 * 2) * 6)] +
                [("shared_output_gate", c_void_p), ("dtype", c_int32), ("expert_ptrs", c_void_p * 3)])


class moe_norm_config(ctypes.Structure):
    _fields_ = [("hidden", c_int64), ("eps", c_float), ("kind", c_int32), ("x_type", c_int32), ("y_type", c_int32),
                ("w_type", c_int32)]


class moe_router_config(ctypes.Structure):
    _fields_ = [("num_experts", c_int64), ("topk", c_int64), ("score", c_int32), ("normalise", c_int32),
                ("scale", c_float), ("aux_coeff", c_float), ("z_coeff", c_float), ("x_type", c_int32)]


class moe_fp8(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("ld", c_int64), ("scales", c_void_p)]


class moe_linear_config(ctypes.Structure):
    _fields_ = [("in_features", c_int64), ("out_features", c_int64), ("x_type", c_int32), ("y_type", c_int32)]


class moe_ffn_config(ctypes.Structure):
    _fields_ = [("hidden", c_int64), ("inter", c_int64), ("swiglu_limit", c_float)]


class moe_ffn_weights(ctypes.Structure):
    _fields_ = [("gate", moe_fp8), ("up", moe_fp8), ("down", moe_fp8)]


class moe_ffn_kept(ctypes.Structure):
    _fields_ = [("x", moe_fp8), ("gate", moe_fp8), ("up", moe_fp8)]


class moe_ffn_grads(ctypes.Structure):
    _fields_ = [("gate", c_void_p), ("up", c_void_p), ("down", c_void_p), ("gate_stride", c_int64), ("up_stride", c_int64),
                ("down_stride", c_int64)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({_status_string(status)})")


_LIB = None
_LOCK = threading.Lock()
EXPORTED = ("moe_workspace_size", "moe_create", "moe_destroy", "moe_saved_size", "moe_saved_create",
            "moe_saved_destroy", "moe_forward", "moe_backward", "moe_export_routing", "moe_device_status",
            "moe_launch_count", "moe_status_string", "moe_profile_enable", "moe_profile_read", "moe_kernel_name",
            "moe_route_noalloc", "moe_prepare_weights", "moe_quantize_mxfp8", "moe_profile_select",
            "moe_forward_topk", "moe_handle_config", "moe_host_pipe_size", "moe_host_pipe_create", "moe_host_step",
            "moe_host_pipe_sync", "moe_host_pipe_destroy", "moe_selftest_timeout",
            "moe_decode_size", "moe_decode_create", "moe_decode_destroy", "moe_decode", "moe_decode_status",
            "moe_norm_forward", "moe_norm_backward_size", "moe_norm_backward",
            "moe_router_size", "moe_router_forward", "moe_router_backward",
            "moe_fp8_quantize", "moe_fp8_dequantize", "moe_linear_size", "moe_linear_forward", "moe_linear_backward",
            "moe_ffn_size", "moe_ffn_forward", "moe_ffn_backward", "moe_fp8_status", "moe_fp8_selftest_timeout")
MOE_K_COUNT = 20


def lib_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libmoe.so")


def load(build_if_missing: bool = True):
    """Loads libmoe.so (building it first if it is absent)."""
    global _LIB
    with _LOCK:
        if _LIB is not None:
            return _LIB
        path = lib_path()
        if not os.path.exists(path):
            if not build_if_missing:
                raise OSError(f"{path} is not built")
            from . import build_lib
            build_lib.build()
        L = ctypes.CDLL(path)
        P = ctypes.POINTER
        L.moe_workspace_size.argtypes = [P(moe_config), P(c_size_t)]
        L.moe_saved_size.argtypes = [P(moe_config), P(c_size_t)]
        L.moe_create.argtypes = [P(moe_config), c_void_p, c_size_t, P(c_void_p)]
        L.moe_destroy.argtypes = [c_void_p]
        L.moe_destroy.restype = None
        L.moe_saved_create.argtypes = [c_void_p, c_void_p, c_size_t, P(c_void_p)]
        L.moe_saved_destroy.argtypes = [c_void_p]
        L.moe_saved_destroy.restype = None
        L.moe_forward.argtypes = [c_void_p, c_int64, c_void_p, c_void_p, c_void_p, P(moe_weights), c_void_p,
                                  c_void_p, c_void_p]
        L.moe_forward_topk.argtypes = [c_void_p, c_int64, c_void_p, c_void_p, c_void_p, P(moe_weights), c_void_p,
                                       c_void_p, c_void_p]
        L.moe_backward.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, P(moe_main_grads), c_void_p]
        L.moe_export_routing.argtypes = [c_void_p, c_void_p] + [c_void_p] * 6 + [c_void_p]
        L.moe_device_status.argtypes = [c_void_p, c_void_p]
        L.moe_selftest_timeout.argtypes = [c_void_p, c_void_p]
        L.moe_launch_count.argtypes = []
        L.moe_launch_count.restype = ctypes.c_uint64
        L.moe_profile_enable.argtypes = [c_void_p, c_int32]
        L.moe_profile_select.argtypes = [c_void_p, ctypes.c_uint32]
        L.moe_profile_read.argtypes = [c_void_p, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(c_int64), c_int32]
        L.moe_kernel_name.argtypes = [c_int32]
        L.moe_kernel_name.restype = ctypes.c_char_p
        L.moe_route_noalloc.argtypes = [c_int64, c_int64, c_int64] + [c_void_p] * 10
        L.moe_prepare_weights.argtypes = [c_void_p, P(moe_weights), c_void_p]
        L.moe_quantize_mxfp8.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_int32, c_void_p, c_int64, c_void_p,
                                         c_void_p]
        L.moe_status_string.argtypes = [c_int32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_handle_config.argtypes = [c_void_p, P(moe_config)]
        L.moe_host_pipe_size.argtypes = [P(moe_config), c_int64, P(c_size_t)]
        L.moe_host_pipe_create.argtypes = [c_void_p, c_int64, c_void_p, c_size_t, P(c_void_p)]
        L.moe_host_step.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, P(moe_weights),
                                    P(moe_main_grads), c_void_p, c_void_p, c_void_p, c_void_p]
        L.moe_host_pipe_sync.argtypes = [c_void_p]
        L.moe_host_pipe_destroy.argtypes = [c_void_p]
        L.moe_host_pipe_destroy.restype = None
        V = c_void_p
        L.moe_decode_size.argtypes = [P(moe_config), P(c_size_t)]
        L.moe_decode_create.argtypes = [P(moe_config), V, c_size_t, P(V)]
        L.moe_decode_destroy.argtypes = [V]
        L.moe_decode_destroy.restype = None
        L.moe_decode.argtypes = [V, c_int64, V, c_int64, V, V, P(moe_weights), V, c_int64, V]
        L.moe_decode_status.argtypes = [V, V]
        L.moe_norm_forward.argtypes = [P(moe_norm_config), c_int64, V, c_int64, V, c_int64, V, V, V, c_int64, V,
                                       c_int64, V, V, V]
        L.moe_norm_backward_size.argtypes = [P(moe_norm_config), c_int64, P(c_size_t)]
        L.moe_norm_backward.argtypes = [P(moe_norm_config), c_int64, V, c_int64, V, c_int64, V, V, V, V, c_int64, V,
                                        c_int64, V, V, c_int32, c_int32, V, c_size_t, V]
        L.moe_router_size.argtypes = [P(moe_router_config), c_int64, P(c_size_t)]
        L.moe_router_forward.argtypes = [P(moe_router_config), c_int64, V, c_int64, V, V, V, V, V, V, c_size_t, V]
        L.moe_router_backward.argtypes = [P(moe_router_config), c_int64, V, c_int64, V, V, V, c_float, V, c_int64, V]
        I64, I32 = c_int64, c_int32
        L.moe_fp8_quantize.argtypes = [V, I32, I64, I64, I64, P(moe_fp8), P(moe_fp8), P(moe_fp8), V]
        L.moe_fp8_dequantize.argtypes = [P(moe_fp8), I32, I64, I64, V, I32, I64, V]
        L.moe_linear_size.argtypes = [P(moe_linear_config), I64, I32, P(c_size_t)]
        L.moe_linear_forward.argtypes = [P(moe_linear_config), I64, V, I64, P(moe_fp8), V, I64, P(moe_fp8), V, c_size_t, V]
        L.moe_linear_backward.argtypes = [P(moe_linear_config), I64, V, I64, P(moe_fp8), P(moe_fp8), V, I64, V, I64, I32, I32,
                                          V, c_size_t, V]
        L.moe_ffn_size.argtypes = [P(moe_ffn_config), I64, I32, P(c_size_t)]
        L.moe_ffn_forward.argtypes = [P(moe_ffn_config), I64, V, I64, P(moe_ffn_weights), V, I64, P(moe_ffn_kept), V, c_size_t, V]
        L.moe_ffn_backward.argtypes = [P(moe_ffn_config), I64, V, I64, P(moe_ffn_weights), P(moe_ffn_kept), V, I64,
                                       P(moe_ffn_grads), I32, I32, V, c_size_t, V]
        L.moe_fp8_status.argtypes = L.moe_fp8_selftest_timeout.argtypes = [V]
        for name in ("moe_fp8_quantize", "moe_fp8_dequantize", "moe_linear_size", "moe_linear_forward", "moe_linear_backward",
                     "moe_ffn_size", "moe_ffn_forward", "moe_ffn_backward", "moe_fp8_status", "moe_fp8_selftest_timeout"):
            getattr(L, name).restype = c_int32
        for name in ("moe_decode_size", "moe_decode_create", "moe_decode", "moe_decode_status", "moe_norm_forward",
                     "moe_norm_backward_size", "moe_norm_backward", "moe_router_size", "moe_router_forward",
                     "moe_router_backward"):
            getattr(L, name).restype = c_int32
        for name in ("moe_workspace_size", "moe_saved_size", "moe_create", "moe_saved_create", "moe_forward",
                     "moe_backward", "moe_export_routing", "moe_device_status", "moe_profile_enable",
                     "moe_profile_read", "moe_route_noalloc", "moe_prepare_weights", "moe_quantize_mxfp8",
                     "moe_profile_select", "moe_handle_config", "moe_host_pipe_size", "moe_host_pipe_create",
                     "moe_host_step", "moe_host_pipe_sync", "moe_selftest_timeout"):
            getattr(L, name).restype = c_int32
        _LIB = L
        return L


def _status_string(status: int) -> str:
    try:
        return load().moe_status_string(status).decode()
    except Exception:  # pragma: no cover
        return "?"


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ------------------------------------------------------------------ the C ABI, same names
def moe_workspace_size(cfg: moe_config) -> int:
    n = c_size_t(0)
    _check(load().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def moe_saved_size(cfg: moe_config) -> int:
    n = c_size_t(0)
    _check(load().moe_saved_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_saved_size")
    return n.value


def moe_create(cfg: moe_config, workspace) -> c_void_p:
    import torch
    # memory that the allocator hands out on this stream may have work of its last owner queued there
    torch.cuda.current_stream(workspace.device).synchronize()
    h = c_void_p()
    _check(load().moe_create(ctypes.byref(cfg), _ptr(workspace), workspace.numel() * workspace.element_size(),
                             ctypes.byref(h)), "moe_create")
    return h


def moe_destroy(h):
    load().moe_destroy(h)


def moe_saved_create(h, memory) -> c_void_p:
    s = c_void_p()
    _check(load().moe_saved_create(h, _ptr(memory), memory.numel() * memory.element_size(), ctypes.byref(s)),
           "moe_saved_create")
    return s


def moe_saved_destroy(s):
    load().moe_saved_destroy(s)


def moe_forward(h, T, hidden, probs, routing_map, weights: moe_weights, out, saved, stream=None):
    _check(load().moe_forward(h, int(T), _ptr(hidden), _ptr(probs), _ptr(routing_map), ctypes.byref(weights),
                              _ptr(out), saved, _stream_ptr(stream)), "moe_forward")


def moe_forward_topk(h, T, hidden, topk_ids, topk_probs, weights: moe_weights, out, saved, stream=None):
    _check(load().moe_forward_topk(h, int(T), _ptr(hidden), _ptr(topk_ids), _ptr(topk_probs), ctypes.byref(weights),
                                   _ptr(out), saved, _stream_ptr(stream)), "moe_forward_topk")


def moe_backward(h, grad_out, saved, dhidden, dprobs, main_grads: moe_main_grads, stream=None):
    _check(load().moe_backward(h, _ptr(grad_out), saved, _ptr(dhidden), _ptr(dprobs), ctypes.byref(main_grads),
                               _stream_ptr(stream)), "moe_backward")


def moe_handle_config(h) -> moe_config:
    c = moe_config()
    _check(load().moe_handle_config(h, ctypes.byref(c)), "moe_handle_config")
    return c


def moe_host_pipe_size(cfg: moe_config, T: int) -> int:
    n = c_size_t(0)
    _check(load().moe_host_pipe_size(ctypes.byref(cfg), int(T), ctypes.byref(n)), "moe_host_pipe_size")
    return n.value


def moe_host_pipe_create(h, T: int, memory) -> c_void_p:
    p = c_void_p()
    _check(load().moe_host_pipe_create(h, int(T), _ptr(memory), memory.numel() * memory.element_size(),
                                       ctypes.byref(p)), "moe_host_pipe_create")
    return p


def moe_host_step(p, hidden, probs, routing_map, grad_out, weights: moe_weights, main_grads: moe_main_grads,
                  out, dhidden, dprobs, stream=None):
    """One forward + backward step from HOST tensors (include/moe.h, moe_host_step)."""
    _check(load().moe_host_step(p, _ptr(hidden), _ptr(probs), _ptr(routing_map), _ptr(grad_out),
                                ctypes.byref(weights), ctypes.byref(main_grads), _ptr(out), _ptr(dhidden),
                                _ptr(dprobs), _stream_ptr(stream)), "moe_host_step")


def moe_host_pipe_sync(p):
    _check(load().moe_host_pipe_sync(p), "moe_host_pipe_sync")


def moe_host_pipe_destroy(p):
    load().moe_host_pipe_destroy(p)


def moe_export_routing(h, saved, ids=None, pp=None, counts=None, offsets=None, perm_src=None, row_of=None,
                       stream=None):
    _check(load().moe_export_routing(h, saved, _ptr(ids), _ptr(pp), _ptr(counts), _ptr(offsets), _ptr(perm_src),
                                     _ptr(row_of), _stream_ptr(stream)), "moe_export_routing")


def moe_device_status(h, stream=None) -> int:
    return int(load().moe_device_status(h, _stream_ptr(stream)))


def moe_selftest_timeout(h, stream=None):
    """Enqueues the timeout-path test: one bounded wait that gives up (2 s) and records
    MOE_ERR_TIMEOUT in the handle's device status."""
    _check(load().moe_selftest_timeout(h, _stream_ptr(stream)), "moe_selftest_timeout")


def moe_route_noalloc(T, E, k, routing_map, probs, ids, pp, counts, offsets, perm_src, row_of, routing_error,
                      stream=None):
    """Routing into caller buffers with no device allocation (see include/moe.h)."""
    _check(load().moe_route_noalloc(int(T), int(E), int(k), _ptr(routing_map), _ptr(probs), _ptr(ids), _ptr(pp),
                                    _ptr(counts), _ptr(offsets), _ptr(perm_src), _ptr(row_of), _ptr(routing_error),
                                    _stream_ptr(stream)), "moe_route_noalloc")


def moe_prepare_weights(h, weights: moe_weights, stream=None):
    _check(load().moe_prepare_weights(h, ctypes.byref(weights), _stream_ptr(stream)), "moe_prepare_weights")


def moe_quantize_mxfp8(x, axis, q, scales, stream=None):
    """MXFP8-quantise a 2-D bf16 tensor x into q (uint8, same shape) and compact scales."""
    rows, cols = x.shape
    _check(load().moe_quantize_mxfp8(_ptr(x), rows, cols, x.stride(0), int(axis), _ptr(q), q.stride(0),
                                     _ptr(scales), _stream_ptr(stream)), "moe_quantize_mxfp8")


def mxfp8_weight(w):
    """Quantises a bf16 weight [E, N, K] (or a combined-FC1 row view of one) on the
    device with moe_quantize_mxfp8: returns (rowwise payload, compact row scales,
    columnwise payload, compact column scales) as [E, N, K], [E, N, K/32],
    [E, N, K], [E, N/32, K] uint8 tensors."""
    import torch
    E, N, K = w.shape
    x = w.reshape(E * N, K).contiguous()
    q = torch.empty((E * N, K), dtype=torch.uint8, device=w.device)
    s = torch.empty((E * N, K // 32), dtype=torch.uint8, device=w.device)
    moe_quantize_mxfp8(x, 1, q, s)
    qc = torch.empty((E * N, K), dtype=torch.uint8, device=w.device)
    sc = torch.empty((E * N // 32, K), dtype=torch.uint8, device=w.device)
    moe_quantize_mxfp8(x, 0, qc, sc)
    return q.view(E, N, K), s.view(E, N, K // 32), qc.view(E, N, K), sc.view(E, N // 32, K)


def mxfp8_view(payload, scale, col_payload, col_scale) -> moe_wview:
    """moe_wview of an MXFP8 routed weight ([E, N, K] payloads, strides in bytes)."""
    return moe_wview(payload.data_ptr(), payload.stride(0), payload.stride(1), scale.data_ptr(),
                     col_payload.data_ptr(), col_scale.data_ptr())


def _addr(t):
    return None if t is None else t.data_ptr()


def _ld(t):
    """Row stride of a [T, n] tensor with contiguous rows; a single row has none of its own."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _raw_stream(stream, device):
    """cudaStream_t of a torch stream, or of the current stream of `device`."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _on_one_device(first, *rest):
    """A context with the CUDA device that every tensor given (None: absent) is on as the current one, where kernels go."""
    import torch
    index = first.get_device()
    if index < 0 or any(t is not None and t.get_device() != index for t in rest):
        raise ValueError("the tensors must be on one CUDA device")
    return torch.cuda.device(index)


def _current_device_of():
    """A function: the index of the current CUDA device."""
    import torch
    return getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _current_stream_of():
    """A function of a device index: its current cudaStream_t."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # a twentieth of current_stream's time
    return raw if raw is not None else (lambda index: torch.cuda.current_stream(index).cuda_stream)


def moe_decode_size(cfg: moe_config) -> int:
    n = c_size_t(0)
    _check(load().moe_decode_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_decode_size")
    return n.value


def moe_decode_create(cfg: moe_config, workspace) -> c_void_p:
    import torch
    # memory that the allocator hands out on this stream may have work of its last owner queued there
    torch.cuda.current_stream(workspace.device).synchronize()
    d = c_void_p()
    _check(load().moe_decode_create(ctypes.byref(cfg), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    ctypes.byref(d)), "moe_decode_create")
    return d


def moe_decode_destroy(d):
    load().moe_decode_destroy(d)


def moe_decode(d, T, hidden, topk_ids, topk_probs, weights: moe_weights, out, stream=None):
    """The layer for up to 64 tokens; hidden and out are 2-D tensors whose rows may be strided."""
    with _on_one_device(hidden, topk_ids, topk_probs, out):
        _check(load().moe_decode(d, T, hidden.data_ptr(), _ld(hidden), topk_ids.data_ptr(), topk_probs.data_ptr(),
                                 weights, out.data_ptr(), _ld(out), _raw_stream(stream, hidden.device)), "moe_decode")


def moe_decode_status(d, stream=None) -> int:
    return int(load().moe_decode_status(d, _stream_ptr(stream)))


def moe_norm_forward(cfg: moe_norm_config, x, weight, y, bias=None, residual=None, sum=None, mean=None, rstd=None,
                     stream=None):
    with _on_one_device(x, weight, y, bias, residual, sum, mean, rstd):
        _check(load().moe_norm_forward(cfg, x.shape[0], x.data_ptr(), _ld(x), _addr(residual),
                                       0 if residual is None else _ld(residual), weight.data_ptr(), _addr(bias),
                                       _addr(sum), 0 if sum is None else _ld(sum), y.data_ptr(), _ld(y),
                                       _addr(mean), _addr(rstd), _raw_stream(stream, x.device)), "moe_norm_forward")


def _sized(size, sizes, cfg, T, index=0):
    """size(cfg, T) from the dict of those asked for before; `index`: the current device, where the size depends on its number of
    SMs (it depends on nothing else)."""
    key = (id(cfg), T, index)  # an object keeps its configurations as long as its sizes
    n = sizes.get(key)
    if n is None:
        if len(sizes) > 4096:
            sizes.clear()
        n = sizes[key] = size(cfg, T)
    return n


def moe_norm_backward_size(cfg: moe_norm_config, T: int) -> int:
    n = c_size_t(0)
    _check(load().moe_norm_backward_size(cfg, T, ctypes.byref(n)), "moe_norm_backward_size")
    return n.value


def moe_norm_backward(cfg: moe_norm_config, dy, x, weight, mean, rstd, dx, dsum=None, dweight=None, dbias=None,
                      g_type=MOE_G_FP32, accumulate=False, workspace=None, stream=None):
    with _on_one_device(dy, x, weight, mean, rstd, dx, dsum, dweight, dbias, workspace):
        _check(load().moe_norm_backward(cfg, x.shape[0], dy.data_ptr(), _ld(dy), x.data_ptr(), _ld(x),
                                        weight.data_ptr(), _addr(mean), rstd.data_ptr(), _addr(dsum),
                                        0 if dsum is None else _ld(dsum), dx.data_ptr(), _ld(dx),
                                        _addr(dweight), _addr(dbias), g_type, 1 if accumulate else 0, _addr(workspace),
                                        0 if workspace is None else workspace.numel() * workspace.element_size(),
                                        _raw_stream(stream, x.device)), "moe_norm_backward")


def moe_router_size(cfg: moe_router_config, T: int) -> int:
    n = c_size_t(0)
    _check(load().moe_router_size(cfg, T, ctypes.byref(n)), "moe_router_size")
    return n.value


def moe_router_forward(cfg: moe_router_config, logits, ids, probs, counts=None, losses=None, select_bias=None,
                       workspace=None, stream=None):
    with _on_one_device(logits, ids, probs, counts, losses, select_bias, workspace):
        _check(load().moe_router_forward(cfg, logits.shape[0], logits.data_ptr(), _ld(logits), _addr(select_bias),
                                         ids.data_ptr(), probs.data_ptr(), _addr(counts), _addr(losses), _addr(workspace),
                                         0 if workspace is None else workspace.numel() * workspace.element_size(),
                                         _raw_stream(stream, logits.device)), "moe_router_forward")


def moe_router_backward(cfg: moe_router_config, logits, ids, dprobs, dlogits, counts=None, loss_grad=1.0,
                        stream=None):
    with _on_one_device(logits, ids, dprobs, dlogits, counts):
        _check(load().moe_router_backward(cfg, logits.shape[0], logits.data_ptr(), _ld(logits), ids.data_ptr(),
                                          dprobs.data_ptr(), _addr(counts), loss_grad, dlogits.data_ptr(),
                                          _ld(dlogits), _raw_stream(stream, logits.device)), "moe_router_backward")


def moe_linear_size(cfg: moe_linear_config, T: int, backward=False) -> int:
    n = c_size_t(0)
    _check(load().moe_linear_size(cfg, T, 1 if backward else 0, ctypes.byref(n)), "moe_linear_size")
    return n.value


def moe_ffn_size(cfg: moe_ffn_config, T: int, backward=False) -> int:
    n = c_size_t(0)
    _check(load().moe_ffn_size(cfg, T, 1 if backward else 0, ctypes.byref(n)), "moe_ffn_size")
    return n.value


def moe_fp8_status(stream=None) -> int:
    """MOE_ERR_TIMEOUT if a wait inside an 8-bit product gave up on the current device since the last call, else 0 (include/moe.h)."""
    return int(load().moe_fp8_status(_stream_ptr(stream)))


def moe_fp8_selftest_timeout(stream=None):
    """Enqueues the test of it: one wait of the 8-bit products' that gives up (2 s)."""
    _check(load().moe_fp8_selftest_timeout(_stream_ptr(stream)), "moe_fp8_selftest_timeout")


def moe_launch_count() -> int:
    return int(load().moe_launch_count())


def moe_profile_enable(h, enable: bool = True):
    _check(load().moe_profile_enable(h, 1 if enable else 0), "moe_profile_enable")


def moe_profile_select(h, classes=None):
    """Time only the given kernel classes (names or indices); None: all of them."""
    if classes is None:
        mask = 0xFFFFFFFF
    else:
        names = [moe_kernel_name(i) for i in range(MOE_K_COUNT)]
        mask = 0
        for c in classes:
            mask |= 1 << (names.index(c) if isinstance(c, str) else int(c))
    _check(load().moe_profile_select(h, mask), "moe_profile_select")


def moe_profile_read(h) -> dict:
    """{kernel name: (summed ms, launches)} since the previous read."""
    ms = (ctypes.c_double * MOE_K_COUNT)()
    n = (c_int64 * MOE_K_COUNT)()
    _check(load().moe_profile_read(h, ms, n, MOE_K_COUNT), "moe_profile_read")
    return {moe_kernel_name(i): (ms[i], n[i]) for i in range(MOE_K_COUNT)}


def moe_kernel_name(i: int) -> str:
    r = load().moe_kernel_name(i)
    return r.decode() if r else None


# ------------------------------------------------------------------ marshalling helpers
def wview(t, scale=None, col_data=None, col_scale=None) -> moe_wview:
    """View of a 2-D [N,K] or 3-D [E,N,K] tensor (strides taken from the tensor)."""
    if t.dim() == 3:
        es, rs = t.stride(0), t.stride(1)
    else:
        es, rs = 0, t.stride(0)
    return moe_wview(t.data_ptr(), es, rs, None if scale is None else scale.data_ptr(),
                     None if col_data is None else col_data.data_ptr(),
                     None if col_scale is None else col_scale.data_ptr())


def weights_from_combined(shared_fc1, shared_fc2, routed_fc1, routed_fc2, shared_output_gate=None) -> moe_weights:
    """Gate/up views of combined FC1 weights ([2I,H], [E,2I,H]): rows [0,I) gate, [I,2I) up;
    optional bf16 [H] shared-expert output gate. shared_fc1 / shared_fc2 None: no shared
    views (a layer without a shared expert ignores them)."""
    inter = routed_fc1.shape[1] // 2
    shared = (moe_wview(), moe_wview(), moe_wview()) if shared_fc1 is None else \
        (wview(shared_fc1[:inter]), wview(shared_fc1[inter:]), wview(shared_fc2))
    return moe_weights(*shared, wview(routed_fc1[:, :inter]), wview(routed_fc1[:, inter:]), wview(routed_fc2),
                       None if shared_output_gate is None else shared_output_gate.data_ptr())


def weights_from_combined_mxfp8(shared_fc1, shared_fc2, routed_q1, routed_scale1, routed_q2, routed_scale2,
                                shared_output_gate=None) -> moe_weights:
    """weights_from_combined with MXFP8 routed weights given by their rowwise payloads
    ([E,2I,H], [E,H,I] uint8) and compact E8M0 scales ([E,2I,H/32], [E,H,I/32]) alone:
    what moe_decode reads (the layer's backward takes the columnwise ones as well)."""
    inter = routed_q1.shape[1] // 2

    def view(q, s):
        if q.stride(-1) != 1 or s.stride(-1) != 1 or s.stride(0) * 32 != q.stride(0) or s.stride(1) * 32 != q.stride(1):
            raise ValueError("MXFP8 scales must have the payload's strides / 32")
        return moe_wview(q.data_ptr(), q.stride(0), q.stride(1), s.data_ptr())

    shared = (moe_wview(), moe_wview(), moe_wview()) if shared_fc1 is None else \
        (wview(shared_fc1[:inter]), wview(shared_fc1[inter:]), wview(shared_fc2))
    return moe_weights(*shared, view(routed_q1[:, :inter], routed_scale1[:, :inter]),
                       view(routed_q1[:, inter:], routed_scale1[:, inter:]), view(routed_q2, routed_scale2),
                       None if shared_output_gate is None else shared_output_gate.data_ptr())


def main_grads_from_combined(shared_fc1, shared_fc2, routed_fc1, routed_fc2, shared_output_gate=None) -> moe_main_grads:
    """Six-buffer main_grad order over combined FC1/FC2 buffers, all fp32 or all
    bf16 (plus the optional [H] main_grad of the shared-expert output gate)."""
    import torch
    inter = routed_fc1.shape[1] // 2
    shared = (None, None, None) if shared_fc1 is None else (shared_fc1[:inter], shared_fc1[inter:], shared_fc2)
    views = shared + (routed_fc1[:, :inter], routed_fc1[:, inter:], routed_fc2)
    present = [v for v in views if v is not None]
    dtypes = {v.dtype for v in present} | ({shared_output_gate.dtype} if shared_output_gate is not None else set())
    if dtypes not in ({torch.float32}, {torch.bfloat16}):
        raise ValueError(f"main_grad buffers must be all fp32 or all bf16, got {dtypes}")
    m = moe_main_grads(*[None if v is None else v.data_ptr() for v in views])
    m.dtype = MOE_G_BF16 if dtypes == {torch.bfloat16} else MOE_G_FP32
    m.shared_output_gate = None if shared_output_gate is None else shared_output_gate.data_ptr()
    for i, v in enumerate(views):
        if v is None:
            continue
        if v.dim() == 3:
            m.strides[i][0], m.strides[i][1] = v.stride(0), v.stride(1)
        else:
            m.strides[i][0], m.strides[i][1] = 0, v.stride(0)
    return m


def _pointer_table(tensors):
    """HOST array of the tensors' device pointers (ctypes), one per expert."""
    return (c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def set_expert_tables(weights: moe_weights, gate=None, up=None, down=None) -> moe_weights:
    """Describes routed BF16 weights expert by expert: each argument a list of E
    [N,K] tensors sharing one row stride (PR #6572 per-expert non-single
    weights). The host pointer arrays are kept alive on ``weights``."""
    keep = list(getattr(weights, "_tables", []))
    for name, ts in (("routed_gate", gate), ("routed_up", up), ("routed_down", down)):
        if ts is None:
            continue
        arr = _pointer_table(ts)
        v = getattr(weights, name)
        v.expert_ptrs = ctypes.cast(arr, c_void_p).value
        v.row_stride = ts[0].stride(0)
        v.data = None
        v.expert_stride = 0
        keep.append(arr)
    weights._tables = keep
    return weights


def set_mx_expert_tables(weights: moe_weights, gate=None, up=None, down=None) -> moe_weights:
    """Describes MXFP8 routed weights expert by expert: each argument a tuple of four
    lists of E tensors -- rowwise payloads [N,K] uint8, columnwise payloads [N,K],
    rowwise scales [N,K/32], columnwise scales [N/32,K] -- with the row strides the
    C ABI expects (payload row stride R; scales R/32 and R). The host pointer
    arrays are kept alive on ``weights``."""
    keep = list(getattr(weights, "_tables", []))
    for name, parts in (("routed_gate", gate), ("routed_up", up), ("routed_down", down)):
        if parts is None:
            continue
        q, cq, sc, csc = parts
        r = q[0].stride(0)
        if any(t.stride(0) != r for t in list(q) + list(cq)) or any(t.stride(0) * 32 != r for t in sc) or \
                any(t.stride(0) != r for t in csc):
            raise ValueError("per-expert MXFP8 tensors with inconsistent row strides")
        arr = _pointer_table(list(q) + list(cq) + list(sc) + list(csc))
        v = getattr(weights, name)
        v.expert_ptrs = ctypes.cast(arr, c_void_p).value
        v.row_stride = r
        v.data = v.col_data = v.scale = v.col_scale = None
        v.expert_stride = 0
        keep.append(arr)
    weights._tables = keep
    return weights


def set_main_grad_tables(main_grads: moe_main_grads, gate=None, up=None, down=None) -> moe_main_grads:
    """Describes the routed main_grads expert by expert: lists of E [N,K] tensors
    (one row stride per list). The host pointer arrays are kept alive on ``main_grads``."""
    keep = list(getattr(main_grads, "_tables", []))
    for i, ts in enumerate((gate, up, down)):
        if ts is None:
            continue
        arr = _pointer_table(ts)
        main_grads.expert_ptrs[i] = ctypes.cast(arr, c_void_p).value
        main_grads.strides[3 + i][1] = ts[0].stride(0)
        keep.append(arr)
    main_grads._tables = keep
    return main_grads


class MoELayer:
    """Holds a handle, its workspace and one saved-state block (all torch device memory)."""

    def __init__(self, max_tokens, hidden, num_experts, topk, inter, device="cuda", routed_wtype=MOE_W_BF16,
                 swiglu_limit=0.0, recompute_dispatch=False, act_precision=None, shared_expert=True, fill=None):
        """fill: a byte value written over the workspace and saved-state memory before the
        handle is created (None: left as allocated); no result may depend on it."""
        import torch
        self.cfg = moe_config(max_tokens, hidden, num_experts, topk, inter, routed_wtype, float(swiglu_limit),
                              int(bool(recompute_dispatch)),
                              MOE_ACT_FP32 if act_precision is None else int(act_precision),
                              0 if shared_expert else 1)
        self.device = torch.device(device)
        self.prepared = None
        ws = moe_workspace_size(self.cfg)
        sv = moe_saved_size(self.cfg)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=self.device)
        self.saved_mem = torch.empty(sv, dtype=torch.uint8, device=self.device)
        if fill is not None:
            self.workspace.fill_(int(fill))
            self.saved_mem.fill_(int(fill))
        with torch.cuda.device(self.device):
            self.handle = moe_create(self.cfg, self.workspace)
            self.saved = moe_saved_create(self.handle, self.saved_mem)

    def prepare_weights(self, weights: moe_weights, stream=None):
        moe_prepare_weights(self.handle, weights, stream)
        if self.cfg.routed_wtype == MOE_W_MXFP8:
            self.prepared = bytes(weights)  # whose scales the handle holds

    def forward(self, hidden, probs, routing_map, weights: moe_weights, out=None, stream=None):
        import torch
        if out is None:
            out = torch.empty_like(hidden)
        moe_forward(self.handle, hidden.shape[0], hidden, probs, routing_map, weights, out, self.saved, stream)
        self._topk = False
        return out

    def forward_topk(self, hidden, topk_ids, topk_probs, weights: moe_weights, out=None, stream=None):
        """Forward from the router's top-k output: int32 ids [T,k] (-1 = empty slot), fp32 probs [T,k]."""
        import torch
        if out is None:
            out = torch.empty_like(hidden)
        moe_forward_topk(self.handle, hidden.shape[0], hidden, topk_ids, topk_probs, weights, out, self.saved, stream)
        self._topk = True
        return out

    def backward(self, grad_out, main_grads: moe_main_grads, dhidden=None, dprobs=None, stream=None):
        import torch
        T = grad_out.shape[0]
        if dhidden is None:
            dhidden = torch.empty_like(grad_out)
        if dprobs is None:  # [T,k] per slot after forward_topk, else dense [T,E]
            n = self.cfg.topk if getattr(self, "_topk", False) else self.cfg.num_experts
            dprobs = torch.empty((T, n), dtype=torch.float32, device=grad_out.device)
        moe_backward(self.handle, grad_out, self.saved, dhidden, dprobs, main_grads, stream)
        return dhidden, dprobs

    def device_status(self, stream=None) -> int:
        return moe_device_status(self.handle, stream)

    def host_pipe(self, T):
        """A HostPipe of forward + backward steps of T tokens from host buffers."""
        return HostPipe(self, T)

    def close(self):
        if getattr(self, "handle", None) is not None:
            moe_saved_destroy(self.saved)
            moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HostPipe:
    """Forward + backward steps of a layer fed from host buffers, through the C
    ABI's host pipeline (moe_host_pipe_create / moe_host_step): every step
    uploads its inputs and downloads its results, the copies overlapped with the
    kernels of the neighbouring steps. Device staging memory is a torch buffer
    held here; the steps apply to main_grad in call order."""

    def __init__(self, layer: "MoELayer", T: int):
        import torch
        self.layer = layer
        self.T = int(T)
        self.compute = torch.cuda.Stream(layer.device)
        self.memory = torch.empty(moe_host_pipe_size(layer.cfg, self.T), dtype=torch.uint8, device=layer.device)
        with torch.cuda.device(layer.device):
            self.pipe = moe_host_pipe_create(layer.handle, self.T, self.memory)

    def step(self, hidden, probs, routing_map, grad_out, weights: moe_weights, main_grads: moe_main_grads,
             out, dhidden, dprobs):
        """Enqueues one step: host hidden[T,H] bf16, probs[T,E] f32, routing_map[T,E]
        (bool or uint8), grad_out[T,H] bf16 in; host out[T,H], dhidden[T,H] bf16 and
        dprobs[T,E] f32 receive the results once `synchronize` returns. Page-locked
        tensors only (pageable ones would make every call wait for its step)."""
        import torch
        for t in (hidden, probs, routing_map, grad_out, out, dhidden, dprobs):
            if t.is_cuda or not t.is_pinned() or not t.is_contiguous():
                raise ValueError("HostPipe.step takes contiguous pinned host tensors")
        if hidden.shape[0] != self.T:
            raise ValueError("token count differs from the pipeline's")
        H, E = self.layer.cfg.hidden, self.layer.cfg.num_experts
        for t, shape, dt in ((hidden, (self.T, H), torch.bfloat16), (grad_out, (self.T, H), torch.bfloat16),
                             (out, (self.T, H), torch.bfloat16), (dhidden, (self.T, H), torch.bfloat16),
                             (probs, (self.T, E), torch.float32), (dprobs, (self.T, E), torch.float32)):
            if tuple(t.shape) != shape or t.dtype != dt:
                raise ValueError("host tensor of the wrong shape or dtype")
        if tuple(routing_map.shape) != (self.T, E) or routing_map.element_size() != 1:
            raise ValueError("routing_map must be [T,E] bytes")
        moe_host_step(self.pipe, hidden, probs, routing_map, grad_out, weights, main_grads, out, dhidden, dprobs,
                      self.compute)

    def synchronize(self):
        """Waits until every enqueued step's results are in host memory."""
        moe_host_pipe_sync(self.pipe)

    def close(self):
        if getattr(self, "pipe", None) is not None:
            moe_host_pipe_destroy(self.pipe)   # waits for the steps in flight
            self.pipe = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass



def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _on_stream(call):
    """Runs a method whose `stream` is given with that stream as the current one, so that new tensors belong to it."""
    @functools.wraps(call)
    def wrapped(self, *args, stream=None, **kw):
        if stream is None:
            return call(self, *args, **kw)
        import torch
        with torch.cuda.stream(stream):
            return call(self, *args, **kw)
    return wrapped


class MoEDecoder:
    """The layer for a few tokens (include/moe.h, moe_decode): holds a decoder and its workspace."""

    def __init__(self, max_tokens, hidden, num_experts, topk, inter, device="cuda", routed_wtype=MOE_W_BF16,
                 swiglu_limit=0.0, shared_expert=True):
        import torch
        self.cfg = moe_config(max_tokens, hidden, num_experts, topk, inter, routed_wtype, float(swiglu_limit), 0,
                              MOE_ACT_FP32, 0 if shared_expert else 1)
        self.hidden, self.topk = int(hidden), int(topk)
        self.device = torch.device(device)
        self._torch, self._call, self._stream, self._current = torch, load().moe_decode, _current_stream_of(), _current_device_of()
        self.workspace = torch.empty(moe_decode_size(self.cfg), dtype=torch.uint8, device=self.device)
        with torch.cuda.device(self.device):
            self.handle = moe_decode_create(self.cfg, self.workspace)
        self.index = self.workspace.get_device()
        self._streams = {self._stream(self.index)}  # those that the allocator knows to use the workspace

    @_on_stream
    def forward_topk(self, hidden, topk_ids, topk_probs, weights: moe_weights, out=None):
        """out [T,H] of bf16 hidden [T,H] (rows may be strided), int32 ids [T,k] (-1 = empty
        slot) and fp32 probs [T,k], for T up to max_tokens; `stream`: where (the current stream)."""
        torch, index = self._torch, self.index
        T, H = shape = hidden.shape
        slots = (T, self.topk)
        if hidden.get_device() != index or topk_ids.get_device() != index or topk_probs.get_device() != index or \
                out is not None and out.get_device() != index:
            raise ValueError("hidden, topk_ids, topk_probs and out must be on the decoder's device")
        if self._current() != index:  # kernels go to the current device
            with torch.cuda.device(index):
                return self.forward_topk(hidden, topk_ids, topk_probs, weights, out)
        if hidden.dtype != torch.bfloat16 or H != self.hidden or hidden.stride(1) != 1:
            raise ValueError("hidden must be [T, H] bf16 with contiguous rows")
        if topk_ids.dtype != torch.int32 or topk_probs.dtype != torch.float32 or topk_ids.shape != slots or \
                topk_probs.shape != slots or not topk_ids.is_contiguous() or not topk_probs.is_contiguous():
            raise ValueError("topk_ids and topk_probs must be contiguous [T, k] int32 and fp32")
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=hidden.device)
        elif out.dtype != torch.bfloat16 or out.shape != shape or out.stride(1) != 1:
            raise ValueError("out must be [T, H] bf16 with contiguous rows")
        stream = self._stream(index)
        if stream not in self._streams:
            self.workspace.record_stream(torch.cuda.current_stream(index))
            self._streams.add(stream)
        status = self._call(self.handle, T, hidden.data_ptr(), _ld(hidden), topk_ids.data_ptr(), topk_probs.data_ptr(),
                            weights, out.data_ptr(), _ld(out), stream)
        if status:
            raise MoeError(status, "moe_decode")
        return out

    def device_status(self, stream=None) -> int:
        with self._torch.cuda.device(self.index):
            return moe_decode_status(self.handle, stream)

    def close(self):
        if getattr(self, "handle", None) is not None:
            moe_decode_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MoENorm:
    """Layer norm or RMS norm in front of the layer (include/moe.h, moe_norm_forward)."""

    def __init__(self, hidden, eps=1e-5, kind=MOE_NORM_LAYER, device="cuda"):
        import torch
        self.hidden, self.eps, self.kind, self.device = int(hidden), float(eps), int(kind), torch.device(device)
        self._types = {torch.bfloat16: MOE_T_BF16, torch.float32: MOE_T_FP32}
        self._cfgs, self._sizes = {}, {}
        self._empty, self._f32, self._row = torch.empty, torch.float32, torch.Size((self.hidden,))
        self._torch, self._stream, self._current = torch, _current_stream_of(), _current_device_of()
        self._forward, self._backward = load().moe_norm_forward, load().moe_norm_backward
        _check(load().moe_norm_forward(moe_norm_config(self.hidden, self.eps, self.kind, 0, 0, 0), 0, None, self.hidden,
                                       None, 0, None, None, None, 0, None, self.hidden, None, None, None), "MoENorm")

    def _cfg(self, x, y, w):
        key = (x, y, w)
        c = self._cfgs.get(key)
        if c is None:
            _require(all(t in self._types for t in key), "tensors must be bf16 or fp32")
            c = self._cfgs[key] = moe_norm_config(self.hidden, self.eps, self.kind, *(self._types[t] for t in key))
        return c

    def _same(self, t, shape, dtype, what):
        if t.shape != shape or t.dtype != dtype or t.stride(1) != 1:
            raise ValueError(f"{what} must be [T, hidden] rows of the right type")

    def _vector(self, t, dtype):
        if t.shape != self._row or t.dtype != dtype or t.stride(0) != 1:
            raise ValueError("weight and bias, and their gradients, must be [hidden] vectors of one type")

    @_on_stream
    def forward(self, x, weight, bias=None, residual=None, out_dtype=None):
        """(y, s, mean, rstd): s = x + residual (x itself without one), y = norm(s) weight + bias in
        out_dtype (x's by default); mean is None for RMS norm. s, mean and rstd are what backward takes.
        `stream`: where (the current stream)."""
        empty = self._empty
        T, H = shape = x.shape
        xt, wt, dev, index = x.dtype, weight.dtype, x.device, x.get_device()
        yt = xt if out_dtype is None else out_dtype
        if index < 0 or weight.get_device() != index or bias is not None and bias.get_device() != index or \
                residual is not None and residual.get_device() != index:
            raise ValueError("the tensors must be on one CUDA device")
        if self._current() != index:  # kernels go to the current device
            with self._torch.cuda.device(index):
                return self.forward(x, weight, bias, residual, out_dtype)
        if H != self.hidden or x.stride(1) != 1:
            raise ValueError("x must be [T, hidden] rows")
        self._vector(weight, wt)
        if bias is not None:
            self._vector(bias, wt)
        cfg = self._cfgs.get((xt, yt, wt)) or self._cfg(xt, yt, wt)
        y = empty(shape, dtype=yt, device=dev)
        rstd = empty(T, dtype=self._f32, device=dev)
        if self.kind == MOE_NORM_LAYER:
            mean = empty(T, dtype=self._f32, device=dev)
            mean_at = mean.data_ptr()
        else:
            mean = mean_at = None
        if residual is None:
            s, res_at, res_ld, s_at, s_ld = x, None, 0, None, 0
        else:
            self._same(residual, shape, xt, "residual")
            s = empty(shape, dtype=xt, device=dev)
            res_at, res_ld, s_at, s_ld = residual.data_ptr(), _ld(residual), s.data_ptr(), H
        status = self._forward(cfg, T, x.data_ptr(), x.stride(0) if T > 1 else H, res_at, res_ld, weight.data_ptr(),
                               None if bias is None else bias.data_ptr(), s_at, s_ld, y.data_ptr(), H, mean_at,
                               rstd.data_ptr(), self._stream(index))
        if status:
            raise MoeError(status, "moe_norm_forward")
        return y, s, mean, rstd

    @_on_stream
    def backward(self, dy, s, weight, mean, rstd, dsum=None, bias=False, dweight=None, dbias=None, accumulate=False):
        """(ds, dweight, dbias) for the gradient dy of y, joined by dsum, the gradient that reaches s
        past the norm. dweight (and, with `bias`, dbias) are new fp32 vectors, or the given
        fp32 / bf16 buffers, overwritten or (accumulate) added to. `stream`: where (the current stream)."""
        torch, empty = self._torch, self._empty
        T, H = shape = s.shape
        st, yt, wt, dev, f32, index = s.dtype, dy.dtype, weight.dtype, s.device, self._f32, s.get_device()
        if H != self.hidden or s.stride(1) != 1:
            raise ValueError("s must be [T, hidden] rows")
        if dy.shape != shape or dy.stride(1) != 1:
            raise ValueError("dy must be [T, hidden] rows of the right type")
        self._vector(weight, wt)
        rows = (T,)
        if rstd is None or rstd.dtype != f32 or rstd.shape != rows or not rstd.is_contiguous() or (
                self.kind == MOE_NORM_LAYER if mean is None else
                mean.dtype != f32 or mean.shape != rows or not mean.is_contiguous()):
            raise ValueError("mean and rstd must be the forward's [T] fp32")
        if accumulate and (dweight is None or (bias and dbias is None)):
            raise ValueError("accumulate adds to given buffers")
        if index < 0 or dy.get_device() != index or weight.get_device() != index or rstd.get_device() != index or \
                mean is not None and mean.get_device() != index or dsum is not None and dsum.get_device() != index or \
                dweight is not None and dweight.get_device() != index or dbias is not None and dbias.get_device() != index:
            raise ValueError("the tensors must be on one CUDA device")
        if self._current() != index:
            with torch.cuda.device(index):
                return self.backward(dy, s, weight, mean, rstd, dsum, bias, dweight, dbias, accumulate)
        if dsum is not None:
            self._same(dsum, shape, st, "dsum")
        cfg = self._cfgs.get((st, yt, wt)) or self._cfg(st, yt, wt)
        ds = empty(shape, dtype=st, device=dev)
        if dweight is None and dbias is None:
            gt = f32
            dweight = empty(H, dtype=f32, device=dev)
            if bias:
                dbias = empty(H, dtype=f32, device=dev)
        else:
            if dweight is None:
                dweight = empty(H, dtype=f32, device=dev)
            gt = dweight.dtype
            if bias and dbias is None:
                dbias = empty(H, dtype=gt, device=dev)
            if gt not in self._types:
                raise ValueError("dweight and dbias must be fp32 or bf16")
            self._vector(dweight, gt)
            if dbias is not None:
                self._vector(dbias, gt)
        size = _sized(moe_norm_backward_size, self._sizes, cfg, T)
        workspace = empty(size, dtype=torch.uint8, device=dev)
        many = T > 1  # a single row has no stride of its own
        status = self._backward(cfg, T, dy.data_ptr(), dy.stride(0) if many else H, s.data_ptr(), s.stride(0) if many else H,
                                weight.data_ptr(), None if mean is None else mean.data_ptr(), rstd.data_ptr(), _addr(dsum),
                                0 if dsum is None else _ld(dsum), ds.data_ptr(), H, dweight.data_ptr(),
                                None if dbias is None else dbias.data_ptr(), MOE_G_FP32 if gt is f32 else MOE_G_BF16,
                                1 if accumulate else 0, workspace.data_ptr(), size, self._stream(index))
        if status:
            raise MoeError(status, "moe_norm_backward")
        return ds, dweight, dbias


class MoERouter:
    """The choice of experts from the router's logits (include/moe.h, moe_router_forward)."""

    def __init__(self, num_experts, topk, score=MOE_SCORE_SOFTMAX, normalise=True, scale=1.0, aux_coeff=0.0,
                 z_coeff=0.0, device="cuda"):
        import torch
        self.E, self.k = int(num_experts), int(topk)
        self.device = torch.device(device)
        args = (self.E, self.k, int(score), int(bool(normalise)), float(scale), float(aux_coeff), float(z_coeff))
        self._sizes, self._empty, self._f32 = {}, torch.empty, torch.float32
        self._cfgs = {torch.bfloat16: moe_router_config(*args, MOE_T_BF16),
                      torch.float32: moe_router_config(*args, MOE_T_FP32)}
        self.losses_wanted = aux_coeff != 0 or z_coeff != 0
        self._torch, self._stream, self._current = torch, _current_stream_of(), _current_device_of()
        self._forward, self._backward = load().moe_router_forward, load().moe_router_backward
        moe_router_size(self._cfgs[torch.float32], 0)      # the library's check of the configuration

    def _cfg(self, logits):
        cfg = self._cfgs.get(logits.dtype)
        if cfg is None or logits.shape[1] != self.E or logits.stride(1) != 1:
            raise ValueError("logits must be [T, E] rows, bf16 or fp32")
        return cfg

    @_on_stream
    def forward(self, logits, select_bias=None):
        """(ids [T,k] int32, probs [T,k] fp32, counts [E] int32, losses [2] fp32 or None): the input of
        forward_topk, the routes per expert, and the balance and z losses where a coefficient asks for them.
        `stream`: where (the current stream)."""
        torch, empty, f32 = self._torch, self._empty, self._f32
        cfg = self._cfgs.get(logits.dtype)
        T, E = logits.shape
        if cfg is None or E != self.E or logits.stride(1) != 1:
            raise ValueError("logits must be [T, E] rows, bf16 or fp32")
        dev, index = logits.device, logits.get_device()
        if index < 0 or select_bias is not None and select_bias.get_device() != index:
            raise ValueError("the tensors must be on one CUDA device")
        if self._current() != index:  # kernels go to the current device
            with torch.cuda.device(index):
                return self.forward(logits, select_bias)
        if select_bias is not None and (select_bias.shape != (E,) or select_bias.dtype != f32 or select_bias.stride(0) != 1):
            raise ValueError("select_bias must be [E] fp32")
        slots = (T, self.k)
        ids = empty(slots, dtype=torch.int32, device=dev)
        probs = empty(slots, dtype=f32, device=dev)
        counts = empty(E, dtype=torch.int32, device=dev)
        losses = empty(2, dtype=f32, device=dev) if self.losses_wanted else None
        size = _sized(moe_router_size, self._sizes, cfg, T)
        workspace = empty(size, dtype=torch.uint8, device=dev)
        status = self._forward(cfg, T, logits.data_ptr(), logits.stride(0) if T > 1 else E,
                               None if select_bias is None else select_bias.data_ptr(), ids.data_ptr(),
                               probs.data_ptr(), counts.data_ptr(), None if losses is None else losses.data_ptr(),
                               workspace.data_ptr(), size, self._stream(index))
        if status:
            raise MoeError(status, "moe_router_forward")
        return ids, probs, counts, losses

    @_on_stream
    def backward(self, logits, ids, dprobs, counts=None, loss_grad=1.0):
        """dlogits of sum(dprobs * probs) + loss_grad * (balance + z); counts: the forward's (needed
        with a balance loss). `stream`: where (the current stream)."""
        torch = self._torch
        cfg = self._cfg(logits)
        shape = logits.shape
        slots = (shape[0], self.k)
        if ids.shape != slots or ids.dtype != torch.int32 or not ids.is_contiguous() or dprobs.shape != slots or \
                dprobs.dtype != torch.float32 or not dprobs.is_contiguous():
            raise ValueError("ids and dprobs must be contiguous [T, k] int32 and fp32")
        if counts is not None and (counts.shape != (self.E,) or counts.dtype != torch.int32 or counts.stride(0) != 1):
            raise ValueError("counts must be [E] int32")
        index = logits.get_device()
        if index < 0 or ids.get_device() != index or dprobs.get_device() != index or \
                counts is not None and counts.get_device() != index:
            raise ValueError("the tensors must be on one CUDA device")
        if self._current() != index:
            with torch.cuda.device(index):
                return self.backward(logits, ids, dprobs, counts, loss_grad)
        dlogits = torch.empty(shape, dtype=logits.dtype, device=logits.device)
        status = self._backward(cfg, shape[0], logits.data_ptr(), _ld(logits), ids.data_ptr(), dprobs.data_ptr(),
                                _addr(counts), float(loss_grad), dlogits.data_ptr(), self.E, self._stream(index))
        if status:
            raise MoeError(status, "moe_router_backward")
        return dlogits


# ------------------------------------------------------------------ dense layers in 8-bit floating point
def fp8_scales_shape(rows, cols, block):
    """Shape of the scales of an 8-bit [rows, cols] matrix (include/moe.h, moe_block)."""
    r, c = -(-rows // 128), -(-cols // 128)
    return (c, rows) if block == MOE_B_ROW else (r, cols) if block == MOE_B_COL else (r, c)


def _new_codes(torch, rows, cols, block, device):
    """A new (codes, scales) pair: codes uint8 [rows, cols] whose row stride is a multiple of 16."""
    ld = (cols + 15) // 16 * 16
    q = torch.empty_strided((rows, cols), (ld, 1), dtype=torch.uint8, device=device)   # half the time of a slice of rows x ld
    return q, torch.empty(fp8_scales_shape(rows, cols, block), dtype=torch.float32, device=device)


def _as_view(pair) -> moe_fp8:
    """The moe_fp8 of a pair that _new_codes made."""
    q, s = pair
    return moe_fp8(q.data_ptr(), q.stride(0), s.data_ptr())


def _codes(torch, pair, rows, cols, block, index, what) -> moe_fp8:
    """The moe_fp8 of a (codes, scales) pair of the given size on the device `index`."""
    q, s = pair
    ld = q.stride(0) if rows > 1 else (cols + 15) // 16 * 16
    if q.dtype is not torch.uint8 or q.shape != (rows, cols) or cols > 1 and q.stride(1) != 1 or ld % 16 or ld < cols or \
            s.dtype is not torch.float32 or s.shape != fp8_scales_shape(rows, cols, block) or not s.is_contiguous():
        raise ValueError(f"{what} must be (codes, scales): uint8 [{rows}, {cols}] with a row stride of a multiple of 16, and contiguous "
                         f"fp32 {list(fp8_scales_shape(rows, cols, block))}")
    if q.get_device() != index or s.get_device() != index:
        raise ValueError("the tensors must be on one CUDA device")
    return moe_fp8(q.data_ptr(), ld, s.data_ptr())


@functools.lru_cache(maxsize=None)
def _fp8_of_torch():
    """(torch, moe_dtype of its types, current device, current stream of a device): looked up once."""
    import torch
    return torch, {torch.bfloat16: MOE_T_BF16, torch.float32: MOE_T_FP32}, _current_device_of(), _current_stream_of()


def _fp8_types(torch):
    return _fp8_of_torch()[1]


def _as_rows(t, what):
    """t, a 2-D tensor, with contiguous elements in its rows."""
    if t.dim() != 2 or t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what} must be rows with contiguous elements, bf16 or fp32")


_BLOCKS = (MOE_B_ROW, MOE_B_COL, MOE_B_SQUARE)


def fp8_quantize(x, block, out=None, stream=None):
    """(codes, scales) of x [rows, cols] (bf16 or fp32, rows of any stride) in blocks of 128: MOE_B_ROW along its rows, MOE_B_COL
    down its columns, MOE_B_SQUARE both (a weight). codes uint8 [rows, cols] (E4M3), scales fp32 of fp8_scales_shape(rows,
    cols, block); `out`: a pair to write. An activation kept like this for a later pass takes half of its bf16 bytes.
    `stream`: where (the current stream)."""
    torch, types, current, streams = _fp8_of_torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return fp8_quantize(x, block, out)
    _as_rows(x, "x")
    xt, index = types.get(x.dtype), x.get_device()
    if xt is None or block not in _BLOCKS:
        raise ValueError("x must be bf16 or fp32, and block one of MOE_B_ROW, MOE_B_COL, MOE_B_SQUARE")
    if index < 0:
        raise ValueError("the tensors must be on one CUDA device")
    if current() != index:  # kernels go to the current device
        with torch.cuda.device(index):
            return fp8_quantize(x, block, out)
    rows, cols = x.shape
    if out is None:
        pair = _new_codes(torch, rows, cols, block, x.device)
        v = _as_view(pair)
    else:
        pair, v = out, _codes(torch, out, rows, cols, block, index, "out")
    status = load().moe_fp8_quantize(x.data_ptr(), xt, rows, cols, _ld(x), v if block == MOE_B_ROW else None, v if block == MOE_B_COL else None,
                                     v if block == MOE_B_SQUARE else None, streams(index))
    if status:
        raise MoeError(status, "moe_fp8_quantize")
    return pair


def fp8_dequantize(codes, scales, block, dtype=None, out=None, stream=None):
    """The values [rows, cols] that codes and scales stand for, in `dtype` (bf16 by default) or the type of `out`.
    `stream`: where (the current stream)."""
    torch, types, current, streams = _fp8_of_torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            return fp8_dequantize(codes, scales, block, dtype, out)
    index = codes.get_device()
    if index < 0 or out is not None and out.get_device() != index:
        raise ValueError("the tensors must be on one CUDA device")
    if block not in _BLOCKS or codes.dim() != 2:
        raise ValueError("codes must be [rows, cols], and block one of MOE_B_ROW, MOE_B_COL, MOE_B_SQUARE")
    if current() != index:
        with torch.cuda.device(index):
            return fp8_dequantize(codes, scales, block, dtype, out)
    rows, cols = codes.shape
    v = _codes(torch, (codes, scales), rows, cols, block, index, "codes and scales")
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.bfloat16 if dtype is None else dtype, device=codes.device)
    yt = types.get(out.dtype)
    if yt is None or out.shape != codes.shape or dtype not in (None, out.dtype):
        raise ValueError("out must be bf16 or fp32, of the codes' shape")
    _as_rows(out, "out")
    status = load().moe_fp8_dequantize(v, block, rows, cols, out.data_ptr(), yt, _ld(out), streams(index))
    if status:
        raise MoeError(status, "moe_fp8_dequantize")
    return out


def _grad_buffer(t, shape, what):
    """Checks the buffer of a weight's gradient."""
    _as_rows(t, what)
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}")


class MoEFp8Linear:
    """y = x W^T with 8-bit products, a scale for each block of 128 (include/moe.h, moe_linear_forward). A weight is a (codes, scales)
    pair of fp8_quantize(w, MOE_B_SQUARE), w [out_features, in_features]."""

    def __init__(self, in_features, out_features, device="cuda"):
        import torch
        self.K, self.N, self.device = int(in_features), int(out_features), torch.device(device)
        self._torch, self._stream, self._current = torch, _current_stream_of(), _current_device_of()
        self._cfgs, self._sizes, self._back_sizes = {}, {}, {}
        self._forward, self._backward = load().moe_linear_forward, load().moe_linear_backward
        moe_linear_size(self._cfg(torch.bfloat16, torch.bfloat16), 0)   # the library's check of the configuration

    def _cfg(self, xt, yt):
        c = self._cfgs.get((xt, yt))
        if c is None:
            types = _fp8_types(self._torch)
            _require(xt in types and yt in types, "tensors must be bf16 or fp32")
            c = self._cfgs[xt, yt] = moe_linear_config(self.K, self.N, types[xt], types[yt])
        return c

    @_on_stream
    def forward(self, x, weight, keep=True, out_dtype=None):
        """(y, kept): y [T, out] in out_dtype (x's by default) of x [T, in] bf16 or fp32; kept, what backward takes in x's place, is
        x in 8 bits, column blocks (None without `keep`). `stream`: where (the current stream)."""
        torch = self._torch
        T, K = x.shape
        index = x.get_device()
        if index < 0:
            raise ValueError("the tensors must be on one CUDA device")
        if self._current() != index:  # kernels go to the current device
            with torch.cuda.device(index):
                return self.forward(x, weight, keep, out_dtype)
        if K != self.K:
            raise ValueError("x must be [T, in_features] rows")
        _as_rows(x, "x")
        xt, dev = x.dtype, x.device
        yt = xt if out_dtype is None else out_dtype
        cfg = self._cfgs.get((xt, yt)) or self._cfg(xt, yt)
        w = _codes(torch, weight, self.N, K, MOE_B_SQUARE, index, "weight")
        y = torch.empty((T, self.N), dtype=yt, device=dev)
        kept = _new_codes(torch, T, K, MOE_B_COL, dev) if keep else None
        size = _sized(moe_linear_size, self._sizes, cfg, T, index)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        status = self._forward(cfg, T, x.data_ptr(), _ld(x), w, y.data_ptr(), self.N, _as_view(kept) if keep else None, _addr(workspace), size,
                               self._stream(index))
        if status:
            raise MoeError(status, "moe_linear_forward")
        return y, kept

    @_on_stream
    def backward(self, dy, weight, kept, dx_dtype=None, dweight=None, accumulate=False, need_dx=True, need_dweight=True):
        """(dx, dweight) for the gradient dy [T, out] of y and the forward's `kept`: dx [T, in] in dx_dtype (dy's by default), dweight
        [out, in], a new fp32 matrix or the given fp32 / bf16 buffer, overwritten or (accumulate) added to. What is not
        needed is None. `stream`: where (the current stream)."""
        torch = self._torch
        T, N = dy.shape
        index = dy.get_device()
        if index < 0 or dweight is not None and dweight.get_device() != index:
            raise ValueError("the tensors must be on one CUDA device")
        if self._current() != index:
            with torch.cuda.device(index):
                return self.backward(dy, weight, kept, dx_dtype, dweight, accumulate, need_dx, need_dweight)
        if N != self.N:
            raise ValueError("dy must be [T, out_features] rows")
        _as_rows(dy, "dy")
        if accumulate and dweight is None:
            raise ValueError("accumulate adds to a given buffer")
        if dweight is not None and not need_dweight:
            raise ValueError("a buffer for a gradient that is not needed")
        yt, dev, K = dy.dtype, dy.device, self.K
        xt = yt if dx_dtype is None else dx_dtype
        cfg = self._cfgs.get((xt, yt)) or self._cfg(xt, yt)
        w = _codes(torch, weight, N, K, MOE_B_SQUARE, index, "weight") if need_dx else None
        k = _codes(torch, kept, T, K, MOE_B_COL, index, "kept") if need_dweight else None
        dx = torch.empty((T, K), dtype=xt, device=dev) if need_dx else None
        gt = MOE_G_FP32
        if need_dweight:
            if dweight is None:
                dweight = torch.empty((N, K), dtype=torch.float32, device=dev)
            else:
                _grad_buffer(dweight, (N, K), "dweight")
                gt = _fp8_types(torch).get(dweight.dtype)
                if gt is None:
                    raise ValueError("dweight must be fp32 or bf16")
                gt = MOE_G_BF16 if gt == MOE_T_BF16 else MOE_G_FP32
        size = _sized(_linear_back_size, self._back_sizes, cfg, T, index)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        status = self._backward(cfg, T, dy.data_ptr(), _ld(dy), w, k, _addr(dx), K, _addr(dweight), _ld(dweight) if need_dweight else 0,
                                gt, 1 if accumulate else 0, workspace.data_ptr(), size, self._stream(index))
        if status:
            raise MoeError(status, "moe_linear_backward")
        return dx, dweight


def _linear_back_size(cfg, T):
    return moe_linear_size(cfg, T, True)


def _ffn_back_size(cfg, T):
    return moe_ffn_size(cfg, T, True)


class FeedForwardWeights:
    """The weights of a MoEFeedForward: (codes, scales) pairs of fp8_quantize(w, MOE_B_SQUARE), gate and up [inter, hidden], down
    [hidden, inter]. It holds the tensors; their contents may change, their places may not."""

    def __init__(self, gate, up, down):
        import torch
        I, H = gate[0].shape
        index = gate[0].get_device()
        self.tensors = (gate, up, down)
        self.hidden, self.inter, self.index = H, I, index
        self.views = moe_ffn_weights(_codes(torch, gate, I, H, MOE_B_SQUARE, index, "gate"),
                                     _codes(torch, up, I, H, MOE_B_SQUARE, index, "up"),
                                     _codes(torch, down, H, I, MOE_B_SQUARE, index, "down"))


class MoEFeedForward:
    """The gated feed-forward network of a dense block with 8-bit products (include/moe.h, moe_ffn_forward):
    y = (silu(x Wg^T) (x Wu^T)) Wd^T, with the layer's clamp where swiglu_limit > 0."""

    def __init__(self, hidden, inter, swiglu_limit=0.0, device="cuda"):
        import torch
        self.cfg = moe_ffn_config(int(hidden), int(inter), float(swiglu_limit))
        self.H, self.I, self.device = int(hidden), int(inter), torch.device(device)
        self._torch, self._stream, self._current = torch, _current_stream_of(), _current_device_of()
        self._sizes, self._back_sizes = {}, {}
        self._forward, self._backward = load().moe_ffn_forward, load().moe_ffn_backward
        moe_ffn_size(self.cfg, 0)   # the library's check of the configuration

    def _weights(self, weights, index):
        if weights.hidden != self.H or weights.inter != self.I:
            raise ValueError("the weights are of another size")
        if index < 0 or weights.index != index:
            raise ValueError("the tensors must be on one CUDA device")
        return weights.views

    @_on_stream
    def forward(self, x, weights: FeedForwardWeights, keep=True):
        """(y, kept): y [T, hidden] bf16 of x [T, hidden] bf16 (rows of any stride); kept, what backward takes: x, g and u in 8 bits,
        three (codes, scales) pairs in column, row and row blocks (None without `keep`). `stream`: where (the current stream)."""
        torch = self._torch
        T, H = x.shape
        index = x.get_device()
        w = self._weights(weights, index)
        if self._current() != index:  # kernels go to the current device
            with torch.cuda.device(index):
                return self.forward(x, weights, keep)
        if H != self.H or x.dtype != torch.bfloat16:
            raise ValueError("x must be [T, hidden] bf16 rows")
        _as_rows(x, "x")
        dev, I = x.device, self.I
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        kept = views = None
        if keep:
            kept = (_new_codes(torch, T, H, MOE_B_COL, dev), _new_codes(torch, T, I, MOE_B_ROW, dev), _new_codes(torch, T, I, MOE_B_ROW, dev))
            views = moe_ffn_kept(*[_as_view(v) for v in kept])
        size = _sized(moe_ffn_size, self._sizes, self.cfg, T, index)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        status = self._forward(self.cfg, T, x.data_ptr(), _ld(x), w, y.data_ptr(), H, views, workspace.data_ptr(), size, self._stream(index))
        if status:
            raise MoeError(status, "moe_ffn_forward")
        return y, kept

    def _kept(self, kept, T, index):
        torch = self._torch
        return moe_ffn_kept(_codes(torch, kept[0], T, self.H, MOE_B_COL, index, "kept x"),
                            _codes(torch, kept[1], T, self.I, MOE_B_ROW, index, "kept gate"),
                            _codes(torch, kept[2], T, self.I, MOE_B_ROW, index, "kept up"))

    @_on_stream
    def backward(self, dy, weights: FeedForwardWeights, kept, grads=None, accumulate=False, need_dx=True, need_grads=True):
        """(dx, (dgate, dup, ddown)) for the gradient dy [T, hidden] bf16 of y and the forward's `kept`: dx bf16, the weights' gradients
        new fp32 matrices or the given ones (`grads`: three buffers, all fp32 or all bf16), overwritten or (accumulate)
        added to. What is not needed is None. `stream`: where (the current stream)."""
        torch = self._torch
        T, H = dy.shape
        index = dy.get_device()
        w = self._weights(weights, index)
        if self._current() != index:
            with torch.cuda.device(index):
                return self.backward(dy, weights, kept, grads, accumulate, need_dx, need_grads)
        if H != self.H or dy.dtype != torch.bfloat16:
            raise ValueError("dy must be [T, hidden] bf16 rows")
        _as_rows(dy, "dy")
        if accumulate and grads is None:
            raise ValueError("accumulate adds to given buffers")
        if grads is not None and not need_grads:
            raise ValueError("buffers for gradients that are not needed")
        dev, I = dy.device, self.I
        views = self._kept(kept, T, index)
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if need_dx else None
        at, gt = None, MOE_G_FP32
        if need_grads:
            shapes = ((I, H), (I, H), (H, I))
            if grads is None:
                grads = tuple(torch.empty(n, dtype=torch.float32, device=dev) for n in shapes)
            for t, n, what in zip(grads, shapes, ("dgate", "dup", "ddown")):
                _grad_buffer(t, n, what)
                if t.get_device() != index:
                    raise ValueError("the tensors must be on one CUDA device")
            dtypes = {t.dtype for t in grads}
            if dtypes not in ({torch.float32}, {torch.bfloat16}) or len(grads) != 3:
                raise ValueError("grads must be three buffers, all fp32 or all bf16")
            gt = MOE_G_BF16 if torch.bfloat16 in dtypes else MOE_G_FP32
            at = moe_ffn_grads(*[t.data_ptr() for t in grads], *[_ld(t) for t in grads])
        size = _sized(_ffn_back_size, self._back_sizes, self.cfg, T, index)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        status = self._backward(self.cfg, T, dy.data_ptr(), _ld(dy), w, views, _addr(dx), H, at, gt, 1 if accumulate else 0,
                                workspace.data_ptr(), size, self._stream(index))
        if status:
            raise MoeError(status, "moe_ffn_backward")
        return dx, grads
