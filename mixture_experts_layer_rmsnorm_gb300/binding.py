"""Python binding of the C ABI in include/moe.h (argument marshalling only).

Every function here has the name of the C entry point it calls and forwards
plain integers / device pointers; all of the layer's work runs in the CUDA
kernels of libmoe_gb300.so.  There is no fallback: if the library cannot be
built or loaded, :func:`load` raises.

:class:`MoeLayer` is a convenience holder for torch tensors (weights and a
workspace on the GPU) that marshals their pointers into :func:`moe_forward`.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import _build

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_TIMEOUT, \
    MOE_ERR_DEVICE = range(7)

_lock = threading.Lock()
_lib = None


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("eps", ctypes.c_float)]


class MoeViews(ctypes.Structure):
    _fields_ = [("error_word", ctypes.c_void_p), ("h", ctypes.c_void_p), ("logits", ctypes.c_void_p),
                ("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("sorted_ids", ctypes.c_void_p), ("slot_of", ctypes.c_void_p),
                ("xg", ctypes.c_void_p), ("act", ctypes.c_void_p), ("out_rows", ctypes.c_void_p),
                ("P_max", ctypes.c_int64)]


class MoeMxViews(ctypes.Structure):
    _fields_ = [("x_codes", ctypes.c_void_p), ("x_scales", ctypes.c_void_p), ("act_codes", ctypes.c_void_p),
                ("act_scales", ctypes.c_void_p), ("x_chunk_rows", ctypes.c_int32), ("act_chunk_rows", ctypes.c_int32),
                ("x_gscale", ctypes.c_void_p), ("act_gscale", ctypes.c_void_p), ("nv_chunk_rows", ctypes.c_int32)]


class MoeGroupedShape(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("type", ctypes.c_int32),
                ("rows", ctypes.c_int64)]


class MoeFp4Shape(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("groups", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("K", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {moe_status_string(status)} (status {status})")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load(build: bool = True):
    """Load libmoe_gb300.so (compiling it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build() if build else _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library {path} is missing; run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            p, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
            sp = ctypes.POINTER(MoeShape)
            lib.moe_workspace_size.argtypes = [sp, ctypes.POINTER(sz)]
            lib.moe_forward.argtypes = [sp, p, p, p, p, p, p, p, p, sz, p]
            lib.moe_forward_events.argtypes = [sp, p, p, p, p, p, p, p, p, sz, p, p, i32]
            lib.moe_route_debug.argtypes = [sp, p, p, p, p, i32, p, p, p, p, i64, p, sz, p]
            lib.moe_forward_static_scratch.argtypes = [sp, p, p, p, p, p, p, p, p]
            lib.moe_static_scratch_bytes.argtypes = [ctypes.POINTER(sz)]
            lib.moe_static_scratch_device_status.argtypes = [p, ctypes.POINTER(ctypes.c_int32)]
            lib.moe_workspace_views.argtypes = [sp, p, sz, ctypes.POINTER(MoeViews)]
            lib.moe_device_status.argtypes = [p, sz, p, ctypes.POINTER(ctypes.c_int32)]
            lib.moe_kernels_per_call.argtypes = [sp, ctypes.POINTER(ctypes.c_int32)]
            lib.moe_kernels_per_call_of.argtypes = [sp, i32, ctypes.POINTER(ctypes.c_int32)]
            lib.moe_selftest_wait_timeout.argtypes = [p, sz, i64, p]
            lib.moe_qk_norm.argtypes = [i64, i32, i32, i32, p, p, p, p, ctypes.c_float, ctypes.c_float, p]
            psz = ctypes.POINTER(sz)
            lib.moe_mx_weight_sizes.argtypes = [sp, psz, psz, psz, psz]
            lib.moe_mx_quantize_weights.argtypes = [sp, p, p, p, p, p, p, p]
            lib.moe_workspace_size_mx.argtypes = [sp, psz]
            lib.moe_workspace_views_mx.argtypes = [sp, p, sz, ctypes.POINTER(MoeViews), ctypes.POINTER(MoeMxViews)]
            lib.moe_forward_mx.argtypes = [sp, p, p, p, p, p, p, p, p, p, p, sz, p, p, i32]
            lib.moe_mxfp4_weight_sizes.argtypes = [sp, psz, psz, psz, psz]
            lib.moe_mxfp4_quantize_weights.argtypes = [sp, p, p, p, p, p, p, p]
            lib.moe_forward_mxfp4.argtypes = [sp, p, p, p, p, p, p, p, p, p, p, sz, p, p, i32]
            lib.moe_forward_mxfp4a4.argtypes = [sp, p, p, p, p, p, p, p, p, p, p, sz, p, p, i32]
            lib.moe_nvfp4_weight_sizes.argtypes = [sp, psz, psz, psz, psz]
            lib.moe_nvfp4_quantize_weights.argtypes = [sp, p, p, p, p, p, p, p, p, p]
            lib.moe_forward_nvfp4.argtypes = [sp, p, p, p, p, p, p, p, p, p, p, p, p, sz, p, p, i32]
            lib.moe_forward_fused_front.argtypes = [sp, p, p, p, p, p, p, p, p, sz, p, p, i32]
            lib.moe_forward_fused_combine.argtypes = [sp, p, p, p, p, p, p, p, p, sz, p, p, i32]
            lib.moe_forward_fused_mlp.argtypes = [sp, p, p, p, p, p, p, p, p, sz, p, p, i32]
            gp = ctypes.POINTER(MoeGroupedShape)
            lib.moe_grouped_workspace_size.argtypes = [gp, psz]
            lib.moe_grouped_gemm.argtypes = [gp, p, i64, p, p, p, p, i64, p, sz, p]
            lib.moe_grouped_gemm_dgrad.argtypes = [gp, p, i64, p, p, p, p, i64, p, sz, p]
            lib.moe_grouped_gemm_wgrad.argtypes = [gp, p, i64, p, i64, p, p, p, i32, i32, p, sz, p]
            lib.moe_swiglu.argtypes = [i32, i64, i32, p, i64, p, i64, p]
            lib.moe_swiglu_grad.argtypes = [i32, i64, i32, p, i64, p, i64, p, i64, p]
            fp = ctypes.POINTER(MoeFp4Shape)
            lib.moe_fp4_sizes.argtypes = [fp, psz, psz]
            lib.moe_fp4_quantize.argtypes = [fp, i32, p, i64, p, p, p, p, p, i32, p]
            lib.moe_fp4_dequantize.argtypes = [fp, p, p, p, i32, p, p, i32, p, i64, p]
            lib.moe_fp4_gemm.argtypes = [gp, i32, p, p, p, p, p, p, p, p, p, i64, p, sz, p]
            lib.moe_status_string.argtypes = [ctypes.c_int]
            lib.moe_status_string.restype = ctypes.c_char_p
            for f in ("moe_workspace_size", "moe_forward", "moe_forward_events", "moe_route_debug",
                      "moe_workspace_views", "moe_device_status", "moe_forward_static_scratch",
                      "moe_static_scratch_bytes", "moe_static_scratch_device_status",
                      "moe_kernels_per_call", "moe_kernels_per_call_of", "moe_forward_fused_front",
                      "moe_selftest_wait_timeout",
                      "moe_qk_norm", "moe_mx_weight_sizes", "moe_mx_quantize_weights", "moe_workspace_size_mx",
                      "moe_workspace_views_mx", "moe_forward_mx", "moe_forward_fused_combine",
                      "moe_mxfp4_weight_sizes", "moe_mxfp4_quantize_weights", "moe_forward_mxfp4",
                      "moe_forward_mxfp4a4", "moe_nvfp4_weight_sizes", "moe_nvfp4_quantize_weights",
                      "moe_forward_nvfp4", "moe_forward_fused_mlp", "moe_grouped_workspace_size",
                      "moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad", "moe_swiglu",
                      "moe_swiglu_grad", "moe_fp4_sizes", "moe_fp4_quantize", "moe_fp4_dequantize", "moe_fp4_gemm"):
                getattr(lib, f).restype = ctypes.c_int
            _lib = lib
    return _lib


def shape(T, H, I, E, top_k, renormalize=True, eps=1e-6) -> MoeShape:
    return MoeShape(int(T), int(H), int(I), int(E), int(top_k), int(bool(renormalize)), float(eps))


def moe_status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


def moe_workspace_size(s: MoeShape) -> tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load().moe_workspace_size(ctypes.byref(s), ctypes.byref(n))
    return st, n.value


def moe_forward(s: MoeShape, x, g_norm, w_router, router_bias, w13, w2, y, workspace, workspace_bytes,
                stream) -> int:
    return load().moe_forward(ctypes.byref(s), x, g_norm, w_router, router_bias, w13, w2, y, workspace,
                              workspace_bytes, stream)


MOE_NUM_KERNELS = 7
MOE_FRONT_MAX_T = 64  # single-launch front end (norm .. gather) up to this many tokens ...
MOE_FRONT_MAX_E = 256  # ... and experts
MOE_FUSED_TOPK_MAX_T = 256  # top-k runs inside the align kernel up to this many tokens ...
MOE_FUSED_TOPK_MAX_E = 256  # ... and experts


def moe_kernels_per_call(s: MoeShape) -> tuple[int, int]:
    n = ctypes.c_int32(0)
    st = load().moe_kernels_per_call(ctypes.byref(s), ctypes.byref(n))
    return st, n.value


(MOE_CALL_FORWARD, MOE_CALL_FORWARD_FUSED_FRONT, MOE_CALL_FORWARD_MX, MOE_CALL_FORWARD_FUSED_COMBINE,
 MOE_CALL_FORWARD_MXFP4, MOE_CALL_FORWARD_MXFP4A4, MOE_CALL_FORWARD_NVFP4, MOE_CALL_FORWARD_FUSED_MLP) = \
    0, 1, 2, 3, 4, 5, 6, 7


def moe_kernels_per_call_of(s: MoeShape, call: int) -> tuple[int, int]:
    n = ctypes.c_int32(0)
    st = load().moe_kernels_per_call_of(ctypes.byref(s), int(call), ctypes.byref(n))
    return st, n.value


def kernels_per_call(T: int, H: int, I: int, E: int, top_k: int, call: int = MOE_CALL_FORWARD) -> int:
    """Kernel launches of one call of the entry point `call` (MOE_CALL_*)."""
    st, n = moe_kernels_per_call_of(shape(T, H, I, E, top_k), call)
    if st != MOE_OK:
        raise MoeError(st, "moe_kernels_per_call_of")
    return n


KERNEL_NAMES = ("norm_router", "topk_softmax", "align", "gather", "gemm_gate_up_swiglu", "gemm_down", "combine")


def moe_forward_events(s: MoeShape, x, g_norm, w_router, router_bias, w13, w2, y, workspace, workspace_bytes,
                       stream, events) -> int:
    """events: a sequence of MOE_NUM_KERNELS + 1 raw cudaEvent_t handles (ints)."""
    arr = (ctypes.c_void_p * len(events))(*events)
    return load().moe_forward_events(ctypes.byref(s), x, g_norm, w_router, router_bias, w13, w2, y, workspace,
                                     workspace_bytes, stream, arr, len(events))


def moe_forward_fused_front(s: MoeShape, x, g_norm, w_router, router_bias, w13, w2, y, workspace,
                            workspace_bytes, stream, events=None) -> int:
    """moe_forward with norm .. gather as one cluster launch (decode shapes only)."""
    if events is None:
        arr, n = None, 0
    else:
        arr, n = (ctypes.c_void_p * len(events))(*events), len(events)
    return load().moe_forward_fused_front(ctypes.byref(s), x, g_norm, w_router, router_bias, w13, w2, y, workspace,
                                          workspace_bytes, stream, arr, n)


def moe_forward_fused_combine(s: MoeShape, x, g_norm, w_router, router_bias, w13, w2, y, workspace,
                              workspace_bytes, stream, events=None) -> int:
    """moe_forward with the top-k weighted combine in the down GEMM's epilogue."""
    if events is None:
        arr, n = None, 0
    else:
        arr, n = (ctypes.c_void_p * len(events))(*events), len(events)
    return load().moe_forward_fused_combine(ctypes.byref(s), x, g_norm, w_router, router_bias, w13, w2, y,
                                            workspace, workspace_bytes, stream, arr, n)


def moe_forward_fused_mlp(s: MoeShape, x, g_norm, w_router, router_bias, w13, w2, y, workspace, workspace_bytes,
                          stream, events=None) -> int:
    """moe_forward with both expert GEMMs in one launch (decode tile plan only)."""
    if events is None:
        arr, n = None, 0
    else:
        arr, n = (ctypes.c_void_p * len(events))(*events), len(events)
    return load().moe_forward_fused_mlp(ctypes.byref(s), x, g_norm, w_router, router_bias, w13, w2, y, workspace,
                                        workspace_bytes, stream, arr, n)


def moe_static_scratch_bytes() -> tuple[int, int]:
    """Size of the library's fixed device scratch array, as compiled into it."""
    n = ctypes.c_size_t(0)
    st = load().moe_static_scratch_bytes(ctypes.byref(n))
    return st, n.value


def moe_static_scratch_device_status(stream) -> tuple[int, list]:
    """moe_device_status for moe_forward_static_scratch (the current device's array)."""
    d = (ctypes.c_int32 * 4)()
    st = load().moe_static_scratch_device_status(stream, d)
    return st, list(d)


def moe_forward_static_scratch(s: MoeShape, x, g_norm, w_router, router_bias, w13, w2, y, stream) -> int:
    """moe_forward with the library's fixed device scratch array instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    return load().moe_forward_static_scratch(ctypes.byref(s), x, g_norm, w_router, router_bias, w13, w2, y, stream)


def moe_route_debug(s: MoeShape, x, g_norm, w_router, router_bias, pad_rows, topk_ids, topk_w, expert_offsets,
                    sorted_ids, sorted_capacity, workspace, workspace_bytes, stream) -> int:
    return load().moe_route_debug(ctypes.byref(s), x, g_norm, w_router, router_bias, pad_rows, topk_ids, topk_w,
                                  expert_offsets, sorted_ids, sorted_capacity, workspace, workspace_bytes, stream)


def moe_workspace_views(s: MoeShape, workspace, workspace_bytes) -> tuple[int, MoeViews]:
    v = MoeViews()
    st = load().moe_workspace_views(ctypes.byref(s), workspace, workspace_bytes, ctypes.byref(v))
    return st, v


def moe_device_status(workspace, workspace_bytes, stream) -> tuple[int, list]:
    d = (ctypes.c_int32 * 4)()
    st = load().moe_device_status(workspace, workspace_bytes, stream, d)
    return st, list(d)


def moe_qk_norm(T, Hq, Hk, D, q, k, q_weight, k_weight, weight_bias, eps, stream) -> int:
    return load().moe_qk_norm(int(T), int(Hq), int(Hk), int(D), q, k, q_weight, k_weight, float(weight_bias),
                              float(eps), stream)


def moe_selftest_wait_timeout(workspace, workspace_bytes, timeout_ns, stream) -> int:
    return load().moe_selftest_wait_timeout(workspace, workspace_bytes, int(timeout_ns), stream)


def moe_mx_weight_sizes(s: MoeShape) -> tuple[int, tuple[int, int, int, int]]:
    v = [ctypes.c_size_t(0) for _ in range(4)]
    st = load().moe_mx_weight_sizes(ctypes.byref(s), *[ctypes.byref(a) for a in v])
    return st, tuple(a.value for a in v)


def moe_mx_quantize_weights(s: MoeShape, w13, w2, w13_codes, w13_scales, w2_codes, w2_scales, stream) -> int:
    return load().moe_mx_quantize_weights(ctypes.byref(s), w13, w2, w13_codes, w13_scales, w2_codes, w2_scales,
                                          stream)


def moe_workspace_size_mx(s: MoeShape) -> tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load().moe_workspace_size_mx(ctypes.byref(s), ctypes.byref(n))
    return st, n.value


def moe_workspace_views_mx(s: MoeShape, workspace, workspace_bytes) -> tuple[int, MoeViews, MoeMxViews]:
    v, mv = MoeViews(), MoeMxViews()
    st = load().moe_workspace_views_mx(ctypes.byref(s), workspace, workspace_bytes, ctypes.byref(v), ctypes.byref(mv))
    return st, v, mv


def moe_forward_mx(s: MoeShape, x, g_norm, w_router, router_bias, w13_codes, w13_scales, w2_codes, w2_scales, y,
                   workspace, workspace_bytes, stream, events=None) -> int:
    if events is None:
        arr, n = None, 0
    else:
        arr, n = (ctypes.c_void_p * len(events))(*events), len(events)
    return load().moe_forward_mx(ctypes.byref(s), x, g_norm, w_router, router_bias, w13_codes, w13_scales, w2_codes,
                                 w2_scales, y, workspace, workspace_bytes, stream, arr, n)


def moe_mxfp4_weight_sizes(s: MoeShape) -> tuple[int, tuple[int, int, int, int]]:
    v = [ctypes.c_size_t(0) for _ in range(4)]
    st = load().moe_mxfp4_weight_sizes(ctypes.byref(s), *[ctypes.byref(a) for a in v])
    return st, tuple(a.value for a in v)


def moe_mxfp4_quantize_weights(s: MoeShape, w13, w2, w13_codes, w13_scales, w2_codes, w2_scales, stream) -> int:
    return load().moe_mxfp4_quantize_weights(ctypes.byref(s), w13, w2, w13_codes, w13_scales, w2_codes, w2_scales,
                                             stream)


def moe_forward_mxfp4(s: MoeShape, x, g_norm, w_router, router_bias, w13_codes, w13_scales, w2_codes, w2_scales, y,
                      workspace, workspace_bytes, stream, events=None) -> int:
    if events is None:
        arr, n = None, 0
    else:
        arr, n = (ctypes.c_void_p * len(events))(*events), len(events)
    return load().moe_forward_mxfp4(ctypes.byref(s), x, g_norm, w_router, router_bias, w13_codes, w13_scales,
                                    w2_codes, w2_scales, y, workspace, workspace_bytes, stream, arr, n)


def moe_forward_mxfp4a4(s: MoeShape, x, g_norm, w_router, router_bias, w13_codes, w13_scales, w2_codes, w2_scales,
                        y, workspace, workspace_bytes, stream, events=None) -> int:
    if events is None:
        arr, n = None, 0
    else:
        arr, n = (ctypes.c_void_p * len(events))(*events), len(events)
    return load().moe_forward_mxfp4a4(ctypes.byref(s), x, g_norm, w_router, router_bias, w13_codes, w13_scales,
                                      w2_codes, w2_scales, y, workspace, workspace_bytes, stream, arr, n)


def moe_nvfp4_weight_sizes(s: MoeShape) -> tuple[int, tuple[int, int, int, int]]:
    v = [ctypes.c_size_t(0) for _ in range(4)]
    st = load().moe_nvfp4_weight_sizes(ctypes.byref(s), *[ctypes.byref(a) for a in v])
    return st, tuple(a.value for a in v)


def moe_nvfp4_quantize_weights(s: MoeShape, w13, w2, w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales,
                               w2_gscale, stream) -> int:
    return load().moe_nvfp4_quantize_weights(ctypes.byref(s), w13, w2, w13_codes, w13_scales, w13_gscale, w2_codes,
                                             w2_scales, w2_gscale, stream)


def moe_forward_nvfp4(s: MoeShape, x, g_norm, w_router, router_bias, w13_codes, w13_scales, w13_gscale, w2_codes,
                      w2_scales, w2_gscale, y, workspace, workspace_bytes, stream, events=None) -> int:
    if events is None:
        arr, n = None, 0
    else:
        arr, n = (ctypes.c_void_p * len(events))(*events), len(events)
    return load().moe_forward_nvfp4(ctypes.byref(s), x, g_norm, w_router, router_bias, w13_codes, w13_scales,
                                    w13_gscale, w2_codes, w2_scales, w2_gscale, y, workspace, workspace_bytes, stream,
                                    arr, n)


def _ptr(t):
    return None if t is None else t.data_ptr()


MOE_TYPE_BF16, MOE_TYPE_FP16, MOE_TYPE_FP32 = range(3)


def grouped_shape(groups, N, K, rows, type=MOE_TYPE_BF16) -> MoeGroupedShape:
    return MoeGroupedShape(int(groups), int(N), int(K), int(type), int(rows))


def moe_grouped_workspace_size(s: MoeGroupedShape) -> tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load().moe_grouped_workspace_size(ctypes.byref(s), ctypes.byref(n))
    return st, n.value


def moe_grouped_gemm(s: MoeGroupedShape, x, ldx, w, offsets, counts, y, ldy, workspace, workspace_bytes,
                     stream) -> int:
    return load().moe_grouped_gemm(ctypes.byref(s), x, ldx, w, offsets, counts, y, ldy, workspace, workspace_bytes,
                                   stream)


def moe_grouped_gemm_dgrad(s: MoeGroupedShape, dy, lddy, w, offsets, counts, dx, lddx, workspace, workspace_bytes,
                           stream) -> int:
    return load().moe_grouped_gemm_dgrad(ctypes.byref(s), dy, lddy, w, offsets, counts, dx, lddx, workspace,
                                         workspace_bytes, stream)


def moe_grouped_gemm_wgrad(s: MoeGroupedShape, dy, lddy, x, ldx, offsets, counts, dw, dw_type, accumulate, workspace,
                           workspace_bytes, stream) -> int:
    return load().moe_grouped_gemm_wgrad(ctypes.byref(s), dy, lddy, x, ldx, offsets, counts, dw, int(dw_type),
                                         int(bool(accumulate)), workspace, workspace_bytes, stream)


def moe_swiglu(type, rows, I, h, ldh, act, ldact, stream) -> int:
    return load().moe_swiglu(int(type), int(rows), int(I), h, ldh, act, ldact, stream)


def moe_swiglu_grad(type, rows, I, h, ldh, dact, lddact, dh, lddh, stream) -> int:
    return load().moe_swiglu_grad(int(type), int(rows), int(I), h, ldh, dact, lddact, dh, lddh, stream)


MOE_FORMAT_MXFP4, MOE_FORMAT_NVFP4 = range(2)
MOE_SCALE_PER_ROW, MOE_SCALE_PER_GROUP = range(2)


def fp4_shape(format, groups, rows, K) -> MoeFp4Shape:
    return MoeFp4Shape(int(format), int(groups), int(rows), int(K))


def moe_fp4_sizes(s: MoeFp4Shape) -> tuple[int, tuple[int, int]]:
    v = [ctypes.c_size_t(0) for _ in range(2)]
    st = load().moe_fp4_sizes(ctypes.byref(s), *[ctypes.byref(a) for a in v])
    return st, tuple(a.value for a in v)


def moe_fp4_quantize(s: MoeFp4Shape, src_type, src, ldsrc, offsets, counts, codes, scales, gscale, gscale_per,
                     stream) -> int:
    return load().moe_fp4_quantize(ctypes.byref(s), int(src_type), src, ldsrc, offsets, counts, codes, scales, gscale,
                                   int(gscale_per), stream)


def moe_fp4_dequantize(s: MoeFp4Shape, codes, scales, gscale, gscale_per, offsets, counts, dst_type, dst, lddst,
                       stream) -> int:
    return load().moe_fp4_dequantize(ctypes.byref(s), codes, scales, gscale, int(gscale_per), offsets, counts,
                                     int(dst_type), dst, lddst, stream)


def moe_fp4_gemm(s: MoeGroupedShape, format, x_codes, x_scales, x_gscale, w_codes, w_scales, w_gscale, offsets, counts,
                 y, ldy, workspace, workspace_bytes, stream) -> int:
    return load().moe_fp4_gemm(ctypes.byref(s), int(format), x_codes, x_scales, x_gscale, w_codes, w_scales, w_gscale,
                               offsets, counts, y, ldy, workspace, workspace_bytes, stream)


_types = {}


def _type_of(dtype) -> int:
    if not _types:
        import torch
        _types.update({torch.bfloat16: MOE_TYPE_BF16, torch.float16: MOE_TYPE_FP16, torch.float32: MOE_TYPE_FP32})
    if dtype not in _types:
        raise TypeError(f"{dtype}: bfloat16, float16 or float32 wanted")
    return _types[dtype]


def _check(what, t, device, dtype, shape_, rows=False):
    """A tensor argument: its device, type and shape; contiguous, or (rows) rows of contiguous elements."""
    if t.dtype == dtype and t.shape == shape_ and t.device == device and (
            t.is_contiguous() or (rows and (t.stride(-1) == 1 or t.shape[-1] == 1))):
        return t
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{what} is {t.dtype}, not {dtype}")
    if t.shape != shape_:
        raise ValueError(f"{what} is {tuple(t.shape)}, not {tuple(shape_)}")
    raise ValueError(f"{what} is not contiguous" + (" along its rows" if rows else ""))


def _lists(of, offsets, counts):
    """The row lists of an object with ``groups`` and ``device``, as pointers."""
    if offsets is not None:
        offsets = _check("offsets", offsets, of.device, of.int32, (of.groups + 1,)).data_ptr()
    if counts is not None:
        counts = _check("counts", counts, of.device, of.int32, (of.groups,)).data_ptr()
    return offsets, counts


def _matrix(what, t, device, dtype, shape_):
    """A matrix argument, rows of contiguous elements: its pointer and row stride."""
    if t.dtype == dtype and t.shape == shape_ and t.device == device:  # (the common way, in few calls)
        ld, one = t.stride()
        if one == 1 and shape_[0] > 1:
            return t.data_ptr(), ld
    _check(what, t, device, dtype, shape_, rows=True)
    return t.data_ptr(), t.stride(0) if shape_[0] > 1 else (shape_[1] + 7) // 8 * 8  # (one row's stride says nothing)


_torch = None


def _empty(shape_, dtype, device):
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch.empty(shape_, dtype=dtype, device=device)


_C = None  # torch's native module, once it is needed


class _Buffers:
    """An object that keeps buffers on ``device``, listed by ``_buffers()``.  A stream that uses them is made known to
    the allocator once, so that the object may go while its work is queued there."""

    _streams = frozenset()

    def _used_on(self, stream):
        import torch
        for t in self._buffers():
            if t is not None:
                t.record_stream(torch.cuda.current_stream(self.device))
        self._streams = self._streams | {stream}  # (one assignment: other host threads may ask too)


def _enqueue(name, device, *args, of=()):
    """name(*args, stream) of the library with ``device`` current, on its current stream; MoeError if it fails.  of:
    the objects whose buffers it uses."""
    global _C
    if device.type != "cuda":
        raise ValueError(f"{name}: tensors on {device}, not on a CUDA device")
    if _C is None:
        from torch import _C as native
        _C = native
    index, fn = device.index, getattr(_lib or load(), name)
    here = _C._cuda_getDevice() == index  # (the tensors exist: CUDA is initialised)
    stream = _C._cuda_getCurrentRawStream(index)
    for o in of:
        if stream not in o._streams:
            o._used_on(stream)
    if here:
        st = fn(*args, stream)
    else:
        from torch import cuda
        with cuda.device(device):
            st = fn(*args, stream)
    if st != MOE_OK:
        raise MoeError(st, name)


def swiglu(h, act=None):
    """SiLU(gate) * up of rows h = [gate | up] (moe_swiglu), on the current stream of h's device."""
    rows, two_i = h.shape
    i, device, dtype = two_i // 2, h.device, h.dtype
    hp, ldh = _matrix("h", h, device, dtype, (rows, 2 * i))
    if act is None:
        act = _empty((rows, i), dtype, device)
    ap, lda = _matrix("act", act, device, dtype, (rows, i))
    _enqueue("moe_swiglu", device, _type_of(dtype), rows, i, hp, ldh, ap, lda)
    return act


def swiglu_grad(h, dact, dh=None):
    """d[gate | up] from dact (moe_swiglu_grad), on the current stream of h's device."""
    rows, two_i = h.shape
    i, device, dtype = two_i // 2, h.device, h.dtype
    hp, ldh = _matrix("h", h, device, dtype, (rows, 2 * i))
    ap, lda = _matrix("dact", dact, device, dtype, (rows, i))
    if dh is None:
        dh = _empty((rows, 2 * i), dtype, device)
    dp, ldd = _matrix("dh", dh, device, dtype, (rows, 2 * i))
    _enqueue("moe_swiglu_grad", device, _type_of(dtype), rows, i, hp, ldh, ap, lda, dp, ldd)
    return dh


class _Workspace(_Buffers):
    """A workspace of the grouped calls, for an object with ``device`` and ``workspace``."""

    called = False  # a call was accepted

    def _new_workspace(self, bytes_):
        import torch
        workspace = torch.empty(bytes_, dtype=torch.uint8, device=self.device)
        workspace[:16].zero_()  # no status yet: a captured call may be replayed later, or never
        return workspace

    def _buffers(self):
        return (self.workspace,)

    def _call(self, name, shape_, *args, of=()):
        if shape_.rows == 0:  # nothing is enqueued: what a call before it reported is not its own
            self.workspace[:16].zero_()
        _enqueue(name, self.device, ctypes.byref(shape_), *args, self.workspace.data_ptr(), self.workspace.numel(),
                 of=(self, *of))
        self.called = True

    def device_status(self):
        """(status, detail) of the last call, after waiting for the current stream (moe_device_status)."""
        if not self.called:  # (what the workspace holds means nothing yet)
            return MOE_OK, [0] * 4
        import torch
        with torch.cuda.device(self.device):
            return moe_device_status(_ptr(self.workspace), self.workspace.numel(),
                                     torch.cuda.current_stream().cuda_stream)


class GroupedProducts(_Workspace):
    """The products of ``groups`` weight matrices [N, K] with the rows of their
    groups, and the gradients (moe_grouped_gemm*), with a workspace of their
    own.  Calls go to the current stream of the tensors' device; calls of one
    object on several streams share its workspace and must not overlap.
    max_rows: rows the workspace is made for; weight gradients into 16 bits of more
    get a larger one (the outgrown one lives as long as the object, for graphs that
    were captured with it and work still queued on other streams).
    offsets: int32 [groups + 1] on the device, or None (equal groups);
    counts: int32 [groups] or None (offsets[g + 1] - offsets[g])."""

    def __init__(self, groups, N, K, dtype, max_rows=0, device=None):
        import torch
        self.groups, self.N, self.K, self.dtype = int(groups), int(N), int(K), dtype
        self.device = torch.empty(0, device=device or "cuda").device
        self._shape, self.int32 = None, torch.int32
        self.workspace, self._outgrown = None, []
        self._ensure_workspace(int(max_rows))

    def _ensure_workspace(self, rows):
        """A workspace for calls of up to ``rows`` rows."""
        st, n = moe_grouped_workspace_size(self.shape(rows))
        if st != MOE_OK:
            raise MoeError(st, "moe_grouped_workspace_size")
        if self.workspace is None or n > self.workspace.numel():
            workspace = self._new_workspace(n)
            if self.workspace is not None:
                self._outgrown.append(self.workspace)
            self.workspace, self.called, self._streams = workspace, False, frozenset()
        self.max_rows = rows

    def shape(self, rows) -> MoeGroupedShape:
        s = self._shape  # (kept by one assignment: other host threads may ask too)
        if s is None or s.rows != rows:
            s = self._shape = grouped_shape(self.groups, self.N, self.K, rows, _type_of(self.dtype))
        return s

    def _weights(self, w):
        return _check("w", w, self.device, self.dtype, (self.groups, self.N, self.K)).data_ptr()

    def forward(self, x, w, offsets=None, counts=None, y=None):
        """y[p] = x[p] w_g^T for the rows p of every group g; other rows of y stay as they are."""
        rows = x.shape[0]
        xp, ldx = _matrix("x", x, self.device, self.dtype, (rows, self.K))
        if y is None:
            y = _empty((rows, self.N), self.dtype, self.device)
        yp, ldy = _matrix("y", y, self.device, self.dtype, (rows, self.N))
        self._call("moe_grouped_gemm", self.shape(rows), xp, ldx, self._weights(w), *_lists(self, offsets, counts), yp,
                   ldy)
        return y

    def dgrad(self, dy, w, offsets=None, counts=None, dx=None):
        """dx[p] = dy[p] w_g."""
        rows = dy.shape[0]
        yp, ldy = _matrix("dy", dy, self.device, self.dtype, (rows, self.N))
        if dx is None:
            dx = _empty((rows, self.K), self.dtype, self.device)
        xp, ldx = _matrix("dx", dx, self.device, self.dtype, (rows, self.K))
        self._call("moe_grouped_gemm_dgrad", self.shape(rows), yp, ldy, self._weights(w),
                   *_lists(self, offsets, counts), xp, ldx)
        return dx

    def wgrad(self, dy, x, offsets=None, counts=None, dw=None, dtype=None, accumulate=False):
        """dw_g = sum over the group's rows of dy[p]^T x[p], in ``dtype`` (fp32 or the operands' type, the default)
        or dw's type; accumulate (fp32): added to dw."""
        rows = x.shape[0]
        yp, ldy = _matrix("dy", dy, self.device, self.dtype, (rows, self.N))
        xp, ldx = _matrix("x", x, self.device, self.dtype, (rows, self.K))
        if dw is None:
            if accumulate:
                raise ValueError("accumulate adds to dw: pass it")
            dw = _empty((self.groups, self.N, self.K), dtype or self.dtype, self.device)
        else:
            _check("dw", dw, self.device, dtype or dw.dtype, (self.groups, self.N, self.K))
        if rows > self.max_rows and dw.dtype == self.dtype:
            self._ensure_workspace(rows)
        self._call("moe_grouped_gemm_wgrad", self.shape(rows), yp, ldy, xp, ldx, *_lists(self, offsets, counts),
                   dw.data_ptr(), _type_of(dw.dtype), 1 if accumulate else 0)
        return dw


def _format_of(name) -> int:
    formats = {"mx": MOE_FORMAT_MXFP4, "nv": MOE_FORMAT_NVFP4}
    if name not in formats:
        raise ValueError(f"format {name!r}: 'mx' (MXFP4) or 'nv' (NVFP4) wanted")
    return formats[name]


class Fp4Rows(_Buffers):
    """Rows of groups in 4 bits (moe_fp4_quantize, moe_fp4_dequantize): buffers
    for up to ``max_rows`` rows of K elements, filled by :meth:`quantize`.
    format: "mx" (MXFP4) or "nv" (NVFP4, one fp32 scale per row).  offsets and
    counts as for :class:`GroupedProducts`; pass the same ones to every call on
    the same rows.  Calls go to the current stream of the device.  More rows than
    ``max_rows`` get larger buffers; the outgrown ones live as long as the object,
    for graphs that were captured with them and work still queued on other streams."""

    def __init__(self, format, K, groups=1, max_rows=0, device=None):
        import torch
        self.format, self.K, self.groups = _format_of(format), int(K), int(groups)
        self.device, self.int32 = torch.empty(0, device=device or "cuda").device, torch.int32
        self.rows = self.max_rows = 0
        self._shape = None
        self._outgrown, self._listed = [], None
        self.ensure_capacity(max_rows)

    def shape(self, rows) -> MoeFp4Shape:
        s = self._shape  # (kept by one assignment: other host threads may ask too)
        if s is None or s.rows != rows:
            s = self._shape = fp4_shape(self.format, self.groups, rows, self.K)
        return s

    def ensure_capacity(self, rows):
        """Buffers for up to ``rows`` rows; new ones hold no rows yet (``rows`` becomes 0)."""
        if rows <= self.max_rows and self.max_rows > 0:
            return
        import torch
        # (by half at least: what outgrown buffers hold stays below twice the last ones)
        rows = max(rows, min(self.max_rows * 3 // 2, 2 ** 31 - 512), 1)
        st, (n_codes, n_scales) = moe_fp4_sizes(fp4_shape(self.format, self.groups, rows, self.K))
        if st != MOE_OK:
            raise MoeError(st, "moe_fp4_sizes")
        # (all of them before any takes its place: where one does not fit, the rows before stay)
        codes = torch.empty(n_codes, dtype=torch.uint8, device=self.device)
        scales = torch.empty(n_scales, dtype=torch.uint8, device=self.device)
        gscale = (torch.empty(rows, dtype=torch.float32, device=self.device)
                  if self.format == MOE_FORMAT_NVFP4 else None)
        if self.max_rows > 0:
            self._outgrown.append((self.codes, self.scales, self.gscale))
        self.codes, self.scales, self.gscale, self.max_rows = codes, scales, gscale, rows
        self.rows, self._listed, self._streams = 0, None, frozenset()

    def _buffers(self):
        return self.codes, self.scales, self.gscale

    def quantize(self, x, offsets=None, counts=None):
        """x [rows, K] (bf16, fp16 or fp32) to 4 bits; returns self."""
        rows = x.shape[0]
        xp, ldx = _matrix("x", x, self.device, x.dtype, (rows, self.K))
        lists, type_ = _lists(self, offsets, counts), _type_of(x.dtype)
        self.ensure_capacity(rows)
        self.rows = 0  # (until they are on their way)
        _enqueue("moe_fp4_quantize", self.device, ctypes.byref(self.shape(rows)), type_, xp, ldx, *lists,
                 self.codes.data_ptr(), self.scales.data_ptr(), _ptr(self.gscale), MOE_SCALE_PER_ROW, of=(self,))
        self.rows, self._listed = rows, offsets is not None
        return self

    def check_lists(self, offsets):
        # (listed groups' scales lie elsewhere than equal groups')
        if self._listed is not None and self._listed != (offsets is not None):
            raise ValueError(f"the rows were quantized {'with' if self._listed else 'without'} offsets")

    def dequantize(self, offsets=None, counts=None, y=None, dtype=None):
        """The values of the rows quantized last, in ``dtype`` (bf16 by default) or y's type."""
        self.check_lists(offsets)
        if y is None:
            import torch
            y = torch.empty((self.rows, self.K), dtype=dtype or torch.bfloat16, device=self.device)
        yp, ldy = _matrix("y", y, self.device, dtype or y.dtype, (self.rows, self.K))
        _enqueue("moe_fp4_dequantize", self.device, ctypes.byref(self.shape(self.rows)), self.codes.data_ptr(),
                 self.scales.data_ptr(), _ptr(self.gscale), MOE_SCALE_PER_ROW, *_lists(self, offsets, counts),
                 _type_of(y.dtype), yp, ldy, of=(self,))
        return y


class Fp4Weights(_Workspace):
    """Weights of ``groups`` matrices [N, K] in 4 bits and their product with 4-bit
    rows (moe_fp4_gemm).  codes: uint8 [groups, N, K / 2]; scales: the tiles of
    moe_fp4_quantize for equal groups of N rows; gscale: fp32 [groups] ("nv") or None."""

    def __init__(self, format, codes, scales, gscale=None):
        import torch
        self.format = _format_of(format)
        self.groups, self.N, half = codes.shape
        self.K, self.device, self.int32 = 2 * half, codes.device, torch.int32
        st, (_, n_scales) = moe_fp4_sizes(fp4_shape(self.format, self.groups, self.groups * self.N, self.K))
        if st != MOE_OK:
            raise MoeError(st, "moe_fp4_sizes")
        chunk = 128 if self.format == MOE_FORMAT_MXFP4 else 64
        need = self.groups * -(-self.N // 128) * -(-self.K // chunk) * 512
        _check("codes", codes, self.device, torch.uint8, codes.shape)
        _check("scales", scales, self.device, torch.uint8, scales.shape)
        if scales.numel() < need:
            raise ValueError(f"scales hold {scales.numel()} bytes, {need} wanted")
        if self.format == MOE_FORMAT_NVFP4:
            if gscale is None:
                raise ValueError("NVFP4 weights have an fp32 scale for each group")
            _check("gscale", gscale, self.device, torch.float32, (self.groups,))
        self.codes, self.scales, self.gscale, self._shape = codes, scales, gscale, None
        st, n = moe_grouped_workspace_size(grouped_shape(self.groups, self.N, self.K, 0))
        if st != MOE_OK:
            raise MoeError(st, "moe_grouped_workspace_size")
        self.workspace = self._new_workspace(n)

    def _buffers(self):
        return self.workspace, self.codes, self.scales, self.gscale

    def shape(self, rows, type) -> MoeGroupedShape:
        s = self._shape  # (kept by one assignment: other host threads may ask too)
        if s is None or s.rows != rows or s.type != type:
            s = self._shape = grouped_shape(self.groups, self.N, self.K, rows, type)
        return s

    @classmethod
    def quantize(cls, w, format):
        """From w [groups, N, K] (bf16, fp16 or fp32)."""
        import torch
        groups, N, K = w.shape
        _check("w", w, w.device, w.dtype, w.shape)
        s = fp4_shape(_format_of(format), groups, groups * N, K)
        st, (_, n_scales) = moe_fp4_sizes(s)
        if st != MOE_OK:
            raise MoeError(st, "moe_fp4_sizes")
        codes = torch.empty((groups, N, K // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty(n_scales, dtype=torch.uint8, device=w.device)
        gscale = torch.empty(groups, dtype=torch.float32, device=w.device) if format == "nv" else None
        _enqueue("moe_fp4_quantize", w.device, ctypes.byref(s), _type_of(w.dtype), _ptr(w), K, None, None,
                 _ptr(codes), _ptr(scales), _ptr(gscale), MOE_SCALE_PER_GROUP)
        return cls(format, codes, scales, gscale)

    def dequantize(self, dtype=None):
        """The values the weights stand for, [groups, N, K] in ``dtype`` (bf16 by default)."""
        import torch
        w = torch.empty((self.groups, self.N, self.K), dtype=dtype or torch.bfloat16, device=self.device)
        _enqueue("moe_fp4_dequantize", self.device,
                 ctypes.byref(fp4_shape(self.format, self.groups, self.groups * self.N, self.K)), _ptr(self.codes),
                 _ptr(self.scales), _ptr(self.gscale), MOE_SCALE_PER_GROUP, None, None, _type_of(w.dtype), _ptr(w),
                 self.K, of=(self,))
        return w

    def forward(self, rows: Fp4Rows, offsets=None, counts=None, y=None, dtype=None):
        """y[p] = x[p] w_g^T in ``dtype`` (bf16 by default, or fp16) or y's type; rows: x quantized for the same lists."""
        if rows.format != self.format or rows.K != self.K or rows.groups != self.groups or rows.device != self.device:
            raise ValueError("rows of another format, K, number of groups or device")
        rows.check_lists(offsets)
        if y is None:
            import torch
            y = torch.empty((rows.rows, self.N), dtype=dtype or torch.bfloat16, device=self.device)
        yp, ldy = _matrix("y", y, self.device, dtype or y.dtype, (rows.rows, self.N))
        self._call("moe_fp4_gemm", self.shape(rows.rows, _type_of(y.dtype)), self.format, rows.codes.data_ptr(),
                   rows.scales.data_ptr(), _ptr(rows.gscale), self.codes.data_ptr(), self.scales.data_ptr(),
                   _ptr(self.gscale), *_lists(self, offsets, counts), yp, ldy, of=(rows,))
        return y


class MoeLayer:
    """One MoE layer's weights on the GPU plus a workspace sized for up to
    ``max_tokens`` tokens.  Inputs and outputs are torch tensors on the same
    device; bf16 tensors may be torch.bfloat16 or raw int16 bit patterns."""

    def __init__(self, g_norm, w_router, w13, w2, top_k, renormalize=True, eps=1e-6, router_bias=None,
                 max_tokens=1):
        import torch
        self.g_norm, self.w_router, self.w13, self.w2, self.bias = g_norm, w_router, w13, w2, router_bias
        self.E, two_i, self.H = w13.shape
        self.I = two_i // 2
        self.top_k, self.renormalize, self.eps = int(top_k), bool(renormalize), float(eps)
        self.device = w13.device
        self.max_tokens = 0
        self.workspace = None
        self.ensure_capacity(max_tokens)
        self._torch = torch

    def shape(self, T) -> MoeShape:
        return shape(T, self.H, self.I, self.E, self.top_k, self.renormalize, self.eps)

    def ensure_capacity(self, T):
        import torch
        if T <= self.max_tokens and self.workspace is not None:
            return
        st, n = moe_workspace_size(self.shape(max(T, 1)))
        if st != MOE_OK:
            raise MoeError(st, "moe_workspace_size")
        st, n_mx = moe_workspace_size_mx(self.shape(max(T, 1)))
        if st == MOE_OK:
            n = max(n, n_mx)  # room for the MXFP8 forward as well
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)
        self.max_tokens = max(T, 1)

    def workspace_bytes(self, T) -> int:
        st, n = moe_workspace_size(self.shape(T))
        if st != MOE_OK:
            raise MoeError(st, "moe_workspace_size")
        return n

    def forward(self, x, y=None, stream=None, events=None, fused_front=False, fused_combine=False, fused_mlp=False):
        """y = layer(x).  events: optional MOE_NUM_KERNELS + 1 cudaEvent_t handles
        recorded around the kernels (moe_forward_events).  fused_front: run the
        norm .. gather steps as one cluster launch (moe_forward_fused_front).
        fused_combine: the combine in the down GEMM's epilogue
        (moe_forward_fused_combine).  fused_mlp: both expert GEMMs in one
        launch (moe_forward_fused_mlp; decode tile plan only)."""
        import torch
        T = x.shape[0]
        self.ensure_capacity(T)
        if y is None:
            y = torch.empty((T, self.H), dtype=x.dtype, device=x.device)
        s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
        args = (self.shape(T), _ptr(x), _ptr(self.g_norm), _ptr(self.w_router), _ptr(self.bias), _ptr(self.w13),
                _ptr(self.w2), _ptr(y), _ptr(self.workspace), self.workspace_bytes(T), s)
        if int(fused_front) + int(fused_combine) + int(fused_mlp) > 1:
            raise ValueError("fused_front, fused_combine and fused_mlp are separate entry points")
        if fused_mlp:
            st = moe_forward_fused_mlp(*args, events)
        elif fused_front:
            st = moe_forward_fused_front(*args, events)
        elif fused_combine:
            st = moe_forward_fused_combine(*args, events)
        elif events is None:
            st = moe_forward(*args)
        else:
            st = moe_forward_events(*args, events)
        if st != MOE_OK:
            raise MoeError(st, "moe_forward")
        return y

    def quantize_mx(self, stream=None):
        """Make the MXFP8 copies of W13 and W2 (moe_mx_quantize_weights) for forward_mx."""
        import torch
        st, (n13c, n13s, n2c, n2s) = moe_mx_weight_sizes(self.shape(1))
        if st != MOE_OK:
            raise MoeError(st, "moe_mx_weight_sizes")
        u8 = dict(dtype=torch.uint8, device=self.device)
        self.w13_codes, self.w13_scales = torch.empty(n13c, **u8), torch.empty(n13s, **u8)
        self.w2_codes, self.w2_scales = torch.empty(n2c, **u8), torch.empty(n2s, **u8)
        s = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        st = moe_mx_quantize_weights(self.shape(1), _ptr(self.w13), _ptr(self.w2), _ptr(self.w13_codes),
                                     _ptr(self.w13_scales), _ptr(self.w2_codes), _ptr(self.w2_scales), s)
        if st != MOE_OK:
            raise MoeError(st, "moe_mx_quantize_weights")

    def quantize_mxfp4(self, stream=None):
        """Make the MXFP4 copies of W13 and W2 (moe_mxfp4_quantize_weights) for forward_mxfp4."""
        import torch
        st, (n13c, n13s, n2c, n2s) = moe_mxfp4_weight_sizes(self.shape(1))
        if st != MOE_OK:
            raise MoeError(st, "moe_mxfp4_weight_sizes")
        u8 = dict(dtype=torch.uint8, device=self.device)
        self.w13_codes4, self.w13_scales4 = torch.empty(n13c, **u8), torch.empty(n13s, **u8)
        self.w2_codes4, self.w2_scales4 = torch.empty(n2c, **u8), torch.empty(n2s, **u8)
        s = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        st = moe_mxfp4_quantize_weights(self.shape(1), _ptr(self.w13), _ptr(self.w2), _ptr(self.w13_codes4),
                                        _ptr(self.w13_scales4), _ptr(self.w2_codes4), _ptr(self.w2_scales4), s)
        if st != MOE_OK:
            raise MoeError(st, "moe_mxfp4_quantize_weights")

    def forward_mxfp4(self, x, y=None, stream=None, events=None, fp4_tokens=False):
        """y = layer(x) with the MXFP4 expert weights (call quantize_mxfp4 first);
        fp4_tokens: the MXFP4 layer, with token rows and activations in MXFP4
        too (moe_forward_mxfp4a4), else MXFP8 tokens (moe_forward_mxfp4)."""
        import torch
        T = x.shape[0]
        self.ensure_capacity(T)
        if y is None:
            y = torch.empty((T, self.H), dtype=x.dtype, device=x.device)
        s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
        fn, name = (moe_forward_mxfp4a4, "moe_forward_mxfp4a4") if fp4_tokens else (moe_forward_mxfp4,
                                                                                   "moe_forward_mxfp4")
        st = fn(self.shape(T), _ptr(x), _ptr(self.g_norm), _ptr(self.w_router), _ptr(self.bias),
                _ptr(self.w13_codes4), _ptr(self.w13_scales4), _ptr(self.w2_codes4), _ptr(self.w2_scales4), _ptr(y),
                _ptr(self.workspace), self.workspace_bytes_mx(T), s, events)
        if st != MOE_OK:
            raise MoeError(st, name)
        return y

    def quantize_nvfp4(self, stream=None):
        """Make the NVFP4 copies of W13 and W2 (moe_nvfp4_quantize_weights) for forward_nvfp4."""
        import torch
        st, (n13c, n13s, n2c, n2s) = moe_nvfp4_weight_sizes(self.shape(1))
        if st != MOE_OK:
            raise MoeError(st, "moe_nvfp4_weight_sizes")
        u8 = dict(dtype=torch.uint8, device=self.device)
        self.w13_codes_nv, self.w13_scales_nv = torch.empty(n13c, **u8), torch.empty(n13s, **u8)
        self.w2_codes_nv, self.w2_scales_nv = torch.empty(n2c, **u8), torch.empty(n2s, **u8)
        self.w13_gscale_nv = torch.empty(self.E, dtype=torch.float32, device=self.device)
        self.w2_gscale_nv = torch.empty(self.E, dtype=torch.float32, device=self.device)
        s = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        st = moe_nvfp4_quantize_weights(self.shape(1), _ptr(self.w13), _ptr(self.w2), _ptr(self.w13_codes_nv),
                                        _ptr(self.w13_scales_nv), _ptr(self.w13_gscale_nv), _ptr(self.w2_codes_nv),
                                        _ptr(self.w2_scales_nv), _ptr(self.w2_gscale_nv), s)
        if st != MOE_OK:
            raise MoeError(st, "moe_nvfp4_quantize_weights")

    def forward_nvfp4(self, x, y=None, stream=None, events=None):
        """y = layer(x), the NVFP4 layer (call quantize_nvfp4 first)."""
        import torch
        T = x.shape[0]
        self.ensure_capacity(T)
        if y is None:
            y = torch.empty((T, self.H), dtype=x.dtype, device=x.device)
        s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
        st = moe_forward_nvfp4(self.shape(T), _ptr(x), _ptr(self.g_norm), _ptr(self.w_router), _ptr(self.bias),
                               _ptr(self.w13_codes_nv), _ptr(self.w13_scales_nv), _ptr(self.w13_gscale_nv),
                               _ptr(self.w2_codes_nv), _ptr(self.w2_scales_nv), _ptr(self.w2_gscale_nv), _ptr(y),
                               _ptr(self.workspace), self.workspace_bytes_mx(T), s, events)
        if st != MOE_OK:
            raise MoeError(st, "moe_forward_nvfp4")
        return y

    def workspace_bytes_mx(self, T) -> int:
        st, n = moe_workspace_size_mx(self.shape(T))
        if st != MOE_OK:
            raise MoeError(st, "moe_workspace_size_mx")
        return n

    def forward_mx(self, x, y=None, stream=None, events=None):
        """y = layer(x) with the MXFP8 expert weights (call quantize_mx first)."""
        import torch
        T = x.shape[0]
        self.ensure_capacity(T)
        if y is None:
            y = torch.empty((T, self.H), dtype=x.dtype, device=x.device)
        s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
        st = moe_forward_mx(self.shape(T), _ptr(x), _ptr(self.g_norm), _ptr(self.w_router), _ptr(self.bias),
                            _ptr(self.w13_codes), _ptr(self.w13_scales), _ptr(self.w2_codes), _ptr(self.w2_scales),
                            _ptr(y), _ptr(self.workspace), self.workspace_bytes_mx(T), s, events)
        if st != MOE_OK:
            raise MoeError(st, "moe_forward_mx")
        return y

    def views_mx(self, T):
        st, v, mv = moe_workspace_views_mx(self.shape(T), _ptr(self.workspace), self.workspace_bytes_mx(T))
        if st != MOE_OK:
            raise MoeError(st, "moe_workspace_views_mx")
        return v, mv

    def views(self, T):
        st, v = moe_workspace_views(self.shape(T), _ptr(self.workspace), self.workspace_bytes(T))
        if st != MOE_OK:
            raise MoeError(st, "moe_workspace_views")
        return v

    def view_tensor(self, T, name, dtype, shape_):
        """A torch view of one intermediate tensor inside the workspace."""
        import torch
        v = self.views(T)
        off = getattr(v, name) - self.workspace.data_ptr()
        n = 1
        for d in shape_:
            n *= d
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.workspace[off:off + nbytes].view(dtype).view(*shape_)

    def device_status(self, T, stream=None):
        import torch
        s = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        return moe_device_status(_ptr(self.workspace), self.workspace_bytes(T), s)
