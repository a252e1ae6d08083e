"""ctypes binding of libmoe_gg.so (declared in include/moe_gg.h).

Argument marshalling only: each function takes torch tensors (or None for nullable pointers),
passes their device pointers and the current CUDA stream to the C entry point of the same name,
and raises MoEError on a non-OK status. Every step runs in the library's CUDA kernels; there is
no fallback of any kind, and loading fails loudly when the library has not been built. The calls of
a decode step are marshalled by a small CPython extension where it has been built (_install_binding).
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gg.so")
DEBUG_LIB_PATH = os.path.join(_HERE, "libmoe_gg_debug.so")  # same ABI, built with MOE_GG_DEBUG
HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe_gg.h")

MOE_OK = 0
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
          3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_TIMEOUT",
          6: "MOE_ERR_UNSUPPORTED_DEVICE"}
MOE_DEV_TIMEOUT = 0x1
MOE_DEV_BAD_OFFSETS = 0x2
OP_ROUTE, OP_FWD, OP_BWD, OP_PADDED_BMM, OP_LOOP, OP_SAVED, OP_MX_WEIGHTS, OP_MX_FWD, OP_MX_BWD, OP_MX_ROW_SCALES = \
    range(10)
OP_MX4_WEIGHTS, OP_MX4_FWD, OP_MX4_ROW_SCALES, OP_GATE, OP_LAYER_NORM_BWD = range(10, 15)
OP_RESIDUAL_NORM_BWD, OP_GRAD_NORM, OP_W4_WEIGHTS, OP_W4_DECODE = range(15, 19)
DTYPE_BF16, DTYPE_F32 = 0, 1
GATE_RENORM = 0x1
NORM_NONE, NORM_LAYER, NORM_RMS = 0, 1, 2
W4_MAX_SLOTS = 4096  # token slots of one call of the 4-bit integer products

_P, _I, _S, _L, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float
_D, _U = ctypes.c_double, ctypes.c_uint32


class AdamWTensor(ctypes.Structure):
    """moe_adamw_tensor_t: one tensor of moe_grad_norm and moe_adamw_step (device pointers)."""
    _fields_ = [("p", _P), ("copy", _P), ("g", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P), ("n", _L),
                ("weight_decay", _F), ("p_dtype", _I), ("g_dtype", _I), ("reserved", _I)]


_PI32, _PI64 = ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_longlong)
SIGNATURES = {
    "moe_workspace_bytes": (_S, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_route_offsets": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _S, _P]),
    "moe_permute": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_grouped_swiglu_fwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _S, _P, _P]),
    "moe_grouped_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P,
                             _P]),
    "moe_unpermute_combine": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_padded_bmm_swiglu_fwd": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _S, _P, _P]),
    "moe_loop_swiglu_fwd": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "moe_grouped_up_swiglu": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_grouped_down": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "moe_grouped_down_dgrad_swiglu": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "moe_routing_weight_grad": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "moe_grouped_up_dgrad": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "moe_grouped_wgrad": (_I, [_P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _P]),
    "moe_grouped_wgrad_dual": (_I, [_P, _P, _I, _P, _I, _P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _P, _P]),
    "moe_mx_prepare_weights": (_I, [_P, _P, _I, _I, _I, _P, _S, _P]),
    "moe_mx_quantize_rows": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _P]),
    "moe_permute_mxfp8": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_grouped_swiglu_fwd_mxfp8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _S, _P, _P]),
    "moe_grouped_bwd_mxfp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                   _S, _P, _P]),
    "moe_grouped_swiglu_fwd_top1_combine": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                                                 _P]),
    "moe_route_offsets_noalloc": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_mx4_prepare_weights": (_I, [_P, _P, _I, _I, _I, _P, _S, _P]),
    "moe_mx4_quantize_rows": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _P]),
    "moe_mx4_dequantize_rows": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_permute_mxfp4": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "moe_grouped_swiglu_fwd_mxfp4": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _S, _P, _P]),
    "moe_gate_fwd": (_I, [_P, _I, _L, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_gate_bwd": (_I, [_P, _I, _L, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _L, _P]),
    "moe_layer_norm_fwd": (_I, [_P, _I, _L, _P, _P, _I, _I, _I, _F, _P, _L, _P, _P, _P]),
    "moe_layer_norm_bwd": (_I, [_P, _L, _P, _L, _I, _P, _I, _P, _P, _I, _I, _P, _L, _P, _P, _P, _S, _P]),
    "moe_residual_norm_fwd": (_I, [_P, _I, _L, _P, _I, _L, _I, _P, _P, _P, _I, _P, _P, _I, _I, _I, _F, _F, _F, _P, _L, _P, _L,
                                   _P, _P]),
    "moe_residual_norm_bwd": (_I, [_P, _L, _P, _L, _P, _L, _I, _P, _L, _I, _I, _P, _P, _P, _I, _P, _I, _P, _I, _I, _F, _F, _P,
                                   _L, _P, _L, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_grad_norm": (_I, [_P, _I, _F, _P, _P, _S, _P]),
    "moe_adamw_step": (_I, [_P, _I, _I, _D, _D, _D, _D, _U, _P, _P, _P, _P]),
    "moe_w4_quantize_rows": (_I, [_P, _L, _I, _I, _P, _P, _P, _P]),
    "moe_w4_pack": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _S, _P]),
    "moe_w4_matvec": (_I, [_P, _L, _P, _I, _I, _I, _I, _I, _I, _P, _P, _I, _L, _P]),
    "moe_w4_swiglu_decode": (_I, [_P, _L, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _L, _P, _S, _P]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_last_cuda_error": (ctypes.c_char_p, []),
    "moe_abi_version": (_I, []),
    "moe_debug_build": (_I, []),
    "moe_debug_report": (_I, [_PI32, _PI32, _PI64, _PI64, _I]),
    "moe_debug_site_name": (ctypes.c_char_p, [_I]),
}
MOE_DEBUG_CALL_ERROR_BIT = 30

_lib = None


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        detail = ""
        if status == 4 and _lib is not None:
            detail = ": " + _lib.moe_last_cuda_error().decode()
        super().__init__(f"{fn} returned {STATUS.get(status, status)}{detail}")


def header_functions(path: str = HEADER):
    """Names of the functions include/moe_gg.h declares."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


def open_library(path: str):
    """A ctypes handle of a build of the library at `path`, every entry point declared."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run __graft_entry__.build() (nvcc, sm_103a)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load(path: str = None):
    """Load the library (once; the first call's path wins, so a process that wants the debug
    build calls load(DEBUG_LIB_PATH) before anything else) and return its handle. Without a
    path: the release build, or the debug build when MOE_GG_DEBUG_LIB=1 is set in the
    environment (to run a whole program or test suite with the debug build's bounds checks)."""
    global _lib
    if _lib is None:
        if path is None:
            path = DEBUG_LIB_PATH if os.environ.get("MOE_GG_DEBUG_LIB") == "1" else LIB_PATH
        _lib = open_library(path)
        _install_binding()
    return _lib


# calls that the compiled binding takes over (csrc/binding.cpp)
COMPILED = ("moe_layer_norm_fwd", "moe_layer_norm_bwd", "moe_gate_fwd", "moe_gate_bwd", "moe_mx4_quantize_rows",
            "moe_mx4_dequantize_rows", "moe_permute_mxfp4", "moe_grouped_swiglu_fwd_mxfp4", "moe_unpermute_combine",
            "moe_route_offsets")
# ... and those of a block's joins, of an optimizer step and of the 4-bit integer experts
COMPILED_STEP = ("moe_residual_norm_fwd", "moe_residual_norm_bwd", "moe_grad_norm", "moe_adamw_step", "moe_w4_matvec",
                 "moe_w4_swiglu_decode")
PYTHON_BINDING = {}       # the functions that they replaced
PYTHON_BINDING_STEP = {}
adamw_pointers = None     # the extension's loop over AdamW's tensors


def _install_binding():
    """Replace the functions of COMPILED and COMPILED_STEP by the CPython extension's, which make the same checks and call
    the same entry points of the loaded library with less marshalling time. Without the extension (or
    without torch, when only host functions are called) the Python functions below stay."""
    import sys
    torch = sys.modules.get("torch")
    if torch is None or not torch.cuda.is_available():
        return
    try:
        from . import _binding
    except ImportError:
        return

    entry_points = COMPILED + COMPILED_STEP + ("moe_workspace_bytes",)
    _binding.bind({n: ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value for n in entry_points}, _check)
    for names, replaced in ((COMPILED, PYTHON_BINDING), (COMPILED_STEP, PYTHON_BINDING_STEP)):
        for n in names:
            replaced[n] = globals()[n]
            globals()[n] = getattr(_binding, n)
    globals()["adamw_pointers"] = _binding.adamw_pointers


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous CUDA tensors")
    return t.data_ptr()


def _rows(t, T, width):
    """(pointer, row pitch in elements) of a [T, width] view whose rows are contiguous. A view with
    one row repeated (row stride 0) is a pitch of 0."""
    shape, stride = t.shape, t.stride()
    if not t.is_cuda or len(shape) != 2 or shape[0] < T or shape[1] != width or (stride[1] != 1 and width > 1):
        raise ValueError(f"expected a CUDA tensor of at least {T} rows of {width} contiguous elements")
    return t.data_ptr(), stride[0] if T > 1 else width


def _dtype(t):
    import torch
    if t.dtype is torch.bfloat16:
        return DTYPE_BF16
    if t.dtype is torch.float32:
        return DTYPE_F32
    raise ValueError(f"expected a bfloat16 or float32 tensor, not {t.dtype}")


def _typed(t, dtype, numel, name):
    """Pointer of a contiguous CUDA tensor of `dtype` with at least `numel` elements (None passes)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() < numel or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of at least {numel} elements of {dtype}")
    return t.data_ptr()


def _bytes(t, nbytes, name):
    """Pointer of a contiguous CUDA tensor of at least `nbytes` bytes, whatever its type: packed codes, scales,
    prepared weights (None passes)."""
    if t is None:
        return None
    if t.numel() * t.element_size() < nbytes or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of at least {nbytes} bytes")
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    # the handle of torch.cuda.current_stream() without its Python object: that takes 3 us, as long
    # as the C call and its launch together
    import torch
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status)


def moe_workspace_bytes(op: int, T: int, top_k: int, E: int, d: int = 0, h: int = 0, capacity_C: int = 0) -> int:
    return int(load().moe_workspace_bytes(op, T, top_k, E, d, h, capacity_C))


def moe_route_offsets(ids, T, top_k, E, counts, offsets, sorted_src, inv_map, ws, stream=None):
    L = load()
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_route_offsets", L.moe_route_offsets(_ptr(ids), T, top_k, E, _ptr(counts), _ptr(offsets),
                                                    _ptr(sorted_src), _ptr(inv_map), _ptr(ws), ws_bytes,
                                                    _stream(stream)))


def moe_route_offsets_noalloc(ids, T, top_k, E, counts, offsets, sorted_src, inv_map, stream=None):
    """moe_route_offsets without a workspace: for callers that cannot allocate device memory; the
    scratch is one fixed 1 MiB array inside the library (calls that overlap on the GPU race)."""
    _check("moe_route_offsets_noalloc", load().moe_route_offsets_noalloc(
        _ptr(ids), T, top_k, E, _ptr(counts), _ptr(offsets), _ptr(sorted_src), _ptr(inv_map), _stream(stream)))


def moe_permute(x, sorted_src, offsets, row_scale, T, top_k, E, d, xp, stream=None):
    _check("moe_permute", load().moe_permute(_ptr(x), _ptr(sorted_src), _ptr(offsets), _ptr(row_scale),
                                             T, top_k, E, d, _ptr(xp), _stream(stream)))


def moe_grouped_swiglu_fwd(xp, offsets, sorted_src, weights, E, cap, d, h, w_ug, w_down, y, a_save,
                           saved=None, ws=None, dev_status=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_grouped_swiglu_fwd", load().moe_grouped_swiglu_fwd(
        _ptr(xp), _ptr(offsets), _ptr(sorted_src), _ptr(weights), E, cap, d, h, _ptr(w_ug), _ptr(w_down),
        _ptr(y), _ptr(a_save), _ptr(saved), _ptr(ws), ws_bytes, _ptr(dev_status), _stream(stream)))


def moe_grouped_bwd(dy, xp, a_save, saved, offsets, sorted_src, weights, E, cap, d, h, w_ug, w_down, dxp,
                    dw_ug, dw_down, ws, dev_status=None, stream=None, inv_map=None, dw_route=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_grouped_bwd", load().moe_grouped_bwd(
        _ptr(dy), _ptr(xp), _ptr(a_save), _ptr(saved), _ptr(offsets), _ptr(sorted_src), _ptr(weights), E,
        cap, d, h, _ptr(w_ug),
        _ptr(w_down), _ptr(dxp), _ptr(dw_ug), _ptr(dw_down), _ptr(inv_map), _ptr(dw_route), _ptr(ws), ws_bytes,
        _ptr(dev_status), _stream(stream)))


def moe_grouped_up_swiglu(xp, offsets, sorted_src, weights, E, cap, d, h, w_ug, a_save, saved=None,
                          dev_status=None, stream=None):
    _check("moe_grouped_up_swiglu", load().moe_grouped_up_swiglu(
        _ptr(xp), _ptr(offsets), _ptr(sorted_src), _ptr(weights), E, cap, d, h, _ptr(w_ug), _ptr(a_save),
        _ptr(saved), _ptr(dev_status), _stream(stream)))


def moe_grouped_down(a, offsets, E, cap, d, h, w_down, y, dev_status=None, stream=None):
    _check("moe_grouped_down", load().moe_grouped_down(
        _ptr(a), _ptr(offsets), E, cap, d, h, _ptr(w_down), _ptr(y), _ptr(dev_status), _stream(stream)))


def moe_grouped_down_dgrad_swiglu(dy, saved, offsets, sorted_src, weights, E, cap, d, h, w_down, du_hi, du_lo,
                                  dev_status=None, stream=None, dw_part=None):
    _check("moe_grouped_down_dgrad_swiglu", load().moe_grouped_down_dgrad_swiglu(
        _ptr(dy), _ptr(saved), _ptr(offsets), _ptr(sorted_src), _ptr(weights), E, cap, d, h, _ptr(w_down),
        _ptr(du_hi), _ptr(du_lo), _ptr(dw_part), _ptr(dev_status), _stream(stream)))


def routing_grad_parts(h):
    """Partial sums per row the dgrad leaves for the routing-weight gradient: 2 ceil(h/256)."""
    return 2 * ((h + 255) // 256)


def moe_routing_weight_grad(dw_part, inv_map, T, top_k, h, dw_route, stream=None):
    _check("moe_routing_weight_grad", load().moe_routing_weight_grad(
        _ptr(dw_part), _ptr(inv_map), T, top_k, h, _ptr(dw_route), _stream(stream)))


def moe_grouped_up_dgrad(du_hi, offsets, E, cap, d, h, w_ug, dxp, dev_status=None, stream=None):
    _check("moe_grouped_up_dgrad", load().moe_grouped_up_dgrad(
        _ptr(du_hi), _ptr(offsets), E, cap, d, h, _ptr(w_ug), _ptr(dxp), _ptr(dev_status), _stream(stream)))


def moe_grouped_wgrad(p_hi, p_lo, p_cols, q, q_cols, offsets, E, cap, dw, dev_status=None, stream=None):
    _check("moe_grouped_wgrad", load().moe_grouped_wgrad(
        _ptr(p_hi), _ptr(p_lo), p_cols, _ptr(q), q_cols, _ptr(offsets), E, cap, _ptr(dw), _ptr(dev_status),
        _stream(stream)))


def moe_grouped_wgrad_dual(p1_hi, p1_lo, p1_cols, q1, q1_cols, dw1, p2_hi, p2_lo, p2_cols, q2, q2_cols, dw2,
                           offsets, E, cap, dev_status=None, stream=None):
    _check("moe_grouped_wgrad_dual", load().moe_grouped_wgrad_dual(
        _ptr(p1_hi), _ptr(p1_lo), p1_cols, _ptr(q1), q1_cols, _ptr(dw1), _ptr(p2_hi), _ptr(p2_lo), p2_cols,
        _ptr(q2), q2_cols, _ptr(dw2), _ptr(offsets), E, cap, _ptr(dev_status), _stream(stream)))


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def moe_mx_prepare_weights(w_ug, w_down, E, d, h, mxw, stream=None):
    _check("moe_mx_prepare_weights", load().moe_mx_prepare_weights(
        _ptr(w_ug), _ptr(w_down), E, d, h, _ptr(mxw), _nbytes(mxw), _stream(stream)))


def moe_permute_mxfp8(x, sorted_src, offsets, T, top_k, E, d, xp, q, sf, dev_status=None, stream=None):
    _check("moe_permute_mxfp8", load().moe_permute_mxfp8(
        _ptr(x), _ptr(sorted_src), _ptr(offsets), T, top_k, E, d, _ptr(xp), _ptr(q), _ptr(sf), _ptr(dev_status),
        _stream(stream)))


def moe_mx_quantize_rows(x, offsets, E, cap, K, q, sf, dev_status=None, stream=None):
    _check("moe_mx_quantize_rows", load().moe_mx_quantize_rows(
        _ptr(x), _ptr(offsets), E, cap, K, _ptr(q), _ptr(sf), _ptr(dev_status), _stream(stream)))


def moe_grouped_swiglu_fwd_mxfp8(xp, offsets, sorted_src, weights, E, cap, d, h, mxw, y, a_save, saved, ws,
                                 dev_status=None, stream=None, xq=None, xsf=None):
    _check("moe_grouped_swiglu_fwd_mxfp8", load().moe_grouped_swiglu_fwd_mxfp8(
        _ptr(xp), _ptr(xq), _ptr(xsf), _ptr(offsets), _ptr(sorted_src), _ptr(weights), E, cap, d, h, _ptr(mxw), _ptr(y), _ptr(a_save),
        _ptr(saved), _ptr(ws), _nbytes(ws), _ptr(dev_status), _stream(stream)))


def moe_grouped_bwd_mxfp8(dy, xp, a_save, saved, offsets, sorted_src, weights, E, cap, d, h, mxw, dxp, dw_ug,
                          dw_down, ws, dev_status=None, stream=None, inv_map=None, dw_route=None, dyq=None, dysf=None):
    _check("moe_grouped_bwd_mxfp8", load().moe_grouped_bwd_mxfp8(
        _ptr(dy), _ptr(dyq), _ptr(dysf), _ptr(xp), _ptr(a_save), _ptr(saved), _ptr(offsets), _ptr(sorted_src), _ptr(weights), E, cap, d,
        h, _ptr(mxw), _ptr(dxp), _ptr(dw_ug), _ptr(dw_down), _ptr(inv_map), _ptr(dw_route), _ptr(ws), _nbytes(ws),
        _ptr(dev_status), _stream(stream)))


def saved_views(saved, cap, h):
    """The parts of the forward's `saved` buffer (a contiguous tensor of any dtype, read as bytes):
    the low half of P = w*A (bf16 [cap, h8]; the high half is a_save) at byte 0, then U rounded to
    24 bits in the kernels' blocked layout (a flat byte view; see the header for the block
    order). h8 = h rounded up to a multiple of 8: widths that are not are stored zero-padded."""
    import torch
    saved = saved.reshape(-1).view(torch.uint8)
    h = (h + 7) // 8 * 8
    pb = cap * h * 2
    off = (pb + 255) // 256 * 256
    p_lo = saved[:pb].view(torch.bfloat16).view(cap, h)
    u = saved[off:]
    return u, p_lo


def moe_unpermute_combine(y, inv_map, weights, T, top_k, d, out, stream=None):
    _check("moe_unpermute_combine", load().moe_unpermute_combine(
        _ptr(y), _ptr(inv_map), _ptr(weights), T, top_k, d, _ptr(out), _stream(stream)))


def moe_grouped_swiglu_fwd_top1_combine(xp, offsets, sorted_src, inv_map, weights, E, T, d, h, w_ug, w_down, out,
                                        a_save, saved=None, dev_status=None, stream=None):
    _check("moe_grouped_swiglu_fwd_top1_combine", load().moe_grouped_swiglu_fwd_top1_combine(
        _ptr(xp), _ptr(offsets), _ptr(sorted_src), _ptr(inv_map), _ptr(weights), E, T, d, h, _ptr(w_ug),
        _ptr(w_down), _ptr(out), _ptr(a_save), _ptr(saved), _ptr(dev_status), _stream(stream)))


def moe_padded_bmm_swiglu_fwd(xp, offsets, E, cap, d, h, capacity_C, w_ug, w_down, y, ws,
                              dev_status=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_padded_bmm_swiglu_fwd", load().moe_padded_bmm_swiglu_fwd(
        _ptr(xp), _ptr(offsets), E, cap, d, h, capacity_C, _ptr(w_ug), _ptr(w_down), _ptr(y), _ptr(ws),
        ws_bytes, _ptr(dev_status), _stream(stream)))


def moe_loop_swiglu_fwd(xp, offsets, E, cap, d, h, w_ug, w_down, y, a_save, saved=None, dev_status=None,
                        stream=None):
    _check("moe_loop_swiglu_fwd", load().moe_loop_swiglu_fwd(
        _ptr(xp), _ptr(offsets), E, cap, d, h, _ptr(w_ug), _ptr(w_down), _ptr(y), _ptr(a_save),
        _ptr(saved), _ptr(dev_status), _stream(stream)))


def moe_mx4_prepare_weights(w_ug, w_down, E, d, h, mxw, stream=None):
    import torch
    bf = torch.bfloat16
    _check("moe_mx4_prepare_weights", load().moe_mx4_prepare_weights(
        _typed(w_ug, bf, 2 * E * h * d, "w_ug"), _typed(w_down, bf, E * h * d, "w_down"), E, d, h, _ptr(mxw),
        _nbytes(mxw), _stream(stream)))


def _mx4_scale_bytes(rows, E, K):
    """Bytes of the scale atoms of `rows` rows of K elements (0 without rows and for sizes that the library refuses)."""
    return 0 if not 0 < rows < 1 << 31 else moe_workspace_bytes(OP_MX4_ROW_SCALES, rows, 1, E, K, 32)


def moe_mx4_quantize_rows(x, offsets, E, cap, K, q, sf, dev_status=None, stream=None):
    import torch
    i32 = torch.int32
    _check("moe_mx4_quantize_rows", load().moe_mx4_quantize_rows(
        _typed(x, torch.bfloat16, cap * K, "x"), _typed(offsets, i32, E, "offsets"), E, cap, K,
        _bytes(q, cap * K // 2, "q"), _bytes(sf, _mx4_scale_bytes(cap, E, K), "sf"),
        _typed(dev_status, i32, 1, "dev_status"), _stream(stream)))


def moe_mx4_dequantize_rows(q, sf, offsets, E, cap, K, x, dev_status=None, stream=None):
    import torch
    i32 = torch.int32
    _check("moe_mx4_dequantize_rows", load().moe_mx4_dequantize_rows(
        _bytes(q, cap * K // 2, "q"), _bytes(sf, _mx4_scale_bytes(cap, E, K), "sf"), _typed(offsets, i32, E, "offsets"),
        E, cap, K, _typed(x, torch.bfloat16, cap * K, "x"), _typed(dev_status, i32, 1, "dev_status"), _stream(stream)))


def moe_permute_mxfp4(x, inv_map, offsets, T, top_k, E, d, q, sf, dev_status=None, stream=None):
    import torch
    i32, n = torch.int32, T * top_k
    _check("moe_permute_mxfp4", load().moe_permute_mxfp4(
        _typed(x, torch.bfloat16, T * d, "x"), _typed(inv_map, i32, n, "inv_map"), _typed(offsets, i32, E, "offsets"),
        T, top_k, E, d, _bytes(q, n * d // 2, "q"), _bytes(sf, _mx4_scale_bytes(n, E, d), "sf"),
        _typed(dev_status, i32, 1, "dev_status"), _stream(stream)))


def moe_grouped_swiglu_fwd_mxfp4(xq, xsf, offsets, E, cap, d, h, mxw, y, ws, dev_status=None, stream=None):
    import torch
    i32 = torch.int32
    _check("moe_grouped_swiglu_fwd_mxfp4", load().moe_grouped_swiglu_fwd_mxfp4(
        _bytes(xq, cap * d // 2, "xq"), _bytes(xsf, _mx4_scale_bytes(cap, E, d), "xsf"),
        _typed(offsets, i32, E, "offsets"), E, cap, d, h,
        _bytes(mxw, moe_workspace_bytes(OP_MX4_WEIGHTS, 0, 1, E, d, h), "mxw"),
        _typed(y, torch.bfloat16, cap * d, "y"), _ptr(ws), _nbytes(ws), _typed(dev_status, i32, 1, "dev_status"),
        _stream(stream)))


def moe_gate_fwd(logits, token_mask, T, top_k, E, flags, ids, weights, lse=None, counts=None, n_valid=None,
                 prob_sum=None, loss=None, ws=None, stream=None):
    """logits [T, E] bf16 or fp32 (any row pitch); token_mask nullable [T] uint8 or bool."""
    import torch
    p, ld = _rows(logits, T, E)
    if token_mask is not None and token_mask.dtype == torch.bool:
        token_mask = token_mask.view(torch.uint8)
    i32, f32 = torch.int32, torch.float32
    _check("moe_gate_fwd", load().moe_gate_fwd(
        p, _dtype(logits), ld, _typed(token_mask, torch.uint8, T, "token_mask"), T, top_k, E, flags,
        _typed(ids, i32, T * top_k, "ids"), _typed(weights, f32, T * top_k, "weights"), _typed(lse, f32, T, "lse"),
        _typed(counts, i32, E, "counts"), _typed(n_valid, i32, 1, "n_valid"), _typed(prob_sum, f32, E, "prob_sum"),
        _typed(loss, f32, 2, "loss"), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_gate_bwd(logits, lse, ids, weights, counts, n_valid, d_weights, d_loss, T, top_k, E, flags, dlogits,
                 stream=None):
    import torch
    p, ld = _rows(logits, T, E)
    o, ldd = _rows(dlogits, T, E)
    if dlogits.dtype != logits.dtype:
        raise ValueError("dlogits has to have the logits' type")
    i32, f32 = torch.int32, torch.float32
    _check("moe_gate_bwd", load().moe_gate_bwd(
        p, _dtype(logits), ld, _typed(lse, f32, T, "lse"), _typed(ids, i32, T * top_k, "ids"),
        _typed(weights, f32, T * top_k, "weights"), _typed(counts, i32, E, "counts"),
        _typed(n_valid, i32, 1, "n_valid"), _typed(d_weights, f32, T * top_k, "d_weights"),
        _typed(d_loss, f32, 2, "d_loss"), T, top_k, E, flags, o, ldd, _stream(stream)))


def _norm_weight(d, *ws):
    """The type of the given weights (all bf16 or all fp32, [d] each; fp32 when there are none)."""
    one = None
    for w in ws:
        if w is None:
            continue
        if w.numel() != d or (one is not None and w.dtype is not one.dtype):
            raise ValueError(f"the weights have to be [{d}] and of one type")
        one = w
    return DTYPE_F32 if one is None else _dtype(one)


def moe_layer_norm_fwd(x, gamma, beta, T, d, eps, y, mean=None, rstd=None, stream=None):
    """x, y [T, d] bf16 or fp32 (any row pitch); gamma, beta nullable [d] bf16 or fp32."""
    import torch
    px, ldx = _rows(x, T, d)
    py, ldy = _rows(y, T, d)
    if x.dtype != y.dtype:
        raise ValueError("y has to have x's type")
    f32 = torch.float32
    _check("moe_layer_norm_fwd", load().moe_layer_norm_fwd(
        px, _dtype(x), ldx, _ptr(gamma), _ptr(beta), _norm_weight(d, gamma, beta), T, d, eps, py, ldy,
        _typed(mean, f32, T, "mean"), _typed(rstd, f32, T, "rstd"), _stream(stream)))


def moe_layer_norm_bwd(dy, x, gamma, mean, rstd, T, d, dx, dgamma=None, dbeta=None, ws=None, stream=None):
    import torch
    pdy, lddy = _rows(dy, T, d)
    px, ldx = _rows(x, T, d)
    pdx, lddx = _rows(dx, T, d)
    if x.dtype != dy.dtype or x.dtype != dx.dtype:
        raise ValueError("x, dy and dx have to have one type")
    f32 = torch.float32
    _check("moe_layer_norm_bwd", load().moe_layer_norm_bwd(
        pdy, lddy, px, ldx, _dtype(x), _ptr(gamma), _norm_weight(d, gamma), _typed(mean, f32, T, "mean"),
        _typed(rstd, f32, T, "rstd"), T, d, pdx, lddx, _typed(dgamma, f32, d, "dgamma"),
        _typed(dbeta, f32, d, "dbeta"), _ptr(ws), _nbytes(ws), _stream(stream)))


def _rows_or_none(t, T, width):
    return (None, 0) if t is None else _rows(t, T, width)


def _same_type(what, *ts):
    if len({t.dtype for t in ts if t is not None}) > 1:
        raise ValueError(f"{what} have to have one type")


def moe_residual_norm_fwd(x, y, post, post_gamma, post_beta, gate, pre, pre_gamma, pre_beta, T, d, eps, res_scale,
                          branch_scale, r, n, stats=None, stream=None):
    """r = res_scale x + branch_scale gate post(y), n = pre(r): x, r [T, d] of one type, y, n of one type (any row
    pitch); the weights nullable [d] of one type; y, r or n nullable (see the header)."""
    import torch
    px, ldx = _rows(x, T, d)
    py, ldy = _rows_or_none(y, T, d)
    pr, ldr = _rows_or_none(r, T, d)
    pn, ldn = _rows_or_none(n, T, d)
    _same_type("x and r", x, r)
    _same_type("y and n", y, n)
    weights = (post_gamma, post_beta, gate, pre_gamma, pre_beta)
    branch = y if y is not None else n if n is not None else x
    _check("moe_residual_norm_fwd", load().moe_residual_norm_fwd(
        px, _dtype(x), ldx, py, _dtype(branch), ldy, post, _ptr(post_gamma), _ptr(post_beta), _ptr(gate), pre,
        _ptr(pre_gamma), _ptr(pre_beta), _norm_weight(d, *weights), T, d, eps, res_scale, branch_scale, pr, ldr, pn, ldn,
        _typed(stats, torch.float32, 4 * T, "stats"), _stream(stream)))


def moe_residual_norm_bwd(dn, dr, r, y, post, post_gamma, post_beta, gate, pre, pre_gamma, stats, T, d, res_scale,
                          branch_scale, dx, dy, d_post_gamma=None, d_post_beta=None, d_gate=None, d_pre_gamma=None,
                          d_pre_beta=None, ws=None, stream=None):
    import torch
    f32 = torch.float32
    pdn, lddn = _rows_or_none(dn, T, d)
    pdr, lddr = _rows_or_none(dr, T, d)
    pr, ldr = _rows_or_none(r, T, d)
    py, ldy = _rows_or_none(y, T, d)
    pdx, lddx = _rows_or_none(dx, T, d)
    pdy, lddy = _rows_or_none(dy, T, d)
    _same_type("dr, r and dx", dr, r, dx)
    _same_type("dn, y and dy", dn, y, dy)
    first = lambda *ts: next((t for t in ts if t is not None), None)  # noqa: E731
    stream_like, branch_like = first(dr, r, dx), first(dn, y, dy)
    stream_like, branch_like = first(stream_like, branch_like), first(branch_like, stream_like)
    if stream_like is None:
        raise ValueError("neither gradients nor rows were given")
    _check("moe_residual_norm_bwd", load().moe_residual_norm_bwd(
        pdn, lddn, pdr, lddr, pr, ldr, _dtype(stream_like), py, ldy, _dtype(branch_like), post, _ptr(post_gamma),
        _ptr(post_beta), _ptr(gate), pre, _ptr(pre_gamma), _norm_weight(d, post_gamma, post_beta, gate, pre_gamma),
        _typed(stats, f32, 4 * T, "stats"), T, d, res_scale, branch_scale, pdx, lddx, pdy, lddy,
        _typed(d_post_gamma, f32, d, "d_post_gamma"), _typed(d_post_beta, f32, d, "d_post_beta"),
        _typed(d_gate, f32, d, "d_gate"), _typed(d_pre_gamma, f32, d, "d_pre_gamma"),
        _typed(d_pre_beta, f32, d, "d_pre_beta"), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_grad_norm(tensors, max_norm, norm, ws, stream=None):
    """tensors: a ctypes array of AdamWTensor; norm [2] fp32 out: the norm and the clipping coefficient."""
    import torch
    _check("moe_grad_norm", load().moe_grad_norm(tensors, len(tensors), max_norm, _typed(norm, torch.float32, 2, "norm"),
                                                 _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_adamw_step(tensors, state_bits, lr, beta1, beta2, eps, seed, steps, lr_scale=None, grad_scale=None, stream=None):
    """tensors: a ctypes array of AdamWTensor; steps [2] int32; lr_scale, grad_scale nullable [1] fp32."""
    import torch
    f32 = torch.float32
    _check("moe_adamw_step", load().moe_adamw_step(
        tensors, len(tensors), state_bits, lr, beta1, beta2, eps, seed, _typed(steps, torch.int32, 2, "steps"),
        _typed(lr_scale, f32, 1, "lr_scale"), _typed(grad_scale, f32, 1, "grad_scale"), _stream(stream)))


def _w4_groups(K, group):
    return (K + group - 1) // group if group > 0 else 0


def moe_w4_quantize_rows(w, rows, K, group, codes, scales, zeros, stream=None):
    import torch
    n = rows * _w4_groups(K, group)
    _check("moe_w4_quantize_rows", load().moe_w4_quantize_rows(
        _typed(w, torch.bfloat16, rows * K, "w"), rows, K, group, _bytes(codes, rows * ((K + 1) // 2), "codes"),
        _typed(scales, torch.bfloat16, n, "scales"), _typed(zeros, torch.uint8, n, "zeros"), _stream(stream)))


def moe_w4_pack(codes, scales, zeros, matrices, N, K, group, packed, stream=None):
    import torch
    n = matrices * N * _w4_groups(K, group)
    _check("moe_w4_pack", load().moe_w4_pack(
        _bytes(codes, matrices * N * ((K + 1) // 2), "codes"), _typed(scales, torch.bfloat16, n, "scales"),
        _typed(zeros, torch.uint8, n, "zeros"), matrices, N, K, group, _ptr(packed), _nbytes(packed), _stream(stream)))


def _w4_weights(t, matrices, K, N, group, name):
    return _bytes(t, moe_workspace_bytes(OP_W4_WEIGHTS, 0, 1, matrices, K, N, group), name)


def moe_w4_matvec(x, ids, T, top_k, matrices, N, K, group, packed, y, stream=None):
    """x [T, K] bf16, y [T * top_k, N] bf16 or fp32 (any row pitch); ids nullable [T * top_k] int32."""
    import torch
    if x.dtype != torch.bfloat16:
        raise ValueError("x has to be bfloat16")
    px, ldx = _rows(x, T, K)
    py, ldy = _rows(y, T * top_k, N)
    _check("moe_w4_matvec", load().moe_w4_matvec(
        px, ldx, _typed(ids, torch.int32, T * top_k, "ids"), T, top_k, matrices, N, K, group,
        _w4_weights(packed, matrices, K, N, group, "packed"), py, _dtype(y), ldy, _stream(stream)))


def moe_w4_swiglu_decode(x, ids, weights, T, top_k, E, d, h, group, w_ug, w_down, out, ws, stream=None):
    """x, out [T, d] bf16 (any row pitch), ids [T * top_k] int32, weights nullable [T * top_k] fp32; w_ug and w_down
    as moe_w4_pack laid them out."""
    import torch
    if x.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise ValueError("x and out have to be bfloat16")
    px, ldx = _rows(x, T, d)
    po, ldo = _rows(out, T, d)
    n = T * top_k
    _check("moe_w4_swiglu_decode", load().moe_w4_swiglu_decode(
        px, ldx, _typed(ids, torch.int32, n, "ids"), _typed(weights, torch.float32, n, "weights"), T, top_k, E, d, h, group,
        _w4_weights(w_ug, 2 * E, d, h, group, "w_ug"), _w4_weights(w_down, E, h, d, group, "w_down"), po, ldo, _ptr(ws),
        _nbytes(ws), _stream(stream)))


def moe_status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


def moe_abi_version() -> int:
    return int(load().moe_abi_version())


def moe_debug_build() -> bool:
    return bool(load().moe_debug_build())


def moe_debug_report(reset: bool = True, lib=None):
    """(site_mask, first_site, index, limit) of the debug build's bounds checks since the last
    reset (waits for the device); (0, -1, 0, 0) from a release build."""
    L = lib if lib is not None else load()
    m, s, i, l = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_longlong(), ctypes.c_longlong()
    _check("moe_debug_report", L.moe_debug_report(ctypes.byref(m), ctypes.byref(s), ctypes.byref(i),
                                                  ctypes.byref(l), int(reset)))
    return m.value, s.value, i.value, l.value


def moe_debug_site_name(site: int) -> str:
    return load().moe_debug_site_name(site).decode()
