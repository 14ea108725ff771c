"""Thin Python binding of libmxfp4 (C ABI in include/mxfp4.h).

Argument marshalling only: every step of the path runs in the library's
sm_100a kernels.  PyTorch supplies device memory and the current CUDA stream.
There is no fallback: if the shared library is missing or fails to load, the
first call raises.

Raw entry points keep the C names (``mxfp4_quantize``, ``mxfp4_rht``,
``mxfp4_deosc_update``, ``mxfp4_grouped_gemm``, ...).  The lower-case helpers
(``quantize``, ``rht``, ``deosc_update``, ``grouped_gemm``, and for the
experts' routing ``route``, ``expert_plan``, ``dispatch``, ``combine``,
``grad_clip``) allocate outputs with torch and call the library.  None of them
records anything for autograd, whatever requires_grad its tensors have: the
gradients are calls of their own (``route_bwd``, ``combine_bwd``; dispatch's is
``combine`` without weights).  Outputs must not overlap inputs unless a call
says so.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxfp4.so")

MXFP4_OK = 0
STATUS_NAMES = {0: "OK", -1: "INVALID_ARG", -2: "UNSUPPORTED_SHAPE", -3: "MISALIGNED", -4: "CUDA_ERROR",
                -5: "DEVICE_TIMEOUT", -6: "DEVICE_BAD_INPUT"}
DTYPE_BF16, DTYPE_F32 = 0, 1
BLOCK_1X32, BLOCK_32X32 = 0, 1
ROUND_NEAREST, ROUND_STOCHASTIC = 0, 1
GEMM_FPROP, GEMM_DGRAD, GEMM_WGRAD = 0, 1, 2
SCORES = {"softmax": 0, "sigmoid": 1}


class QuantParams(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int), ("along_rows", ctypes.c_int), ("rht_d", ctypes.c_int),
                ("rht_seed", ctypes.c_uint64), ("rounding", ctypes.c_int), ("sr_seed", ctypes.c_uint64),
                ("sr_offset", ctypes.c_uint32)]


class QuantOutputs(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("scales_mma", ctypes.c_void_p),
                ("codes_t", ctypes.c_void_p), ("scales_mma_t", ctypes.c_void_p)]


class DeoscParams(ctypes.Structure):
    _fields_ = [("flip_threshold", ctypes.c_uint32), ("reset_period", ctypes.c_uint32),
                ("freeze_lower", ctypes.c_uint32)]


class Operand(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales_mma", ctypes.c_void_p)]


class RouteParams(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("top_k", ctypes.c_int), ("groups", ctypes.c_int),
                ("top_groups", ctypes.c_int), ("group_best", ctypes.c_int), ("renormalise", ctypes.c_int),
                ("scale", ctypes.c_float)]


class GradTensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


class MXFP4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s (%d): %s" % (STATUS_NAMES.get(status, "?"), status, message))
        self.status = status


_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Load libmxfp4.so (raises if it is absent: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libmxfp4.so not built (%s); run python -m fp4_precision_numerics_b200.build"
                                   % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            L.mxfp4_quantize.argtypes = [vp, st, i64, i64, i64, i64, ctypes.POINTER(QuantParams),
                                         ctypes.POINTER(QuantOutputs), vp]
            L.mxfp4_quantize.restype = st
            L.mxfp4_quantize_dual.argtypes = [vp, st, i64, i64, i64, i64, ctypes.POINTER(QuantParams),
                                              ctypes.POINTER(QuantParams), ctypes.POINTER(QuantOutputs),
                                              ctypes.POINTER(QuantOutputs), vp]
            L.mxfp4_quantize_dual.restype = st
            L.mxfp4_rht.argtypes = [vp, st, i64, i64, i64, st, st, ctypes.c_uint64, vp, st, vp]
            L.mxfp4_rht.restype = st
            L.mxfp4_deosc_update.argtypes = [vp, i64, i64, i64, ctypes.c_uint32, ctypes.POINTER(DeoscParams), vp,
                                             ctypes.POINTER(QuantOutputs), vp]
            L.mxfp4_deosc_update.restype = st
            L.mxfp4_grouped_gemm.argtypes = [st, st, vp, Operand, Operand, i64, i64, i64, vp, i64, vp]
            L.mxfp4_grouped_gemm.restype = st
            L.mxfp4_grouped_gemm_fused.argtypes = [st, st, vp, Operand, Operand, i64, i64, i64, vp, i64,
                                                   ctypes.POINTER(QuantOutputs), ctypes.POINTER(QuantParams), vp]
            L.mxfp4_grouped_gemm_fused.restype = st
            sz = ctypes.c_size_t
            L.mxfp4_route.argtypes = [vp, st, i64, i64, i64, vp, vp, ctypes.POINTER(RouteParams), vp, vp, vp]
            L.mxfp4_route.restype = st
            L.mxfp4_route_bwd.argtypes = [vp, st, i64, i64, i64, vp, vp, ctypes.POINTER(RouteParams), vp, i64, vp]
            L.mxfp4_route_bwd.restype = st
            L.mxfp4_expert_plan_rows.argtypes = [i64, i64, i64, i64]
            L.mxfp4_expert_plan_rows.restype = i64
            L.mxfp4_expert_plan_workspace.argtypes = [i64, i64, i64]
            L.mxfp4_expert_plan_workspace.restype = sz
            L.mxfp4_expert_plan.argtypes = [vp, i64, i64, i64, i64, i64, st, vp, vp, vp, vp, vp, sz, vp]
            L.mxfp4_expert_plan.restype = st
            L.mxfp4_dispatch.argtypes = [vp, st, i64, i64, i64, i64, vp, vp, i64, vp, i64, vp]
            L.mxfp4_dispatch.restype = st
            L.mxfp4_combine.argtypes = [vp, st, i64, i64, i64, vp, vp, i64, i64, vp, st, i64, vp]
            L.mxfp4_combine.restype = st
            L.mxfp4_combine_bwd.argtypes = [vp, st, i64, vp, st, i64, i64, i64, vp, vp, vp, i64, i64, vp, i64, vp, vp]
            L.mxfp4_combine_bwd.restype = st
            L.mxfp4_grad_clip_workspace.argtypes = [ctypes.POINTER(GradTensor), st]
            L.mxfp4_grad_clip_workspace.restype = sz
            L.mxfp4_grad_clip.argtypes = [ctypes.POINTER(GradTensor), st, ctypes.c_float, vp, vp, sz, vp]
            L.mxfp4_grad_clip.restype = st
            L.mxfp4_mma_peak_probe.argtypes = [i64, ctypes.POINTER(ctypes.c_double), vp]
            L.mxfp4_mma_peak_probe.restype = st
            L.mxfp4_selftest_wait_timeout.argtypes = [vp]
            L.mxfp4_selftest_wait_timeout.restype = st
            L.mxfp4_mma_scale_bytes.argtypes = [i64, i64]
            L.mxfp4_mma_scale_bytes.restype = ctypes.c_size_t
            L.mxfp4_last_error.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
            L.mxfp4_last_error.restype = ctypes.c_size_t
            L.mxfp4_check_device_status.argtypes = [vp]
            L.mxfp4_check_device_status.restype = st
            L.mxfp4_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


def last_error() -> str:
    buf = ctypes.create_string_buffer(1024)
    lib().mxfp4_last_error(buf, len(buf))
    return buf.value.decode(errors="replace")


def _check(status: int):
    if status != MXFP4_OK:
        raise MXFP4Error(status, last_error())


def _stream(stream=None) -> ctypes.c_void_p:
    """The handle of a torch stream (the current one by default)."""
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the current stream's handle without building a Stream object (3 us a call)
    return ctypes.c_void_p(_current(torch.cuda.current_device()))


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError("expected bfloat16 or float32, got %s" % t.dtype)


# ---------------------------------------------------------------------------
# Raw entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def mxfp4_mma_scale_bytes(rows: int, nscales: int) -> int:
    return int(lib().mxfp4_mma_scale_bytes(rows, nscales))


def mxfp4_quantize(x_ptr, in_dtype, groups, rows, cols, ld, params: QuantParams, outputs: QuantOutputs,
                   stream=None):
    _check(lib().mxfp4_quantize(x_ptr, in_dtype, groups, rows, cols, ld, ctypes.byref(params),
                                ctypes.byref(outputs), _stream(stream)))


def mxfp4_quantize_dual(x_ptr, in_dtype, groups, rows, cols, ld, row_params: QuantParams, col_params: QuantParams,
                        row_outputs: QuantOutputs, col_outputs: QuantOutputs, stream=None):
    _check(lib().mxfp4_quantize_dual(x_ptr, in_dtype, groups, rows, cols, ld, ctypes.byref(row_params),
                                     ctypes.byref(col_params), ctypes.byref(row_outputs), ctypes.byref(col_outputs),
                                     _stream(stream)))


def mxfp4_rht(x_ptr, in_dtype, rows, cols, ld, axis, d, seed, out_ptr, out_dtype, stream=None):
    _check(lib().mxfp4_rht(x_ptr, in_dtype, rows, cols, ld, axis, d, seed, out_ptr, out_dtype, _stream(stream)))


def mxfp4_deosc_update(master_ptr, groups, rows, cols, step, params: DeoscParams, state_ptr,
                       outputs: QuantOutputs, stream=None):
    _check(lib().mxfp4_deosc_update(master_ptr, groups, rows, cols, step, ctypes.byref(params), state_ptr,
                                    ctypes.byref(outputs), _stream(stream)))


def mxfp4_grouped_gemm(op, num_groups, offsets_ptr, a: Operand, b: Operand, M, N, K, out_ptr, ldo, stream=None):
    _check(lib().mxfp4_grouped_gemm(op, num_groups, offsets_ptr, a, b, M, N, K, out_ptr, ldo, _stream(stream)))


def mxfp4_grouped_gemm_fused(op, num_groups, offsets_ptr, a: Operand, b: Operand, M, N, K, y_ptr, ldy,
                             q: QuantOutputs, qp: QuantParams | None = None, stream=None):
    _check(lib().mxfp4_grouped_gemm_fused(op, num_groups, offsets_ptr, a, b, M, N, K, y_ptr, ldy, ctypes.byref(q),
                                          ctypes.byref(qp) if qp is not None else None, _stream(stream)))


def mxfp4_route(logits_ptr, dtype, tokens, experts, ld, bias_ptr, mask_ptr, params: RouteParams, ids_ptr, weights_ptr,
                stream=None):
    _check(lib().mxfp4_route(logits_ptr, dtype, tokens, experts, ld, bias_ptr, mask_ptr, ctypes.byref(params), ids_ptr,
                             weights_ptr, _stream(stream)))


def mxfp4_route_bwd(logits_ptr, dtype, tokens, experts, ld, ids_ptr, d_weights_ptr, params: RouteParams, d_logits_ptr,
                    ldd, stream=None):
    _check(lib().mxfp4_route_bwd(logits_ptr, dtype, tokens, experts, ld, ids_ptr, d_weights_ptr, ctypes.byref(params),
                                 d_logits_ptr, ldd, _stream(stream)))


def mxfp4_expert_plan_rows(tokens: int, top_k: int, experts: int, align: int = 128) -> int:
    return int(lib().mxfp4_expert_plan_rows(tokens, top_k, experts, align))


def mxfp4_expert_plan_workspace(tokens: int, top_k: int, experts: int) -> int:
    return int(lib().mxfp4_expert_plan_workspace(tokens, top_k, experts))


def mxfp4_expert_plan(ids_ptr, tokens, top_k, experts, align, rows, fill, counts_ptr, offsets_ptr, row_of_slot_ptr,
                      slot_of_row_ptr, workspace_ptr, workspace_bytes, stream=None):
    _check(lib().mxfp4_expert_plan(ids_ptr, tokens, top_k, experts, align, rows, fill, counts_ptr, offsets_ptr,
                                   row_of_slot_ptr, slot_of_row_ptr, workspace_ptr, workspace_bytes, _stream(stream)))


def mxfp4_dispatch(x_ptr, dtype, tokens, top_k, cols, ldx, row_of_slot_ptr, slot_of_row_ptr, rows, out_ptr, ldo,
                   stream=None):
    _check(lib().mxfp4_dispatch(x_ptr, dtype, tokens, top_k, cols, ldx, row_of_slot_ptr, slot_of_row_ptr, rows, out_ptr,
                                ldo, _stream(stream)))


def mxfp4_combine(y_ptr, y_dtype, rows, cols, ldy, row_of_slot_ptr, weights_ptr, tokens, top_k, out_ptr, out_dtype, ldo,
                  stream=None):
    _check(lib().mxfp4_combine(y_ptr, y_dtype, rows, cols, ldy, row_of_slot_ptr, weights_ptr, tokens, top_k, out_ptr,
                               out_dtype, ldo, _stream(stream)))


def mxfp4_combine_bwd(d_out_ptr, d_dtype, ldd, y_ptr, y_dtype, rows, cols, ldy, row_of_slot_ptr, slot_of_row_ptr,
                      weights_ptr, tokens, top_k, dy_ptr, lddy, d_weights_ptr, stream=None):
    _check(lib().mxfp4_combine_bwd(d_out_ptr, d_dtype, ldd, y_ptr, y_dtype, rows, cols, ldy, row_of_slot_ptr,
                                   slot_of_row_ptr, weights_ptr, tokens, top_k, dy_ptr, lddy, d_weights_ptr,
                                   _stream(stream)))


def mxfp4_grad_clip_workspace(tensors, count: int) -> int:
    return int(lib().mxfp4_grad_clip_workspace(tensors, count))


def mxfp4_grad_clip(tensors, count, max_norm, norm_ptr, workspace_ptr, workspace_bytes, stream=None):
    _check(lib().mxfp4_grad_clip(tensors, count, max_norm, norm_ptr, workspace_ptr, workspace_bytes, _stream(stream)))


def mxfp4_mma_peak_probe(mmas_per_pair: int, stream=None) -> float:
    """Launch the tensor-pipe peak probe on `stream`; returns the launch's
    floating-point operations (the caller times the launch)."""
    flops = ctypes.c_double(0.0)
    _check(lib().mxfp4_mma_peak_probe(int(mmas_per_pair), ctypes.byref(flops), _stream(stream)))
    return flops.value


def mxfp4_selftest_wait_timeout(stream=None):
    """Launch the failure-detection self-test (a bounded wait that expires
    after about 2 s); read its result with mxfp4_check_device_status."""
    _check(lib().mxfp4_selftest_wait_timeout(_stream(stream)))


def mxfp4_check_device_status(stream=None):
    _check(lib().mxfp4_check_device_status(_stream(stream)))


def version() -> str:
    return lib().mxfp4_version().decode()


# ---------------------------------------------------------------------------
# Tensor helpers
# ---------------------------------------------------------------------------
def _require(cond: bool, msg: str) -> None:
    """Argument checks of the tensor helpers.  They raise (and survive
    `python -O`): a wrong dtype, layout or size would otherwise reach the
    library as a pointer and become an out-of-bounds device access."""
    if not cond:
        raise ValueError(msg)


def _check_buf(t, nbytes: int, name: str, dtype=torch.uint8) -> None:
    """`t` is a contiguous CUDA tensor of `dtype` holding at least `nbytes`."""
    _require(isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous(),
             "%s: a contiguous CUDA %s tensor is required" % (name, dtype))
    have = t.numel() * t.element_size()
    _require(have >= nbytes, "%s: %d bytes, at least %d required" % (name, have, nbytes))


def _check_input(x: torch.Tensor, name: str = "x") -> torch.Tensor:
    if isinstance(x, torch.Tensor) and x.dim() == 2:
        x = x.unsqueeze(0)
    _require(isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 3 and x.stride(2) == 1,
             "%s: a [rows, cols] or [groups, rows, cols] CUDA tensor with unit column stride is required" % name)
    _require(x.dtype in (torch.bfloat16, torch.float32), "%s: bf16 or float32 required" % name)
    _require(x.shape[0] == 1 or x.stride(0) == x.shape[1] * x.stride(1), "%s: groups must be back to back" % name)
    return x


def _check_offsets(offsets) -> None:
    _require(isinstance(offsets, torch.Tensor) and offsets.is_cuda and offsets.dtype == torch.int32
             and offsets.dim() == 1 and offsets.is_contiguous() and offsets.numel() >= 1,
             "offsets: a contiguous 1D int32 CUDA tensor of G + 1 entries")


def _check_quant_outputs(o: dict, G: int, Ro: int, Co: int, two_d: bool, R: int, C: int) -> None:
    """Sizes of a quantiser's output buffers (those present in `o`): codes
    [G, Ro, Co/2]; scales [G, Ro, Co/32] (2D: [G, R/32, C/32]); tensor-core
    scales per group; for 2D the transpose's codes [G, C, R/2] and scales."""
    _check_buf(o["codes"], G * Ro * (Co // 2), "codes")
    if o.get("scales") is not None:
        _check_buf(o["scales"], G * ((R // 32) * (C // 32) if two_d else Ro * (Co // 32)), "scales")
    if o.get("scales_mma") is not None:
        _check_buf(o["scales_mma"], G * mxfp4_mma_scale_bytes(Ro, Co // 32), "scales_mma")
    if o.get("codes_t") is not None:
        _check_buf(o["codes_t"], G * C * (R // 2), "codes_t")
    if o.get("scales_mma_t") is not None:
        _check_buf(o["scales_mma_t"], G * mxfp4_mma_scale_bytes(C, R // 32), "scales_mma_t")


def _check_operands(op: int, G: int, M: int, N: int, K: int, a_codes, a_scales, b_codes, b_scales) -> None:
    """Sizes of the GEMM operands as include/mxfp4.h lays them out."""
    _check_buf(a_codes, M * K // 2, "a_codes")
    _check_buf(a_scales, mxfp4_mma_scale_bytes(M, K // 32), "a_scales_mma")
    groups_b = 1 if op == GEMM_WGRAD else G
    _check_buf(b_codes, groups_b * N * K // 2, "b_codes")
    _check_buf(b_scales, groups_b * mxfp4_mma_scale_bytes(N, K // 32), "b_scales_mma")


def quantize(x: torch.Tensor, block: str = "1x32", along_rows: bool = False, rht_seed=None, sr_seed=None,
             sr_offset: int = 0, scales: bool = True, scales_mma: bool = False, transposed: bool = False,
             out: dict | None = None, stream=None) -> dict:
    """Quantise a [rows, cols] or [groups, rows, cols] bf16/f32 CUDA tensor.

    Returns a dict with 'codes', and as requested 'scales' (canonical),
    'scales_mma', 'codes_t' and 'scales_mma_t' (2D: the transpose's codes
    and tensor-core scales).  `out` may supply preallocated tensors."""
    x = _check_input(x)
    G, R, C = x.shape
    ld = x.stride(1)
    two_d = block == "32x32"
    p = QuantParams(BLOCK_32X32 if two_d else BLOCK_1X32, int(bool(along_rows) and not two_d),
                    16 if rht_seed is not None else 0, int(rht_seed or 0),
                    ROUND_STOCHASTIC if sr_seed is not None else ROUND_NEAREST, int(sr_seed or 0), int(sr_offset))
    Ro, Co = (C, R) if (along_rows and not two_d) else (R, C)
    o = dict(out or {})
    dev = x.device
    if "codes" not in o:
        o["codes"] = torch.empty((G, Ro, Co // 2), dtype=torch.uint8, device=dev)
    if scales and "scales" not in o:
        shape = (G, R // 32, C // 32) if two_d else (G, Ro, Co // 32)
        o["scales"] = torch.empty(shape, dtype=torch.uint8, device=dev)
    if scales_mma and "scales_mma" not in o:
        o["scales_mma"] = torch.empty((G, mxfp4_mma_scale_bytes(Ro, Co // 32)), dtype=torch.uint8, device=dev)
    if transposed and two_d:
        if "codes_t" not in o:
            o["codes_t"] = torch.empty((G, C, R // 2), dtype=torch.uint8, device=dev)
        if scales_mma and "scales_mma_t" not in o:
            o["scales_mma_t"] = torch.empty((G, mxfp4_mma_scale_bytes(C, R // 32)), dtype=torch.uint8, device=dev)
    _check_quant_outputs(o, G, Ro, Co, two_d, R, C)
    outs = QuantOutputs(o["codes"].data_ptr(), _ptr(o.get("scales")), _ptr(o.get("scales_mma")),
                        _ptr(o.get("codes_t")), _ptr(o.get("scales_mma_t")))
    mxfp4_quantize(ctypes.c_void_p(x.data_ptr()), _dtype_code(x), G, R, C, ld, p, outs, stream)
    return o


def quantize_dual(x: torch.Tensor, row_rht_seed=None, col_rht_seed=None, sr_seed=None, row_sr_offset: int = 0,
                  col_sr_offset: int = 0, scales: bool = True, scales_mma: bool = False, out_row: dict | None = None,
                  out_col: dict | None = None, stream=None) -> tuple:
    """Quantise a [rows, cols] or [groups, rows, cols] bf16/f32 CUDA tensor
    in both 1D directions from one read: returns (row, col), the outputs of
    quantize(x, ...) along the last dim and quantize(x, along_rows=True, ...),
    each a dict like quantize's."""
    x = _check_input(x)
    G, R, C = x.shape
    rounding = ROUND_STOCHASTIC if sr_seed is not None else ROUND_NEAREST
    rp = QuantParams(BLOCK_1X32, 0, 16 if row_rht_seed is not None else 0, int(row_rht_seed or 0), rounding,
                     int(sr_seed or 0), int(row_sr_offset))
    cp = QuantParams(BLOCK_1X32, 1, 16 if col_rht_seed is not None else 0, int(col_rht_seed or 0), rounding,
                     int(sr_seed or 0), int(col_sr_offset))
    dev = x.device
    outs = []
    for (o, Ro, Co) in ((dict(out_row or {}), R, C), (dict(out_col or {}), C, R)):
        if "codes" not in o:
            o["codes"] = torch.empty((G, Ro, Co // 2), dtype=torch.uint8, device=dev)
        if scales and "scales" not in o:
            o["scales"] = torch.empty((G, Ro, Co // 32), dtype=torch.uint8, device=dev)
        if scales_mma and "scales_mma" not in o:
            o["scales_mma"] = torch.empty((G, mxfp4_mma_scale_bytes(Ro, Co // 32)), dtype=torch.uint8, device=dev)
        _check_quant_outputs(o, G, Ro, Co, False, R, C)
        outs.append(o)
    ro, co = outs
    qo_r = QuantOutputs(ro["codes"].data_ptr(), _ptr(ro.get("scales")), _ptr(ro.get("scales_mma")), None, None)
    qo_c = QuantOutputs(co["codes"].data_ptr(), _ptr(co.get("scales")), _ptr(co.get("scales_mma")), None, None)
    mxfp4_quantize_dual(ctypes.c_void_p(x.data_ptr()), _dtype_code(x), G, R, C, x.stride(1), rp, cp, qo_r, qo_c,
                        stream)
    return ro, co


def rht(x: torch.Tensor, seed: int, out_dtype=torch.float32, axis: int = 1, stream=None) -> torch.Tensor:
    """RHT-16 of a 2D tensor along the last dim (axis 1) or along dim 0
    (axis 0); the output keeps x's shape."""
    _require(isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2 and x.stride(1) == 1
             and x.dtype in (torch.bfloat16, torch.float32), "x: a 2D bf16/float32 CUDA tensor with unit column stride")
    _require(axis in (0, 1), "axis: 0 or 1")
    R, C = x.shape
    y = torch.empty((R, C), dtype=out_dtype, device=x.device)
    mxfp4_rht(ctypes.c_void_p(x.data_ptr()), _dtype_code(x), R, C, x.stride(0), int(axis), 16, int(seed),
              ctypes.c_void_p(y.data_ptr()), _dtype_code(y), stream)
    return y


def deosc_update(master: torch.Tensor, step: int, state: torch.Tensor, flip_threshold: int = 4,
                 reset_period: int = 0, scales: bool = True, scales_mma: bool = False, transposed: bool = False,
                 out: dict | None = None, stream=None, freeze_lower: bool = False) -> dict:
    if isinstance(master, torch.Tensor) and master.dim() == 2:
        master = master.unsqueeze(0)
    _require(isinstance(master, torch.Tensor) and master.is_cuda and master.dtype == torch.float32
             and master.dim() == 3 and master.is_contiguous(), "master: a contiguous float32 CUDA tensor")
    _check_buf(state, master.numel(), "state")
    _require(state.numel() == master.numel(), "state: one byte per weight")
    G, R, C = master.shape
    o = dict(out or {})
    dev = master.device
    if "codes" not in o:
        o["codes"] = torch.empty((G, R, C // 2), dtype=torch.uint8, device=dev)
    if scales and "scales" not in o:
        o["scales"] = torch.empty((G, R // 32, C // 32), dtype=torch.uint8, device=dev)
    if scales_mma and "scales_mma" not in o:
        o["scales_mma"] = torch.empty((G, mxfp4_mma_scale_bytes(R, C // 32)), dtype=torch.uint8, device=dev)
    if transposed:
        if "codes_t" not in o:
            o["codes_t"] = torch.empty((G, C, R // 2), dtype=torch.uint8, device=dev)
        if scales_mma and "scales_mma_t" not in o:
            o["scales_mma_t"] = torch.empty((G, mxfp4_mma_scale_bytes(C, R // 32)), dtype=torch.uint8, device=dev)
    _check_quant_outputs(o, G, R, C, True, R, C)
    outs = QuantOutputs(o["codes"].data_ptr(), _ptr(o.get("scales")), _ptr(o.get("scales_mma")),
                        _ptr(o.get("codes_t")), _ptr(o.get("scales_mma_t")))
    mxfp4_deosc_update(ctypes.c_void_p(master.data_ptr()), G, R, C, int(step),
                       DeoscParams(int(flip_threshold), int(reset_period), int(bool(freeze_lower))),
                       ctypes.c_void_p(state.data_ptr()), outs,
                       stream)
    return o


def grouped_gemm(op: int, offsets: torch.Tensor, a_codes, a_scales_mma, b_codes, b_scales_mma, M: int, N: int,
                 K: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """FPROP/DGRAD: out [M, N]; WGRAD: out [G, M, N] (see include/mxfp4.h)."""
    _check_offsets(offsets)
    G = offsets.numel() - 1
    if out is None:
        shape = (G, M, N) if op == GEMM_WGRAD else (M, N)
        out = torch.empty(shape, dtype=torch.float32, device=offsets.device)
    _require(isinstance(out, torch.Tensor) and out.is_cuda and out.dtype == torch.float32 and out.stride(-1) == 1,
             "out: a float32 CUDA tensor with unit column stride")
    ldo = out.stride(-2)
    if op == GEMM_WGRAD:
        _require(out.dim() == 3 and out.shape[0] >= G and out.shape[1] == M and out.shape[2] >= N
                 and (G <= 1 or out.stride(0) == M * ldo), "out: [G, M, >= N] with group stride M * row stride")
    else:
        _require(out.dim() == 2 and out.shape[0] >= M and out.shape[1] >= N, "out: [>= M, >= N]")
    _check_operands(op, G, M, N, K, a_codes, a_scales_mma, b_codes, b_scales_mma)
    mxfp4_grouped_gemm(op, G, ctypes.c_void_p(offsets.data_ptr()),
                       Operand(a_codes.data_ptr(), a_scales_mma.data_ptr()),
                       Operand(b_codes.data_ptr(), b_scales_mma.data_ptr()), M, N, K,
                       ctypes.c_void_p(out.data_ptr()), ldo, stream)
    return out


def grouped_gemm_fused(op: int, offsets: torch.Tensor, a_codes, a_scales_mma, b_codes, b_scales_mma, M: int, N: int,
                       K: int, scales: bool = True, scales_mma: bool = True, y: torch.Tensor | None = None,
                       out: dict | None = None, sr_seed=None, sr_offset: int = 0, stream=None) -> tuple:
    """FPROP/DGRAD with the fused epilogue: returns (y, q) with y the [M, N]
    bf16 output and q the dict ('codes', 'scales', 'scales_mma') of its
    1x32-along-N MXFP4 quantisation, nearest rounding or, with sr_seed,
    stochastic rounding as quantize(y, sr_seed=..., sr_offset=...)."""
    _check_offsets(offsets)
    G = offsets.numel() - 1
    dev = offsets.device
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _require(isinstance(y, torch.Tensor) and y.is_cuda and y.dtype == torch.bfloat16 and y.dim() == 2
             and y.stride(-1) == 1 and y.shape[0] >= M and y.shape[1] >= N,
             "y: a [>= M, >= N] bf16 CUDA tensor with unit column stride")
    _check_operands(op, G, M, N, K, a_codes, a_scales_mma, b_codes, b_scales_mma)
    o = dict(out or {})
    if "codes" not in o:
        o["codes"] = torch.empty((M, N // 2), dtype=torch.uint8, device=dev)
    if scales and "scales" not in o:
        o["scales"] = torch.empty((M, N // 32), dtype=torch.uint8, device=dev)
    if scales_mma and "scales_mma" not in o:
        o["scales_mma"] = torch.empty((mxfp4_mma_scale_bytes(M, N // 32),), dtype=torch.uint8, device=dev)
    _check_quant_outputs(o, 1, M, N, False, M, N)
    q = QuantOutputs(o["codes"].data_ptr(), _ptr(o.get("scales")), _ptr(o.get("scales_mma")), None, None)
    qp = QuantParams(BLOCK_1X32, 0, 0, 0, ROUND_STOCHASTIC if sr_seed is not None else ROUND_NEAREST,
                     int(sr_seed or 0), int(sr_offset))
    mxfp4_grouped_gemm_fused(op, G, ctypes.c_void_p(offsets.data_ptr()),
                             Operand(a_codes.data_ptr(), a_scales_mma.data_ptr()),
                             Operand(b_codes.data_ptr(), b_scales_mma.data_ptr()), M, N, K,
                             ctypes.c_void_p(y.data_ptr()), y.stride(0), q, qp, stream)
    return y, o


# ---------------------------------------------------------------------------
# Routing of tokens to experts
# ---------------------------------------------------------------------------
def _home(t, stream, what: str) -> int:
    """The device of `t` if it is the current one and no stream is named,
    else -1 (then _elsewhere makes the call)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError("%s: a CUDA tensor is required" % what)
    dev = t.get_device()
    return dev if stream is None and dev == torch.cuda.current_device() else -1


def _elsewhere(fn, t, stream, *args, **kw):
    """Call a helper on its tensor's device and, if a stream is named, under
    that stream: what it allocates belongs to the stream that uses it, and the
    launch goes to the device that holds the tensors."""
    if stream is None:
        with torch.cuda.device(t.device):
            return fn(*args, **kw)
    _require(stream.device == t.device, "%s: stream and tensors on different devices" % fn.__name__)
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _current(device: int) -> int:
    """The handle of a device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device)


def _check_matrix(t, name: str, dev: int) -> int:
    """`t` is a 2D bf16/f32 tensor on CUDA device `dev` with unit column
    stride; returns its row stride."""
    if not (isinstance(t, torch.Tensor) and t.dim() == 2 and t.dtype in _FLOATS and t.get_device() == dev):
        raise ValueError("%s: a 2D bf16/float32 tensor on cuda:%d is required" % (name, dev))
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError("%s: unit column stride is required" % name)
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError("%s: rows must not overlap" % name)
    return ld


def _check_vector(t, numel: int, name: str, dev: int, dtype) -> int:
    """`t` is a contiguous tensor of `numel` elements of `dtype` on CUDA device
    `dev`; returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == numel and t.is_contiguous()
            and t.get_device() == dev):
        raise ValueError("%s: a contiguous %s tensor of %d elements on cuda:%d is required" % (name, dtype, numel, dev))
    return t.data_ptr()


_FLOATS = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


@functools.lru_cache(maxsize=256)
def _route_struct(score, *values) -> RouteParams:   # a name and plain numbers only
    _require(score in SCORES, "score: 'softmax' or 'sigmoid'")
    _require(all(-2 ** 31 <= v < 2 ** 31 for v in values[:-1]), "top_k, groups, top_groups, group_best: out of range")
    return RouteParams(SCORES[score], *values)


def _route_params(score, top_k, groups, top_groups, group_best, renormalise, scale) -> RouteParams:
    if not (type(top_k) is type(groups) is type(top_groups) is type(group_best) is int and type(scale) is float):
        top_k, groups, top_groups, group_best = int(top_k), int(groups), int(top_groups), int(group_best)
        scale = float(scale)
    return _route_struct(score, top_k, groups, top_groups, group_best, True if renormalise else False, scale)


def route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None,
          mask: torch.Tensor | None = None, groups: int = 1, top_groups: int | None = None, group_best: int = 1,
          renormalise: bool = True, scale: float = 1.0, out: dict | None = None, stream=None) -> dict:
    """Choose top_k experts for each row of the [tokens, experts] bf16/f32
    logits (include/mxfp4.h, mxfp4_route).  bias: f32 [experts], for the
    choice only; mask: bool or uint8 [tokens], False for a token without
    experts (ids -1, weights 0); groups, top_groups (all by default),
    group_best: choice within the best groups.  Returns 'ids' (int32) and
    'weights' (f32), both [tokens, top_k]; `out` may supply them.  `stream`
    names a stream to use instead of the current one, here and below."""
    dev = _home(logits, stream, "route")
    if dev < 0:
        return _elsewhere(route, logits, stream, logits, top_k, score, bias, mask, groups, top_groups, group_best, renormalise,
                          scale, out)
    ld = _check_matrix(logits, "logits", dev)
    T, E = logits.shape
    p = _route_params(score, top_k, groups, groups if top_groups is None else top_groups, group_best, renormalise, scale)
    k = p.top_k
    o = dict(out or {})
    if "ids" not in o:
        o["ids"] = torch.empty((T, max(k, 0)), dtype=torch.int32, device=dev)
    if "weights" not in o:
        o["weights"] = torch.empty((T, max(k, 0)), dtype=torch.float32, device=dev)
    ids = _check_vector(o["ids"], T * k, "ids", dev, torch.int32)
    weights = _check_vector(o["weights"], T * k, "weights", dev, torch.float32)
    b = m = None
    if bias is not None:
        b = _check_vector(bias, E, "bias", dev, torch.float32)
    if mask is not None:
        _require(isinstance(mask, torch.Tensor) and mask.dtype in (torch.bool, torch.uint8), "mask: bool or uint8")
        m = _check_vector(mask, T, "mask", dev, mask.dtype)
    _check(lib().mxfp4_route(logits.data_ptr(), _FLOATS[logits.dtype], T, E, ld, b, m, ctypes.byref(p), ids, weights,
                             _current(dev)))
    return o


def route_bwd(logits: torch.Tensor, ids: torch.Tensor, d_weights: torch.Tensor, score: str = "softmax",
              renormalise: bool = True, scale: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of route's weights with respect to its logits: [tokens,
    experts] in the logits' dtype.  ids and d_weights are [tokens, top_k];
    score, renormalise and scale as in the forward call."""
    dev = _home(logits, stream, "route_bwd")
    if dev < 0:
        return _elsewhere(route_bwd, logits, stream, logits, ids, d_weights, score, renormalise, scale, out)
    ld = _check_matrix(logits, "logits", dev)
    T, E = logits.shape
    _require(isinstance(ids, torch.Tensor) and ids.dim() == 2 and ids.shape[0] == T, "ids: [tokens, top_k]")
    k = ids.shape[1]
    p = _route_params(score, k, 1, 1, 1, renormalise, scale)
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=dev)
    ldd = _check_matrix(out, "out", dev)
    _require(out.dtype == logits.dtype and out.shape == logits.shape, "out: shape and dtype of the logits")
    _check(lib().mxfp4_route_bwd(
        logits.data_ptr(), _FLOATS[logits.dtype], T, E, ld, _check_vector(ids, T * k, "ids", dev, torch.int32),
        _check_vector(d_weights, T * k, "d_weights", dev, torch.float32), ctypes.byref(p), out.data_ptr(), ldd,
        _current(dev)))
    return out


_PLAN_PARTS = {"counts", "offsets", "row_of_slot", "slot_of_row"}
_plan_workspace = functools.lru_cache(maxsize=256)(lambda T, k, E: mxfp4_expert_plan_workspace(T, k, E))


def expert_plan(ids: torch.Tensor, experts: int, align: int = 128, rows: int | None = None, fill: bool = False,
                out: dict | None = None, stream=None) -> dict:
    """Lay the slots of the int32 ids [tokens, top_k] out in one segment per
    expert, padded to `align` rows (include/mxfp4.h, mxfp4_expert_plan).
    rows: length of slot_of_row, by default the least that holds every split
    (mxfp4_expert_plan_rows).  fill: the last segment ends at `rows`, so that
    the grouped GEMMs' M is `rows` without reading the device.  Returns
    int32 'counts' [experts], 'offsets' [experts + 1], 'row_of_slot' [tokens,
    top_k] and 'slot_of_row' [rows]."""
    dev = _home(ids, stream, "expert_plan")
    if dev < 0:
        return _elsewhere(expert_plan, ids, stream, ids, experts, align, rows, fill, out)
    _require(ids.dim() == 2 and ids.dtype == torch.int32 and ids.is_contiguous(),
             "ids: a contiguous int32 [tokens, top_k] tensor is required")
    T, k = ids.shape
    E = int(experts)
    _require(E >= 1, "experts: at least 1")
    o = dict(out or {})
    if rows is None:
        rows = o["slot_of_row"].numel() if "slot_of_row" in o else mxfp4_expert_plan_rows(T, k, E, align)
    if not _PLAN_PARTS <= o.keys():
        for name, shape in (("counts", (E,)), ("offsets", (E + 1,)), ("row_of_slot", (T, k)), ("slot_of_row", (rows,))):
            if name not in o:
                o[name] = torch.empty(shape, dtype=torch.int32, device=dev)
    i32 = torch.int32
    counts = _check_vector(o["counts"], E, "counts", dev, i32)
    offsets = _check_vector(o["offsets"], E + 1, "offsets", dev, i32)
    row_of_slot = _check_vector(o["row_of_slot"], T * k, "row_of_slot", dev, i32)
    slot_of_row = _check_vector(o["slot_of_row"], rows, "slot_of_row", dev, i32)
    need = _plan_workspace(T, k, E)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None   # held until the launch
    _check(lib().mxfp4_expert_plan(ids.data_ptr(), T, k, E, int(align), rows, int(bool(fill)), counts, offsets,
                                   row_of_slot, slot_of_row, None if ws is None else ws.data_ptr(), need, _current(dev)))
    return o


def _plan_part(plan: dict, name: str, dev: int) -> torch.Tensor:
    t = plan[name]
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.get_device() == dev and t.is_contiguous()
            and t.dim() == (2 if name == "row_of_slot" else 1)):
        raise ValueError("plan: '%s' of expert_plan on cuda:%d" % (name, dev))
    return t


def dispatch(x: torch.Tensor, plan: dict, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The [tokens, cols] bf16/f32 rows of x in the plan's segments: [rows,
    cols], zeros on rows without a slot.  Its gradient is combine(d_rows,
    plan)."""
    dev = _home(x, stream, "dispatch")
    if dev < 0:
        return _elsewhere(dispatch, x, stream, x, plan, out)
    ldx = _check_matrix(x, "x", dev)
    slot_of_row, row_of_slot = _plan_part(plan, "slot_of_row", dev), _plan_part(plan, "row_of_slot", dev)
    T, k = row_of_slot.shape
    _require(x.shape[0] == T, "x: one row per token of the plan")
    rows, cols = slot_of_row.numel(), x.shape[1]
    if out is None:
        out = torch.empty((rows, cols), dtype=x.dtype, device=dev)
    ldo = _check_matrix(out, "out", dev)
    _require(out.shape == (rows, cols) and out.dtype == x.dtype, "out: [rows, cols] in the dtype of x")
    _check(lib().mxfp4_dispatch(x.data_ptr(), _FLOATS[x.dtype], T, k, cols, ldx, row_of_slot.data_ptr(),
                                slot_of_row.data_ptr(), rows, out.data_ptr(), ldo, _current(dev)))
    return out


def combine(y: torch.Tensor, plan: dict, weights: torch.Tensor | None = None, out_dtype=None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Each token's rows of y [rows, cols] (bf16/f32) added up with its f32
    weights [tokens, top_k] (ones by default): [tokens, cols] in out_dtype
    (y's by default), binary32 sums rounded once."""
    dev = _home(y, stream, "combine")
    if dev < 0:
        return _elsewhere(combine, y, stream, y, plan, weights, out_dtype, out)
    ldy = _check_matrix(y, "y", dev)
    row_of_slot = _plan_part(plan, "row_of_slot", dev)
    (T, k), (rows, cols) = row_of_slot.shape, y.shape
    _require(rows == _plan_part(plan, "slot_of_row", dev).numel(), "y: one row per row of the plan")
    w = None if weights is None else _check_vector(weights, T * k, "weights", dev, torch.float32)
    if out is None:
        out = torch.empty((T, cols), dtype=y.dtype if out_dtype is None else out_dtype, device=dev)
    ldo = _check_matrix(out, "out", dev)
    _require(out.shape == (T, cols) and out_dtype in (None, out.dtype), "out: [tokens, cols] in out_dtype")
    _check(lib().mxfp4_combine(y.data_ptr(), _FLOATS[y.dtype], rows, cols, ldy, row_of_slot.data_ptr(), w, T, k,
                               out.data_ptr(), _FLOATS[out.dtype], ldo, _current(dev)))
    return out


def combine_bwd(d_out: torch.Tensor, y: torch.Tensor, plan: dict, weights: torch.Tensor,
                out: dict | None = None, stream=None) -> dict:
    """Gradient of combine: 'dy' [rows, cols] in d_out's dtype (zeros on rows
    without a slot) and 'd_weights' f32 [tokens, top_k]."""
    dev = _home(d_out, stream, "combine_bwd")
    if dev < 0:
        return _elsewhere(combine_bwd, d_out, stream, d_out, y, plan, weights, out)
    ldd, ldy = _check_matrix(d_out, "d_out", dev), _check_matrix(y, "y", dev)
    row_of_slot, slot_of_row = _plan_part(plan, "row_of_slot", dev), _plan_part(plan, "slot_of_row", dev)
    (T, k), (rows, cols) = row_of_slot.shape, y.shape
    _require(rows == slot_of_row.numel(), "y: one row per row of the plan")
    _require(d_out.shape == (T, cols), "d_out: [tokens, cols]")
    o = dict(out or {})
    if "dy" not in o:
        o["dy"] = torch.empty((rows, cols), dtype=d_out.dtype, device=dev)
    if "d_weights" not in o:
        o["d_weights"] = torch.empty((T, k), dtype=torch.float32, device=dev)
    lddy = _check_matrix(o["dy"], "dy", dev)
    _require(o["dy"].shape == y.shape and o["dy"].dtype == d_out.dtype, "dy: [rows, cols] in the dtype of d_out")
    _check(lib().mxfp4_combine_bwd(
        d_out.data_ptr(), _FLOATS[d_out.dtype], ldd, y.data_ptr(), _FLOATS[y.dtype], rows, cols, ldy,
        row_of_slot.data_ptr(), slot_of_row.data_ptr(), _check_vector(weights, T * k, "weights", dev, torch.float32), T, k,
        o["dy"].data_ptr(), lddy, _check_vector(o["d_weights"], T * k, "d_weights", dev, torch.float32), _current(dev)))
    return o


class GradList:
    """The gradients of one grad_clip call, checked once and kept for later
    calls: contiguous bf16/f32 CUDA tensors of one device.  out: None to scale
    in place, else as many tensors of the same shapes and dtypes.  The list
    shares the tensors' storages and keeps them alive; a tensor whose storage
    was resized, freed or exchanged since is refused at the call.  A parameter
    whose .grad is another tensor by then (zero_grad(set_to_none=True)) needs a
    new list: this one goes on with the tensors it was given."""

    def __init__(self, grads, out=None):
        grads = list(grads)
        outs = grads if out is None else list(out)
        _require(len(grads) > 0, "grads: at least one tensor")
        _require(len(outs) == len(grads), "out: one tensor per gradient")
        for name, ts in (("grads", grads), ("out", outs)):
            for t in ts:
                _require(isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in _FLOATS and t.is_contiguous()
                         and t.device == grads[0].device, "%s: contiguous bf16/float32 CUDA tensors of one device" % name)
        for g, o in zip(grads, outs):
            _require(o.shape == g.shape and o.dtype == g.dtype, "out: shapes and dtypes of the gradients")
        spans = []   # (begin, end, tensor, is output)
        for i, (g, o) in enumerate(zip(grads, outs)):
            n = g.numel() * g.element_size()
            if n:
                spans.append((o.data_ptr(), o.data_ptr() + n, i, True))
                if o.data_ptr() != g.data_ptr():
                    spans.append((g.data_ptr(), g.data_ptr() + n, i, False))
        spans.sort()
        end, end_out = 0, 0   # furthest end of any span so far, and of an output's
        for b, e, i, is_out in spans:
            _require(b >= (end if is_out else end_out), "grads, out: the outputs overlap each other or a gradient")
            end = max(end, e)
            end_out = max(end_out, e) if is_out else end_out
        self.anchor = grads[0].detach()
        self._tensors = grads + ([] if out is None else outs)
        self._storages = [t.detach() for t in self._tensors]   # kept alive even if a tensor leaves its own
        self._addresses = [t.data_ptr() for t in self._tensors]
        self.count = len(grads)
        self._table = (GradTensor * self.count)(*[
            GradTensor(g.data_ptr(), o.data_ptr(), g.numel(), _FLOATS[g.dtype]) for g, o in zip(grads, outs)])
        self.workspace_bytes = mxfp4_grad_clip_workspace(self._table, self.count)

    def table(self):
        """The library's descriptors, after a look at the storages."""
        if list(map(torch.Tensor.data_ptr, self._tensors)) != self._addresses:
            raise ValueError("grads: a storage was resized, freed or exchanged")
        return self._table


def _grad_clip(grads: GradList, max_norm: float, norm: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    dev = _home(grads.anchor, stream, "grad_clip")
    if dev < 0:
        return _elsewhere(_grad_clip, grads.anchor, stream, grads, max_norm, norm)
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
    need = grads.workspace_bytes
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None   # held until the launch
    _check(lib().mxfp4_grad_clip(grads.table(), grads.count, float(max_norm),
                                 _check_vector(norm, 1, "norm", dev, torch.float32),
                                 None if ws is None else ws.data_ptr(), need, _current(dev)))
    return norm


def grad_clip(grads, max_norm: float, norm: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scale the gradients so that their global norm is at most max_norm, and
    return the norm they had (f32 [1] on the device; `norm` may supply it).
    grads: a GradList, or a sequence of tensors, which are scaled in place.
    Nothing is scaled when the norm is not finite; max_norm = inf gives the
    norm alone.  A sequence is checked and laid out on every call (3 us a
    tensor of host time), a GradList once."""
    return _grad_clip(grads if isinstance(grads, GradList) else GradList(grads), max_norm, norm=norm, stream=stream)
