"""Quantized GEMV with fused dequantization for GB300 (sm_103a), and the
operators around it in a serving step: the block-scaled fp8 products, norms and
gates, attention over a paged cache, the upkeep of its pages and token log
probabilities.

The compute lives in the CUDA library libqgemv.so (C ABI in include/qgemv.h);
this module is a thin binding over it with the same names, by ctypes and, for
the serving operators, by the compiled module _serving. It only marshals
arguments: torch supplies device memory and the current stream, every step of
the computation runs in the library's kernels. The library is loaded on first
use, and every call raises if it has not been built or no CUDA device is
present: there is no CPU fallback. Calls run on the current device, and tensors
of another one are refused.

Workspace: calls that need device scratch (split-K partial sums) get it from
a torch buffer per (device, stream) that grows on demand, unless the caller
passes one. Calls on different streams therefore never share scratch; calls
on one stream are ordered by the stream. A call that torch.cuda.graph captures
takes its scratch from the graph's own memory, so that graphs may run beside
each other; under another kind of capture the caller passes a workspace.

A serving operator given a stream runs as under torch.cuda.stream(stream): its
new outputs belong to that stream.
"""
from __future__ import annotations

import ctypes as C
import importlib
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemv.so")

QG_OK, QG_ERR_INVALID_ARG, QG_ERR_UNSUPPORTED, QG_ERR_MISALIGNED = 0, 1, 2, 3
QG_ERR_CUDA, QG_ERR_WORKSPACE, QG_ERR_DEVICE = 4, 5, 6
QG_OP_Q4_0, QG_OP_DUAL_Q4_0, QG_OP_Q4_K, QG_OP_AFFINE, QG_OP_AF4_G64 = 0, 1, 2, 3, 4
QG_OP_DUAL_Q4_0_HOST = 5
QG_F32, QG_F16, QG_BF16 = 0, 1, 2
QG_OPT_PDL = 1
QG_OPT_PREFILL_MIN_M = 2
QG_OPT_STREAM, QG_OPT_STREAM_WARPS, QG_OPT_STREAM_SLOTS = 3, 4, 5
QG_OPT_STAGES_AHEAD = 6
QG_OPT_STAGED_WARPS = 7
QG_OPT_PREFILL_FOLD = 8
QG_OPT_XREG = 9
QG_OPT_XREG_AHEAD = 10
QG_OPT_XREG_WARPS = 11
QG_OPT_XREG_CTAS = 12

EXPORTS = ("qgemv_q4_0", "qgemv_dual_q4_0", "qgemv_q4_k", "qmm_affine", "qkv_split",
           "dequant_q4_0", "dequant_q4_k", "dequant_affine", "qg_workspace_size",
           "qg_status_string", "qg_last_cuda_error", "qg_device_error",
           "qg_selftest_wait_timeout", "qg_set_option", "qg_get_option",
           "qgemv_q4_k_noalloc", "qg_prepare_af4_g64", "qmm_af4_g64", "qgemv_dual_q4_0_host",
           "quantize_fp8_b128", "qmm_fp8_b128", "qmm_fp8_b128_workspace_size", "qmm_fp8_b128_grouped",
           "qmm_fp8_b128_grouped_workspace_size", "rms_norm", "rms_norm_fp8_b128", "silu_mul", "silu_mul_fp8_b128",
           "attn_paged", "attn_paged_workspace_size", "kv_append", "kv_append_rope", "kv_copy_pages", "kv_fork", "kv_fork_workspace_size", "kv_free",
           "kv_compact", "kv_compact_workspace_size", "token_logprobs")

_LIB = None
_LOCK = threading.Lock()


class QGError(RuntimeError):
    def __init__(self, what: str, status: int):
        self.status = status
        msg = f"{what}: {status_string(status)}"
        if status == QG_ERR_CUDA:
            msg += f" (cudaError {lib().qg_last_cuda_error()})"
        super().__init__(msg)


def lib():
    """The loaded library (ctypes.CDLL), typed. Raises if it was not built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    with _LOCK:
        if _LIB is not None:
            return _LIB
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = C.CDLL(LIB_PATH)
        P, I64, I, SZ = C.c_void_p, C.c_int64, C.c_int, C.c_size_t
        sig = {
            "qgemv_q4_0": [P, P, P, I64, I64, I64, P, SZ, P],
            "qgemv_dual_q4_0": [P, P, P, P, P, I64, I64, I64, P, SZ, P],
            "qgemv_dual_q4_0_host": [P, P, P, P, P, I64, I64, I64, P, SZ, P],
            "qgemv_q4_k": [P, P, P, I64, I64, I64, P, SZ, P],
            "qmm_affine": [P, P, P, P, P, I64, I64, I64, I, I, P, SZ, P],
            "qkv_split": [P, P, P, P, I64, I64, I64, I64, P],
            "dequant_q4_0": [P, P, I64, I64, P],
            "dequant_q4_k": [P, P, I64, I64, P],
            "dequant_affine": [P, P, P, P, I64, I64, I, I, P],
            "qg_workspace_size": [I, I64, I64, I64, I, I, C.POINTER(SZ)],
            "qg_status_string": [I],
            "qg_last_cuda_error": [],
            "qg_device_error": [I, C.POINTER(C.c_uint)],
            "qg_selftest_wait_timeout": [I64, P],
            "qg_set_option": [I, I64],
            "qg_get_option": [I, C.POINTER(I64)],
            "qgemv_q4_k_noalloc": [P, P, P, I64, I64, I64, P],
            "qg_prepare_af4_g64": [P, P, P, P, P, I64, I64, P],
            "qmm_af4_g64": [P, P, P, P, I64, I64, I64, P, SZ, P],
            "quantize_fp8_b128": [P, I, I64, P, P, I64, I64, P],
            "qmm_fp8_b128": [P, P, P, P, P, I, I64, I64, I64, P, SZ, P],
            "qmm_fp8_b128_workspace_size": [I64, I64, I64, C.POINTER(SZ)],
            "qmm_fp8_b128_grouped": [P, P, P, P, P, P, I, I64, I64, I64, I64, P, SZ, P],
            "qmm_fp8_b128_grouped_workspace_size": [I64, I64, I64, I64, C.POINTER(SZ)],
            "rms_norm": [P, I, I64, P, I, I64, P, I, C.c_float, C.c_float, P, I, P, I64, I64, I64, P],
            "rms_norm_fp8_b128": [P, I, I64, P, I, I64, P, I, C.c_float, C.c_float, P, P, P, I64, I64, I64, P],
            "silu_mul": [P, I64, P, I64, I, P, I, I64, I64, P],
            "silu_mul_fp8_b128": [P, I64, P, I64, I, P, P, I64, I64, P],
            "attn_paged": [P, I64] + [P] * 7 + [I] + [I64] * 9 + [C.c_float] * 2 + [I64, P, SZ, P],
            "attn_paged_workspace_size": [I64] * 6 + [C.POINTER(SZ)],
            "kv_append": [P, P, I64, I64, I, P, P, I, P] + [I64] * 5 + [P],
            "kv_append_rope": [P, P, P, I64, I64, I64, I, P, P, I64, I, P, P, P, I, P] + [I64] * 6 + [P],
            "kv_copy_pages": [P, I64, I64, I64, P, P, I64, P],
            "kv_fork": [P] + [I64] * 4 + [P] * 3 + [I64, I64, P, I64, P, P, P, P, SZ, P],
            "kv_fork_workspace_size": [I64, C.POINTER(SZ)],
            "kv_free": [P] * 4 + [I64] * 3 + [P] * 4,
            "kv_compact": [P, I64, I64, I64, P, I64, I64] + [P] * 6 + [SZ, P],
            "kv_compact_workspace_size": [I64, C.POINTER(SZ)],
            "token_logprobs": [P, I, I64, P, I64, I64, I] + [P] * 6,
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = C.c_char_p if name == "qg_status_string" else C.c_int
        _LIB = L
        return L


def status_string(status: int) -> str:
    return lib().qg_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != QG_OK:
        raise QGError(what, rc)


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current device ({torch._C._cuda_getDevice()}), got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _host(t: torch.Tensor, name: str, dtype) -> int:
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise ValueError(f"{name} must be a CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        if torch.cuda.is_initialized():  # the current stream, without building an object for it
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# --------------------------------------------------------------- workspace
_WS = {}


def workspace_size(op: int, M: int, N: int, K: int, group_size: int = 0, packed: int = 0) -> int:
    n = C.c_size_t(0)
    _check(lib().qg_workspace_size(op, M, N, K, group_size, packed, C.byref(n)), "qg_workspace_size")
    return int(n.value)


def _workspace(op, M, N, K, gs, packed, device, workspace, stream):
    return _scratch(workspace_size(op, M, N, K, gs, packed), device, workspace, stream)


def _scratch(need, device, workspace, stream):
    if workspace is not None:
        return _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    if need == 0:
        return None, 0
    if torch.cuda.is_current_stream_capturing():
        # The graph may run on any stream, beside other graphs: scratch of its own.
        buf = torch.empty(need, dtype=torch.uint8, device=device)
        return buf.data_ptr(), need
    # One buffer per (device, stream): two calls on different streams may run
    # at the same time and must not share split-K scratch.
    key = (device.index, stream)
    buf = _WS.get(key)
    if buf is None or buf.numel() < need:
        with _LOCK:
            buf = _WS.get(key)
            if buf is None or buf.numel() < need:
                buf = _WS[key] = torch.empty(need, dtype=torch.uint8, device=device)
    return buf.data_ptr(), buf.numel()


# ------------------------------------------------------------------- calls
def qgemv_q4_0(w, x, y=None, *, N=None, workspace=None, stream=None):
    """y[M,N] = x[M,K] . dequant_q4_0(w)^T. w: uint8 Q4_0 bytes of N rows."""
    M, K = x.shape
    N = N if N is not None else w.numel() // (K // 32 * 18)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    st = _stream(stream)
    ws, wsb = _workspace(QG_OP_Q4_0, M, N, K, 0, 0, x.device, workspace, st)
    _check(lib().qgemv_q4_0(_dev(w, "w", torch.uint8), _dev(x, "x", torch.float32),
                            _dev(y, "y", torch.float32), M, N, K, ws, wsb, st),
           "qgemv_q4_0")
    return y


def qgemv_dual_q4_0(w_a, w_b, x, y_a=None, y_b=None, *, N=None, workspace=None, stream=None):
    """(y_a, y_b) = (x . dequant(w_a)^T, x . dequant(w_b)^T) in one launch."""
    M, K = x.shape
    N = N if N is not None else w_a.numel() // (K // 32 * 18)
    if y_a is None:
        y_a = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if y_b is None:
        y_b = torch.empty((M, N), dtype=torch.float32, device=x.device)
    st = _stream(stream)
    ws, wsb = _workspace(QG_OP_DUAL_Q4_0, M, N, K, 0, 0, x.device, workspace, st)
    _check(lib().qgemv_dual_q4_0(_dev(w_a, "w_a", torch.uint8), _dev(w_b, "w_b", torch.uint8),
                                 _dev(x, "x", torch.float32), _dev(y_a, "y_a", torch.float32),
                                 _dev(y_b, "y_b", torch.float32), M, N, K, ws, wsb,
                                 st), "qgemv_dual_q4_0")
    return y_a, y_b


def qgemv_dual_q4_0_host(w_a, w_b, x, y_a=None, y_b=None, *, N=None, workspace=None,
                         stream=None):
    """qgemv_dual_q4_0 with x, y_a, y_b in host memory (CPU tensors); returns
    once y_a and y_b hold the result. Page-locked buffers (pin_memory()) are
    read and written in place for M <= 2; other buffers pass through device
    staging. New outputs are page-locked when x is."""
    M, K = x.shape
    N = N if N is not None else w_a.numel() // (K // 32 * 18)
    pin = x.is_pinned()
    if y_a is None:
        y_a = torch.empty((M, N), dtype=torch.float32, pin_memory=pin)
    if y_b is None:
        y_b = torch.empty((M, N), dtype=torch.float32, pin_memory=pin)
    st = _stream(stream)
    ws, wsb = _workspace(QG_OP_DUAL_Q4_0_HOST, M, N, K, 0, 0, w_a.device, workspace, st)
    _check(lib().qgemv_dual_q4_0_host(_dev(w_a, "w_a", torch.uint8), _dev(w_b, "w_b", torch.uint8),
                                      _host(x, "x", torch.float32), _host(y_a, "y_a", torch.float32),
                                      _host(y_b, "y_b", torch.float32), M, N, K, ws, wsb, st),
           "qgemv_dual_q4_0_host")
    return y_a, y_b


def qgemv_q4_k(w, x, y=None, *, N=None, workspace=None, stream=None):
    """y[M,N] = x[M,K] . dequant_q4_k(w)^T. w: uint8 Q4_K bytes of N rows."""
    M, K = x.shape
    N = N if N is not None else w.numel() // (K // 256 * 144)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    st = _stream(stream)
    ws, wsb = _workspace(QG_OP_Q4_K, M, N, K, 0, 0, x.device, workspace, st)
    _check(lib().qgemv_q4_k(_dev(w, "w", torch.uint8), _dev(x, "x", torch.float32),
                            _dev(y, "y", torch.float32), M, N, K, ws, wsb, st),
           "qgemv_q4_k")
    return y


def qgemv_q4_k_noalloc(w, x, y=None, *, N=None, stream=None):
    """qgemv_q4_k without a caller workspace: split-K scratch lives in a fixed
    4 MiB device array inside the library (see include/qgemv.h)."""
    M, K = x.shape
    N = N if N is not None else w.numel() // (K // 256 * 144)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(lib().qgemv_q4_k_noalloc(_dev(w, "w", torch.uint8), _dev(x, "x", torch.float32),
                                    _dev(y, "y", torch.float32), M, N, K, _stream(stream)),
           "qgemv_q4_k_noalloc")
    return y


def qmm_affine(x, q, scales, biases, group_size, packed, y=None, *, workspace=None, stream=None):
    """y = x . dequant_affine(q, scales, biases)^T; q uint8 codes ([N,K] or [N,K/2])."""
    M, K = x.shape
    N = scales.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    st = _stream(stream)
    ws, wsb = _workspace(QG_OP_AFFINE, M, N, K, group_size, int(packed), x.device, workspace, st)
    _check(lib().qmm_affine(_dev(x, "x", torch.float32), _dev(q, "q", torch.uint8),
                            _dev(scales, "scales", torch.float32),
                            _dev(biases, "biases", torch.float32), _dev(y, "y", torch.float32),
                            M, N, K, int(group_size), int(packed), ws, wsb, st),
           "qmm_affine")
    return y


def prepare_af4_g64(codes, scales, biases, *, stream=None):
    """(plane, metadata) of the prepared AF4-g64 layout (int32 tensors holding
    the u32 words): codes uint8 [N, K] (0..15), scales and biases bfloat16
    [N, K/64]."""
    N, K = codes.shape
    plane = torch.empty(N * K // 8, dtype=torch.int32, device=codes.device)
    meta = torch.empty(N * K // 64, dtype=torch.int32, device=codes.device)
    _check(lib().qg_prepare_af4_g64(_dev(codes, "codes", torch.uint8),
                                    _dev(scales, "scales", torch.bfloat16),
                                    _dev(biases, "biases", torch.bfloat16), plane.data_ptr(),
                                    meta.data_ptr(), N, K, _stream(stream)), "qg_prepare_af4_g64")
    return plane, meta


def qmm_af4_g64(x, plane, metadata, N, y=None, *, workspace=None, stream=None):
    """y[M,N] = x[M,K] . w^T from the prepared AF4-g64 layout (M <= 32; no workspace)."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    st = _stream(stream)
    ws, wsb = _workspace(QG_OP_AF4_G64, M, N, K, 0, 0, x.device, workspace, st)
    _check(lib().qmm_af4_g64(_dev(x, "x", torch.float32), _dev(plane, "plane", torch.int32),
                             _dev(metadata, "metadata", torch.int32), _dev(y, "y", torch.float32),
                             M, N, K, ws, wsb, st), "qmm_af4_g64")
    return y


def qkv_split(qkv, q_sp, k_sp, v_sp, q=None, k=None, v=None, *, stream=None):
    """Split [seq, q_sp+k_sp+v_sp] f32 into q [seq,q_sp], k [seq,k_sp], v [seq,v_sp]."""
    seq = qkv.shape[0]
    dev = qkv.device
    q = torch.empty((seq, q_sp), dtype=torch.float32, device=dev) if q is None else q
    k = torch.empty((seq, k_sp), dtype=torch.float32, device=dev) if k is None else k
    v = torch.empty((seq, v_sp), dtype=torch.float32, device=dev) if v is None else v
    _check(lib().qkv_split(_dev(qkv, "qkv", torch.float32), _dev(q, "q", torch.float32),
                           _dev(k, "k", torch.float32), _dev(v, "v", torch.float32), seq, q_sp,
                           k_sp, v_sp, _stream(stream)), "qkv_split")
    return q, k, v


def dequant_q4_0(w, N, K, out=None, *, stream=None):
    out = torch.empty((N, K), dtype=torch.float32, device=w.device) if out is None else out
    _check(lib().dequant_q4_0(_dev(w, "w", torch.uint8), _dev(out, "out", torch.float32), N, K,
                              _stream(stream)), "dequant_q4_0")
    return out


def dequant_q4_k(w, N, K, out=None, *, stream=None):
    out = torch.empty((N, K), dtype=torch.float32, device=w.device) if out is None else out
    _check(lib().dequant_q4_k(_dev(w, "w", torch.uint8), _dev(out, "out", torch.float32), N, K,
                              _stream(stream)), "dequant_q4_k")
    return out


def dequant_affine(q, scales, biases, N, K, group_size, packed, out=None, *, stream=None):
    out = torch.empty((N, K), dtype=torch.float32, device=q.device) if out is None else out
    _check(lib().dequant_affine(_dev(q, "q", torch.uint8), _dev(scales, "scales", torch.float32),
                                _dev(biases, "biases", torch.float32),
                                _dev(out, "out", torch.float32), N, K, int(group_size),
                                int(packed), _stream(stream)), "dequant_affine")
    return out


# ------------------------------------------------------- serving operators
# Through the module _serving (csrc/serving.cpp), which does for these calls what
# the functions above do, in less time: tensors are checked (ValueError), new
# outputs allocated, and a status that is not QG_OK raises QGError.
_SERVING = None


def _calls():
    global _SERVING
    if _SERVING is None:
        lib()
        if not os.path.exists(os.path.join(_HERE, "_serving.so")):
            raise RuntimeError("_serving.so is missing: build it with __graft_entry__.build()")
        module = importlib.import_module(__name__ + "._serving")
        module.set_error(QGError)
        _SERVING = module
    return _SERVING


def quantize_fp8_b128(x, codes=None, scales=None, *, stream=None):
    """(codes, scales) of x [M, K] (float32, float16 or bfloat16; its rows may
    lie apart): e4m3 codes [M, K] and one float32 scale per 128 values of a
    row, [M, ceil(K / 128)]."""
    return (_SERVING or _calls()).quantize_fp8_b128(x, codes, scales, stream)


def qmm_fp8_b128(a, a_scales, w, w_scales, y=None, *, out_dtype=torch.float32, workspace=None,
                 stream=None):
    """y[M, N] = (a * a_scales) . (w * w_scales)^T: e4m3 codes a [M, K] with a
    scale per row and 128 values of K, w [N, K] with one per 128 x 128 values;
    y is float32 or bfloat16."""
    return (_SERVING or _calls()).qmm_fp8_b128(a, a_scales, w, w_scales, y, out_dtype, workspace, stream)


def qmm_fp8_b128_grouped(a, a_scales, w, w_scales, offsets, y=None, *, out_dtype=torch.float32, workspace=None,
                         stream=None):
    """qmm_fp8_b128 for a layer of experts: rows offsets[e] .. offsets[e + 1] - 1
    of a [M, K] times w[e] of w [experts, N, K] (scales [experts, ceil(N / 128),
    ceil(K / 128)]); offsets int32 [experts + 1]. Rows of y [M, N] that no expert
    has are left as they are. With K % 16 != 0, or a weight that does not begin on 16
    bytes, the scratch that stays with the stream is as large as all weights: lay them
    out with rows of a multiple of 16 bytes, or pass a workspace."""
    return (_SERVING or _calls()).qmm_fp8_b128_grouped(a, a_scales, w, w_scales, offsets, y, out_dtype, workspace,
                                                       stream)


def rms_norm(x, weight=None, residual=None, out=None, residual_out=None, *, eps=1e-6, weight_offset=0.0,
             out_dtype=None, stream=None):
    """h / sqrt(mean(h^2) + eps) * (weight_offset + weight) of the rows h = x (+
    residual) of x [M, K] (its and the residual's rows may lie apart), in
    out_dtype (default: x's); weight [K], or None for a factor of 1. With a
    residual (of x's type or float32): (out, residual_out), the latter h in the
    residual's type, which may be the residual itself."""
    return (_SERVING or _calls()).rms_norm(x, weight, residual, out, residual_out, eps, weight_offset, out_dtype, stream)


def rms_norm_fp8_b128(x, weight=None, residual=None, codes=None, scales=None, residual_out=None, *, eps=1e-6,
                      weight_offset=0.0, stream=None):
    """rms_norm with its output as quantize_fp8_b128 gives it: (codes, scales), or
    (codes, scales, residual_out) with a residual."""
    return (_SERVING or _calls()).rms_norm_fp8_b128(x, weight, residual, codes, scales, residual_out, eps, weight_offset,
                                                    stream)


def silu_mul(gate, up, out=None, *, out_dtype=None, stream=None):
    """up * gate / (1 + exp(-gate)) of gate, up [M, K] of one type (rows may lie
    apart, as halves of one product's rows), in out_dtype (default: theirs)."""
    return (_SERVING or _calls()).silu_mul(gate, up, out, out_dtype, stream)


def silu_mul_fp8_b128(gate, up, codes=None, scales=None, *, stream=None):
    """silu_mul with its output as quantize_fp8_b128 gives it: (codes, scales)."""
    return (_SERVING or _calls()).silu_mul_fp8_b128(gate, up, codes, scales, stream)


def attn_paged(q, k_cache, v_cache, page_table, q_offsets, context_lens, out=None, lse=None, *,
               max_new=None, scale=None, softcap=0.0, window=0, return_lse=False, workspace=None,
               stream=None):
    """Attention of new tokens over a paged cache that holds their keys and
    values already; out [tokens, q_heads, head_dim], and with return_lse (or a
    tensor lse) also the log of each row's sum, float32 [tokens, q_heads].

    q [tokens, q_heads, head_dim] float16 or bfloat16 (rows may lie apart);
    k_cache, v_cache [num_pages, kv_heads, page_size, head_dim]; page_table
    int32 [batch, width]; q_offsets int32 [batch + 1]: sequence b's new tokens
    are rows q_offsets[b] .. q_offsets[b + 1] - 1; context_lens int32 [batch]:
    its keys, the new ones included. max_new: the most new tokens that any
    sequence has (default: all of q's rows); the kernel is chosen by it, so say
    1 for a batch of single tokens (a quarter faster than the default for 128).
    scale: default head_dim ** -0.5. softcap > 0 caps the scores, window > 0
    limits how far back a row sees. Rows at or after q_offsets[batch] are left as
    they are."""
    return (_SERVING or _calls()).attn_paged(q, k_cache, v_cache, page_table, q_offsets, context_lens, out, lse,
                                                max_new, scale, softcap, window, return_lse, workspace, stream)


def kv_append(k, v, k_cache, v_cache, slots, *, stream=None):
    """Rows of k and v [tokens, kv_heads, head_dim] (rows may lie apart, as
    parts of one fused projection) into a layer's k_cache and v_cache
    [num_pages, kv_heads, page_size, head_dim], rounded to their type. slots
    int64 [tokens]: page * page_size + place of each row; negative: skipped."""
    return (_SERVING or _calls()).kv_append(k, v, k_cache, v_cache, slots, stream)


def kv_append_rope(q, k, v, positions, inv_freq, k_cache, v_cache, slots, q_out=None, *, interleaved=False,
                   stream=None):
    """kv_append with keys, and queries, rotated on the way: pair i of row t of q
    [tokens, q_heads, head_dim] (or None) and k by the angle positions[t] (int64)
    * inv_freq[i] (float32). The pairs are the first 2 * len(inv_freq) values of a
    head: i and i + len(inv_freq), or with interleaved 2 i and 2 i + 1. Returns
    the rotated q, dense, in the cache's type (None without q)."""
    return (_SERVING or _calls()).kv_append_rope(q, k, v, positions, inv_freq, k_cache, v_cache, slots, q_out, interleaved,
                                                 stream)


def kv_copy_pages(cache, src, dst, *, stream=None):
    """In every plane of cache [planes, num_pages, ...]: page dst[i] = page
    src[i] (int32). Pairs with a negative member are skipped."""
    return (_SERVING or _calls()).kv_copy_pages(cache, src, dst, stream)


def kv_fork(cache, page_table, lens, ref_counts, parents, page_size, *, workspace=None, stream=None):
    """Continuations of sequences: child c shares the whole pages of row
    parents[c] of page_table and gets a copy of its partly filled last page, in
    the lowest free pages. Returns (child_table [children, width], child_lens,
    new ref_counts); cache [planes, num_pages, ...] is changed in place."""
    return (_SERVING or _calls()).kv_fork(cache, page_table, lens, ref_counts, parents, page_size, workspace,
                                             stream)


def kv_free(page_table, lens, ref_counts, drop, *, stream=None):
    """New (page_table, lens, ref_counts) without the rows where drop (uint8
    [rows]) is not 0: their entries are -1, their length 0, and each page that
    they held counts one holder less."""
    return (_SERVING or _calls()).kv_free(page_table, lens, ref_counts, drop, stream)


def kv_compact(cache, page_table, ref_counts, *, workspace=None, stream=None):
    """Moves the pages of cache [planes, num_pages, ...] so that those in use
    are 0 .. live - 1. Returns (page_table, ref_counts, page_map, live) in the
    new numbers; page_map[p] is page p's new number, -1 if it was free."""
    return (_SERVING or _calls()).kv_compact(cache, page_table, ref_counts, workspace, stream)


def token_logprobs(logits, targets, top_k=0, *, stream=None):
    """(logprobs, entropy, ranks, top_values, top_ids) of rows of logits [M, V]
    (rows may lie apart): the log probability of each row's target (int64;
    negative: none, 0 and rank -1), the row's entropy, how many logits are
    greater than the target's, and the min(top_k, V) largest alternatives as log
    probabilities and ids, ties to the lower id."""
    return (_SERVING or _calls()).token_logprobs(logits, targets, top_k, stream)


def device_error(clear: bool = True) -> int:
    """Synchronize and return (optionally clearing) the device error word."""
    code = C.c_uint(0)
    rc = lib().qg_device_error(int(clear), C.byref(code))
    if rc not in (QG_OK, QG_ERR_DEVICE):
        raise QGError("qg_device_error", rc)
    return int(code.value)


def selftest_wait_timeout(timeout_ns: int, *, stream=None):
    _check(lib().qg_selftest_wait_timeout(int(timeout_ns), _stream(stream)),
           "qg_selftest_wait_timeout")


def set_option(option: int, value: int):
    """qg_set_option: e.g. set_option(QG_OPT_PDL, 1) (see include/qgemv.h)."""
    _check(lib().qg_set_option(int(option), int(value)), "qg_set_option")


def get_option(option: int) -> int:
    v = C.c_int64(0)
    _check(lib().qg_get_option(int(option), C.byref(v)), "qg_get_option")
    return int(v.value)
