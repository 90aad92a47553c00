"""Python binding of libqffn (FP8 SwiGLU FFN block for one GB300).

Argument marshalling only: each function here has the name of a C entry
point of ``include/qffn.h``, turns torch tensors (or raw integer device
addresses) into pointers, passes the current torch CUDA stream unless one is
given, and raises ``QffnError`` on a non-zero status.  The norm, linear and
gated-linear functions also refuse tensors that are too small, of another
type, not contiguous or not on the current device.  Every step of the
block runs in the CUDA kernels of ``libqffn.so``; there is no fallback.  If
the library is missing the import fails (run ``build()`` first).
"""
from __future__ import annotations

import ctypes
import os
import sys
import threading

from ._build import LIB as LIB_PATH
from ._build import build

__all__ = [
    "QffnError", "lib", "build", "LIB_PATH", "STATUS",
    "qffn_status_string", "qffn_abi_version", "qffn_check_status", "qffn_selftest_bounded_wait",
    "qffn_gemm_clock_sample",
    "qffn_rmsnorm_absmax", "qffn_absmax", "qffn_quantize", "qffn_quantize_rows",
    "qffn_fp8_gemm_scaled", "qffn_qmm", "qffn_gate_up_swiglu", "qffn_swiglu_quant",
    "qffn_swiglu_forward_quant", "qffn_gate_up_swiglu_quant",
    "qffn_forward_workspace_size", "qffn_forward_workspace_offsets", "qffn_forward",
    "qffn_forward_recompute", "qffn_transpose_e4m3", "qffn_swiglu_backward",
    "qffn_backward_qmm_workspace_size", "qffn_backward_qmm", "qffn_ffn_backward_workspace_size",
    "qffn_ffn_backward_workspace_offsets", "qffn_ffn_backward", "qffn_gate_up_swiglu_backward",
    "qffn_layernorm_absmax", "qffn_norm_backward_workspace_size", "qffn_layernorm_backward",
    "qffn_rmsnorm_backward", "qffn_linear_workspace_size", "qffn_linear", "qffn_linear_fp8_workspace_size",
    "qffn_linear_fp8", "qffn_linear_backward_workspace_size", "qffn_linear_backward",
    "qffn_gated_linear_workspace_size", "qffn_gated_linear", "qffn_gated_linear_backward_workspace_size",
    "qffn_gated_linear_backward", "QFFN_ACT_NONE", "QFFN_ACT_RELU", "QFFN_ACT_GELU", "QFFN_ACT_GELU_TANH",
    "QFFN_ACT_SILU",
    "qffn_quantize_blocks", "qffn_quantize_weight_blocks", "qffn_rmsnorm_quantize_blocks",
    "qffn_swiglu_quantize_blocks", "qffn_linear_fp8_blocks", "qffn_grouped_linear", "qffn_grouped_linear_backward",
    "qffn_grouped_linear_fp8_blocks",
    "qffn_gemv_dual", "qffn_gemv", "qffn_gemv_silu_input", "qffn_silu_mul", "qffn_decode_workspace_size",
    "qffn_decode_workspace_offsets", "qffn_decode_forward", "qffn_decode_forward_ex", "qffn_decode_forward_gu",
    "qffn_decode_forward_noalloc", "QFFN_DECODE_WEIGHTS_STABLE",
]

QFFN_DECODE_WEIGHTS_STABLE = 1
QFFN_ACT_NONE, QFFN_ACT_RELU, QFFN_ACT_GELU, QFFN_ACT_GELU_TANH, QFFN_ACT_SILU = range(5)

STATUS = {0: "QFFN_OK", 1: "QFFN_ERR_INVALID_ARG", 2: "QFFN_ERR_UNSUPPORTED_SHAPE",
          3: "QFFN_ERR_MISALIGNED", 4: "QFFN_ERR_CUDA", 5: "QFFN_ERR_TIMEOUT"}

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run transformer_ffn_block_gb300._build.build() "
        "(or __graft_entry__.build()) first")

lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_S = ctypes.c_int

_SIGS = {
    "qffn_status_string": ([_S], ctypes.c_char_p),
    "qffn_abi_version": ([], ctypes.c_int),
    "qffn_check_status": ([_P], _S),
    "qffn_selftest_bounded_wait": ([_P, _S, _I64, _P], _S),
    "qffn_gemm_clock_sample": ([_P, _P], _S),
    "qffn_rmsnorm_absmax": ([_P, _P, _P, _P, _P, _P, _P, _F, _I64, _I64, _P], _S),
    "qffn_absmax": ([_P, _P, _I64, _P], _S),
    "qffn_quantize": ([_P, _P, _P, _I64, _P], _S),
    "qffn_quantize_rows": ([_P, _P, _P, _I64, _I64, _P], _S),
    "qffn_fp8_gemm_scaled": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P], _S),
    "qffn_qmm": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], _S),
    "qffn_gate_up_swiglu": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], _S),
    "qffn_swiglu_quant": ([_P, _P, _P, _P, _I64, _I64, _P], _S),
    "qffn_swiglu_forward_quant": ([_P, _P, _P, _I64, _I64, _P], _S),
    "qffn_gate_up_swiglu_quant": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], _S),
    "qffn_forward_workspace_size": ([_I64, _I64, _I64, _I64], _SZ),
    "qffn_forward_workspace_offsets": ([_I64, _I64, _I64, _I64, ctypes.POINTER(_SZ)], _S),
    "qffn_forward": ([_P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P,
                      _I64, _I64, _I64, _I64, _P, _SZ, _P], _S),
    "qffn_forward_recompute": ([_P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P,
                                _I64, _I64, _I64, _I64, _P, _SZ, _P], _S),
    "qffn_transpose_e4m3": ([_P, _P, _I64, _I64, _P], _S),
    "qffn_swiglu_backward": ([_P, _P, _P, _P, _I64, _I64, _P], _S),
    "qffn_backward_qmm_workspace_size": ([_I64, _I64, _I64], _SZ),
    "qffn_backward_qmm": ([_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _S, _P, _SZ, _P], _S),
    "qffn_ffn_backward_workspace_size": ([_I64, _I64, _I64], _SZ),
    "qffn_gate_up_swiglu_backward": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], _S),
    "qffn_ffn_backward_workspace_offsets": ([_I64, _I64, _I64, ctypes.POINTER(_SZ)], _S),
    "qffn_ffn_backward": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                           _I64, _I64, _I64, _S, _P, _SZ, _P], _S),
    "qffn_layernorm_absmax": ([_P] * 9 + [_F, _I64, _I64, _P], _S),
    "qffn_norm_backward_workspace_size": ([_I64, _I64], _SZ),
    "qffn_layernorm_backward": ([_P] * 10 + [_I64, _I64, _S, _P, _SZ, _P], _S),
    "qffn_rmsnorm_backward": ([_P] * 8 + [_I64, _I64, _S, _P, _SZ, _P], _S),
    "qffn_linear_workspace_size": ([_I64] * 3, _SZ),
    "qffn_linear": ([_P] * 6 + [_S, _I64, _I64, _I64, _P, _SZ, _P], _S),
    "qffn_linear_fp8_workspace_size": ([_I64] * 3, _SZ),
    "qffn_linear_fp8": ([_P] * 8 + [_S, _I64, _I64, _I64, _P, _SZ, _P], _S),
    "qffn_linear_backward_workspace_size": ([_I64] * 3, _SZ),
    "qffn_linear_backward": ([_P] * 7 + [_S, _I64, _I64, _I64, _S, _P, _SZ, _P], _S),
    "qffn_gated_linear_workspace_size": ([_I64] * 3, _SZ),
    "qffn_gated_linear": ([_P] * 3 + [_S, _I64, _I64, _I64, _P, _SZ, _P], _S),
    "qffn_gated_linear_backward_workspace_size": ([_I64] * 3, _SZ),
    "qffn_gated_linear_backward": ([_P] * 5 + [_S, _I64, _I64, _I64, _S, _P, _SZ, _P], _S),
    "qffn_quantize_blocks": ([_P] * 3 + [_I64] * 2 + [_P], _S),
    "qffn_quantize_weight_blocks": ([_P] * 3 + [_I64] * 3 + [_P], _S),
    "qffn_rmsnorm_quantize_blocks": ([_P] * 8 + [_F, _I64, _I64, _P], _S),
    "qffn_swiglu_quantize_blocks": ([_P] * 4 + [_I64] * 2 + [_P], _S),
    "qffn_linear_fp8_blocks": ([_P] * 7 + [_I64] * 3 + [_P], _S),
    "qffn_grouped_linear": ([_P] * 4 + [_I64] * 4 + [_P], _S),
    "qffn_grouped_linear_backward": ([_P] * 6 + [_I64] * 4 + [_S, _P], _S),
    "qffn_grouped_linear_fp8_blocks": ([_P] * 6 + [_I64] * 4 + [_P], _S),
    "qffn_gemv_dual": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P], _S),
    "qffn_gemv": ([_P, _P, _P, _P, _I64, _I64, _P], _S),
    "qffn_gemv_silu_input": ([_P, _P, _P, _P, _P, _I64, _I64, _P], _S),
    "qffn_silu_mul": ([_P, _P, _I64, _P], _S),
    "qffn_decode_workspace_size": ([_I64, _I64], _SZ),
    "qffn_decode_workspace_offsets": ([_I64, _I64, _P], _S),
    "qffn_decode_forward": ([_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _SZ, _P], _S),
    "qffn_decode_forward_ex": ([_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _SZ, ctypes.c_uint, _P], _S),
    "qffn_decode_forward_gu": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _P, _SZ, _P], _S),
    "qffn_decode_forward_noalloc": ([_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P], _S),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class QffnError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({detail or qffn_status_string(status)})")


def _ptr(t):
    """torch tensor -> device address; int -> itself; None -> NULL."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the tensor types that hold each (filled with torch)
_BF16, _F32, _E4M3, _E8M0, _I32 = set(), set(), set(), set(), set()
_KINDS = ((_BF16, "bf16"), (_F32, "fp32"), (_E4M3, "E4M3"), (_E8M0, "E8M0"), (_I32, "int32"))


def _buf(fn, device, name, t, types, n):
    """_ptr of a tensor after the checks that a bare address cannot have: ``n`` elements at least of one
    of ``types``, contiguous, on the current device.  bf16 may come as int16 or uint16 bits and E4M3
    and E8M0 as uint8 codes, as in the other functions."""
    if t is None:
        return None
    if t.__class__ is int:
        return t
    if t.is_contiguous() and t.dtype in types and t.numel() >= n and (t.get_device() == device or n <= 0):
        return t.data_ptr()
    kind = next(name for held, name in _KINDS if held is types)
    raise QffnError(fn, 1, f"{name}: expected {n} contiguous {kind} elements on cuda:{device}, got "
                           f"{tuple(t.shape)} {t.dtype} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


_torch = None                # imported on first use: calls with bare addresses and a stream do not need it
_get_device = _get_stream = None
_load_lock = threading.Lock()


def _load_torch():
    global _torch, _get_device, _get_stream
    import torch
    with _load_lock:         # first calls from several threads: the others wait
        if _torch is not None:
            return
        _BF16.update((torch.bfloat16, torch.int16, torch.uint16))
        _F32.add(torch.float32)
        _E4M3.update((torch.float8_e4m3fn, torch.uint8))
        _E8M0.update((getattr(torch, "float8_e8m0fnu", torch.uint8), torch.uint8))   # (not in every torch)
        _I32.add(torch.int32)
        if torch.cuda.is_available():
            torch.cuda.init()
            _get_stream, _get_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        _torch = torch       # last: with it set, the two above are what they stay


def _current_device():
    if _get_device is not None:
        return _get_device()
    if _torch is None:
        if "torch" not in sys.modules:       # then no argument is a tensor
            return -2
        _load_torch()
    return _get_device() if _get_device is not None else -2      # (-1 is a CPU tensor's)


def _workspace(fn, device, workspace, workspace_bytes):
    if workspace_bytes is not None and workspace_bytes < 0:      # (as a size_t it would be enough for anything)
        raise QffnError(fn, 1, f"workspace_bytes: {workspace_bytes}")
    if workspace is None or workspace.__class__ is int:
        return workspace, int(workspace_bytes or 0)
    nbytes = workspace.numel() * workspace.element_size()
    if not (workspace.is_contiguous() and nbytes > 0 and workspace.get_device() == device):
        raise QffnError(fn, 1, f"workspace: expected contiguous memory on cuda:{device}, got "
                               f"{tuple(workspace.shape)} {workspace.dtype} on {workspace.device}")
    if workspace_bytes is not None:
        nbytes = min(nbytes, int(workspace_bytes))
    return workspace.data_ptr(), nbytes


def _stream(stream):
    if stream is None:
        # torch.cuda.current_stream().cuda_stream without the Stream object (2.8 us -> 0.1 us a call)
        if _get_device is None:
            _load_torch()
        return _get_stream(_get_device()) if _get_device is not None else _torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != 0:
        raise QffnError(fn, status)


def qffn_status_string(status: int) -> str:
    return lib.qffn_status_string(status).decode()


def qffn_abi_version() -> int:
    return lib.qffn_abi_version()


def qffn_check_status(stream=None):
    _check("qffn_check_status", lib.qffn_check_status(_stream(stream)))


def qffn_selftest_bounded_wait(out, arrive, limit_ns, stream=None):
    _check("qffn_selftest_bounded_wait", lib.qffn_selftest_bounded_wait(
        _ptr(out), int(bool(arrive)), int(limit_ns), _stream(stream)))


def qffn_gemm_clock_sample(stream=None):
    """(SM clock cycles, nanoseconds) of the first CTA of the most recent FP8 GEMM launch."""
    out = (ctypes.c_uint64 * 2)()
    _check("qffn_gemm_clock_sample", lib.qffn_gemm_clock_sample(
        ctypes.cast(out, ctypes.c_void_p), _stream(stream)))
    return int(out[0]), int(out[1])


def qffn_rmsnorm_absmax(res_out, y, rstd, stats, res_in, x, gain, eps, N, C, stream=None):
    _check("qffn_rmsnorm_absmax", lib.qffn_rmsnorm_absmax(
        _ptr(res_out), _ptr(y), _ptr(rstd), _ptr(stats), _ptr(res_in), _ptr(x), _ptr(gain),
        float(eps), int(N), int(C), _stream(stream)))


def qffn_absmax(stats, inp, n, stream=None):
    _check("qffn_absmax", lib.qffn_absmax(_ptr(stats), _ptr(inp), int(n), _stream(stream)))


def qffn_quantize(q, stats, inp, n, stream=None):
    _check("qffn_quantize", lib.qffn_quantize(_ptr(q), _ptr(stats), _ptr(inp), int(n), _stream(stream)))


def qffn_quantize_rows(q, row_scale, w, rows, cols, stream=None):
    _check("qffn_quantize_rows", lib.qffn_quantize_rows(
        _ptr(q), _ptr(row_scale), _ptr(w), int(rows), int(cols), _stream(stream)))


def qffn_fp8_gemm_scaled(out, a, a_scale, w, w_scale, M, N, K, stream=None):
    _check("qffn_fp8_gemm_scaled", lib.qffn_fp8_gemm_scaled(
        _ptr(out), _ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale), int(M), int(N), int(K),
        _stream(stream)))


def qffn_qmm(out, q, stats, inp, bias, w, w_scale, M, N, K, stream=None):
    _check("qffn_qmm", lib.qffn_qmm(
        _ptr(out), _ptr(q), _ptr(stats), _ptr(inp), _ptr(bias), _ptr(w), _ptr(w_scale),
        int(M), int(N), int(K), _stream(stream)))


def qffn_gate_up_swiglu(h, stats_h, yq, y_scale, w1, w1_scale, N, C, H, stream=None):
    _check("qffn_gate_up_swiglu", lib.qffn_gate_up_swiglu(
        _ptr(h), _ptr(stats_h), _ptr(yq), _ptr(y_scale), _ptr(w1), _ptr(w1_scale),
        int(N), int(C), int(H), _stream(stream)))


def qffn_swiglu_quant(h, hq, stats, gate_up, N, H, stream=None):
    _check("qffn_swiglu_quant", lib.qffn_swiglu_quant(
        _ptr(h), _ptr(hq), _ptr(stats), _ptr(gate_up), int(N), int(H), _stream(stream)))


def qffn_swiglu_forward_quant(hq, stats, gate_up, N, H, stream=None):
    _check("qffn_swiglu_forward_quant", lib.qffn_swiglu_forward_quant(
        _ptr(hq), _ptr(stats), _ptr(gate_up), int(N), int(H), _stream(stream)))


def qffn_gate_up_swiglu_quant(hq, stats_h, yq, y_scale, w1, w1_scale, N, C, H, stream=None):
    _check("qffn_gate_up_swiglu_quant", lib.qffn_gate_up_swiglu_quant(
        _ptr(hq), _ptr(stats_h), _ptr(yq), _ptr(y_scale), _ptr(w1), _ptr(w1_scale),
        int(N), int(C), int(H), _stream(stream)))


def qffn_forward_workspace_size(B, T, C, H) -> int:
    return int(lib.qffn_forward_workspace_size(int(B), int(T), int(C), int(H)))


def qffn_forward_workspace_offsets(B, T, C, H) -> list[int]:
    off = (_SZ * 4)()
    _check("qffn_forward_workspace_offsets",
           lib.qffn_forward_workspace_offsets(int(B), int(T), int(C), int(H), off))
    return [int(v) for v in off]


def qffn_forward(res_out, out, rstd, stats_y, stats_h, res_in, x, gain, eps, w1, w1_scale,
                 w2, w2_scale, B, T, C, H, workspace, workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("qffn_forward", lib.qffn_forward(
        _ptr(res_out), _ptr(out), _ptr(rstd), _ptr(stats_y), _ptr(stats_h), _ptr(res_in),
        _ptr(x), _ptr(gain), float(eps), _ptr(w1), _ptr(w1_scale), _ptr(w2), _ptr(w2_scale),
        int(B), int(T), int(C), int(H), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def qffn_forward_recompute(res_out, out, rstd, stats_y, stats_h, res_in, x, gain, eps, w1,
                           w1_scale, w2, w2_scale, B, T, C, H, workspace, workspace_bytes=None,
                           stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("qffn_forward_recompute", lib.qffn_forward_recompute(
        _ptr(res_out), _ptr(out), _ptr(rstd), _ptr(stats_y), _ptr(stats_h), _ptr(res_in),
        _ptr(x), _ptr(gain), float(eps), _ptr(w1), _ptr(w1_scale), _ptr(w2), _ptr(w2_scale),
        int(B), int(T), int(C), int(H), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def qffn_transpose_e4m3(out, inp, rows, cols, stream=None):
    _check("qffn_transpose_e4m3", lib.qffn_transpose_e4m3(
        _ptr(out), _ptr(inp), int(rows), int(cols), _stream(stream)))


def qffn_swiglu_backward(d_gate_up, stats, dh, gate_up, N, H, stream=None):
    _check("qffn_swiglu_backward", lib.qffn_swiglu_backward(
        _ptr(d_gate_up), _ptr(stats), _ptr(dh), _ptr(gate_up), int(N), int(H), _stream(stream)))


def qffn_backward_qmm_workspace_size(N, IC, OC) -> int:
    return int(lib.qffn_backward_qmm_workspace_size(int(N), int(IC), int(OC)))


def qffn_backward_qmm(dinp, dw, stats_dout, dout, inp_q, inp_scale, w, w_scale, N, IC, OC,
                      accumulate, workspace, workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("qffn_backward_qmm", lib.qffn_backward_qmm(
        _ptr(dinp), _ptr(dw), _ptr(stats_dout), _ptr(dout), _ptr(inp_q), _ptr(inp_scale), _ptr(w),
        _ptr(w_scale), int(N), int(IC), int(OC), int(bool(accumulate)), _ptr(workspace),
        int(workspace_bytes), _stream(stream)))


def qffn_ffn_backward_workspace_size(N, C, H) -> int:
    return int(lib.qffn_ffn_backward_workspace_size(int(N), int(C), int(H)))


def qffn_gate_up_swiglu_backward(d_gate_up, stats, dh, yq, y_scale, w1, w1_scale, N, C, H,
                                 stream=None):
    _check("qffn_gate_up_swiglu_backward", lib.qffn_gate_up_swiglu_backward(
        _ptr(d_gate_up), _ptr(stats), _ptr(dh), _ptr(yq), _ptr(y_scale), _ptr(w1), _ptr(w1_scale),
        int(N), int(C), int(H), _stream(stream)))


def qffn_ffn_backward_workspace_offsets(N, C, H) -> list[int]:
    off = (_SZ * 2)()
    _check("qffn_ffn_backward_workspace_offsets",
           lib.qffn_ffn_backward_workspace_offsets(int(N), int(C), int(H), off))
    return [int(v) for v in off]


def qffn_ffn_backward(d_ln2, dw1, dw2, stats_dout, stats_dgu, dout, yq, y_scale, hq, h_scale, w1,
                      w1_scale, w2, w2_scale, N, C, H, accumulate, workspace, workspace_bytes=None,
                      stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("qffn_ffn_backward", lib.qffn_ffn_backward(
        _ptr(d_ln2), _ptr(dw1), _ptr(dw2), _ptr(stats_dout), _ptr(stats_dgu), _ptr(dout), _ptr(yq),
        _ptr(y_scale), _ptr(hq), _ptr(h_scale), _ptr(w1), _ptr(w1_scale), _ptr(w2), _ptr(w2_scale),
        int(N), int(C), int(H), int(bool(accumulate)), _ptr(workspace), int(workspace_bytes),
        _stream(stream)))


def qffn_layernorm_absmax(res_out, y, mean, rstd, stats, res_in, x, gain, shift, eps, N, C, stream=None):
    fn, d, n = "qffn_layernorm_absmax", _current_device(), N * C
    _check(fn, lib.qffn_layernorm_absmax(
        _buf(fn, d, "res_out", res_out, _BF16, n), _buf(fn, d, "y", y, _BF16, n), _buf(fn, d, "mean", mean, _F32, N),
        _buf(fn, d, "rstd", rstd, _F32, N), _buf(fn, d, "stats", stats, _F32, 1),
        _buf(fn, d, "res_in", res_in, _BF16, n), _buf(fn, d, "x", x, _BF16, n),
        _buf(fn, d, "gain", gain, _BF16, C), _buf(fn, d, "shift", shift, _BF16, C), eps, N, C, _stream(stream)))


def qffn_norm_backward_workspace_size(N, C) -> int:
    return int(lib.qffn_norm_backward_workspace_size(int(N), int(C)))


def qffn_layernorm_backward(dx, dgain, dshift, stats, dy, dres, r, mean, rstd, gain, N, C, accumulate, workspace,
                            workspace_bytes=None, stream=None):
    fn, d, n = "qffn_layernorm_backward", _current_device(), N * C
    ws, nbytes = _workspace(fn, d, workspace, workspace_bytes)
    _check(fn, lib.qffn_layernorm_backward(
        _buf(fn, d, "dx", dx, _BF16, n), _buf(fn, d, "dgain", dgain, _F32, C), _buf(fn, d, "dshift", dshift, _F32, C),
        _buf(fn, d, "stats", stats, _F32, 1), _buf(fn, d, "dy", dy, _BF16, n), _buf(fn, d, "dres", dres, _BF16, n),
        _buf(fn, d, "r", r, _BF16, n), _buf(fn, d, "mean", mean, _F32, N), _buf(fn, d, "rstd", rstd, _F32, N),
        _buf(fn, d, "gain", gain, _BF16, C), N, C, bool(accumulate), ws, nbytes, _stream(stream)))


def qffn_rmsnorm_backward(dx, dgain, stats, dy, dres, r, rstd, gain, N, C, accumulate, workspace,
                          workspace_bytes=None, stream=None):
    fn, d, n = "qffn_rmsnorm_backward", _current_device(), N * C
    ws, nbytes = _workspace(fn, d, workspace, workspace_bytes)
    _check(fn, lib.qffn_rmsnorm_backward(
        _buf(fn, d, "dx", dx, _BF16, n), _buf(fn, d, "dgain", dgain, _F32, C), _buf(fn, d, "stats", stats, _F32, 1),
        _buf(fn, d, "dy", dy, _BF16, n), _buf(fn, d, "dres", dres, _BF16, n), _buf(fn, d, "r", r, _BF16, n),
        _buf(fn, d, "rstd", rstd, _F32, N), _buf(fn, d, "gain", gain, _BF16, C), N, C, bool(accumulate), ws, nbytes,
        _stream(stream)))


def qffn_linear_workspace_size(M, N, K) -> int:
    return int(lib.qffn_linear_workspace_size(int(M), int(N), int(K)))


def qffn_linear(out, z, x, w, bias, residual, act, M, N, K, workspace, workspace_bytes=None, stream=None):
    fn, d = "qffn_linear", _current_device()
    ws, nbytes = _workspace(fn, d, workspace, workspace_bytes)
    _check(fn, lib.qffn_linear(
        _buf(fn, d, "out", out, _BF16, M * N), _buf(fn, d, "z", z, _BF16, M * N), _buf(fn, d, "x", x, _BF16, M * K),
        _buf(fn, d, "w", w, _BF16, N * K), _buf(fn, d, "bias", bias, _BF16, N),
        _buf(fn, d, "residual", residual, _BF16, M * N), act, M, N, K, ws, nbytes, _stream(stream)))


def qffn_linear_fp8_workspace_size(M, N, K) -> int:
    return int(lib.qffn_linear_fp8_workspace_size(int(M), int(N), int(K)))


def qffn_linear_fp8(out, z, x, x_scale, w, w_scale, bias, residual, act, M, N, K, workspace, workspace_bytes=None,
                    stream=None):
    fn, d = "qffn_linear_fp8", _current_device()
    ws, nbytes = _workspace(fn, d, workspace, workspace_bytes)
    _check(fn, lib.qffn_linear_fp8(
        _buf(fn, d, "out", out, _BF16, M * N), _buf(fn, d, "z", z, _BF16, M * N), _buf(fn, d, "x", x, _E4M3, M * K),
        _buf(fn, d, "x_scale", x_scale, _F32, 1), _buf(fn, d, "w", w, _E4M3, N * K),
        _buf(fn, d, "w_scale", w_scale, _F32, 1), _buf(fn, d, "bias", bias, _BF16, N),
        _buf(fn, d, "residual", residual, _BF16, M * N), act, M, N, K, ws, nbytes, _stream(stream)))


def qffn_linear_backward_workspace_size(M, N, K) -> int:
    return int(lib.qffn_linear_backward_workspace_size(int(M), int(N), int(K)))


def qffn_linear_backward(dx, dw, dbias, dout, z, x, w, act, M, N, K, accumulate, workspace, workspace_bytes=None,
                         stream=None):
    fn, d = "qffn_linear_backward", _current_device()
    ws, nbytes = _workspace(fn, d, workspace, workspace_bytes)
    _check(fn, lib.qffn_linear_backward(
        _buf(fn, d, "dx", dx, _BF16, M * K), _buf(fn, d, "dw", dw, _BF16, N * K), _buf(fn, d, "dbias", dbias, _F32, N),
        _buf(fn, d, "dout", dout, _BF16, M * N), _buf(fn, d, "z", z, _BF16, M * N), _buf(fn, d, "x", x, _BF16, M * K),
        _buf(fn, d, "w", w, _BF16, N * K), act, M, N, K, bool(accumulate), ws, nbytes, _stream(stream)))


def qffn_gated_linear_workspace_size(N, C, H) -> int:
    return int(lib.qffn_gated_linear_workspace_size(int(N), int(C), int(H)))


def qffn_gated_linear(h, x, w1, act, N, C, H, workspace, workspace_bytes=None, stream=None):
    fn, d = "qffn_gated_linear", _current_device()
    ws, nbytes = _workspace(fn, d, workspace, workspace_bytes)
    _check(fn, lib.qffn_gated_linear(
        _buf(fn, d, "h", h, _BF16, N * H), _buf(fn, d, "x", x, _BF16, N * C), _buf(fn, d, "w1", w1, _BF16, 2 * H * C),
        act, N, C, H, ws, nbytes, _stream(stream)))


def qffn_gated_linear_backward_workspace_size(N, C, H) -> int:
    return int(lib.qffn_gated_linear_backward_workspace_size(int(N), int(C), int(H)))


def qffn_gated_linear_backward(dx, dw1, dh, x, w1, act, N, C, H, accumulate, workspace, workspace_bytes=None,
                               stream=None):
    fn, d = "qffn_gated_linear_backward", _current_device()
    ws, nbytes = _workspace(fn, d, workspace, workspace_bytes)
    _check(fn, lib.qffn_gated_linear_backward(
        _buf(fn, d, "dx", dx, _BF16, N * C), _buf(fn, d, "dw1", dw1, _BF16, 2 * H * C),
        _buf(fn, d, "dh", dh, _BF16, N * H), _buf(fn, d, "x", x, _BF16, N * C), _buf(fn, d, "w1", w1, _BF16, 2 * H * C),
        act, N, C, H, bool(accumulate), ws, nbytes, _stream(stream)))


def _blocks(n):
    return (n + 127) // 128


def qffn_quantize_blocks(q, scale, inp, rows, cols, stream=None):
    fn, d, n = "qffn_quantize_blocks", _current_device(), rows * cols
    _check(fn, lib.qffn_quantize_blocks(
        _buf(fn, d, "q", q, _E4M3, n), _buf(fn, d, "scale", scale, _E8M0, rows * _blocks(cols)),
        _buf(fn, d, "inp", inp, _BF16, n), rows, cols, _stream(stream)))


def qffn_quantize_weight_blocks(q, scale, w, count, rows, cols, stream=None):
    fn, d, n = "qffn_quantize_weight_blocks", _current_device(), count * rows * cols
    _check(fn, lib.qffn_quantize_weight_blocks(
        _buf(fn, d, "q", q, _E4M3, n), _buf(fn, d, "scale", scale, _E8M0, count * _blocks(rows) * _blocks(cols)),
        _buf(fn, d, "w", w, _BF16, n), count, rows, cols, _stream(stream)))


def qffn_rmsnorm_quantize_blocks(res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C, stream=None):
    fn, d, n = "qffn_rmsnorm_quantize_blocks", _current_device(), N * C
    _check(fn, lib.qffn_rmsnorm_quantize_blocks(
        _buf(fn, d, "res_out", res_out, _BF16, n), _buf(fn, d, "y", y, _BF16, n), _buf(fn, d, "q", q, _E4M3, n),
        _buf(fn, d, "scale", scale, _E8M0, N * _blocks(C)), _buf(fn, d, "rstd", rstd, _F32, N),
        _buf(fn, d, "res_in", res_in, _BF16, n), _buf(fn, d, "x", x, _BF16, n), _buf(fn, d, "gain", gain, _BF16, C),
        eps, N, C, _stream(stream)))


def qffn_swiglu_quantize_blocks(h, q, scale, gate_up, N, H, stream=None):
    fn, d, n = "qffn_swiglu_quantize_blocks", _current_device(), N * H
    _check(fn, lib.qffn_swiglu_quantize_blocks(
        _buf(fn, d, "h", h, _BF16, n), _buf(fn, d, "q", q, _E4M3, n), _buf(fn, d, "scale", scale, _E8M0, N * _blocks(H)),
        _buf(fn, d, "gate_up", gate_up, _BF16, 2 * n), N, H, _stream(stream)))


def qffn_linear_fp8_blocks(out, x, x_scale, w, w_scale, bias, residual, M, N, K, stream=None):
    fn, d = "qffn_linear_fp8_blocks", _current_device()
    _check(fn, lib.qffn_linear_fp8_blocks(
        _buf(fn, d, "out", out, _BF16, M * N), _buf(fn, d, "x", x, _E4M3, M * K),
        _buf(fn, d, "x_scale", x_scale, _E8M0, M * _blocks(K)), _buf(fn, d, "w", w, _E4M3, N * K),
        _buf(fn, d, "w_scale", w_scale, _E8M0, _blocks(N) * _blocks(K)), _buf(fn, d, "bias", bias, _BF16, N),
        _buf(fn, d, "residual", residual, _BF16, M * N), M, N, K, _stream(stream)))


def qffn_grouped_linear(out, x, w, offsets, G, M, N, K, stream=None):
    fn, d = "qffn_grouped_linear", _current_device()
    _check(fn, lib.qffn_grouped_linear(
        _buf(fn, d, "out", out, _BF16, M * N), _buf(fn, d, "x", x, _BF16, M * K), _buf(fn, d, "w", w, _BF16, G * N * K),
        _buf(fn, d, "offsets", offsets, _I32, G + 1), G, M, N, K, _stream(stream)))


def qffn_grouped_linear_backward(dx, dw, dout, x, w, offsets, G, M, N, K, accumulate, stream=None):
    fn, d = "qffn_grouped_linear_backward", _current_device()
    _check(fn, lib.qffn_grouped_linear_backward(
        _buf(fn, d, "dx", dx, _BF16, M * K), _buf(fn, d, "dw", dw, _BF16, G * N * K), _buf(fn, d, "dout", dout, _BF16, M * N),
        _buf(fn, d, "x", x, _BF16, M * K), _buf(fn, d, "w", w, _BF16, G * N * K),
        _buf(fn, d, "offsets", offsets, _I32, G + 1), G, M, N, K, bool(accumulate), _stream(stream)))


def qffn_grouped_linear_fp8_blocks(out, x, x_scale, w, w_scale, offsets, G, M, N, K, stream=None):
    fn, d = "qffn_grouped_linear_fp8_blocks", _current_device()
    _check(fn, lib.qffn_grouped_linear_fp8_blocks(
        _buf(fn, d, "out", out, _BF16, M * N), _buf(fn, d, "x", x, _E4M3, M * K),
        _buf(fn, d, "x_scale", x_scale, _E8M0, M * _blocks(K)), _buf(fn, d, "w", w, _E4M3, G * N * K),
        _buf(fn, d, "w_scale", w_scale, _E8M0, G * _blocks(N) * _blocks(K)),
        _buf(fn, d, "offsets", offsets, _I32, G + 1), G, M, N, K, _stream(stream)))


def qffn_gemv_dual(g, u, x, w_gate, s_gate, w_up, s_up, H, C, stream=None):
    _check("qffn_gemv_dual", lib.qffn_gemv_dual(
        _ptr(g), _ptr(u), _ptr(x), _ptr(w_gate), _ptr(s_gate), _ptr(w_up), _ptr(s_up),
        int(H), int(C), _stream(stream)))


def qffn_gemv(out, x, w, row_scale, rows, cols, stream=None):
    _check("qffn_gemv", lib.qffn_gemv(
        _ptr(out), _ptr(x), _ptr(w), _ptr(row_scale), int(rows), int(cols), _stream(stream)))


def qffn_gemv_silu_input(out, g, u, w, row_scale, rows, cols, stream=None):
    _check("qffn_gemv_silu_input", lib.qffn_gemv_silu_input(
        _ptr(out), _ptr(g), _ptr(u), _ptr(w), _ptr(row_scale), int(rows), int(cols),
        _stream(stream)))


def qffn_silu_mul(g, u, n, stream=None):
    _check("qffn_silu_mul", lib.qffn_silu_mul(_ptr(g), _ptr(u), int(n), _stream(stream)))


def qffn_decode_workspace_size(C, H) -> int:
    return int(lib.qffn_decode_workspace_size(int(C), int(H)))


def qffn_decode_workspace_offsets(C, H):
    """Byte offsets of h and u in the decode workspace."""
    off = (ctypes.c_size_t * 2)()
    _check("qffn_decode_workspace_offsets", lib.qffn_decode_workspace_offsets(int(C), int(H), off))
    return [int(off[0]), int(off[1])]


def qffn_decode_forward(out, x, w_gate, s_gate, w_up, s_up, w_down, s_down, C, H, workspace,
                        workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("qffn_decode_forward", lib.qffn_decode_forward(
        _ptr(out), _ptr(x), _ptr(w_gate), _ptr(s_gate), _ptr(w_up), _ptr(s_up), _ptr(w_down),
        _ptr(s_down), int(C), int(H), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def qffn_decode_forward_ex(out, x, w_gate, s_gate, w_up, s_up, w_down, s_down, C, H, workspace, flags,
                           workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("qffn_decode_forward_ex", lib.qffn_decode_forward_ex(
        _ptr(out), _ptr(x), _ptr(w_gate), _ptr(s_gate), _ptr(w_up), _ptr(s_up), _ptr(w_down),
        _ptr(s_down), int(C), int(H), _ptr(workspace), int(workspace_bytes), int(flags), _stream(stream)))


def qffn_decode_forward_gu(out, x, w_gu, gu_row_scale, w_down, s_down, C, H, workspace,
                           workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("qffn_decode_forward_gu", lib.qffn_decode_forward_gu(
        _ptr(out), _ptr(x), _ptr(w_gu), _ptr(gu_row_scale), _ptr(w_down), _ptr(s_down), int(C), int(H),
        _ptr(workspace), int(workspace_bytes), _stream(stream)))


def qffn_decode_forward_noalloc(out, x, w_gate, s_gate, w_up, s_up, w_down, s_down, C, H,
                                stream=None):
    """qffn_decode_forward for callers that cannot allocate: the scratch is a fixed array
    inside the library (C, H <= 32768); calls overlapping on the GPU race on it."""
    _check("qffn_decode_forward_noalloc", lib.qffn_decode_forward_noalloc(
        _ptr(out), _ptr(x), _ptr(w_gate), _ptr(s_gate), _ptr(w_up), _ptr(s_up), _ptr(w_down),
        _ptr(s_down), int(C), int(H), _stream(stream)))
