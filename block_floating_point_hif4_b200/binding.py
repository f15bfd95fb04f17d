"""ctypes binding of libhif4.so — argument marshalling only.

Every function here forwards to the C ABI declared in ``include/hif4.h`` with
the same name (minus the ``hif4_`` prefix).  torch is used for device memory
and the current CUDA stream; all HiF4 arithmetic runs in the library's CUDA
kernels.  There is no CPU fallback: if ``libhif4.so`` is missing or fails to
load, :func:`lib` raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libhif4.so")

OK = 0
ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_SHAPE, ERR_WORKSPACE = 1, 2, 3, 4
ERR_CUDA, ERR_NONFINITE, ERR_TIMEOUT, ERR_UNSUPPORTED, ERR_FORMAT = 5, 6, 7, 8, 9
F32, BF16 = 0, 1
FLAG_NONFINITE, FLAG_TIMEOUT, FLAG_BAD_INDEX = 1, 2, 4
E4M3, E5M2 = 0, 1
LINEAR_GELU_TANH = 1
LINEAR_OUT_F32 = 2
LINEAR_FAKE_QUANT_OUT = 4

# (name, restype, argtypes) of every exported entry point
_P, _I64, _U32, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int32, ctypes.c_size_t
SIGNATURES = {
    "hif4_quantize": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "hif4_dequantize": (ctypes.c_int, [_P, _P, _I64, _I64, ctypes.c_int, _P, _I64, _P]),
    "hif4_fake_quantize": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _P]),
    "hif4_linear_w4a4_workspace": (_SZ, [_I64, _I64, _I64]),
    "hif4_linear_w4a4": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _I32, _P, _P, _P, _I64,
                                        _U32, _P, _SZ, _P, _P]),
    "hif4_weight_decode": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _I32, _P, _P, _I64, _P, _P]),
    "hif4_gemm_bf16": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _U32, _P, _P]),
    "hif4_gemm_bf16_fq": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _U32, _P, _P]),
    "hif4_ffn_w4a4_workspace": (_SZ, [_I64, _I64, _I64]),
    "hif4_ffn_w4a4_host_workspace": (_SZ, [_I64, _I64, _I64, _I64, _U32]),
    "hif4_ffn_w4a4_host": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _I32, _P, _P, _P, _P, _P, _I32,
                                          _P, _P, _P, _I64, _I64, _U32, _P, _SZ, _P, _P]),
    "hif4_ffn_w4a4": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _I32, _P, _P, _P, _P, _P, _I32, _P,
                                     _P, _P, _I64, _U32, _P, _SZ, _P, _P]),
    "hif4_calib_workspace": (_SZ, [_I64, _I64]),
    "hif4_calib_percentile_mask": (ctypes.c_int, [_P, _I64, _I64, _I64, _U32, _U32, _U32, _U32, _P, _P, _P,
                                                  _P, _P, _SZ, _P]),
    "hif4_calib_noalloc_scratch_bytes": (_SZ, []),
    "hif4_calib_percentile_mask_noalloc": (ctypes.c_int, [_P, _I64, _I64, _I64, _U32, _U32, _U32, _U32, _P, _P,
                                                          _P, _P, _P]),
    "hif4_hessian_workspace": (_SZ, [_I64, _I64]),
    "hif4_hessian": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _SZ, _P, _P]),
    "hif4_higptq1_workspace": (_SZ, [_I64, _I64, _I64]),
    "hif4_higptq1_group_inputs_offset": (_SZ, [_I64, _I64, _I64]),
    "hif4_higptq1": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I32, ctypes.c_double, _I64, _P, _P, _P, _P,
                                    _SZ, _P, _P]),
    "hif4_ptq_state_bytes": (_SZ, [_I64, _I64, _I32]),
    "hif4_ptq_state_pack": (ctypes.c_int, [_I64, _I64, _P, _P, _P, _I32, _P, _P, _SZ]),
    "hif4_ptq_state_info": (ctypes.c_int, [_P, _SZ, _P, _P, _P]),
    "hif4_ptq_state_unpack": (ctypes.c_int, [_P, _SZ, _P, _P, _P, _P]),
    "hif4_to_e4m3": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "hif4_gemm_f8": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _U32, _P,
                                    _P]),
    "hif4_quantize_f8": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, ctypes.c_int, _I32, _P, _I64, _P, _I64,
                                        _P, _I64, _P, _I64, _P, _P]),
    "hif4_gemm_f8_block": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _I64, _P, ctypes.c_int, _I64, _I64,
                                          _P, _I64, _I32, _P, _P, _I64, _U32, _P, _P]),
    "hif4_layer_norm": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, ctypes.c_int, ctypes.c_float, _P,
                                       ctypes.c_int, _I64, _P, _P, _P]),
    "hif4_layer_norm_f8": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, ctypes.c_int, ctypes.c_float,
                                          ctypes.c_int, _P, _I64, _P, _I64, _P, _P, _P, _P]),
    "hif4_layer_norm_backward_workspace": (_SZ, [_I64, _I64]),
    "hif4_layer_norm_backward": (ctypes.c_int, [_P, _I64, _P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P,
                                                ctypes.c_int, _P, _I64, _P, _P, _P, _SZ, _P]),
    "hif4_debug_wait_test": (None, [ctypes.c_uint32, ctypes.c_uint64]),
    "hif4_debug_gemm_f8_block_tiles": (ctypes.c_int, [_I64, _I64, _I64, _I32, ctypes.POINTER(ctypes.c_int32)]),
    "hif4_get_status": (ctypes.c_int, [_P, _P]),
    "hif4_reset_status": (ctypes.c_int, [_P, _P]),
    "hif4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "hif4_last_cuda_error": (ctypes.c_char_p, []),
    "hif4_version": (ctypes.c_int, []),
}

_lock = threading.Lock()
_lib = None


class Hif4Error(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        msg = lib().hif4_status_string(code).decode()
        if code == ERR_CUDA:
            msg += ": " + lib().hif4_last_cuda_error().decode()
        super().__init__("%s failed: status %d (%s)" % (fn, code, msg))


def lib() -> ctypes.CDLL:
    """Load libhif4.so (built in-tree by ``build.py``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libhif4.so is not built (run python -m block_floating_point_hif4_b200.build); "
                                   "there is no CPU fallback")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, code):
    if code != OK:
        raise Hif4Error(fn, code)


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t


# ------------------------------------------------------------------ calls

def quantize(x: torch.Tensor, chan_mask: torch.Tensor | None = None, *, codes=None, meta=None,
             status=None, stream=None):
    """HiF4 codes (uint8 [rows, cols/2]) and meta (int32 bit patterns [rows, cols/64])."""
    _dev(x, "x")
    assert x.dim() == 2 and x.stride(1) == 1
    dt = {torch.bfloat16: BF16, torch.float32: F32}[x.dtype]
    rows, cols = x.shape
    if codes is None:
        codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device)
    if meta is None:
        meta = torch.empty(rows, cols // 64, dtype=torch.int32, device=x.device)
    _check("hif4_quantize", lib().hif4_quantize(_ptr(x), dt, rows, cols, x.stride(0), _ptr(chan_mask),
                                                _ptr(codes), _ptr(meta), _ptr(status), _stream(stream)))
    return codes, meta


def dequantize(codes: torch.Tensor, meta: torch.Tensor, cols: int, dtype=torch.bfloat16, *, out=None,
               stream=None):
    _dev(codes, "codes")
    rows = codes.shape[0]
    if out is None:
        out = torch.empty(rows, cols, dtype=dtype, device=codes.device)
    dt = {torch.bfloat16: BF16, torch.float32: F32}[out.dtype]
    _check("hif4_dequantize", lib().hif4_dequantize(_ptr(codes), _ptr(meta), rows, cols, dt, _ptr(out),
                                                    out.stride(0), _stream(stream)))
    return out


def fake_quantize(x: torch.Tensor, chan_mask: torch.Tensor | None = None, *, out=None, status=None,
                  stream=None):
    _dev(x, "x")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out is None:
        out = torch.empty(rows, cols, dtype=torch.bfloat16, device=x.device)
    _check("hif4_fake_quantize", lib().hif4_fake_quantize(_ptr(x), rows, cols, x.stride(0), _ptr(chan_mask),
                                                          _ptr(out), out.stride(0), _ptr(status),
                                                          _stream(stream)))
    return out


def linear_w4a4_workspace(M: int, N: int, K: int) -> int:
    return int(lib().hif4_linear_w4a4_workspace(M, N, K))


def linear_w4a4(x: torch.Tensor, w_codes: torch.Tensor, w_meta: torch.Tensor, N: int,
                mask_idx: torch.Tensor | None = None, w_masked: torch.Tensor | None = None,
                bias: torch.Tensor | None = None, gelu: bool = False, *, out=None, workspace=None,
                status=None, stream=None):
    """y = fakequant(x) · deq(w)ᵀ + bias (BF16 out); protected columns in BF16."""
    _dev(x, "x")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    need = linear_w4a4_workspace(M, N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    n_m = 0 if mask_idx is None else int(mask_idx.numel())
    flags = (LINEAR_GELU_TANH if gelu else 0) | (LINEAR_OUT_F32 if out.dtype == torch.float32 else 0)
    _check("hif4_linear_w4a4", lib().hif4_linear_w4a4(
        _ptr(x), M, K, x.stride(0), _ptr(w_codes), _ptr(w_meta), N, _ptr(mask_idx) if n_m else None, n_m,
        _ptr(w_masked) if n_m else None, _ptr(bias), _ptr(out), out.stride(0), flags, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)))
    return out


def weight_decode(w_codes: torch.Tensor, w_meta: torch.Tensor, N: int, K: int,
                  mask_idx: torch.Tensor | None = None, w_masked: torch.Tensor | None = None, *, out=None,
                  status=None, stream=None):
    """BF16 N x K decoded weight with the protected columns restored."""
    _dev(w_codes, "w_codes")
    if out is None:
        out = torch.empty(N, K, dtype=torch.bfloat16, device=w_codes.device)
    n_m = 0 if mask_idx is None else int(mask_idx.numel())
    _check("hif4_weight_decode", lib().hif4_weight_decode(
        _ptr(w_codes), _ptr(w_meta), N, K, _ptr(mask_idx) if n_m else None, n_m, _ptr(w_masked) if n_m else None,
        _ptr(out), out.stride(0), _ptr(status), _stream(stream)))
    return out


def gemm_bf16(a: torch.Tensor, b: torch.Tensor, bias: torch.Tensor | None = None, gelu: bool = False, *,
              out=None, status=None, stream=None):
    """y = a · bᵀ + bias on BF16 operands (tcgen05, FP32 accumulate, BF16 out)."""
    _dev(a, "a")
    assert a.dtype == torch.bfloat16 and b.dtype == torch.bfloat16 and a.stride(1) == 1 and b.stride(1) == 1
    M, K = a.shape
    N = b.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    flags = (LINEAR_GELU_TANH if gelu else 0) | (LINEAR_OUT_F32 if out.dtype == torch.float32 else 0)
    _check("hif4_gemm_bf16", lib().hif4_gemm_bf16(
        _ptr(a), M, K, a.stride(0), _ptr(b), N, b.stride(0), _ptr(bias), _ptr(out), out.stride(0),
        flags, _ptr(status), _stream(stream)))
    return out


def to_e4m3(codes: torch.Tensor, meta: torch.Tensor, cols: int, *, pad_rows: int = 1, out=None, stream=None):
    """HiF4 codes -> (E4M3 bytes uint8 [rows, cols], unit scales FP32 [cols/64, lds]),
    lds = rows rounded up to `pad_rows` (128 for the FP8 GEMM's A, 256 for its B)."""
    _dev(codes, "codes")
    rows = codes.shape[0]
    lds = -(-rows // pad_rows) * pad_rows
    if out is None:
        out = (torch.empty(rows, cols, dtype=torch.uint8, device=codes.device),
               torch.zeros(cols // 64, lds, dtype=torch.float32, device=codes.device))
    q8, sc = out
    _check("hif4_to_e4m3", lib().hif4_to_e4m3(_ptr(codes), _ptr(meta), rows, cols, _ptr(q8), q8.stride(0),
                                              _ptr(sc), sc.stride(0), _stream(stream)))
    return q8, sc


def gemm_f8(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, *, out=None, out_f32=False,
            status=None, stream=None):
    """y = sum over units of sa sb (a_u · b_uᵀ) on the FP8 tensor cores (E4M3
    operands from to_e4m3, FP32 unit scales, FP32 promotion)."""
    _dev(a, "a")
    M, K = a.shape
    N = b.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=torch.float32 if out_f32 else torch.bfloat16, device=a.device)
    flags = LINEAR_OUT_F32 if out.dtype == torch.float32 else 0
    _check("hif4_gemm_f8", lib().hif4_gemm_f8(_ptr(a), M, K, a.stride(0), _ptr(sa), sa.stride(0), _ptr(b), N,
                                              b.stride(0), _ptr(sb), sb.stride(0), _ptr(out), out.stride(0), flags,
                                              _ptr(status), _stream(stream)))
    return out


def gemm_bf16_fq(a: torch.Tensor, b: torch.Tensor, bias: torch.Tensor | None = None, gelu: bool = False,
                 out_chan_mask: torch.Tensor | None = None, *, out=None, status=None, stream=None):
    """hfq = fakequant(bf16(a · bᵀ + bias), optionally GELU'd) along N in the
    GEMM epilogue; out_chan_mask (u8 [N], nonzero = protected) columns kept."""
    _dev(a, "a")
    assert a.dtype == torch.bfloat16 and b.dtype == torch.bfloat16 and a.stride(1) == 1 and b.stride(1) == 1
    M, K = a.shape
    N = b.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    flags = LINEAR_GELU_TANH if gelu else 0
    _check("hif4_gemm_bf16_fq", lib().hif4_gemm_bf16_fq(
        _ptr(a), M, K, a.stride(0), _ptr(b), N, b.stride(0), _ptr(bias), _ptr(out_chan_mask), _ptr(out),
        out.stride(0), flags, _ptr(status), _stream(stream)))
    return out


def ffn_w4a4_workspace(M: int, D: int, F: int) -> int:
    return int(lib().hif4_ffn_w4a4_workspace(M, D, F))


def ffn_w4a4(x: torch.Tensor, w1_codes: torch.Tensor, w1_meta: torch.Tensor, F: int,
             w2_codes: torch.Tensor, w2_meta: torch.Tensor,
             mask1_idx: torch.Tensor | None = None, w1_masked: torch.Tensor | None = None,
             b1: torch.Tensor | None = None, mask2_idx: torch.Tensor | None = None,
             w2_masked: torch.Tensor | None = None, b2: torch.Tensor | None = None, *, out=None,
             workspace=None, status=None, stream=None):
    """y = fq(gelu(fq(x) · ŵ1ᵀ + b1)) · ŵ2ᵀ + b2, the W4A4 HiF4 FFN block (BF16 or FP32 out)."""
    _dev(x, "x")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, D = x.shape
    if out is None:
        out = torch.empty(M, D, dtype=torch.bfloat16, device=x.device)
    need = ffn_w4a4_workspace(M, D, F)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    n1 = 0 if mask1_idx is None else int(mask1_idx.numel())
    n2 = 0 if mask2_idx is None else int(mask2_idx.numel())
    flags = LINEAR_OUT_F32 if out.dtype == torch.float32 else 0
    _check("hif4_ffn_w4a4", lib().hif4_ffn_w4a4(
        _ptr(x), M, D, x.stride(0), _ptr(w1_codes), _ptr(w1_meta), F, _ptr(mask1_idx) if n1 else None, n1,
        _ptr(w1_masked) if n1 else None, _ptr(b1), _ptr(w2_codes), _ptr(w2_meta),
        _ptr(mask2_idx) if n2 else None, n2, _ptr(w2_masked) if n2 else None, _ptr(b2), _ptr(out),
        out.stride(0), flags, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream)))
    return out


def ffn_w4a4_host_workspace(M: int, D: int, F: int, chunk_rows: int = 0, out_f32: bool = False) -> int:
    return int(lib().hif4_ffn_w4a4_host_workspace(M, D, F, chunk_rows, LINEAR_OUT_F32 if out_f32 else 0))


def ffn_w4a4_host(x_host: torch.Tensor, w1_codes: torch.Tensor, w1_meta: torch.Tensor, F: int,
                  w2_codes: torch.Tensor, w2_meta: torch.Tensor,
                  mask1_idx: torch.Tensor | None = None, w1_masked: torch.Tensor | None = None,
                  b1: torch.Tensor | None = None, mask2_idx: torch.Tensor | None = None,
                  w2_masked: torch.Tensor | None = None, b2: torch.Tensor | None = None, *, out=None,
                  chunk_rows: int = 0, workspace=None, status=None, stream=None):
    """The FFN block on HOST (ideally pinned) x; y returned in a host tensor.
    Copies overlap compute chunk by chunk.  Asynchronous on `stream`."""
    assert x_host.device.type == "cpu" and x_host.dtype == torch.bfloat16 and x_host.stride(1) == 1
    M, D = x_host.shape
    if out is None:
        out = torch.empty(M, D, dtype=torch.bfloat16, pin_memory=x_host.is_pinned())
    assert out.device.type == "cpu" and out.stride(1) == 1
    f32 = out.dtype == torch.float32
    dev = w1_codes.device
    if workspace is None:
        need = ffn_w4a4_host_workspace(M, D, F, chunk_rows, f32)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    n1 = 0 if mask1_idx is None else int(mask1_idx.numel())
    n2 = 0 if mask2_idx is None else int(mask2_idx.numel())
    _check("hif4_ffn_w4a4_host", lib().hif4_ffn_w4a4_host(
        ctypes.c_void_p(x_host.data_ptr()), M, D, x_host.stride(0), _ptr(w1_codes), _ptr(w1_meta), F,
        _ptr(mask1_idx) if n1 else None, n1, _ptr(w1_masked) if n1 else None, _ptr(b1), _ptr(w2_codes),
        _ptr(w2_meta), _ptr(mask2_idx) if n2 else None, n2, _ptr(w2_masked) if n2 else None, _ptr(b2),
        ctypes.c_void_p(out.data_ptr()), out.stride(0), chunk_rows, LINEAR_OUT_F32 if f32 else 0,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)))
    return out


def calib_workspace(T: int, C: int) -> int:
    return int(lib().hif4_calib_workspace(T, C))


def calib_percentile_mask(acts: torch.Tensor, q=(999, 1000), frac=(1, 100), *, workspace=None, out=None,
                          stream=None):
    """-> (pct bf16 [C], ratio f32 [C], mask uint8 [C], mask_idx int32 [n_top])."""
    _dev(acts, "acts")
    assert acts.dtype == torch.bfloat16 and acts.dim() == 2 and acts.stride(1) == 1
    T, C = acts.shape
    n_top = (C * frac[0]) // frac[1]
    dev = acts.device
    if out is None:
        out = (torch.empty(C, dtype=torch.bfloat16, device=dev), torch.empty(C, dtype=torch.float32, device=dev),
               torch.empty(C, dtype=torch.uint8, device=dev), torch.empty(max(n_top, 1), dtype=torch.int32,
                                                                            device=dev))
    pct, ratio, mask, midx = out
    need = calib_workspace(T, C)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check("hif4_calib_percentile_mask", lib().hif4_calib_percentile_mask(
        _ptr(acts), T, C, acts.stride(0), q[0], q[1], frac[0], frac[1], _ptr(pct), _ptr(ratio), _ptr(mask),
        _ptr(midx), _ptr(workspace), workspace.numel(), _stream(stream)))
    return pct, ratio, mask, midx[:n_top]


def hessian(x: torch.Tensor, *, out=None, workspace=None, status=None, stream=None):
    """H = XᵀX (FP32 K x K) of BF16 activations X (T x K)."""
    _dev(x, "x")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    T, K = x.shape
    if out is None:
        out = torch.empty(K, K, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(1, int(lib().hif4_hessian_workspace(T, K))), dtype=torch.uint8, device=x.device)
    _check("hif4_hessian", lib().hif4_hessian(_ptr(x), T, K, x.stride(0), _ptr(out), _ptr(workspace),
                                              workspace.numel(), _ptr(status), _stream(stream)))
    return out


def higptq1(w: torch.Tensor, H: torch.Tensor, mask_idx: torch.Tensor | None = None, damp: float = 0.01,
            blocksize: int = 128, *, workspace=None, status=None, stream=None):
    """HiGPTQ scheme one -> (codes u8 [N, K/2], meta i32 [N, K/64], w_masked bf16 [N, n] or None)."""
    _dev(w, "w")
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
    assert H.dtype == torch.float32 and H.is_contiguous()
    N, K = w.shape
    n = 0 if mask_idx is None else int(mask_idx.numel())
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=w.device)
    meta = torch.empty(N, K // 64, dtype=torch.int32, device=w.device)
    wm = torch.empty(N, n, dtype=torch.bfloat16, device=w.device) if n else None
    if workspace is None:
        need = int(lib().hif4_higptq1_workspace(N, K, blocksize))
        workspace = torch.empty(max(1, need), dtype=torch.uint8, device=w.device)
    _check("hif4_higptq1", lib().hif4_higptq1(
        _ptr(w), N, K, w.stride(0), _ptr(H), _ptr(mask_idx) if n else None, n, float(damp), blocksize,
        _ptr(codes), _ptr(meta), _ptr(wm), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)))
    return codes, meta, wm


def higptq1_group_inputs(workspace: torch.Tensor, N: int, K: int, blocksize: int = 128) -> torch.Tensor:
    """FP32 [N, K] view of a hif4_higptq1 workspace: after the call, the
    weights each 64-column group was quantized from (stream-ordered)."""
    off = int(lib().hif4_higptq1_group_inputs_offset(N, K, blocksize))
    if off == ctypes.c_size_t(-1).value:
        raise ValueError("invalid HiGPTQ shape")
    assert workspace.dtype == torch.uint8 and workspace.numel() >= off + N * K * 4
    return workspace[off:off + N * K * 4].view(torch.float32).view(N, K)


def ptq_state_pack(codes: torch.Tensor, meta: torch.Tensor, mask_idx: torch.Tensor | None = None,
                   w_masked: torch.Tensor | None = None) -> bytes:
    """Compact PTQ state record of one layer (see hif4.h) from its HiF4 codes
    [N, K/2] u8, meta [N, K/64] i32, protected indices [n] i32 and their BF16
    weight columns [N, n]; tensors on any device (copied to host memory)."""
    c = codes.detach().to("cpu").contiguous()
    m = meta.detach().to("cpu").contiguous()
    N, K = c.shape[0], c.shape[1] * 2
    n = 0 if mask_idx is None else int(mask_idx.numel())
    idx = None if n == 0 else mask_idx.detach().to("cpu", torch.int32).contiguous()
    wm = None if n == 0 else w_masked.detach().to("cpu").contiguous()
    size = int(lib().hif4_ptq_state_bytes(N, K, n))
    if size == 0:
        raise Hif4Error("hif4_ptq_state_bytes", ERR_INVALID_ARG)
    out = ctypes.create_string_buffer(size)
    _check("hif4_ptq_state_pack", lib().hif4_ptq_state_pack(
        N, K, _ptr(c), _ptr(m), _ptr(idx), n, _ptr(wm), ctypes.cast(out, ctypes.c_void_p), size))
    return out.raw


def ptq_state_unpack(record: bytes, device=None):
    """-> (codes u8 [N, K/2], meta i32 [N, K/64], mask_idx i32 [n] or None,
    w_masked bf16 [N, n] or None), on `device` (default: host)."""
    buf = ctypes.create_string_buffer(bytes(record), len(record))
    N, K, n = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
    _check("hif4_ptq_state_info", lib().hif4_ptq_state_info(
        ctypes.cast(buf, ctypes.c_void_p), len(record), ctypes.byref(N), ctypes.byref(K), ctypes.byref(n)))
    N, K, n = N.value, K.value, n.value
    codes = torch.empty(N, K // 2, dtype=torch.uint8)
    meta = torch.empty(N, K // 64, dtype=torch.int32)
    idx = torch.empty(n, dtype=torch.int32) if n else None
    wm = torch.empty(N, n, dtype=torch.bfloat16) if n else None
    _check("hif4_ptq_state_unpack", lib().hif4_ptq_state_unpack(
        ctypes.cast(buf, ctypes.c_void_p), len(record), _ptr(codes), _ptr(meta), _ptr(idx), _ptr(wm)))
    if device is not None:
        codes, meta = codes.to(device), meta.to(device)
        idx = None if idx is None else idx.to(device)
        wm = None if wm is None else wm.to(device)
    return codes, meta, idx, wm


# ------------------------------------------------- block-scaled FP8, layer norm
#
# These calls are short enough for their marshalling to count: pointers are
# passed as integers, padded tensors are allocated as such, and no context is
# entered where device and stream are the current ones.
#
# Like every call here they are outside autograd: results carry no graph, whether
# or not an input requires a gradient.  A training step makes the backward calls
# itself (gemm_f8_block on transposed codes, layer_norm_backward).

_DTYPE = {torch.float32: F32, torch.bfloat16: BF16}
_F8 = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
_SCALE = {torch.float32: F32}
_BIAS = {torch.bfloat16: BF16}

# the public calls build a Stream object, or check for a lazy start, each time
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _cdiv(n, m):
    return -(-n // m)


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _matrix(t, name, dtypes, shape=None):
    """Checks a 2-D CUDA tensor whose rows are contiguous -> (rows, cols, leading dimension).  The leading
    dimension of a single row, which no address depends on, is rounded up to a multiple of 16."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s has dtype %s" % (name, t.dtype))
    size = t.shape
    if len(size) != 2:
        raise ValueError("%s must be 2-D" % name)
    if shape is not None and size != shape:
        raise ValueError("%s must be %s, is %s" % (name, tuple(shape), tuple(size)))
    rows, cols = size
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError("%s must have contiguous rows" % name)
    return rows, cols, (ld if rows > 1 else (cols + 15) // 16 * 16)


def _vector(t, name, dtypes, n):
    """Checks an optional contiguous vector -> its address or None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s has dtype %s" % (name, t.dtype))
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d elements" % (name, n))
    return t.data_ptr()


def _status(t):
    if t is None:
        return None
    if not t.is_cuda or t.element_size() != 4 or t.numel() < 1:
        raise ValueError("status must be a 32-bit word on the GPU")
    return t.data_ptr()


def _padded(rows, cols, dtype, multiple, device):
    """rows x cols whose leading dimension is a multiple of `multiple` elements."""
    return torch.empty_strided((rows, cols), ((cols + multiple - 1) // multiple * multiple, 1), dtype=dtype,
                               device=device)


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield stream.cuda_stream


def _place(stream, *tensors):
    """Context of a call: its tensors' device current, `stream` (default: that
    device's current stream) current, so that what the call allocates belongs
    to the stream it runs on.  Yields the stream's handle."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors of one call must be on one device")
    if stream is None:
        if index == _raw_device():
            return contextlib.nullcontext(_raw_stream(index))
        stream = torch.cuda.current_stream(index)
    _need(stream.device.index == index, "the stream is on another device than the tensors")
    return _switched(tensors[0].device, stream)


def quantize_f8(x: torch.Tensor, fmt=torch.float8_e4m3fn, *, block_rows: int = 1, layout: str = "rows", out=None,
                status=None, stream=None):
    """FP8 codes with one FP32 scale per block of 128 (see hif4.h).

    layout "rows": (q [rows, cols], scale); "cols": (qt [cols, rows], scale_t);
    "both": (q, scale, qt, scale_t) from one read of x.  scale is
    [ceil(cols/128), rows] for block_rows 1 and [ceil(rows/128),
    ceil(cols/128)] for 128; scale_t likewise for the transposed matrix.
    `out` is a tuple of those tensors to write into."""
    rows, cols, ldx = _matrix(x, "x", _DTYPE)
    _need(fmt in _F8, "fmt must be torch.float8_e4m3fn or torch.float8_e5m2")
    _need(block_rows in (1, 128), "block_rows must be 1 or 128")
    _need(layout in ("rows", "cols", "both"), "layout must be rows, cols or both")
    sizes = []
    for r, c in ((rows, cols),) * (layout != "cols") + ((cols, rows),) * (layout != "rows"):
        sizes += [(r, c), (_cdiv(c, 128), r) if block_rows == 1 else (_cdiv(r, 128), _cdiv(c, 128))]
    f8 = {fmt: _F8[fmt]}
    with _place(stream, x, status, *(out if out is not None else ())) as s:
        if out is None:
            dev = x.device
            out = tuple([_padded(r, c, torch.float32, 4, dev) if i & 1 else _padded(r, c, fmt, 16, dev)
                         for i, (r, c) in enumerate(sizes)])
        _need(len(out) == len(sizes), "out must hold %d tensors" % len(sizes))
        args = []
        for i, size in enumerate(sizes):
            ld = _matrix(out[i], "out[%d]" % i, _SCALE if i & 1 else f8, size)[2]
            args += [out[i].data_ptr(), ld]
        if layout == "rows":
            args += [None, 0, None, 0]
        elif layout == "cols":
            args = [None, 0, None, 0] + args
        _check("hif4_quantize_f8", lib().hif4_quantize_f8(
            x.data_ptr(), _DTYPE[x.dtype], rows, cols, ldx, _F8[fmt], block_rows, *args, _status(status), s))
    return out


def gemm_f8_block(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                  bias: torch.Tensor | None = None, *, b_block_rows: int = 128, out=None, out_f32: bool = False,
                  status=None, stream=None):
    """y = (a, sa) · (b, sb)ᵀ + bias for FP8 operands with a scale per block of
    128 along K: a [M, K] with 1 x 128 blocks, b [N, K] with 128 x 128 blocks
    (b_block_rows 128) or 1 x 128 blocks (1), as quantize_f8 leaves them."""
    M, K, lda = _matrix(a, "a", _F8)
    N, Kb, ldb = _matrix(b, "b", _F8)
    _need(Kb == K, "a and b must have the same number of columns")
    _need(b_block_rows in (1, 128), "b_block_rows must be 1 or 128")
    units = _cdiv(K, 128)
    ldsa = _matrix(sa, "sa", _SCALE, (units, M))[2]
    ldsb = _matrix(sb, "sb", _SCALE, (units, N) if b_block_rows == 1 else (_cdiv(N, 128), units))[2]
    pbias = _vector(bias, "bias", _BIAS, N)
    with _place(stream, a, sa, b, sb, bias, out, status) as s:
        if out is None:
            out = _padded(M, N, torch.float32, 4, a.device) if out_f32 else _padded(M, N, torch.bfloat16, 8, a.device)
        ldy = _matrix(out, "out", _DTYPE, (M, N))[2]
        _check("hif4_gemm_f8_block", lib().hif4_gemm_f8_block(
            a.data_ptr(), _F8[a.dtype], M, K, lda, sa.data_ptr(), ldsa, b.data_ptr(), _F8[b.dtype], N, ldb,
            sb.data_ptr(), ldsb, b_block_rows, pbias, out.data_ptr(), ldy,
            LINEAR_OUT_F32 if out.dtype == torch.float32 else 0, _status(status), s))
    return out


def _norm_params(gamma, beta, cols):
    """-> (gamma's address, beta's, their dtype)."""
    pg, pb = _vector(gamma, "gamma", _DTYPE, cols), _vector(beta, "beta", _DTYPE, cols)
    _need(gamma is None or beta is None or gamma.dtype == beta.dtype, "gamma and beta must have the same dtype")
    given = gamma if gamma is not None else beta
    return pg, pb, F32 if given is None else _DTYPE[given.dtype]


def layer_norm(x: torch.Tensor, gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
               eps: float = 1e-6, *, out=None, out_dtype=None, save_stats: bool = False, stream=None):
    """Layer norm of the rows of x -> y, or (y, mean, rstd) with save_stats;
    y has out_dtype (default: x's)."""
    rows, cols, ldx = _matrix(x, "x", _DTYPE)
    pg, pb, pdt = _norm_params(gamma, beta, cols)
    with _place(stream, x, gamma, beta, out) as s:
        if out is None:
            dt = out_dtype if out_dtype is not None else x.dtype
            _need(dt in _DTYPE, "out_dtype must be float32 or bfloat16")
            out = _padded(rows, cols, dt, 8, x.device)
        ldy = _matrix(out, "out", _DTYPE, (rows, cols))[2]
        mean = rstd = None
        if save_stats:
            mean = torch.empty(rows, dtype=torch.float32, device=x.device)
            rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
        _check("hif4_layer_norm", lib().hif4_layer_norm(
            x.data_ptr(), _DTYPE[x.dtype], rows, cols, ldx, pg, pb, pdt, eps, out.data_ptr(), _DTYPE[out.dtype], ldy,
            mean.data_ptr() if save_stats else None, rstd.data_ptr() if save_stats else None, s))
    return (out, mean, rstd) if save_stats else out


def layer_norm_f8(x: torch.Tensor, gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                  eps: float = 1e-6, fmt=torch.float8_e4m3fn, *, out=None, save_stats: bool = False, status=None,
                  stream=None):
    """layer_norm in FP32 followed by quantize_f8 in 1 x 128 blocks, in one
    pass -> (q, scale), or (q, scale, mean, rstd) with save_stats."""
    rows, cols, ldx = _matrix(x, "x", _DTYPE)
    _need(fmt in _F8, "fmt must be torch.float8_e4m3fn or torch.float8_e5m2")
    pg, pb, pdt = _norm_params(gamma, beta, cols)
    units = _cdiv(cols, 128)
    with _place(stream, x, gamma, beta, status, *(out if out is not None else ())) as s:
        if out is None:
            out = _padded(rows, cols, fmt, 16, x.device), _padded(units, rows, torch.float32, 4, x.device)
        q, sc = out
        ldq = _matrix(q, "out[0]", {fmt: 0}, (rows, cols))[2]
        lds = _matrix(sc, "out[1]", _SCALE, (units, rows))[2]
        mean = rstd = None
        if save_stats:
            mean = torch.empty(rows, dtype=torch.float32, device=x.device)
            rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
        _check("hif4_layer_norm_f8", lib().hif4_layer_norm_f8(
            x.data_ptr(), _DTYPE[x.dtype], rows, cols, ldx, pg, pb, pdt, eps, _F8[fmt], q.data_ptr(), ldq,
            sc.data_ptr(), lds, mean.data_ptr() if save_stats else None, rstd.data_ptr() if save_stats else None,
            _status(status), s))
    return (q, sc, mean, rstd) if save_stats else (q, sc)


def layer_norm_backward_workspace(rows: int, cols: int) -> int:
    return int(lib().hif4_layer_norm_backward_workspace(rows, cols))


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        gamma: torch.Tensor | None = None, *, out=None, workspace=None, stream=None):
    """Gradients of layer_norm -> (dx, dgamma, dbeta), from the statistics it
    saved.  dx has x's dtype, dgamma and dbeta are FP32.  `out` is a tuple of
    the three, None in the place of one that is not wanted."""
    rows, cols, ldx = _matrix(x, "x", _DTYPE)
    lddy = _matrix(dy, "dy", {x.dtype: 0}, (rows, cols))[2]
    _need(mean is not None and rstd is not None, "mean and rstd are needed")
    pmean, prstd = _vector(mean, "mean", _SCALE, rows), _vector(rstd, "rstd", _SCALE, rows)
    pg, _, pdt = _norm_params(gamma, None, cols)
    with _place(stream, x, dy, mean, rstd, gamma, workspace, *(out if out is not None else ())) as s:
        if out is None:
            dev = x.device
            out = (_padded(rows, cols, x.dtype, 8, dev), torch.empty(cols, dtype=torch.float32, device=dev),
                   torch.empty(cols, dtype=torch.float32, device=dev))
        dx, dgamma, dbeta = out
        lddx = 0 if dx is None else _matrix(dx, "out[0]", {x.dtype: 0}, (rows, cols))[2]
        pdg, pdb = _vector(dgamma, "out[1]", _SCALE, cols), _vector(dbeta, "out[2]", _SCALE, cols)
        if workspace is None and (dgamma is not None or dbeta is not None):
            need = layer_norm_backward_workspace(rows, cols)
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
        pws, nws = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                        workspace.numel() * workspace.element_size())
        _check("hif4_layer_norm_backward", lib().hif4_layer_norm_backward(
            dy.data_ptr(), lddy, x.data_ptr(), _DTYPE[x.dtype], rows, cols, ldx, pmean, prstd, pg, pdt,
            None if dx is None else dx.data_ptr(), lddx, pdg, pdb, pws, nws, s))
    return dx, dgamma, dbeta


def get_status(status: torch.Tensor, stream=None) -> int:
    return int(lib().hif4_get_status(_ptr(status), _stream(stream)))


def reset_status(status: torch.Tensor, stream=None) -> None:
    _check("hif4_reset_status", lib().hif4_reset_status(_ptr(status), _stream(stream)))


def version() -> int:
    return int(lib().hif4_version())
