"""Thin ctypes binding of libbq.so (C ABI in include/bq.h).

Argument marshalling only: every function checks dtypes/devices/shapes of
torch tensors, allocates outputs when none are given, and calls the C entry
point of the same name on the current torch stream of the tensors' device.
All compute runs in the HIP kernels of libbq.so; there is no fallback: if the
library is missing or the device is not gfx950 the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbq.so")

BQ_OK, BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_ALIGN, BQ_ERR_HIP, BQ_ERR_DEVICE, BQ_ERR_ARG = range(7)
PATH_AUTO, PATH_STREAM, PATH_TILED, PATH_GEMV = 0, 1, 2, 3
MAX_K = 65536
_PATHS = {"auto": PATH_AUTO, "stream": PATH_STREAM, "tiled": PATH_TILED, "gemv": PATH_GEMV}

# (name, argtypes) for every entry point declared in include/bq.h
_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
SIGNATURES = {
    "bq_version": [],
    "bq_status_string": [_I],
    "bq_quantize_rows": [_P, _I64, _I64, _P, _P, _P],
    "bq_pack_int4": [_P, _I64, _I64, _P, _P],
    "bq_pack_int2": [_P, _I64, _I64, _P, _P],
    "bq_gemm_w8a8_dequant": [_P, _P, _P, _P, _I64, _I64, _I64, _P],
    "bq_gemm_w4a8_dequant": [_P, _P, _P, _P, _I64, _I64, _I64, _P],
    "bq_gemm_w2a8_dequant": [_P, _P, _P, _P, _I64, _I64, _I64, _P],
    "bq_gemm_w8a8_i32": [_P, _P, _P, _I64, _I64, _I64, _P],
    "bq_gemm_w4a8_i32": [_P, _P, _P, _I64, _I64, _I64, _P],
    "bq_gemm_w2a8_i32": [_P, _P, _P, _I64, _I64, _I64, _P],
    "bq_gemm": [_P, _P, _I, _P, _P, _I64, _I64, _I64, _I, _P],
    "bq_gemm_dual_scale": [_P, _P, _I, _P, _P, _P, _I64, _I64, _I64, _I, _P],
    "bq_gemm_batched": [_P, _I64, _P, _I64, _I, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _I64, _I, _P],
    "bq_gemm_act": [_P, _P, _I, _P, _P, _I, _P, _I64, _I64, _I64, _I, _P],
    "bq_quantize_rows_bits": [_P, _I64, _I64, _I, _P, _P, _P],
    "bq_quantize_pack": [_P, _I64, _I64, _I, _P, _P, _P],
    "bq_gemm_select_path": [_I64, _I64, _I64, _I],
    "bq_gemm_nf4_a16": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P],
    "bq_gemm_splitk_workspace_bytes": [_I64, _I64, _I64, _I],
    "bq_gemm_splitk": [_P, _P, _I, _P, _P, _I64, _I64, _I64, _P, _I64, _P],
    "bq_gemm_splitk_static": [_P, _P, _I, _P, _P, _I64, _I64, _I64, _P],
}
_F32, _F64 = ctypes.c_float, ctypes.c_double
# the same for include/bq_layer.h
LAYER_SIGNATURES = {
    "bq_gemm_w4g_a16": [_P, _I, _P, _P, _P, _I, _P, _I64, _I64, _I64, _P, _I64, _P],
    "bq_gemm_w4g_workspace_bytes": [_I64, _I64, _I64],
    "bq_qk_norm_rope": [_P, _I64, _P, _I64, _I, _I64, _I, _I, _I, _P, _P, _F64, _P, _P, _I64, _I, _I, _P, _P, _P, _P],
    "bq_kv4_page_bytes": [_I, _I, _I],
    "bq_qk_norm_rope_kv4": [_P, _I64, _P, _I64, _P, _I64, _I, _I64, _I, _I, _I, _P, _P, _F64, _P, _P, _I64, _I, _I, _P,
                            _P, _P, _I64, _I, _P, _P],
    "bq_kv4_read": [_P, _I64, _I, _I, _I, _P, _I64, _I, _P, _P, _P],
    "bq_attn_kv4": [_P, _I64, _I, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _I64, _I, _I64, _F32, _I64, _P, _P, _P,
                    _I64, _P],
    "bq_attn_kv4_workspace_bytes": [_I64, _I64, _I, _I, _I, _I64],
}
_RESTYPES = {"bq_status_string": ctypes.c_char_p, "bq_gemm_splitk_workspace_bytes": ctypes.c_int64,
             "bq_gemm_w4g_workspace_bytes": ctypes.c_int64, "bq_kv4_page_bytes": ctypes.c_int64,
             "bq_attn_kv4_workspace_bytes": ctypes.c_int64}


class BQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libbq.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build the HIP library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        handle = ctypes.CDLL(LIB_PATH)
        for name, args in {**SIGNATURES, **LAYER_SIGNATURES}.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = _RESTYPES.get(name, ctypes.c_int)
        _lib = handle
    return _lib


def version() -> int:
    return lib().bq_version()


def status_string(status: int) -> str:
    return lib().bq_status_string(status).decode()


def select_path(M: int, N: int, K: int, bits: int) -> str:
    p = lib().bq_gemm_select_path(M, N, K, bits)
    return {PATH_STREAM: "stream", PATH_TILED: "tiled", PATH_GEMV: "gemv"}[p]


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------

def _check_tensor(t: torch.Tensor, name: str, dtype, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _call(name: str, device: torch.device, *args):
    with torch.cuda.device(device):
        st = getattr(lib(), name)(*args, _stream(device))
    if st != BQ_OK:
        raise BQError(st, name)


# --------------------------------------------------------------------------
# public functions (same names as the C entry points, without the prefix)
# --------------------------------------------------------------------------

def quantize_rows(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None):
    """Per-row int8 quantization of fp16 x [rows, cols] -> (q int8, scale fp16 [rows])."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    rows, cols = x.shape
    _check_tensor(x, "x", torch.float16)
    dev = x.device
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.int8, device=dev)
    if scale is None:
        scale = torch.empty((rows,), dtype=torch.float16, device=dev)
    _check_tensor(q, "q", torch.int8, (rows, cols), dev)
    _check_tensor(scale, "scale", torch.float16, (rows,), dev)
    _call("bq_quantize_rows", dev, _ptr(x), rows, cols, _ptr(q), _ptr(scale))
    return q, scale


def quantize_rows_bits(x: torch.Tensor, bits: int, q: Optional[torch.Tensor] = None,
                       scale: Optional[torch.Tensor] = None):
    """Per-row quantization of fp16 x [rows, cols] to the code range of a
    weight format, qmax = 2^(bits-1) - 1 (bits 8, 4, 2) -> (q int8, scale fp16
    [rows]); the codes feed pack_int4 / pack_int2."""
    if bits not in (8, 4, 2):
        raise ValueError("bits must be 8, 4 or 2")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    rows, cols = x.shape
    _check_tensor(x, "x", torch.float16)
    dev = x.device
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.int8, device=dev)
    if scale is None:
        scale = torch.empty((rows,), dtype=torch.float16, device=dev)
    _check_tensor(q, "q", torch.int8, (rows, cols), dev)
    _check_tensor(scale, "scale", torch.float16, (rows,), dev)
    _call("bq_quantize_rows_bits", dev, _ptr(x), rows, cols, bits, _ptr(q), _ptr(scale))
    return q, scale


def quantize_pack(x: torch.Tensor, bits: int, out: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None):
    """Per-row quantization of fp16 x [rows, cols] to the int4 (bits 4) or
    ternary (bits 2) code range, written packed -> (packed uint8 [rows,
    cols*bits/8], scale fp16 [rows]); equal to quantize_rows_bits followed by
    pack_int4 / pack_int2, in one pass."""
    if bits not in (4, 2):
        raise ValueError("bits must be 4 or 2")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    rows, cols = x.shape
    if cols % (8 // bits):
        raise ValueError(f"cols must be a multiple of {8 // bits}")
    _check_tensor(x, "x", torch.float16)
    dev = x.device
    if out is None:
        out = torch.empty((rows, cols * bits // 8), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty((rows,), dtype=torch.float16, device=dev)
    _check_tensor(out, "out", torch.uint8, (rows, cols * bits // 8), dev)
    _check_tensor(scale, "scale", torch.float16, (rows,), dev)
    _call("bq_quantize_pack", dev, _ptr(x), rows, cols, bits, _ptr(out), _ptr(scale))
    return out, scale


def _pack(name: str, factor: int, v: torch.Tensor, out: Optional[torch.Tensor]):
    if v.dim() != 2:
        raise ValueError("v must be 2-D [n, k]")
    n, k = v.shape
    _check_tensor(v, "v", torch.int8)
    if k % factor:
        raise ValueError(f"k must be a multiple of {factor}")
    if out is None:
        out = torch.empty((n, k // factor), dtype=torch.uint8, device=v.device)
    _check_tensor(out, "out", torch.uint8, (n, k // factor), v.device)
    _call(name, v.device, _ptr(v), n, k, _ptr(out))
    return out


def pack_int4(v: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8 values in [-8, 7] [n, k] -> uint8 [n, k/2] (low nibble = even k)."""
    return _pack("bq_pack_int4", 2, v, out)


def pack_int2(v: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8 values in [-2, 1] [n, k] -> uint8 [n, k/4] (code v+2, bits 2j = k%4 j)."""
    return _pack("bq_pack_int2", 4, v, out)


def _gemm_args(A, B, bits, scale, out):
    if bits not in (8, 4, 2):
        raise ValueError("bits must be 8, 4 or 2")
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = A.shape
    N = B.shape[0]
    dev = A.device
    _check_tensor(A, "A", torch.int8)
    _check_tensor(B, "B", torch.int8 if bits == 8 else torch.uint8, (N, K * bits // 8), dev)
    if scale is not None:
        _check_tensor(scale, "scale", torch.float16, (N,), dev)
    odt = torch.float16 if scale is not None else torch.int32
    if out is None:
        out = torch.empty((M, N), dtype=odt, device=dev)
    _check_tensor(out, "out", odt, (M, N), dev)
    return M, N, K, dev, out


def gemm(A: torch.Tensor, B: torch.Tensor, bits: int, scale: Optional[torch.Tensor] = None,
         out: Optional[torch.Tensor] = None, path: str = "auto") -> torch.Tensor:
    """C = A . B^T (int32), or fp16(C * scale[n]) when scale is given, with an
    explicit kernel path ("auto", "gemv", "stream" or "tiled").

    A int8 [M, K]; B int8 [N, K] (bits=8) or uint8 [N, K*bits/8] (bits=4, 2).
    """
    M, N, K, dev, out = _gemm_args(A, B, bits, scale, out)
    _call("bq_gemm", dev, _ptr(A), _ptr(B), bits, _ptr(scale), _ptr(out), M, N, K, _PATHS[path])
    return out


def gemm_splitk_workspace_bytes(M: int, N: int, K: int, bits: int) -> int:
    """Device workspace bytes gemm_splitk uses to split K for this shape (0:
    it would not split)."""
    n = lib().bq_gemm_splitk_workspace_bytes(M, N, K, bits)
    if n < 0:
        raise BQError(-n, "bq_gemm_splitk_workspace_bytes")
    return n


def gemm_splitk(A: torch.Tensor, B: torch.Tensor, bits: int, scale: Optional[torch.Tensor],
                workspace: Optional[torch.Tensor], out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gemm on the tiled path with K split over workgroups when the output
    has few tiles, using the caller's workspace (a uint8 device tensor whose
    first 4096 bytes are zero before the first call, e.g. torch.zeros of
    gemm_splitk_workspace_bytes(M, N, K, bits) bytes; None: no split)."""
    M, N, K, dev, out = _gemm_args(A, B, bits, scale, out)
    nbytes = 0
    if workspace is not None:
        _check_tensor(workspace, "workspace", torch.uint8, None, dev)
        nbytes = workspace.numel()
    _call("bq_gemm_splitk", dev, _ptr(A), _ptr(B), bits, _ptr(scale), _ptr(out), M, N, K, _ptr(workspace),
          nbytes)
    return out


def gemm_splitk_static(A: torch.Tensor, B: torch.Tensor, bits: int, scale: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gemm_splitk with the library's own static scratch (no device memory
    is allocated by the call; pass `out` as well to allocate nothing here).
    Calls that may overlap on one GPU race: order them on one stream."""
    M, N, K, dev, out = _gemm_args(A, B, bits, scale, out)
    _call("bq_gemm_splitk_static", dev, _ptr(A), _ptr(B), bits, _ptr(scale), _ptr(out), M, N, K)
    return out


def gemm_dual_scale(A: torch.Tensor, B: torch.Tensor, bits: int, w_scale: torch.Tensor,
                    x_scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                    path: str = "auto") -> torch.Tensor:
    """fp16(acc[m,n] * w_scale[n] * x_scale[m]): the GEMM of a linear layer
    whose M activation rows were quantized per token (codes A, scales x_scale
    from quantize_rows)."""
    M, N, K, dev, out = _gemm_args(A, B, bits, w_scale, out)
    _check_tensor(x_scale, "x_scale", torch.float16, (M,), dev)
    _call("bq_gemm_dual_scale", dev, _ptr(A), _ptr(B), bits, _ptr(w_scale), _ptr(x_scale),
          _ptr(out), M, N, K, _PATHS[path])
    return out


ACTS = {"none": 0, "relu": 1, "gelu": 2}


def gemm_act(A: torch.Tensor, B: torch.Tensor, bits: int, w_scale: torch.Tensor,
             x_scale: Optional[torch.Tensor] = None, act: str = "gelu",
             out: Optional[torch.Tensor] = None, path: str = "auto") -> torch.Tensor:
    """fp16(act(acc[m,n] * w_scale[n] * x_scale[m])) with act "none", "relu"
    or "gelu" fused into the epilogue (x_scale None = 1)."""
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    M, N, K, dev, out = _gemm_args(A, B, bits, w_scale, out)
    if x_scale is not None:
        _check_tensor(x_scale, "x_scale", torch.float16, (M,), dev)
    _call("bq_gemm_act", dev, _ptr(A), _ptr(B), bits, _ptr(w_scale), _ptr(x_scale), ACTS[act],
          _ptr(out), M, N, K, _PATHS[path])
    return out


def linear(x: torch.Tensor, B: torch.Tensor, bits: int, w_scale: torch.Tensor,
           act: str = "none", path: str = "auto") -> torch.Tensor:
    """fp16 activations x [M, K] through a quantized weight: per-token int8
    quantization of x (quantize_rows), then the two-scale GEMM with the
    activation act fused."""
    q, xs = quantize_rows(x)
    if act == "none":
        return gemm_dual_scale(q, B, bits, w_scale, xs, path=path)
    return gemm_act(q, B, bits, w_scale, xs, act=act, path=path)


def gemm_batched(A: torch.Tensor, B: torch.Tensor, bits: int, scale: Optional[torch.Tensor] = None,
                 x_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 path: str = "auto") -> torch.Tensor:
    """Batched GEMM in one launch: B [batch, N, K*bits/8]; A [M, K] shared by
    every batch (broadcast, the fused-QKV shape) or [batch, M, K]; scale
    [batch, N] for the fp16 output (times x_scale [M], shared, when given),
    else int32.  Returns [batch, M, N]."""
    if bits not in (8, 4, 2):
        raise ValueError("bits must be 8, 4 or 2")
    if B.dim() != 3 or A.dim() not in (2, 3):
        raise ValueError("B must be [batch, N, K*bits/8] and A [M, K] or [batch, M, K]")
    batch, N, Kb = B.shape
    M, K = A.shape[-2:]
    dev = A.device
    _check_tensor(A, "A", torch.int8, (M, K) if A.dim() == 2 else (batch, M, K), dev)
    _check_tensor(B, "B", torch.int8 if bits == 8 else torch.uint8, (batch, N, K * bits // 8), dev)
    if scale is not None:
        _check_tensor(scale, "scale", torch.float16, (batch, N), dev)
    if x_scale is not None:
        if scale is None:
            raise ValueError("x_scale needs scale")
        _check_tensor(x_scale, "x_scale", torch.float16, (M,), dev)
    odt = torch.float16 if scale is not None else torch.int32
    if out is None:
        out = torch.empty((batch, M, N), dtype=odt, device=dev)
    _check_tensor(out, "out", odt, (batch, M, N), dev)
    strideA = 0 if A.dim() == 2 else M * K
    _call("bq_gemm_batched", dev, _ptr(A), strideA, _ptr(B), N * Kb, bits, _ptr(scale),
          N if scale is not None else 0, _ptr(x_scale), _ptr(out), M * N, batch, M, N, K, _PATHS[path])
    return out


def _named_dequant(bits, A, B, scale, out):
    if scale is None:
        raise ValueError("scale is required")
    M, N, K, dev, out = _gemm_args(A, B, bits, scale, out)
    _call(f"bq_gemm_w{bits}a8_dequant", dev, _ptr(A), _ptr(B), _ptr(scale), _ptr(out), M, N, K)
    return out


def _named_i32(bits, A, B, out):
    M, N, K, dev, out = _gemm_args(A, B, bits, None, out)
    _call(f"bq_gemm_w{bits}a8_i32", dev, _ptr(A), _ptr(B), _ptr(out), M, N, K)
    return out


def gemm_w8a8_dequant(A, B, scale, out=None):
    """fp16((A . B^T) * scale), B int8 [N, K]."""
    return _named_dequant(8, A, B, scale, out)


def gemm_w4a8_dequant(A, B, scale, out=None):
    """fp16((A . B^T) * scale), B packed int4 uint8 [N, K/2]."""
    return _named_dequant(4, A, B, scale, out)


def gemm_w2a8_dequant(A, B, scale, out=None):
    """fp16((A . B^T) * scale), B packed int2 uint8 [N, K/4]."""
    return _named_dequant(2, A, B, scale, out)


def gemm_w8a8_i32(A, B, out=None):
    return _named_i32(8, A, B, out)


def gemm_w4a8_i32(A, B, out=None):
    return _named_i32(4, A, B, out)


def gemm_w2a8_i32(A, B, out=None):
    return _named_i32(2, A, B, out)


def gemm_nf4_a16(A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                 zero: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """W4A16 GEMM with NF4 weight codes: C = fp16(sum_k A[m,k] W[n,k]) with
    W[n,k] = fp16((nf4[code] - zero[n]) * scale[n]) and fp32 accumulation.

    A fp16 [M, K]; B uint8 [N, K/2] (code of k even in the low nibble);
    scale fp16 [N]; zero fp16 [N] or None (0)."""
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = A.shape
    N = B.shape[0]
    dev = A.device
    _check_tensor(A, "A", torch.float16)
    _check_tensor(B, "B", torch.uint8, (N, K // 2), dev)
    _check_tensor(scale, "scale", torch.float16, (N,), dev)
    if zero is not None:
        _check_tensor(zero, "zero", torch.float16, (N,), dev)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=dev)
    _check_tensor(out, "out", torch.float16, (M, N), dev)
    _call("bq_gemm_nf4_a16", dev, _ptr(A), _ptr(B), _ptr(scale), _ptr(zero), _ptr(out), M, N, K)
    return out


# --------------------------------------------------------------------------
# decoder-layer operators (include/bq_layer.h)
# --------------------------------------------------------------------------

# These calls are made many times per token, so their marshalling is kept
# short: one combined test per tensor (the named checks only say what failed),
# plain integers for pointers, sizes that depend on integers alone remembered.

_DTYPES16 = {torch.float16: 0, torch.bfloat16: 1}


def _dtype16(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES16:
        raise ValueError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return _DTYPES16[t.dtype]


def _dense(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    """The address of a dense GPU tensor of this type, shape (None: any) and
    device."""
    try:
        if t.dtype is dtype and t.device == device and t.is_contiguous() and (shape is None or t.shape == shape) and t.is_cuda:
            return t.data_ptr()
    except AttributeError:
        pass
    _check_tensor(t, name, dtype, shape, device)
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    """A [tokens, heads, dim] tensor, dense within a token; the elements
    between its tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not (t.dtype is dtype and t.device == device and t.is_cuda and t.shape == shape):
        _check_tensor(t, name, dtype, shape, device)  # says which, and raises
    stride, by_head, by_dim = t.stride()
    if by_dim != 1 or (by_head != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must be dense within a token")
    return stride if shape[0] > 1 else shape[1] * shape[2]


def _enqueue(name: str, device: torch.device, *args):
    """The C call of this name on the device's current torch stream."""
    if torch._C._cuda_getDevice() != device.index:
        _call(name, device, *args)
        return
    st = getattr(_lib or lib(), name)(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if st != BQ_OK:
        raise BQError(st, name)


@functools.lru_cache(maxsize=4096)
def _host_bytes(name: str, *args) -> int:
    """A size that the library computes from integers alone."""
    n = getattr(lib(), name)(*args)
    if n < 0:
        raise BQError(-n, name)
    return n


def _output(t: Optional[torch.Tensor], name: str, dtype, shape, device):
    """(tensor, address) of the output given, or of a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _dense(t, name, dtype, shape, device)


def _workspace(t: Optional[torch.Tensor], nbytes: int, device):
    """(tensor, address, bytes) of the workspace given or allocated; the
    tensor is held until the call is enqueued."""
    if t is None:
        if not nbytes:
            return None, None, 0
        t = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return t, t.data_ptr(), nbytes
    return t, _dense(t, "workspace", torch.uint8, None, device), t.numel()


def gemm_w4g_workspace_bytes(M: int, N: int, K: int) -> int:
    """Device workspace bytes with which gemm_w4g_a16 splits K for this shape
    (0: it does not)."""
    return _host_bytes("bq_gemm_w4g_workspace_bytes", M, N, K)


def gemm_w4g_a16(A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor, zero: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """4-bit weights with group scales: C = sum_k A[m,k] (c[n,k] - zero[n,g])
    scale[n,g], g = k // group, with fp32 accumulation, of A's type.

    A fp16 or bf16 [M, K]; B uint8 [N, K/2] (pack_int4's layout, codes
    -8..7); scale, zero fp16 [N, K/group], group 32, 64 or 128 (quantize_pack
    of the weight viewed as [N * K/group, group] gives B and scale).  A
    workspace is allocated for the call when it needs one and none is given."""
    dt = _dtype16(A, "A")
    if A.dim() != 2 or B.dim() != 2 or scale.dim() != 2:
        raise ValueError("A, B and scale must be 2-D")
    M, K = A.shape
    N, groups = scale.shape
    dev, dtype = A.device, A.dtype
    a = _dense(A, "A", dtype, None, dev)
    b = _dense(B, "B", torch.uint8, (N, K // 2), dev)
    if K and (groups == 0 or K % groups):
        raise ValueError("scale must have K/group columns")
    group = K // groups if K else 32
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    s = _dense(scale, "scale", torch.float16, None, dev)
    z = None if zero is None else _dense(zero, "zero", torch.float16, (N, groups), dev)
    out, c = _output(out, "out", dtype, (M, N), dev)
    ws, wp, wn = _workspace(workspace, gemm_w4g_workspace_bytes(M, N, K), dev)
    _enqueue("bq_gemm_w4g_a16", dev, a, dt, b, s, z, group, c, M, N, K, wp, wn)
    return out


def _rope_args(q, k, cos, sin, positions, q_weight, k_weight):
    dt = _dtype16(k, "k")
    if k.dim() != 3 or (q is not None and q.dim() != 3):
        raise ValueError("q and k must be 3-D [tokens, heads, head_dim]")
    shape = tokens, hkv, dim = k.shape
    dev, dtype = k.device, k.dtype
    ks = _rows(k, "k", dtype, shape, dev)
    hq, qs, qp = 0, 0, None
    if q is not None:
        hq, qp = q.shape[1], q.data_ptr()
        qs = _rows(q, "q", dtype, (tokens, hq, dim), dev)
    wq = None if q_weight is None else _dense(q_weight, "q_weight", dtype, (dim,), dev)
    wk = None if k_weight is None else _dense(k_weight, "k_weight", dtype, (dim,), dev)
    rot, max_pos, c, s, at = 0, 0, None, None, None
    if cos is not None:
        if sin is None or positions is None:
            raise ValueError("cos needs sin and positions")
        if cos.dim() != 2:
            raise ValueError("cos must be 2-D [max_pos, rot_dim/2]")
        max_pos, half = cos.shape
        rot = 2 * half
        c = _dense(cos, "cos", torch.float32, None, dev)
        s = _dense(sin, "sin", torch.float32, (max_pos, half), dev)
        at = _dense(positions, "positions", torch.int32, (tokens,), dev)
    return dt, dtype, dev, tokens, hq, hkv, dim, qp, qs, k.data_ptr(), ks, wq, wk, c, s, max_pos, rot, at


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, cos: Optional[torch.Tensor], sin: Optional[torch.Tensor],
                 positions: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """The norm of each head of q [tokens, q_heads, head_dim] and k [tokens,
    kv_heads, head_dim] (fp16 or bf16, dense within a token) with weights
    [head_dim] (None: no norm), and the rotation of the first rot_dim channels
    by cos / sin fp32 [max_pos, rot_dim/2] at positions int32 [tokens] (None:
    no rotation), in one pass -> (q_out, k_out).  A token whose position is
    outside the table is left out: its outputs are not written."""
    dt, dtype, dev, tokens, hq, hkv, dim, qp, qs, kp, ks, wq, wk, c, s, max_pos, rot, at = _rope_args(
        q, k, cos, sin, positions, q_weight, k_weight)
    q_out, qo = _output(q_out, "q_out", dtype, (tokens, hq, dim), dev)
    k_out, ko = _output(k_out, "k_out", dtype, (tokens, hkv, dim), dev)
    _enqueue("bq_qk_norm_rope", dev, qp, qs, kp, ks, dt, tokens, hq, hkv, dim, wq, wk, eps, c, s, max_pos, rot, interleaved, at,
             qo, ko)
    return q_out, k_out


def kv4_page_bytes(kv_heads: int, head_dim: int, page_size: int) -> int:
    """Bytes of a page of the 4-bit cache; a cache is a uint8 tensor
    [num_pages, kv4_page_bytes(...)] (its layout: include/bq_layer.h)."""
    return _host_bytes("bq_kv4_page_bytes", kv_heads, head_dim, page_size)


def _cache_ptr(cache, kv_heads, head_dim, page_size, dev) -> int:
    if not isinstance(cache, torch.Tensor) or cache.dim() != 2:
        raise ValueError("cache must be a 2-D tensor [num_pages, page bytes]")
    return _dense(cache, "cache", torch.uint8, (cache.shape[0], kv4_page_bytes(kv_heads, head_dim, page_size)), dev)


def qk_norm_rope_kv4(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, cos: Optional[torch.Tensor],
                     sin: Optional[torch.Tensor], positions: Optional[torch.Tensor], cache: torch.Tensor,
                     slots: torch.Tensor, page_size: int, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                     q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """qk_norm_rope with the keys (rounded to their type) and the values v
    written to the 4-bit cache at slots int64 [tokens] (page * page_size +
    offset, each at most once; outside the cache: not written) -> q_out.  q
    None: keys and values only."""
    dt, dtype, dev, tokens, hq, hkv, dim, qp, qs, kp, ks, wq, wk, c, s, max_pos, rot, at = _rope_args(
        q, k, cos, sin, positions, q_weight, k_weight)
    vs = _rows(v, "v", dtype, (tokens, hkv, dim), dev)
    pages = _cache_ptr(cache, hkv, dim, page_size, dev)
    sl = _dense(slots, "slots", torch.int64, (tokens,), dev)
    qo = None
    if q is not None:
        q_out, qo = _output(q_out, "q_out", dtype, (tokens, hq, dim), dev)
    _enqueue("bq_qk_norm_rope_kv4", dev, qp, qs, kp, ks, v.data_ptr(), vs, dt, tokens, hq, hkv, dim, wq, wk, eps, c, s, max_pos,
             rot, interleaved, at, qo, pages, cache.shape[0], page_size, sl)
    return q_out


def kv4_read(cache: torch.Tensor, slots: torch.Tensor, page_size: int, kv_heads: int, head_dim: int,
             dtype: torch.dtype = torch.float16, k_out: Optional[torch.Tensor] = None,
             v_out: Optional[torch.Tensor] = None):
    """The keys and values at slots int64 [tokens] of the 4-bit cache, dense
    [tokens, kv_heads, head_dim] of dtype -> (k, v).  A slot outside the cache
    leaves its rows as they were."""
    if dtype not in _DTYPES16:
        raise ValueError("dtype must be float16 or bfloat16")
    dev = cache.device
    pages = _cache_ptr(cache, kv_heads, head_dim, page_size, dev)
    if slots.dim() != 1:
        raise ValueError("slots must be 1-D")
    sl = _dense(slots, "slots", torch.int64, None, dev)
    shape = (slots.shape[0], kv_heads, head_dim)
    k_out, ko = _output(k_out, "k_out", dtype, shape, dev)
    v_out, vo = _output(v_out, "v_out", dtype, shape, dev)
    _enqueue("bq_kv4_read", dev, pages, cache.shape[0], page_size, kv_heads, head_dim, sl, shape[0], _DTYPES16[dtype], ko, vo)
    return k_out, v_out


def attn_kv4_workspace_bytes(batch: int, max_q_len: int, q_heads: int, kv_heads: int, head_dim: int, max_len: int) -> int:
    """Device workspace bytes with which attn_kv4 splits sequences of up to
    max_len keys (0: it does not)."""
    return _host_bytes("bq_attn_kv4_workspace_bytes", batch, max_q_len, q_heads, kv_heads, head_dim, max_len)


def attn_kv4(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, page_size: int,
             kv_heads: int, scale: Optional[float] = None, q_start: Optional[torch.Tensor] = None,
             max_q_len: Optional[int] = None, window: int = 0, out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None, return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """Attention of q [total_q, q_heads, head_dim] (fp16 or bf16, dense within
    a token) over the 4-bit cache: sequence b's queries stand at the end of
    its seq_lens[b] cached keys (int32 [batch]), found through block_table
    int32 [batch, max_blocks]; causal, within the last `window` keys if
    window > 0.  q_start int32 [batch + 1] gives each sequence's queries, of
    which the first max_q_len are computed (the others' outputs are not
    written); None: total_q / batch each.  scale None: head_dim ** -0.5.

    -> out, of q's shape and type; (out, lse) with return_lse or lse given:
    lse fp32 [total_q, q_heads].  A row with no keys gives zeros (lse -inf).
    A workspace is allocated for the call when it needs one and none is
    given."""
    dt = _dtype16(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be 3-D [total_q, q_heads, head_dim]")
    shape = total, hq, dim = q.shape
    dev, dtype = q.device, q.dtype
    qs = _rows(q, "q", dtype, shape, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be 2-D [batch, max_blocks]")
    batch, blocks = block_table.shape
    tab = _dense(block_table, "block_table", torch.int32, None, dev)
    lens = _dense(seq_lens, "seq_lens", torch.int32, (batch,), dev)
    pages = _cache_ptr(cache, kv_heads, dim, page_size, dev)
    starts = None
    if q_start is None:
        if total % batch if batch else total:
            raise ValueError("without q_start every sequence has total_q / batch queries")
        each = total // batch if batch else 0
        if max_q_len is not None and max_q_len != each:
            raise ValueError("max_q_len must be total_q / batch without q_start")
        max_q_len = each
    else:
        if max_q_len is None:
            raise ValueError("q_start needs max_q_len")
        starts = _dense(q_start, "q_start", torch.int32, (batch + 1,), dev)
    out, o = _output(out, "out", dtype, shape, dev)
    e = None
    if lse is not None or return_lse:
        lse, e = _output(lse, "lse", torch.float32, (total, hq), dev)
    ws, wp, wn = _workspace(workspace, attn_kv4_workspace_bytes(batch, max_q_len, hq, kv_heads, dim, blocks * page_size), dev)
    _enqueue("bq_attn_kv4", dev, q.data_ptr(), qs, dt, starts, lens, tab, batch, total, max_q_len, hq, kv_heads, dim, pages,
             cache.shape[0], page_size, blocks, dim ** -0.5 if scale is None else scale, window, o, e, wp, wn)
    return out if lse is None else (out, lse)
