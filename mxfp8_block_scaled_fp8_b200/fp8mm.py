"""Python binding of ``libfp8mm.so`` (the C ABI in ``include/fp8mm.h``).

Argument marshalling only: every step of the quantizers and GEMMs runs in the
library's CUDA kernels.  torch supplies device memory and the current stream.
There is no fallback: if the library is missing or a call fails, an
``Fp8mmError`` is raised.

E4M3 operands are uint8 tensors holding the codes (a ``torch.float8_e4m3fn``
tensor is accepted too and viewed as uint8).  B is passed as [n, k] (K
contiguous), i.e. the transpose of the pages' logical [k, n].
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8mm.so")

FP8MM_OK = 0
FP8MM_ERR_DEVICE = 7
KERNEL_AUTO, KERNEL_TILED, KERNEL_SMALL_M, KERNEL_TILED_1SM, KERNEL_TILED_2SM, KERNEL_TILED_1SM_N128 = 0, 1, 2, 3, 4, 5


class Fp8mmError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        msg = f"{fn} failed: status {status}"
        if _lib is not None:
            msg += f" ({_lib.fp8mm_status_str(status).decode()})"
        if detail:
            msg += f"; {detail}"
        super().__init__(msg)


FLAG_WEIGHTS_READY = 1
FLAG_SPLIT_VIA_WORKSPACE = 2
FLAG_SF_A_8X4 = 4


class Opts(ctypes.Structure):
    _fields_ = [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("kernel", ctypes.c_int32), ("small_m_ctas", ctypes.c_int32), ("flags", ctypes.c_uint32)]


# fp8mm_kv_cache of the header: pages, page_stride, num_pages, page_size, kv_heads, head_dim, page_table,
# table_stride, max_pages, batch
KV_CACHE_DESC = struct.Struct("@PqqqqqPqqq")


_lib = None
_P, _I64, _U8P = ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p

_SIGNATURES = {
    "fp8_quantize_rowwise": ([_P, _I64, _I64, _I64, _P, _I64, _P, _P], ctypes.c_int),
    "mxfp8_quantize": ([_P, _I64, _I64, _I64, _P, _I64, _P, _P], ctypes.c_int),
    "fp8_gemm": ([_P, _P, _I64, _I64, _I64, _P, _P, _P, _I64, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "fp8_tensor_scale": ([_P, _I64, _I64, _I64, _P, _P], ctypes.c_int),
    "fp8_quantize_static": ([_P, _I64, _I64, _I64, _P, _P, _I64, _P], ctypes.c_int),
    "fp8_gemm_e4m3_out": ([_P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _I64, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mxfp8_gemm": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mxfp8_quantize_gemm": ([_P, _I64, _P, _P, _I64, _I64, _I64, _P, _I64, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "concat_mla_k": ([_P, _P, _P] + [_I64] * 11 + [_P], ctypes.c_int),
    "qk_norm_rope": ([_P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, ctypes.c_float, _P, _I64, _I64,
                      _I64, ctypes.c_int32, _P, _P, _I64, _I64, _P, _I64, _I64, _P], ctypes.c_int),
    "mxfp4_kv_page_bytes": ([_I64, _I64, _I64], ctypes.c_size_t),
    "mxfp4_kv_append": ([_P, _I64, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _P], ctypes.c_int),
    "mxfp4_kv_gather": ([_P, _P, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, _P], ctypes.c_int),
    "mxfp4_kv_attention": ([_P, _I64, _I64, _I64, _I64, _P, _P, _P, ctypes.c_float, _P, _I64,
                            _I64, _P, _I64, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "mxfp4_kv_attention_workspace_bytes": ([_I64], ctypes.c_size_t),
    "kv_copy_pages": ([_P, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64, _P], ctypes.c_int),
    "fp8mm_sf_bytes": ([_I64, _I64], ctypes.c_size_t),
    "fp8mm_sf_offset": ([_I64, _I64, _I64, _I64], ctypes.c_int64),
    "fp8mm_sf8x4_bytes": ([_I64, _I64], ctypes.c_size_t),
    "fp8mm_sf8x4_offset": ([_I64, _I64, _I64, _I64], ctypes.c_int64),
    "mxfp8_quantize_8x4": ([_P, _I64, _I64, _I64, _P, _I64, _P, _P], ctypes.c_int),
    "fp8mm_sf_to_canonical": ([_P, _I64, _I64, _P], ctypes.c_int),
    "fp8mm_sf_from_canonical": ([_P, _I64, _I64, _P], ctypes.c_int),
    "fp8mm_workspace_bytes": ([_I64, _I64, _I64, ctypes.c_int32], ctypes.c_size_t),
    "fp8mm_pair_split_plan": ([_I64, _I64, _I64, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int32),
    "fp8mm_quantize_gemm_workspace_bytes": ([_I64, _I64, _I64, ctypes.c_int32], ctypes.c_size_t),
    "fp8mm_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "fp8mm_last_cuda_error": ([], ctypes.c_int),
    "fp8mm_last_device_error": ([], ctypes.c_uint),
    "fp8mm_selftest_wait_timeout": ([ctypes.c_uint32, _P], ctypes.c_int),
    "fp8mm_version": ([], ctypes.c_int),
}


def lib():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise Fp8mmError("load", -1, f"{LIB_PATH} is not built; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != FP8MM_OK:
        raise Fp8mmError(fn, status, f"cuda error {lib().fp8mm_last_cuda_error()}")


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _u8(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _need(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name}: expected a CUDA {dtype} tensor, got {t.dtype} on {t.device}")


def _ld(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name}: expected a 2-D tensor with unit column stride")
    return t.stride(0)


# ----------------------------------------------------------------- mode 1

def fp8_quantize_rowwise(x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                         stream=None):
    """bf16 [rows, k] -> (E4M3 codes uint8 [rows, k], fp32 scale [rows])."""
    _need(x, torch.bfloat16, "x")
    rows, k = x.shape
    if q is None:
        q = torch.empty((rows, k), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty((rows,), dtype=torch.float32, device=x.device)
    q = _u8(q)
    _check("fp8_quantize_rowwise", lib().fp8_quantize_rowwise(
        x.data_ptr(), rows, k, _ld(x, "x"), q.data_ptr(), _ld(q, "q"), scale.data_ptr(), _stream(stream)))
    return q, scale


def _ws_opts(workspace, kernel, small_m_ctas=0, flags=0):
    return Opts(workspace.data_ptr() if workspace is not None else None,
                workspace.numel() * workspace.element_size() if workspace is not None else 0,
                kernel, small_m_ctas, flags)


def fp8_gemm(a: torch.Tensor, b: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
             c: torch.Tensor | None = None, kernel: int = KERNEL_AUTO, stream=None,
             workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C bf16 [m, n] = diag(scale_a) (A x B^T) diag(scale_b); a [m,k], b [n,k] E4M3 codes.
    workspace (zeroed once, workspace_bytes(m, n, k) bytes): lets m > 64 shapes split the K range of the
    tiles of their last, partly filled wave of SM pairs over the pairs."""
    a, b = _u8(a), _u8(b)
    _need(a, torch.uint8, "a"); _need(b, torch.uint8, "b")
    _need(scale_a, torch.float32, "scale_a"); _need(scale_b, torch.float32, "scale_b")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a [m,k] and b [n,k] must be contiguous with the same k")
    if c is None:
        c = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    opts = _ws_opts(workspace, kernel)
    _check("fp8_gemm", lib().fp8_gemm(a.data_ptr(), b.data_ptr(), m, n, k, scale_a.data_ptr(), scale_b.data_ptr(),
                                      c.data_ptr(), _ld(c, "c"), ctypes.byref(opts), _stream(stream)))
    return c


# ----------------------------------------------------------------- per tensor, FP8 out

def fp8_tensor_scale(x: torch.Tensor, scale: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 [rows, k] -> fp32 [1] device scale = max|x| / 448 over the whole tensor (1 if all zero)."""
    _need(x, torch.bfloat16, "x")
    rows, k = x.shape
    if scale is None:
        scale = torch.empty((1,), dtype=torch.float32, device=x.device)
    _check("fp8_tensor_scale", lib().fp8_tensor_scale(x.data_ptr(), rows, k, _ld(x, "x") if k else k,
                                                      scale.data_ptr(), _stream(stream)))
    return scale


def fp8_quantize_static(x: torch.Tensor, scale: torch.Tensor, q: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """bf16 [rows, k] and a device fp32 scale -> E4M3 codes uint8 [rows, k] of x / scale."""
    _need(x, torch.bfloat16, "x"); _need(scale, torch.float32, "scale")
    rows, k = x.shape
    if q is None:
        q = torch.empty((rows, k), dtype=torch.uint8, device=x.device)
    q = _u8(q)
    _check("fp8_quantize_static", lib().fp8_quantize_static(x.data_ptr(), rows, k, _ld(x, "x"), scale.data_ptr(),
                                                            q.data_ptr(), _ld(q, "q"), _stream(stream)))
    return q


def fp8_gemm_e4m3_out(a: torch.Tensor, b: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
                      scale_out: torch.Tensor, c: torch.Tensor | None = None, kernel: int = KERNEL_AUTO,
                      stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """E4M3 codes uint8 [m, n] of diag(scale_a) (A x B^T) diag(scale_b) / scale_out (workspace as fp8_gemm)."""
    a, b = _u8(a), _u8(b)
    _need(a, torch.uint8, "a"); _need(b, torch.uint8, "b")
    _need(scale_a, torch.float32, "scale_a"); _need(scale_b, torch.float32, "scale_b")
    _need(scale_out, torch.float32, "scale_out")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a [m,k] and b [n,k] must be contiguous with the same k")
    if c is None:
        c = torch.empty((m, n), dtype=torch.uint8, device=a.device)
    c = _u8(c)
    opts = _ws_opts(workspace, kernel)
    _check("fp8_gemm_e4m3_out", lib().fp8_gemm_e4m3_out(
        a.data_ptr(), b.data_ptr(), m, n, k, scale_a.data_ptr(), scale_b.data_ptr(), scale_out.data_ptr(),
        c.data_ptr(), _ld(c, "c"), ctypes.byref(opts), _stream(stream)))
    return c


# ----------------------------------------------------------------- mode 2

def sf_bytes(rows: int, k: int) -> int:
    return int(lib().fp8mm_sf_bytes(rows, k))


def sf_offset(rows: int, k: int, row: int, block: int) -> int:
    return int(lib().fp8mm_sf_offset(rows, k, row, block))


def sf_to_canonical(sf: torch.Tensor, rows: int, k: int) -> torch.Tensor:
    """Library scale layout (CPU uint8 tensor) -> canonical [rows, k/32] (CPU)."""
    src = sf.detach().cpu().contiguous()
    out = torch.empty((rows, k // 32), dtype=torch.uint8)
    _check("fp8mm_sf_to_canonical", lib().fp8mm_sf_to_canonical(src.data_ptr(), rows, k, out.data_ptr()))
    return out


def sf_from_canonical(canonical: torch.Tensor, rows: int, k: int) -> torch.Tensor:
    """Canonical [rows, k/32] (CPU uint8) -> library scale layout (CPU)."""
    src = canonical.detach().cpu().contiguous()
    out = torch.empty((sf_bytes(rows, k),), dtype=torch.uint8)
    _check("fp8mm_sf_from_canonical", lib().fp8mm_sf_from_canonical(src.data_ptr(), rows, k, out.data_ptr()))
    return out


def mxfp8_quantize(x: torch.Tensor, q: torch.Tensor | None = None, sf: torch.Tensor | None = None, stream=None):
    """bf16 [rows, k] -> (E4M3 codes uint8 [rows, k], scales uint8 [sf_bytes] in the library layout)."""
    _need(x, torch.bfloat16, "x")
    rows, k = x.shape
    if q is None:
        q = torch.empty((rows, k), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty((max(sf_bytes(rows, k), 1),), dtype=torch.uint8, device=x.device)
    q = _u8(q)
    _check("mxfp8_quantize", lib().mxfp8_quantize(x.data_ptr(), rows, k, _ld(x, "x"), q.data_ptr(), _ld(q, "q"),
                                                  sf.data_ptr(), _stream(stream)))
    return q, sf


def sf8x4_bytes(rows: int, k: int) -> int:
    return int(lib().fp8mm_sf8x4_bytes(rows, k))


def sf8x4_offset(rows: int, k: int, row: int, block: int) -> int:
    return int(lib().fp8mm_sf8x4_offset(rows, k, row, block))


def mxfp8_quantize_8x4(x: torch.Tensor, q: torch.Tensor | None = None, sf: torch.Tensor | None = None,
                       stream=None):
    """mxfp8_quantize with the scales in the small-M (8x4) layout: (codes uint8 [rows, k],
    scales uint8 [sf8x4_bytes]); for activations of a few token rows fed to mxfp8_gemm(sf_a_8x4=True)."""
    _need(x, torch.bfloat16, "x")
    rows, k = x.shape
    if q is None:
        q = torch.empty((rows, k), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty((max(sf8x4_bytes(rows, k), 1),), dtype=torch.uint8, device=x.device)
    q = _u8(q)
    _check("mxfp8_quantize_8x4", lib().mxfp8_quantize_8x4(x.data_ptr(), rows, k, _ld(x, "x"), q.data_ptr(),
                                                          _ld(q, "q"), sf.data_ptr(), _stream(stream)))
    return q, sf


def workspace_bytes(m: int, n: int, k: int, ctas: int = 0) -> int:
    return int(lib().fp8mm_workspace_bytes(m, n, k, ctas))


def pair_split_plan(m: int, n: int, k: int, pairs: int) -> tuple[int, int]:
    """(K parts per split tile, tiles run whole) of the paired kernel's split with `pairs` SM pairs."""
    dp = ctypes.c_int32(0)
    split = int(lib().fp8mm_pair_split_plan(m, n, k, pairs, ctypes.byref(dp)))
    return split, int(dp.value)


def quantize_gemm_workspace_bytes(m: int, n: int, k: int, ctas: int = 0) -> int:
    return int(lib().fp8mm_quantize_gemm_workspace_bytes(m, n, k, ctas))


def mxfp8_gemm(a: torch.Tensor, sf_a: torch.Tensor, b: torch.Tensor, sf_b: torch.Tensor,
               c: torch.Tensor | None = None, workspace: torch.Tensor | None = None, kernel: int = KERNEL_AUTO,
               small_m_ctas: int = 0, weights_ready: bool = False, stream=None,
               split_via_workspace: bool = False, sf_a_8x4: bool = False) -> torch.Tensor:
    """C bf16 [m, n] = block-scaled A x B^T; a [m,k], b [n,k] codes with their library-layout scales.
    workspace (zeroed once, workspace_bytes(m, n, k, small_m_ctas) bytes): the small-M kernel's stream-K
    split for m <= 64 where the CTA count is not tile-aligned (aligned splits reduce inside clusters);
    for m > 64 the K split of the tiles of the last, partly filled wave of SM pairs.
    weights_ready: b and sf_b were complete before the preceding kernel on the stream started (see
    FP8MM_FLAG_WEIGHTS_READY).  split_via_workspace: FP8MM_FLAG_SPLIT_VIA_WORKSPACE.  sf_a_8x4: sf_a is in
    the small-M layout of mxfp8_quantize_8x4 (m <= 64 only)."""
    a, b = _u8(a), _u8(b)
    _need(a, torch.uint8, "a"); _need(b, torch.uint8, "b")
    _need(sf_a, torch.uint8, "sf_a"); _need(sf_b, torch.uint8, "sf_b")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a [m,k] and b [n,k] must be contiguous with the same k")
    if c is None:
        c = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    flags = ((FLAG_WEIGHTS_READY if weights_ready else 0) | (FLAG_SPLIT_VIA_WORKSPACE if split_via_workspace else 0)
             | (FLAG_SF_A_8X4 if sf_a_8x4 else 0))
    opts = _ws_opts(workspace, kernel, small_m_ctas, flags)
    _check("mxfp8_gemm", lib().mxfp8_gemm(a.data_ptr(), sf_a.data_ptr(), b.data_ptr(), sf_b.data_ptr(), m, n, k,
                                          c.data_ptr(), _ld(c, "c"), ctypes.byref(opts), _stream(stream)))
    return c


def mxfp8_quantize_gemm(a: torch.Tensor, b: torch.Tensor, sf_b: torch.Tensor, c: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, kernel: int = KERNEL_AUTO, small_m_ctas: int = 0,
                        weights_ready: bool = False, stream=None, split_via_workspace: bool = False) -> torch.Tensor:
    """C bf16 [m, n] = mxfp8_gemm(mxfp8_quantize(a), b) for m <= 64 from the bf16 activation a [m, k]:
    quantized inside the GEMM kernel for m <= 8, else by its own launch into the workspace tail
    (workspace of quantize_gemm_workspace_bytes(m, n, k, small_m_ctas) bytes, required for m > 8)."""
    b = _u8(b)
    _need(a, torch.bfloat16, "a"); _need(b, torch.uint8, "b"); _need(sf_b, torch.uint8, "sf_b")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or not b.is_contiguous():
        raise ValueError("b [n,k] must be contiguous with the k of a")
    if c is None:
        c = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    opts = Opts(workspace.data_ptr() if workspace is not None else None,
                workspace.numel() * workspace.element_size() if workspace is not None else 0,
                kernel, small_m_ctas,
                (FLAG_WEIGHTS_READY if weights_ready else 0) | (FLAG_SPLIT_VIA_WORKSPACE if split_via_workspace else 0))
    _check("mxfp8_quantize_gemm", lib().mxfp8_quantize_gemm(
        a.data_ptr(), _ld(a, "a"), b.data_ptr(), sf_b.data_ptr(), m, n, k, c.data_ptr(), _ld(c, "c"),
        ctypes.byref(opts), _stream(stream)))
    return c


# ----------------------------------------------------------------- KV cache

def concat_mla_k(k_nope: torch.Tensor, k_rope: torch.Tensor, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """k_nope [T, H, nope], k_rope [T, H or 1, rope] (1 = one rope vector per token for all heads)
    -> out [T, H, nope + rope]; 1-byte (float8 / uint8) or 2-byte elements, any 16-byte-aligned strides."""
    if k_nope.dim() != 3 or k_rope.dim() != 3 or not k_nope.is_cuda or not k_rope.is_cuda:
        raise ValueError("k_nope and k_rope must be 3-D CUDA tensors")
    if k_nope.element_size() != k_rope.element_size() or k_nope.dtype != k_rope.dtype:
        raise TypeError("k_nope and k_rope must have the same dtype")
    T, H, dn = k_nope.shape
    dr = k_rope.shape[2]
    if k_rope.shape[0] != T or k_rope.shape[1] not in (1, H) or k_nope.stride(2) != 1 or k_rope.stride(2) != 1:
        raise ValueError("k_rope must be [T, H or 1, rope] with unit element stride, k_nope unit element stride")
    if out is None:
        out = torch.empty((T, H, dn + dr), dtype=k_nope.dtype, device=k_nope.device)
    if out.shape != (T, H, dn + dr) or out.stride(2) != 1 or out.dtype != k_nope.dtype:
        raise ValueError("out must be [T, H, nope + rope] of the input dtype with unit element stride")
    rope_sh = 0 if k_rope.shape[1] == 1 else k_rope.stride(1)
    _check("concat_mla_k", lib().concat_mla_k(
        k_nope.data_ptr(), k_rope.data_ptr(), out.data_ptr(), T, H, dn, dr, k_nope.element_size(),
        k_nope.stride(0), k_nope.stride(1), k_rope.stride(0), rope_sh, out.stride(0), out.stride(1),
        _stream(stream)))
    return out


# ----------------------------------------------------------------- MXFP4 key/value cache in pages

# These calls run on the tensors' device and, with stream=None, on its current stream, whichever device is
# current.  Their checks are written for a call every few microseconds: a decode step makes three per layer.
_BF16, _I32, _F32, _BYTE = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_current, _raw = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


class _on:
    """Makes device ``index`` and ``stream`` (None: the device's current one) current, also for the allocator."""

    def __init__(self, index: int, stream):
        if stream is not None and stream.device.index != index:
            raise ValueError(f"stream of {stream.device}, tensors on cuda:{index}")
        self.ctx = torch.cuda.device(index) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        return self.ctx.__enter__()

    def __exit__(self, *exc):
        return self.ctx.__exit__(*exc)


def _device(t: torch.Tensor, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise TypeError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return index


def _tensor(t, dtype, index: int, name: str, shape=None, dims: int = 1):
    """Checks of one tensor argument: type, device, shape (or dimensions), unit stride of the last dimension."""
    if t.dtype is not dtype or t.get_device() != index:
        raise TypeError(f"{name}: expected a {dtype} tensor on cuda:{index}, got {t.dtype} on {t.device}")
    got = t.shape
    if shape is not None and got != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(got)}")
    if shape is None and len(got) != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got shape {tuple(got)}")
    if got[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: expected unit stride in the last dimension")


def _heads(t, index: int, name: str, shape=None):
    """[rows, heads, dim] bf16 -> pointer, row stride, head stride; those of one row, or one head, say nothing."""
    _tensor(t, _BF16, index, name, shape, 3)
    n, h, d = t.shape
    st = t.stride()
    return t.data_ptr(), st[0] if n > 1 else h * d, st[1] if h > 1 else d


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, cos_sin: torch.Tensor, positions: torch.Tensor,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 stream=None):
    """RMS norm (with both weights [dim] bf16, or without a norm) and position rotation of each head of
    q [T, q_heads, dim] and k [T, k_heads, dim] bf16 (strided views are taken): (q_out, k_out), new tensors unless
    given (q and k themselves: in place).  cos_sin [max_pos, rot] fp32: rot / 2 cosines, then the sines;
    positions int32 [T], negative for a padding row, which is left as it was."""
    dev = _device(q, "q")
    if stream is not None or _current() != dev:
        with _on(dev, stream):
            return qk_norm_rope(q, k, cos_sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out)
    qa, ka = _heads(q, dev, "q"), _heads(k, dev, "k")
    (t, hq, d), (tk, hk, dk) = q.shape, k.shape
    if tk != t or dk != d:
        raise ValueError("q and k must have the same tokens and dim")
    _tensor(cos_sin, _F32, dev, "cos_sin", None, 2)
    _tensor(positions, _I32, dev, "positions", (t,))
    qw = kw = None
    if q_weight is not None:
        _tensor(q_weight, _BF16, dev, "q_weight", (d,))
        qw = q_weight.data_ptr()
    if k_weight is not None:
        _tensor(k_weight, _BF16, dev, "k_weight", (d,))
        kw = k_weight.data_ptr()
    if q_out is None:
        q_out = q.new_empty((t, hq, d))
        qo = q_out.data_ptr(), hq * d, d
    else:
        qo = _heads(q_out, dev, "q_out", q.shape)
    if k_out is None:
        k_out = k.new_empty((t, hk, d))
        ko = k_out.data_ptr(), hk * d, d
    else:
        ko = _heads(k_out, dev, "k_out", k.shape)
    cs = cos_sin.shape
    _check("qk_norm_rope", lib().qk_norm_rope(
        *qa, *ka, t, hq, hk, d, qw, kw, eps, cos_sin.data_ptr(), cs[0], cs[1], cos_sin.stride(0) if cs[0] > 1 else cs[1],
        1 if interleaved else 0, positions.data_ptr(), *qo, *ko, _raw(dev)))
    return q_out, k_out


def mxfp4_kv_page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of a cache page of page_size tokens (0: not supported)."""
    return int(lib().mxfp4_kv_page_bytes(page_size, kv_heads, head_dim))


def _kv_cache(cache, page_table, page_size: int, head_dim: int, dev: int):
    """(heads, batch, the cache's description for the library) of cache uint8 [pages, page_bytes] and page_table
    int32 [batch, pages]."""
    _tensor(cache, _BYTE, dev, "cache", None, 2)
    _tensor(page_table, _I32, dev, "page_table", None, 2)
    (pages, size), (batch, most) = cache.shape, page_table.shape
    one = page_size // 16 * 17 * head_dim
    if one <= 0 or size % one != 0 or size == 0:
        raise ValueError(f"cache: pages of {size} bytes do not hold {page_size} tokens of whole heads of {head_dim}")
    return size // one, batch, KV_CACHE_DESC.pack(
        cache.data_ptr(), cache.stride(0) if pages > 1 else size, pages, page_size, size // one, head_dim,
        page_table.data_ptr(), page_table.stride(0) if batch > 1 else most, most, batch)


def mxfp4_kv_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor,
                    seq_lens: torch.Tensor, page_size: int, cu_seqlens: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Quantizes new keys and values [T, kv_heads, dim] bf16 into the MXFP4 cache uint8 [pages, page_bytes]: rows
    cu_seqlens[s]..cu_seqlens[s + 1] (None: row s) become the last tokens of sequence s, whose length with them
    is seq_lens[s] (int32; 0: a padding sequence).  Returns the cache."""
    dev = _device(cache, "cache")
    if stream is not None or _current() != dev:
        with _on(dev, stream):
            return mxfp4_kv_append(k, v, cache, page_table, seq_lens, page_size, cu_seqlens)
    ka, va = _heads(k, dev, "k"), _heads(v, dev, "v", k.shape)
    t, h, d = k.shape
    heads, batch, desc = _kv_cache(cache, page_table, page_size, d, dev)
    if heads != h:
        raise ValueError(f"cache: pages hold {heads} heads, not {h}")
    cu = None
    if cu_seqlens is not None:
        _tensor(cu_seqlens, _I32, dev, "cu_seqlens", (batch + 1,))
        cu = cu_seqlens.data_ptr()
    _tensor(seq_lens, _I32, dev, "seq_lens", (batch,))
    _check("mxfp4_kv_append", lib().mxfp4_kv_append(*ka, *va, t, cu, seq_lens.data_ptr(), desc, _raw(dev)))
    return cache


def mxfp4_kv_gather(cache: torch.Tensor, page_table: torch.Tensor, cu_seqlens: torch.Tensor, page_size: int,
                    head_dim: int, total: int, starts: torch.Tensor | None = None, k: torch.Tensor | None = None,
                    v: torch.Tensor | None = None, stream=None):
    """Cached keys and values as bf16 [total, kv_heads, head_dim] each: rows cu_seqlens[s]..cu_seqlens[s + 1] are
    the tokens of sequence s from starts[s] (None: 0) on."""
    dev = _device(cache, "cache")
    if stream is not None or _current() != dev:
        with _on(dev, stream):
            return mxfp4_kv_gather(cache, page_table, cu_seqlens, page_size, head_dim, total, starts, k, v)
    heads, batch, desc = _kv_cache(cache, page_table, page_size, head_dim, dev)
    _tensor(cu_seqlens, _I32, dev, "cu_seqlens", (batch + 1,))
    st = None
    if starts is not None:
        _tensor(starts, _I32, dev, "starts", (batch,))
        st = starts.data_ptr()
    shape = (total, heads, head_dim)
    if k is None:
        k = cache.new_empty(shape, dtype=_BF16)
        ka = k.data_ptr(), heads * head_dim, head_dim
    else:
        ka = _heads(k, dev, "k", shape)
    if v is None:
        v = cache.new_empty(shape, dtype=_BF16)
        va = v.data_ptr(), heads * head_dim, head_dim
    else:
        va = _heads(v, dev, "v", shape)
    _check("mxfp4_kv_gather", lib().mxfp4_kv_gather(desc, st, cu_seqlens.data_ptr(), total, *ka, *va, _raw(dev)))
    return k, v


def mxfp4_kv_attention_workspace_bytes(head_dim: int) -> int:
    return int(lib().mxfp4_kv_attention_workspace_bytes(head_dim))


def mxfp4_kv_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                       page_size: int, cu_seqlens: torch.Tensor | None = None, scale: float | None = None,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of q [T, q_heads, dim] bf16, the last tokens of each sequence, over the MXFP4 cache: bf16
    [T, q_heads, dim].  Rows cu_seqlens[s]..cu_seqlens[s + 1] (None: row s) stand at the last positions of
    sequence s, whose length is seq_lens[s]; scale None: dim ** -0.5.  lse: fp32 [T, q_heads] to fill.
    workspace (zeroed once, mxfp4_kv_attention_workspace_bytes(dim) bytes): lets long sequences be cut over the SMs."""
    dev = _device(cache, "cache")
    if stream is not None or _current() != dev:
        with _on(dev, stream):
            return mxfp4_kv_attention(q, cache, page_table, seq_lens, page_size, cu_seqlens, scale, out, lse, workspace)
    qa = _heads(q, dev, "q")
    t, hq, d = q.shape
    _, batch, desc = _kv_cache(cache, page_table, page_size, d, dev)
    cu = lp = ws = None
    lst = wsb = 0
    if cu_seqlens is not None:
        _tensor(cu_seqlens, _I32, dev, "cu_seqlens", (batch + 1,))
        cu = cu_seqlens.data_ptr()
    _tensor(seq_lens, _I32, dev, "seq_lens", (batch,))
    if lse is not None:
        _tensor(lse, _F32, dev, "lse", (t, hq))
        lp, lst = lse.data_ptr(), lse.stride(0) if t > 1 else hq
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise TypeError(f"workspace: expected a contiguous tensor on cuda:{dev}")
        ws, wsb = workspace.data_ptr(), workspace.nbytes
    if out is None:
        out = q.new_empty((t, hq, d))
        oa = out.data_ptr(), hq * d, d
    else:
        oa = _heads(out, dev, "out", q.shape)
    _check("mxfp4_kv_attention", lib().mxfp4_kv_attention(
        *qa, t, hq, cu, seq_lens.data_ptr(), desc, d ** -0.5 if scale is None else scale,
        *oa, lp, lst, ws, wsb, _raw(dev)))
    return out


def kv_copy_pages(cache: torch.Tensor, src, dst, stream=None) -> torch.Tensor:
    """Copies pages dst[i] <- src[i] (sequences or CPU tensors of page ids) in every layer of the cache
    [pages, n] or [layers, pages, n] of any type.  No page may be written twice, or read and written.
    Returns the cache."""
    dev = _device(cache, "cache")
    if stream is not None or _current() != dev:
        with _on(dev, stream):
            return kv_copy_pages(cache, src, dst)
    shape, st = cache.shape, cache.stride()
    if len(shape) not in (2, 3) or (shape[-1] > 1 and st[-1] != 1):
        raise ValueError("cache: expected [pages, n] or [layers, pages, n] with unit stride in n")
    n = len(src)
    if len(dst) != n:
        raise ValueError("src and dst must have the same length")
    try:
        ids = struct.pack(f"@{2 * n}i", *_ids(src), *_ids(dst))
    except struct.error as e:
        raise ValueError(f"page ids: {e}") from None
    at = ctypes.cast(ids, _P).value
    size = cache.element_size()
    layers = shape[0] if len(shape) == 3 else 1
    layer_stride = st[0] * size if layers > 1 else 0
    _check("kv_copy_pages", lib().kv_copy_pages(cache.data_ptr(), shape[-2], shape[-1] * size, st[-2] * size, layers,
                                                layer_stride, at, at + 4 * n, n, _raw(dev)))
    return cache


def _ids(x):
    return x.tolist() if hasattr(x, "tolist") else x


# ----------------------------------------------------------------- misc

def last_device_error() -> int:
    return int(lib().fp8mm_last_device_error())


def selftest_wait_timeout(timeout_us: int = 2000, stream=None) -> int:
    return int(lib().fp8mm_selftest_wait_timeout(timeout_us, _stream(stream)))


def version() -> int:
    return int(lib().fp8mm_version())
