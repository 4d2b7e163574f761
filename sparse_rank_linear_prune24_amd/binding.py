"""Thin ctypes binding of libsplr.so (C ABI in include/splr.h).

Argument marshalling only: tensors are passed as device pointers together with torch's current
HIP stream; every step of the computation runs in the library's kernels. There is no fallback:
if the library is missing or a call fails, an exception is raised.

Conventions: bf16 tensors are torch.bfloat16, fp32 tensors torch.float32; metadata is int32
(the bits of the library's uint32 words). Packed S uses the library's tiled layout (16 rows x 64
input columns per tile, see include/splr.h): values are shaped (TR, TK, 64, 8) and metadata
(TR, TKB, 64, 4) (blocks of 8 tile columns), TR = ceil(n_out / 16), TK = ceil(n_in / 64),
TKB = ceil(TK / 8). The layer's n_out is passed
explicitly where it cannot be read off U.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import List, Optional, Sequence, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsplr.so")

SPLR_FP32, SPLR_BF16, SPLR_E4M3 = 0, 1, 2
STATUS = {0: "SPLR_OK", 1: "SPLR_ERR_NULL", 2: "SPLR_ERR_SHAPE", 3: "SPLR_ERR_DTYPE", 4: "SPLR_ERR_ALIGN",
          5: "SPLR_ERR_HIP", 6: "SPLR_ERR_WORKSPACE", 7: "SPLR_ERR_SCRATCH", 8: "SPLR_ERR_OVERLAP"}
EXPORTS = ("splr_prune24_pack", "splr_prune_nm_pack", "splr_linear_ex", "splr_prune24_pack_scaled", "splr_prune24_pack_residual", "splr_packed_bytes", "splr_linear_workspace_bytes", "splr_linear",
           "splr_linear_stage1", "splr_linear_stage2", "splr_linear_stage2_dense", "splr_linear_group",
           "splr_linear_stage2_group", "splr_linear_noalloc", "splr_linear_fused", "splr_linear_experts",
           "splr_linear_fused_workspace_bytes", "splr_linear_experts_workspace_bytes", "splr_linear_fused_tile", "splr_dense_reconstruct",
           "splr_tokens_dispatch", "splr_tokens_dispatch_workspace_bytes", "splr_tokens_gather", "splr_tokens_combine",
           "splr_tokens_combine_backward", "splr_fp8_quantize", "splr_linear_fp8", "splr_linear_fp8_experts",
           "splr_linear_fp8_workspace_bytes", "splr_linear_fp8_tile",
           "splr_gram_workspace_bytes", "splr_gram_f64", "splr_chol_rinv", "splr_status_string", "splr_version")

_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_lib = None


class SplrError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")


def lib() -> ctypes.CDLL:
    """The loaded library with argument types declared (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_rank_linear_prune24_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.splr_prune24_pack.argtypes = [_P, _I64, _I64, _I32, _P, _P, _P]
        L.splr_prune24_pack.restype = _I32
        L.splr_prune24_pack_scaled.argtypes = [_P, _P, _I64, _I64, _I32, _P, _P, _P]
        L.splr_prune_nm_pack.argtypes = [_P, _I64, _I64, _I32, _I32, _I32, _P, _P, _P]
        L.splr_prune_nm_pack.restype = _I32
        L.splr_prune24_pack_scaled.restype = _I32
        L.splr_prune24_pack_residual.argtypes = [_P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P]
        L.splr_prune24_pack_residual.restype = _I32
        L.splr_packed_bytes.argtypes = [_I64, _I64, _I32, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]
        L.splr_packed_bytes.restype = _I32
        L.splr_linear_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, _I32]
        L.splr_linear_workspace_bytes.restype = _SZ
        L.splr_linear.argtypes = [_P, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _I32, _P, _P, _SZ, _P]
        L.splr_linear_ex.argtypes = [_P, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _I32, _I32, _P, _P, _SZ, _P]
        L.splr_linear_ex.restype = _I32
        L.splr_linear.restype = _I32
        L.splr_linear_stage1.argtypes = [_P, _I64, _I64, _P, _I64, _I32, _P, _SZ, _P]
        L.splr_linear_stage1.restype = _I32
        L.splr_linear_stage2.argtypes = [_P, _I64, _I64, _P, _P, _I64, _P, _I64, _I32, _P, _P, _SZ, _P]
        L.splr_linear_stage2.restype = _I32
        L.splr_linear_stage2_dense.argtypes = [_P, _I64, _I64, _P, _P, _I64, _P, _I64, _I32, _P, _P, _SZ, _P]
        L.splr_linear_stage2_dense.restype = _I32
        L.splr_linear_group.argtypes = [_I32, _P, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _I32, _P, _P, _SZ, _P]
        L.splr_linear_group.restype = _I32
        L.splr_linear_stage2_group.argtypes = [_I32, _P, _I64, _I64, _P, _P, _I64, _P, _I64, _I32, _P, _P, _SZ, _P]
        L.splr_linear_stage2_group.restype = _I32
        L.splr_linear_noalloc.argtypes = [_P, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _I32, _P, _P]
        L.splr_linear_noalloc.restype = _I32
        L.splr_linear_fused.argtypes = [_P, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _I32, _P, _I32, _P, _P, _SZ, _P]
        L.splr_linear_fused.restype = _I32
        L.splr_linear_fused_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, _I32]
        L.splr_linear_fused_workspace_bytes.restype = _SZ
        L.splr_linear_experts_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, _I64, _I32]
        L.splr_linear_experts_workspace_bytes.restype = _SZ
        L.splr_linear_fused_tile.argtypes = [_I64, _I64, _I64, _I64, _I64, _I32, _P, _P]
        L.splr_linear_fused_tile.restype = _I32
        L.splr_linear_experts.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P, _I64, _P, _P, _I64, _I32, _P, _I32, _P,
                                          _P, _SZ, _P]
        L.splr_linear_experts.restype = _I32
        L.splr_tokens_dispatch.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _I64, _I32, _P, _P, _P, _P, _SZ, _P]
        L.splr_tokens_dispatch.restype = _I32
        L.splr_tokens_dispatch_workspace_bytes.argtypes = [_I64, _I64, _I64]
        L.splr_tokens_dispatch_workspace_bytes.restype = _SZ
        L.splr_tokens_gather.argtypes = [_P, _I64, _I64, _I32, _P, _I64, _P, _I64, _P]
        L.splr_tokens_gather.restype = _I32
        L.splr_tokens_combine.argtypes = [_P, _I64, _I64, _I32, _P, _I64, _I64, _P, _P, _P, _P]
        L.splr_tokens_combine.restype = _I32
        L.splr_tokens_combine_backward.argtypes = [_P, _P, _I64, _I64, _I32, _P, _I64, _I64, _P, _P, _P, _P]
        L.splr_tokens_combine_backward.restype = _I32
        L.splr_fp8_quantize.argtypes = [_P, _I64, _I64, _I32, _I32, _I32, _P, _P, _P]
        L.splr_fp8_quantize.restype = _I32
        L.splr_linear_fp8.argtypes = [_P, _P, _I64, _I64, _I32, _P, _P, _I32, _I64, _P, _I32, _P, _P, _SZ, _P]
        L.splr_linear_fp8.restype = _I32
        L.splr_linear_fp8_experts.argtypes = [_P, _P, _I64, _I64, _I32, _P, _I64, _P, _P, _I32, _I64, _P, _I32, _P, _P, _SZ, _P]
        L.splr_linear_fp8_experts.restype = _I32
        L.splr_linear_fp8_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, _I32, _I32]
        L.splr_linear_fp8_workspace_bytes.restype = _SZ
        L.splr_linear_fp8_tile.argtypes = [_I64, _I64, _I64, _I64, _I32, _I32, _P, _P]
        L.splr_linear_fp8_tile.restype = _I32
        L.splr_dense_reconstruct.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P]
        L.splr_dense_reconstruct.restype = _I32
        L.splr_gram_workspace_bytes.argtypes = [_I64, _I64]
        L.splr_gram_workspace_bytes.restype = _SZ
        L.splr_gram_f64.argtypes = [_P, _I64, _I64, _P, _P, _SZ, _P]
        L.splr_gram_f64.restype = _I32
        L.splr_chol_rinv.argtypes = [_P, _I64, _P, _P]
        L.splr_chol_rinv.restype = _I32
        L.splr_status_string.argtypes = [_I32]
        L.splr_status_string.restype = ctypes.c_char_p
        L.splr_version.argtypes = []
        L.splr_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPLR_BF16
    if t.dtype == torch.float32:
        return SPLR_FP32
    raise TypeError(f"unsupported dtype {t.dtype} (use torch.bfloat16 or torch.float32)")


def _is_device(t: torch.Tensor) -> bool:
    return t.is_cuda


def _dev(t: Optional[torch.Tensor], name: str) -> Optional[int]:
    if t is None:
        return None
    if not _is_device(t):
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    return _the_stream(stream).cuda_stream


def _the_stream(stream):
    return torch.cuda.current_stream() if stream is None else stream


def _expect(t: Optional[torch.Tensor], name: str, dtype, numel: int, device, shape=None):
    """Raise ValueError unless `t` is a contiguous device tensor of `dtype` on `device` holding
    exactly `numel` elements (and of `shape`, when given). The C ABI sees only pointers, so a
    buffer of the wrong size would be read or written out of bounds: every tensor is checked here,
    before the call."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not _is_device(t):
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.numel() != numel:
        raise ValueError(f"{name} holds {t.numel()} elements, expected {numel}")


def _matrix(t: torch.Tensor, name: str) -> Tuple[int, int]:
    if not isinstance(t, torch.Tensor) or not _is_device(t):
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.shape[0], t.shape[1]


def _packed_out(values, meta, n_out, n_in, dtype, device, stream):
    """Check caller-supplied packed buffers (or allocate them on the call's stream)."""
    TR, TK = tiles(n_out, n_in)
    if values is None or meta is None:
        with torch.cuda.stream(_the_stream(stream)):
            if values is None:
                values = torch.empty((TR, TK, 64, 8), dtype=dtype, device=device)
            if meta is None:
                meta = torch.empty(meta_shape(n_out, n_in), dtype=torch.int32, device=device)
    _expect(values, "values", dtype, TR * TK * 512, device)
    _expect(meta, "meta", torch.int32, _meta_words(n_out, n_in), device)
    return values, meta


def _meta_words(n_out: int, n_in: int) -> int:
    TR, TKB, lanes, words = meta_shape(n_out, n_in)
    return TR * TKB * lanes * words


def _check_packed_in(values, meta, n_out, n_in, dtype, device):
    TR, TK = tiles(n_out, n_in)
    _expect(values, "values", dtype, TR * TK * 512, device)
    _expect(meta, "meta", torch.int32, _meta_words(n_out, n_in), device)


def _check_factors(U, V, n_out, n_in, dtype, device):
    """U [n_out, r] and V [r, n_in] of the storage type (both or neither); returns r."""
    if (U is None) != (V is None):
        raise ValueError("U and V are given together (or neither, for no low-rank part)")
    if U is None:
        return 0
    r = U.shape[1] if U.dim() == 2 else -1
    _expect(U, "U", dtype, n_out * max(r, 0), device, (n_out, r))
    _expect(V, "V", dtype, r * n_in, device, (r, n_in))
    return r


def _check(fn: str, status: int):
    if status != 0:
        raise SplrError(fn, status)


def tiles(n_out: int, n_in: int) -> Tuple[int, int]:
    return (n_out + 15) // 16, (n_in + 63) // 64


def meta_shape(n_out: int, n_in: int) -> Tuple[int, int, int, int]:
    """Shape of the packed metadata (int32 words): (TR, TKB, 64, 4), blocks of 8 tile columns."""
    TR, TK = tiles(n_out, n_in)
    return TR, (TK + 7) // 8, 64, 4


def packed_bytes(n_out: int, n_in: int, dtype: torch.dtype) -> Tuple[int, int]:
    """(values bytes, metadata bytes) of the packed layout, as the library reports them."""
    vb, mb = ctypes.c_size_t(), ctypes.c_size_t()
    code = SPLR_BF16 if dtype == torch.bfloat16 else SPLR_FP32
    _check("splr_packed_bytes", lib().splr_packed_bytes(n_out, n_in, code, ctypes.byref(vb), ctypes.byref(mb)))
    return vb.value, mb.value


def prune24_pack(R: torch.Tensor, values: Optional[torch.Tensor] = None, meta: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """2:4 projection + pack of R [n_out, n_in] -> (values (TR, TK, 64, 8), meta int32 (TR, TKB, 64, 4))."""
    n_out, n_in = _matrix(R, "R")
    _dtype_code(R)
    values, meta = _packed_out(values, meta, n_out, n_in, R.dtype, R.device, stream)
    _check("splr_prune24_pack", lib().splr_prune24_pack(_dev(R, "R"), n_out, n_in, _dtype_code(R),
                                                        _dev(values, "values"), _dev(meta, "meta"), _stream(stream)))
    return values, meta


def prune_nm_pack(R: torch.Tensor, n: int, m: int, values: Optional[torch.Tensor] = None,
                  meta: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """N:M projection (n in {1, 2}, m in {4, 8, 16}) of R [n_out, n_in], stored in the 2:4 packed
    layout -> (values, meta) as prune24_pack returns them."""
    n_out, n_in = _matrix(R, "R")
    _dtype_code(R)
    values, meta = _packed_out(values, meta, n_out, n_in, R.dtype, R.device, stream)
    _check("splr_prune_nm_pack", lib().splr_prune_nm_pack(_dev(R, "R"), n_out, n_in, n, m, _dtype_code(R),
                                                          _dev(values, "values"), _dev(meta, "meta"), _stream(stream)))
    return values, meta


def prune24_pack_residual(W: torch.Tensor, U: Optional[torch.Tensor], V: Optional[torch.Tensor],
                          values: Optional[torch.Tensor] = None, meta: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """2:4 projection + pack of R = W - U V, formed in the kernel (pinned fused multiply-add order)."""
    n_out, n_in = _matrix(W, "W")
    _dtype_code(W)
    r = _check_factors(U, V, n_out, n_in, W.dtype, W.device)
    values, meta = _packed_out(values, meta, n_out, n_in, W.dtype, W.device, stream)
    _check("splr_prune24_pack_residual",
           lib().splr_prune24_pack_residual(_dev(W, "W"), _dev(U, "U"), _dev(V, "V"), n_out, n_in, r, _dtype_code(W),
                                            _dev(values, "values"), _dev(meta, "meta"), _stream(stream)))
    return values, meta


def prune24_pack_scaled(R: torch.Tensor, d: torch.Tensor, values: Optional[torch.Tensor] = None,
                        meta: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Activation-aware 2:4 projection + pack of R [n_out, n_in] with per-column scales d (float32
    [n_in]): keeps the two entries of largest |R[n][k]| * |d[k]| per group. Same outputs as
    prune24_pack."""
    n_out, n_in = _matrix(R, "R")
    _dtype_code(R)
    _expect(d, "d", torch.float32, n_in, R.device, (n_in,))
    values, meta = _packed_out(values, meta, n_out, n_in, R.dtype, R.device, stream)
    _check("splr_prune24_pack_scaled",
           lib().splr_prune24_pack_scaled(_dev(R, "R"), _dev(d, "d"), n_out, n_in, _dtype_code(R),
                                          _dev(values, "values"), _dev(meta, "meta"), _stream(stream)))
    return values, meta


def workspace_bytes(M: int, n_out: int, n_in: int, r: int, dtype: torch.dtype) -> int:
    code = SPLR_BF16 if dtype == torch.bfloat16 else SPLR_FP32
    return int(lib().splr_linear_workspace_bytes(M, n_out, n_in, r, code))


def new_workspace(M: int, n_out: int, n_in: int, r: int, dtype: torch.dtype, device="cuda",
                  stream=None) -> Optional[torch.Tensor]:
    """A workspace for splr_linear with these sizes (None when none is needed), allocated on
    `stream` (default: the current stream). Any workspace of at least workspace_bytes() serves any
    call, and its contents need no initialisation: every byte the second stage reads is written by
    the first stage of the same call."""
    need = workspace_bytes(M, n_out, n_in, r, dtype)
    if not need:
        return None
    with torch.cuda.stream(_the_stream(stream)):
        return torch.empty(need, dtype=torch.uint8, device=device)


def _linear_args(X, values, meta, U, V, n_out, out, workspace, stream, y_dtype=torch.float32, with_workspace=True,
                 need_v=True):
    """Checks every tensor of a layer-product call against the sizes passed to the C ABI, and
    allocates what is missing on the call's stream."""
    M, n_in = _matrix(X, "X")
    _dtype_code(X)
    if n_out is None:
        n_out = U.shape[0] if U is not None else values.shape[0] * 16
    _check_packed_in(values, meta, n_out, n_in, X.dtype, X.device)
    if need_v:
        r = _check_factors(U, V, n_out, n_in, X.dtype, X.device)
    else:
        r = 0 if U is None else (U.shape[1] if U.dim() == 2 else -1)
        if U is not None:
            _expect(U, "U", X.dtype, n_out * max(r, 0), X.device, (n_out, r))
    if out is None:
        with torch.cuda.stream(_the_stream(stream)):
            out = torch.empty((M, n_out), dtype=y_dtype, device=X.device)
    if workspace is None and with_workspace:
        workspace = new_workspace(M, n_out, n_in, r, X.dtype, X.device, stream)
    _expect(out, "out", y_dtype, M * n_out, X.device, (M, n_out))
    if workspace is not None:
        if not _is_device(workspace) or workspace.device != X.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of X")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return M, n_in, n_out, r, out, workspace, ws_bytes


def linear(X: torch.Tensor, values: torch.Tensor, meta: torch.Tensor, U: Optional[torch.Tensor],
           V: Optional[torch.Tensor], n_out: Optional[int] = None, out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y [M, n_out] float32 = X S^T + (X V^T) U^T (n_out defaults to U's rows, else 16 * TR)."""
    M, n_in, n_out, r, out, workspace, ws_bytes = _linear_args(X, values, meta, U, V, n_out, out, workspace, stream)
    _check("splr_linear", lib().splr_linear(_dev(X, "X"), M, n_in, _dev(values, "values"), _dev(meta, "meta"), n_out,
                                            _dev(U, "U"), _dev(V, "V"), r, _dtype_code(X), _dev(out, "out"),
                                            _dev(workspace, "workspace"), ws_bytes, _stream(stream)))
    return out


def linear_ex(X: torch.Tensor, values: torch.Tensor, meta: torch.Tensor, U: Optional[torch.Tensor],
              V: Optional[torch.Tensor], y_dtype: torch.dtype = torch.float32, n_out: Optional[int] = None,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """splr_linear with the output type chosen: float32, or bfloat16 (each result rounded to nearest
    even)."""
    if y_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"y_dtype must be float32 or bfloat16, got {y_dtype}")
    M, n_in, n_out, r, out, workspace, ws_bytes = _linear_args(X, values, meta, U, V, n_out, out, workspace, stream,
                                                               y_dtype=y_dtype)
    ycode = SPLR_BF16 if y_dtype == torch.bfloat16 else SPLR_FP32
    _check("splr_linear_ex", lib().splr_linear_ex(_dev(X, "X"), M, n_in, _dev(values, "values"), _dev(meta, "meta"),
                                                  n_out, _dev(U, "U"), _dev(V, "V"), r, _dtype_code(X), ycode,
                                                  _dev(out, "out"), _dev(workspace, "workspace"), ws_bytes,
                                                  _stream(stream)))
    return out


def linear_stage1(X: torch.Tensor, V: Optional[torch.Tensor], workspace: torch.Tensor, n_out: int = 0,
                  stream=None) -> torch.Tensor:
    """First low-rank stage T = X V^T into `workspace` (sized by workspace_bytes); returns it."""
    M, n_in = _matrix(X, "X")
    _dtype_code(X)
    r = 0
    if V is not None:
        r = V.shape[0] if V.dim() == 2 else -1
        _expect(V, "V", X.dtype, max(r, 0) * n_in, X.device, (r, n_in))
    if workspace is not None and (not _is_device(workspace) or workspace.device != X.device
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the device of X")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("splr_linear_stage1", lib().splr_linear_stage1(_dev(X, "X"), M, n_in, _dev(V, "V"), r, _dtype_code(X),
                                                          _dev(workspace, "workspace"), ws_bytes, _stream(stream)))
    return workspace


def linear_stage2(X: torch.Tensor, values: torch.Tensor, meta: torch.Tensor, U: Optional[torch.Tensor],
                  workspace: Optional[torch.Tensor], n_out: Optional[int] = None, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Y = X S^T + T U^T with T left in `workspace` by linear_stage1 (same X and r)."""
    M, n_in, n_out, r, out, workspace, ws_bytes = _linear_args(X, values, meta, U, None, n_out, out, workspace, stream,
                                                               with_workspace=False, need_v=False)
    _check("splr_linear_stage2",
           lib().splr_linear_stage2(_dev(X, "X"), M, n_in, _dev(values, "values"), _dev(meta, "meta"), n_out,
                                    _dev(U, "U"), r, _dtype_code(X), _dev(out, "out"), _dev(workspace, "workspace"),
                                    ws_bytes, _stream(stream)))
    return out


GROUP_MAX = 4  # SPLR_GROUP_MAX


def _ptr_array(ts, name):
    """A host array of the tensors' device pointers (None for a missing list)."""
    if ts is None:
        return None
    return (ctypes.c_void_p * len(ts))(*[_dev(t, f"{name}[{i}]") for i, t in enumerate(ts)])


def _group_args(Xs, values, metas, Us, Vs, n_out, outs, workspaces, stream, with_stage1):
    """Checks every layer as the single-layer call would (allocating missing outputs and workspaces
    on the call's stream) and that the layers share their sizes and type."""
    count = len(Xs)
    if not 1 <= count <= GROUP_MAX:
        raise ValueError(f"a group holds 1..{GROUP_MAX} layers, got {count}")
    for name, lst in (("values", values), ("meta", metas), ("U", Us), ("V", Vs), ("outs", outs),
                      ("workspaces", workspaces)):
        if lst is not None and len(lst) != count:
            raise ValueError(f"{name} has {len(lst)} entries for {count} layers")
    per = []
    for i in range(count):
        U = None if Us is None else Us[i]
        V = None if Vs is None else Vs[i]
        out = None if outs is None else outs[i]
        ws = None if workspaces is None else workspaces[i]
        per.append(_linear_args(Xs[i], values[i], metas[i], U, V if with_stage1 else None, n_out, out, ws, stream,
                                with_workspace=with_stage1, need_v=with_stage1))
    shape = per[0][:4]
    if any(p[:4] != shape for p in per) or any(X.dtype != Xs[0].dtype for X in Xs):
        raise ValueError("the layers of a group share M, n_in, n_out, r and the storage type")
    M, n_in, n_out, r = shape
    outs = [p[4] for p in per]
    wss = [p[5] for p in per]
    ws_bytes = min(p[6] for p in per)
    return count, M, n_in, n_out, r, outs, wss, ws_bytes


def linear_group(Xs: Sequence[torch.Tensor], values: Sequence[torch.Tensor], metas: Sequence[torch.Tensor],
                 Us: Optional[Sequence[torch.Tensor]], Vs: Optional[Sequence[torch.Tensor]],
                 n_out: Optional[int] = None, outs: Optional[Sequence[torch.Tensor]] = None,
                 workspaces: Optional[Sequence[torch.Tensor]] = None, stream=None) -> List[torch.Tensor]:
    """splr_linear for up to GROUP_MAX layers of one shape, stage 2 of all of them in one launch
    (splr_linear_group); returns the layers' Y, each bit for bit its splr_linear result."""
    count, M, n_in, n_out, r, outs, wss, ws_bytes = _group_args(Xs, values, metas, Us, Vs, n_out, outs, workspaces,
                                                                stream, True)
    ws_arr = _ptr_array(wss, "workspace") if r > 0 else (ctypes.c_void_p * count)()
    _check("splr_linear_group",
           lib().splr_linear_group(count, _ptr_array(Xs, "X"), M, n_in, _ptr_array(values, "values"),
                                   _ptr_array(metas, "meta"), n_out, _ptr_array(Us, "U") if r > 0 else None,
                                   _ptr_array(Vs, "V") if r > 0 else None, r, _dtype_code(Xs[0]),
                                   _ptr_array(outs, "out"), ws_arr, ws_bytes, _stream(stream)))
    return outs


def linear_stage2_group(Xs: Sequence[torch.Tensor], values: Sequence[torch.Tensor], metas: Sequence[torch.Tensor],
                        Us: Optional[Sequence[torch.Tensor]], workspaces: Optional[Sequence[torch.Tensor]],
                        n_out: Optional[int] = None, outs: Optional[Sequence[torch.Tensor]] = None,
                        stream=None) -> List[torch.Tensor]:
    """linear_stage2 for up to GROUP_MAX layers of one shape in one launch (splr_linear_stage2_group),
    each layer's T left in its workspace by linear_stage1."""
    count, M, n_in, n_out, r, outs, wss, ws_bytes = _group_args(Xs, values, metas, Us, None, n_out, outs, workspaces,
                                                                stream, False)
    ws_arr = _ptr_array(wss, "workspace") if r > 0 else (ctypes.c_void_p * count)()
    _check("splr_linear_stage2_group",
           lib().splr_linear_stage2_group(count, _ptr_array(Xs, "X"), M, n_in, _ptr_array(values, "values"),
                                          _ptr_array(metas, "meta"), n_out, _ptr_array(Us, "U") if r > 0 else None,
                                          r, _dtype_code(Xs[0]), _ptr_array(outs, "out"), ws_arr, ws_bytes,
                                          _stream(stream)))
    return outs


def linear_stage2_dense(X: torch.Tensor, values: torch.Tensor, meta: torch.Tensor, U: Optional[torch.Tensor],
                        workspace: Optional[torch.Tensor], n_out: Optional[int] = None,
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """linear_stage2 with S expanded to dense bfloat16 on chip and multiplied by dense MFMA
    (splr_linear_stage2_dense; bfloat16 only): the measured alternative to the structured-sparse
    instruction."""
    M, n_in, n_out, r, out, workspace, ws_bytes = _linear_args(X, values, meta, U, None, n_out, out, workspace, stream,
                                                               with_workspace=False, need_v=False)
    _check("splr_linear_stage2_dense",
           lib().splr_linear_stage2_dense(_dev(X, "X"), M, n_in, _dev(values, "values"), _dev(meta, "meta"), n_out,
                                          _dev(U, "U"), r, _dtype_code(X), _dev(out, "out"),
                                          _dev(workspace, "workspace"), ws_bytes, _stream(stream)))
    return out


def linear_noalloc(X: torch.Tensor, values: torch.Tensor, meta: torch.Tensor, U: Optional[torch.Tensor],
                   V: Optional[torch.Tensor], n_out: Optional[int] = None, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """splr_linear with the library's built-in workspace (splr_linear_noalloc): nothing is allocated
    when `out` is given. Calls on one GPU share that workspace, so they must not overlap in time."""
    M, n_in, n_out, r, out, _, _ = _linear_args(X, values, meta, U, V, n_out, out, None, stream,
                                                with_workspace=False)
    _check("splr_linear_noalloc",
           lib().splr_linear_noalloc(_dev(X, "X"), M, n_in, _dev(values, "values"), _dev(meta, "meta"), n_out,
                                     _dev(U, "U"), _dev(V, "V"), r, _dtype_code(X), _dev(out, "out"),
                                     _stream(stream)))
    return out


ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}  # splr_activation_t
EXPERTS_MAX = 1024  # SPLR_EXPERTS_MAX


class _Epilogue(ctypes.Structure):
    """splr_epilogue_t."""
    _fields_ = [("activation", _I32), ("bias", _P), ("gate", _P), ("residual", _P)]


def _stream_handle(stream, index: int) -> int:
    """The HIP stream of a call on device number `index`: the given one's, or the current one's as a
    plain number (building torch's stream object for it takes 2.7 us, a fifth of a small call)."""
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _fused_call(X, offsets, values, meta, U, V, bias, activation, gate, residual, y_dtype, n_out, out, workspace,
                stream):
    """linear_fused (offsets None) and linear_experts: checks every tensor, allocates what is missing
    on the call's stream and calls the library, with X's device current.

    Each tensor is asked in one expression whether it is contiguous, of the right type, shape and
    device; `_expect` says what is wrong (or takes another shape of the right size) when it is not. The
    calls of a serving loop are right, and their checks are most of what the host adds to a launch."""
    if not isinstance(X, torch.Tensor) or not _is_device(X):
        raise ValueError("X must be a device tensor")
    index, device, dt = X.get_device(), X.device, X.dtype
    if index >= 0 and index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _fused_call(X, offsets, values, meta, U, V, bias, activation, gate, residual, y_dtype, n_out, out,
                               workspace, stream)
    if X.dim() != 2 or not X.is_contiguous():
        raise ValueError(f"X must be 2-D and contiguous, got shape {tuple(X.shape)}")
    M, n_in = X.shape
    code = _dtype_code(X)
    if stream is not None and getattr(stream, "device", device) != device:
        raise ValueError(f"the stream belongs to {stream.device}, X to {device}")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    if y_dtype is not torch.bfloat16 and y_dtype is not torch.float32:
        raise ValueError(f"y_dtype must be float32 or bfloat16, got {y_dtype}")
    if values is None or meta is None:
        raise ValueError("values and meta are required")
    if (U is None) != (V is None):
        raise ValueError("U and V are given together (or neither, for no low-rank part)")
    experts = offsets is not None
    if experts:
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or not 2 <= offsets.numel() <= EXPERTS_MAX + 1:
            raise ValueError(f"offsets must be a vector of 2 .. {EXPERTS_MAX + 1} entries")
        E = offsets.numel() - 1
        if not (offsets.dtype is torch.int32 and offsets.get_device() == index and offsets.is_contiguous()):
            _expect(offsets, "offsets", torch.int32, E + 1, device)
    else:
        E = 1
    rank_dim = 3 if experts else 2
    if n_out is None:
        if U is not None and U.dim() == rank_dim:
            n_out = U.shape[-2]
        elif values.dim() == rank_dim + 2:
            n_out = values.shape[rank_dim - 2] * 16
        else:
            raise ValueError("n_out is required when neither U's nor values' shape tells it")
    r = 0 if U is None else U.shape[-1] if U.dim() == rank_dim else -1
    TR, TK = (n_out + 15) // 16, (n_in + 63) // 64
    s_shape, m_shape, u_shape, v_shape, b_shape = ((TR, TK, 64, 8), (TR, (TK + 7) // 8, 64, 4), (n_out, r), (r, n_in),
                                                   (n_out,))
    if experts:
        s_shape, m_shape, u_shape, v_shape, b_shape = (E, *s_shape), (E, *m_shape), (E, *u_shape), (E, *v_shape), (E, n_out)
    rows = (M, n_out)
    if not (values.dtype is dt and values.shape == s_shape and values.get_device() == index and values.is_contiguous()):
        _expect(values, "values", dt, E * TR * TK * 512, device)
    if not (meta.dtype is torch.int32 and meta.shape == m_shape and meta.get_device() == index and meta.is_contiguous()):
        _expect(meta, "meta", torch.int32, E * _meta_words(n_out, n_in), device)
    u = v = b = g = s = ws = None   # device addresses
    if U is not None:
        if not (U.dtype is dt and U.shape == u_shape and U.get_device() == index and U.is_contiguous()):
            _expect(U, "U", dt, E * n_out * max(r, 0), device, u_shape)
        if not (V.dtype is dt and V.shape == v_shape and V.get_device() == index and V.is_contiguous()):
            _expect(V, "V", dt, E * max(r, 0) * n_in, device, v_shape)
        u, v = U.data_ptr(), V.data_ptr()
    if bias is not None:
        if not (bias.dtype is dt and bias.shape == b_shape and bias.get_device() == index and bias.is_contiguous()):
            _expect(bias, "bias", dt, E * n_out, device, b_shape)
        b = bias.data_ptr()
    if gate is not None:
        if not (gate.dtype is y_dtype and gate.shape == rows and gate.get_device() == index and gate.is_contiguous()):
            _expect(gate, "gate", y_dtype, M * n_out, device, rows)
        g = gate.data_ptr()
    if residual is not None:
        if not (residual.dtype is y_dtype and residual.shape == rows and residual.get_device() == index
                and residual.is_contiguous()):
            _expect(residual, "residual", y_dtype, M * n_out, device, rows)
        s = residual.data_ptr()
    L = _lib or lib()
    if out is None or (workspace is None and r > 0):
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            if out is None:
                out = torch.empty(rows, dtype=y_dtype, device=device)
            if workspace is None and r > 0:
                need = (L.splr_linear_experts_workspace_bytes(M, E, n_out, n_in, r, code) if experts else
                        L.splr_linear_fused_workspace_bytes(M, n_out, n_in, r, code))
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if not (out.dtype is y_dtype and out.shape == rows and out.get_device() == index and out.is_contiguous()):
        _expect(out, "out", y_dtype, M * n_out, device, rows)
    ws_bytes = 0
    if workspace is not None:
        if not _is_device(workspace) or workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of X")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    epilogue = ctypes.byref(_Epilogue(act, b, g, s))
    ycode = SPLR_BF16 if y_dtype is torch.bfloat16 else SPLR_FP32
    handle = _stream_handle(stream, index)
    if experts:
        status = L.splr_linear_experts(X.data_ptr(), M, n_in, offsets.data_ptr(), E, values.data_ptr(),
                                       meta.data_ptr(), n_out, u, v, r, code, epilogue, ycode, out.data_ptr(), ws,
                                       ws_bytes, handle)
    else:
        status = L.splr_linear_fused(X.data_ptr(), M, n_in, values.data_ptr(), meta.data_ptr(), n_out, u, v, r, code,
                                     epilogue, ycode, out.data_ptr(), ws, ws_bytes, handle)
    if status:
        raise SplrError("splr_linear_experts" if experts else "splr_linear_fused", status)
    return out


def linear_fused(X: torch.Tensor, values: torch.Tensor, meta: torch.Tensor, U: Optional[torch.Tensor],
                 V: Optional[torch.Tensor], bias: Optional[torch.Tensor] = None, activation: str = "none",
                 gate: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                 y_dtype: torch.dtype = torch.float32, n_out: Optional[int] = None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Y [M, n_out] of y_dtype = act(X S^T + (X V^T) U^T + bias) * gate + residual, with everything
    after the products in the kernels' epilogue (splr_linear_fused). bias [n_out] of X's type; gate
    and residual [M, n_out] of y_dtype; `out` may be gate or residual itself, and overlap nothing else. The
    workspace holds fused_workspace_bytes()."""
    return _fused_call(X, None, values, meta, U, V, bias, activation, gate, residual, y_dtype, n_out, out, workspace,
                       stream)


def fused_workspace_bytes(M: int, n_out: int, n_in: int, r: int, dtype: torch.dtype) -> int:
    code = SPLR_BF16 if dtype == torch.bfloat16 else SPLR_FP32
    return int(lib().splr_linear_fused_workspace_bytes(M, n_out, n_in, r, code))


def experts_workspace_bytes(M: int, n_experts: int, n_out: int, n_in: int, r: int, dtype: torch.dtype) -> int:
    code = SPLR_BF16 if dtype == torch.bfloat16 else SPLR_FP32
    return int(lib().splr_linear_experts_workspace_bytes(M, n_experts, n_out, n_in, r, code))


def fused_tile(M: int, n_out: int, n_in: int, r: int, dtype: torch.dtype,
               n_experts: Optional[int] = None) -> Tuple[int, int]:
    """The workgroup tile (rows of S, tokens) of the kernel that linear_fused, or linear_experts with
    n_experts experts, takes for these sizes (splr_linear_fused_tile)."""
    code = SPLR_BF16 if dtype == torch.bfloat16 else SPLR_FP32
    rows, tokens = ctypes.c_int32(), ctypes.c_int32()
    _check("splr_linear_fused_tile", lib().splr_linear_fused_tile(M, n_experts or 0, n_out, n_in, r, code,
                                                                  ctypes.byref(rows), ctypes.byref(tokens)))
    return rows.value, tokens.value


def linear_experts(X: torch.Tensor, offsets: torch.Tensor, values: torch.Tensor, meta: torch.Tensor,
                   U: Optional[torch.Tensor], V: Optional[torch.Tensor], bias: Optional[torch.Tensor] = None,
                   activation: str = "none", gate: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.float32,
                   n_out: Optional[int] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """linear_fused for rows grouped by expert (splr_linear_experts): rows offsets[e] .. offsets[e+1]-1
    of X, gate, residual and Y go through expert e's packed S, U, V and bias.

    offsets: int32 [E + 1] on the device, non-decreasing, within 0 .. M; it is read by the kernels
    only, so nothing waits for it. values (E, TR, TK, 64, 8) and meta (E, TR, TKB, 64, 4): the experts'
    packed S one after the other; U [E, n_out, r], V [E, r, n_in], bias [E, n_out]. M may be 0. Rows
    outside offsets[0] .. offsets[E]-1 of `out` are left as they were."""
    if offsets is None:
        raise ValueError("offsets is required")
    return _fused_call(X, offsets, values, meta, U, V, bias, activation, gate, residual, y_dtype, n_out, out,
                       workspace, stream)


SLOTS_MAX = 64  # SPLR_SLOTS_MAX
E4M3 = torch.float8_e4m3fn
_CODES = {torch.float32: SPLR_FP32, torch.bfloat16: SPLR_BF16, E4M3: SPLR_E4M3}


def _on_device_of(t, name, stream):
    """The device number and device of `t`, the call's leading tensor, and whether its device has to be made current."""
    if not isinstance(t, torch.Tensor) or not _is_device(t):
        raise ValueError(f"{name} must be a device tensor")
    device = t.device
    if stream is not None and getattr(stream, "device", device) != device:
        raise ValueError(f"the stream belongs to {stream.device}, {name} to {device}")
    index = t.get_device()
    return index, device, index >= 0 and index != torch.cuda.current_device()


def _fits(t, name, dtype, shape, index, device) -> int:
    """The address of a contiguous tensor of this type, shape and device; `_expect` says what is wrong with another."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()
            and _is_device(t)):
        if t is not None and not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a device tensor")
        _expect(t, name, dtype, math.prod(shape), device, shape)
    return t.data_ptr()


def _workspace(t, index):
    """(address, bytes) of a caller's workspace, or of none."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or not _is_device(t) or t.get_device() != index or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of the operands")
    return t.data_ptr(), t.nbytes


def _new(shape, dtype, device, stream):
    """An output or workspace, allocated on the call's stream."""
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _slots(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not 1 <= t.shape[1] <= SLOTS_MAX:
        raise ValueError(f"{name} must be 2-D with 1 .. {SLOTS_MAX} columns")
    return t.shape


def _rows_type(t, name, types):
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be 2-D and contiguous, got shape {tuple(t.shape)}")
    if t.dtype not in types:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {', '.join(str(d) for d in types)}")
    return _CODES[t.dtype]


def tokens_dispatch(ids: torch.Tensor, n_experts: int, X: Optional[torch.Tensor] = None,
                    offsets: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """The slots of ids [T, slots] (int32 or int64) sorted by expert (splr_tokens_dispatch): offsets int32 [n_experts + 1] as
    linear_experts takes them, positions int32 [T, slots] (-1 where the id is outside 0 .. n_experts - 1) and, with X [T, D],
    the sorted rows `out` [T * slots, D], of which those behind offsets[n_experts] are left as they were."""
    index, device, other = _on_device_of(ids, "ids", stream)
    if other:
        with torch.cuda.device(device):
            return tokens_dispatch(ids, n_experts, X, offsets, positions, out, workspace, stream)
    T, k = _slots(ids, "ids")
    if ids.dtype is not torch.int64 and ids.dtype is not torch.int32 or not ids.is_contiguous():
        raise ValueError(f"ids must be contiguous int32 or int64, got {ids.dtype}")
    if not 1 <= n_experts <= EXPERTS_MAX:
        raise ValueError(f"n_experts must be 1 .. {EXPERTS_MAX}, got {n_experts}")
    if X is None and out is not None:
        raise ValueError("out is given without X")
    L = _lib or lib()
    if offsets is None:
        offsets = _new((n_experts + 1,), torch.int32, device, stream)
    if positions is None:
        positions = _new((T, k), torch.int32, device, stream)
    o = _fits(offsets, "offsets", torch.int32, (n_experts + 1,), index, device)
    p = _fits(positions, "positions", torch.int32, (T, k), index, device)
    x = y = None
    D = code = 0
    if X is not None:
        code = _rows_type(X, "X", _CODES)
        D = X.shape[1]
        x = _fits(X, "X", X.dtype, (T, D), index, device)
        if out is None:
            out = _new((T * k, D), X.dtype, device, stream)
        y = _fits(out, "out", X.dtype, (T * k, D), index, device)
    if workspace is None:
        need = L.splr_tokens_dispatch_workspace_bytes(T, k, n_experts)
        workspace = _new((need,), torch.uint8, device, stream) if need else None
    ws, ws_bytes = _workspace(workspace, index)
    status = L.splr_tokens_dispatch(ids.data_ptr(), ids.element_size(), T, k, n_experts, x, D, code, o, p, y, ws, ws_bytes,
                                    _stream_handle(stream, index))
    if status:
        raise SplrError("splr_tokens_dispatch", status)
    return offsets, positions, out


def tokens_gather(X: torch.Tensor, positions: torch.Tensor, rows: Optional[int] = None, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """out[positions[t][j]] = X[t] (splr_tokens_gather): the rows of X [T, D] at the places that tokens_dispatch gave them. `out`
    [rows, D], by default a new one of T * slots rows; rows that no position names are left as they were."""
    index, device, other = _on_device_of(X, "X", stream)
    if other:
        with torch.cuda.device(device):
            return tokens_gather(X, positions, rows, out, stream)
    code = _rows_type(X, "X", _CODES)
    T, D = X.shape
    k = _slots(positions, "positions")[1]
    p = _fits(positions, "positions", torch.int32, (T, k), index, device)
    if rows is None:
        rows = T * k if out is None else out.shape[0]
    if out is None:
        out = _new((rows, D), X.dtype, device, stream)
    y = _fits(out, "out", X.dtype, (rows, D), index, device)
    status = (_lib or lib()).splr_tokens_gather(X.data_ptr(), T, D, code, p, k, y, rows, _stream_handle(stream, index))
    if status:
        raise SplrError("splr_tokens_gather", status)
    return out


def tokens_combine(Z: torch.Tensor, positions: torch.Tensor, weights: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = residual[t] + sum_j weights[t][j] Z[positions[t][j]] (splr_tokens_combine): Z [rows, D] float32 or bfloat16,
    positions int32 [T, slots], weights float32 [T, slots] (None: ones), residual and out [T, D] of Z's type; `out` may be
    residual itself. Without weights and residual it is the gradient of tokens_dispatch and tokens_gather."""
    index, device, other = _on_device_of(Z, "Z", stream)
    if other:
        with torch.cuda.device(device):
            return tokens_combine(Z, positions, weights, residual, out, stream)
    code = _rows_type(Z, "Z", (torch.float32, torch.bfloat16))
    rows, D = Z.shape
    T, k = _slots(positions, "positions")
    p = _fits(positions, "positions", torch.int32, (T, k), index, device)
    w = None if weights is None else _fits(weights, "weights", torch.float32, (T, k), index, device)
    r = None if residual is None else _fits(residual, "residual", Z.dtype, (T, D), index, device)
    if out is None:
        out = _new((T, D), Z.dtype, device, stream)
    y = _fits(out, "out", Z.dtype, (T, D), index, device)
    status = (_lib or lib()).splr_tokens_combine(Z.data_ptr(), rows, D, code, p, T, k, w, r, y, _stream_handle(stream, index))
    if status:
        raise SplrError("splr_tokens_combine", status)
    return out


def tokens_combine_backward(dY: torch.Tensor, Z: torch.Tensor, positions: torch.Tensor, weights: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dZ, dweights) of tokens_combine for dY [T, D] (splr_tokens_combine_backward): dZ[positions[t][j]] = weights[t][j] dY[t]
    in `out` [rows, D], which may be Z itself and whose other rows are left as they were (a new one starts as zeros), and
    dweights[t][j] = <dY[t], Z[positions[t][j]]>, float32 [T, slots]. The gradient of residual is dY."""
    index, device, other = _on_device_of(dY, "dY", stream)
    if other:
        with torch.cuda.device(device):
            return tokens_combine_backward(dY, Z, positions, weights, out, dweights, stream)
    code = _rows_type(dY, "dY", (torch.float32, torch.bfloat16))
    T, D = dY.shape
    if not isinstance(Z, torch.Tensor) or Z.dim() != 2:
        raise ValueError("Z must be 2-D")
    rows, k = Z.shape[0], _slots(positions, "positions")[1]
    z = _fits(Z, "Z", dY.dtype, (rows, D), index, device)
    p = _fits(positions, "positions", torch.int32, (T, k), index, device)
    w = None if weights is None else _fits(weights, "weights", torch.float32, (T, k), index, device)
    if out is None:
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            out = torch.zeros((rows, D), dtype=dY.dtype, device=device)
    if dweights is None:
        dweights = _new((T, k), torch.float32, device, stream)
    dz = _fits(out, "out", dY.dtype, (rows, D), index, device)
    dw = _fits(dweights, "dweights", torch.float32, (T, k), index, device)
    status = (_lib or lib()).splr_tokens_combine_backward(dY.data_ptr(), z, rows, D, code, p, T, k, w, dz, dw,
                                                          _stream_handle(stream, index))
    if status:
        raise SplrError("splr_tokens_combine_backward", status)
    return out, dweights


def fp8_quantize(X: torch.Tensor, block_rows: int = 1, transposed: bool = False, out: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """X [rows, cols] (float32 or bfloat16) in e4m3 with a float32 scale for each block of block_rows (1 or 128) x 128
    (splr_fp8_quantize) -> (Q, scales). Q [rows, cols] with scales [ceil(cols/128), rows] for block_rows 1 and
    [ceil(rows/128), ceil(cols/128)] for 128; transposed, of X^T: Q [cols, rows rounded up to 32] with scales
    [ceil(rows/128), cols] or [ceil(cols/128), ceil(rows/128)]. As linear_fp8 takes them."""
    index, device, other = _on_device_of(X, "X", stream)
    if other:
        with torch.cuda.device(device):
            return fp8_quantize(X, block_rows, transposed, out, scales, stream)
    code = _rows_type(X, "X", (torch.float32, torch.bfloat16))
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows must be 1 or 128, got {block_rows}")
    n, K = reversed(X.shape) if transposed else X.shape   # Q's rows and the entries that blocks run along
    KB = (K + 127) // 128
    shape = (n, (K + 31) // 32 * 32) if transposed else (n, K)
    s_shape = (KB, n) if block_rows == 1 else ((n + 127) // 128, KB)
    if out is None:
        out = _new(shape, E4M3, device, stream)
    if scales is None:
        scales = _new(s_shape, torch.float32, device, stream)
    q = _fits(out, "out", E4M3, shape, index, device)
    s = _fits(scales, "scales", torch.float32, s_shape, index, device)
    status = (_lib or lib()).splr_fp8_quantize(X.data_ptr(), X.shape[0], X.shape[1], code, block_rows, int(transposed), q, s,
                                               _stream_handle(stream, index))
    if status:
        raise SplrError("splr_fp8_quantize", status)
    return out, scales


def _fp8_call(X, offsets, W, w_scales, x_scales, bias, activation, gate, residual, y_dtype, out, workspace, stream):
    """linear_fp8 (offsets None) and linear_fp8_experts."""
    index, device, other = _on_device_of(X, "X", stream)
    if other:
        with torch.cuda.device(device):
            return _fp8_call(X, offsets, W, w_scales, x_scales, bias, activation, gate, residual, y_dtype, out, workspace, stream)
    code = _rows_type(X, "X", _CODES)
    M, n_in = X.shape
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    if y_dtype is not torch.bfloat16 and y_dtype is not torch.float32:
        raise ValueError(f"y_dtype must be float32 or bfloat16, got {y_dtype}")
    experts = offsets is not None
    E = o = 0
    lead = ()
    if experts:
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or not 2 <= offsets.numel() <= EXPERTS_MAX + 1:
            raise ValueError(f"offsets must be a vector of 2 .. {EXPERTS_MAX + 1} entries")
        E = offsets.numel() - 1
        o = _fits(offsets, "offsets", torch.int32, (E + 1,), index, device)
        lead = (E,)
    if not isinstance(W, torch.Tensor) or W.dim() != 2 + len(lead):
        raise ValueError("W must be [experts, n_out, n_in]" if experts else "W must be [n_out, n_in]")
    n_out = W.shape[-2]
    w = _fits(W, "W", E4M3, (*lead, n_out, n_in), index, device)
    KB = (n_in + 127) // 128
    blocks, by_row = (*lead, (n_out + 127) // 128, KB), (*lead, KB, n_out)
    block_rows = 1 if isinstance(w_scales, torch.Tensor) and w_scales.shape == by_row != blocks else 128
    ws_ = _fits(w_scales, "w_scales", torch.float32, by_row if block_rows == 1 else blocks, index, device)
    xs = None
    if X.dtype is E4M3:
        xs = _fits(x_scales, "x_scales", torch.float32, (KB, M), index, device)
    elif x_scales is not None:
        raise ValueError("x_scales is for an X in e4m3")
    rows = (M, n_out)
    b = None if bias is None else _fits(bias, "bias", y_dtype, (*lead, n_out), index, device)
    g = None if gate is None else _fits(gate, "gate", y_dtype, rows, index, device)
    r = None if residual is None else _fits(residual, "residual", y_dtype, rows, index, device)
    L = _lib or lib()
    ycode = _CODES[y_dtype]
    if out is None:
        out = _new(rows, y_dtype, device, stream)
    y = _fits(out, "out", y_dtype, rows, index, device)
    if workspace is None:
        need = L.splr_linear_fp8_workspace_bytes(M, E, n_out, n_in, code, ycode)
        workspace = _new((need,), torch.uint8, device, stream) if need else None
    ws, ws_bytes = _workspace(workspace, index)
    epilogue = ctypes.byref(_Epilogue(act, b, g, r))
    handle = _stream_handle(stream, index)
    if experts:
        status = L.splr_linear_fp8_experts(X.data_ptr(), xs, M, n_in, code, o, E, w, ws_, block_rows, n_out, epilogue, ycode, y,
                                           ws, ws_bytes, handle)
    else:
        status = L.splr_linear_fp8(X.data_ptr(), xs, M, n_in, code, w, ws_, block_rows, n_out, epilogue, ycode, y, ws, ws_bytes,
                                   handle)
    if status:
        raise SplrError("splr_linear_fp8_experts" if experts else "splr_linear_fp8", status)
    return out


def linear_fp8(X: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor, x_scales: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, activation: str = "none", gate: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.float32,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y [M, n_out] of y_dtype = act(X W^T + bias) * gate + residual with W [n_out, n_in] in e4m3 (splr_linear_fp8). w_scales
    [ceil(n_out/128), ceil(n_in/128)] (blocks of 128 x 128) or [ceil(n_in/128), n_out] (of 1 x 128). X [M, n_in] float32 or
    bfloat16 is quantised by the call; in e4m3 it comes with x_scales [ceil(n_in/128), M]. bias [n_out], gate and residual
    [M, n_out] of y_dtype; `out` may be gate or residual itself. The workspace holds linear_fp8_workspace_bytes(). The gradient dX =
    dY W is linear_fp8 of dY and fp8_quantize(w, 128, transposed=True), dY's rows padded with zeros to a multiple of 32."""
    return _fp8_call(X, None, W, w_scales, x_scales, bias, activation, gate, residual, y_dtype, out, workspace, stream)


def linear_fp8_experts(X: torch.Tensor, offsets: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor,
                       x_scales: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, activation: str = "none",
                       gate: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                       y_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """linear_fp8 for rows grouped by expert (splr_linear_fp8_experts): rows offsets[e] .. offsets[e+1]-1 go through W[e] (W
    [E, n_out, n_in], w_scales and bias with a leading E). offsets as linear_experts takes it, M may be 0, and rows outside
    offsets[0] .. offsets[E]-1 of `out` are left as they were."""
    if offsets is None:
        raise ValueError("offsets is required")
    return _fp8_call(X, offsets, W, w_scales, x_scales, bias, activation, gate, residual, y_dtype, out, workspace, stream)


def linear_fp8_workspace_bytes(M: int, n_out: int, n_in: int, dtype: torch.dtype, y_dtype: torch.dtype,
                               n_experts: Optional[int] = None) -> int:
    return int(lib().splr_linear_fp8_workspace_bytes(M, n_experts or 0, n_out, n_in, _CODES[dtype], _CODES[y_dtype]))


def linear_fp8_tile(M: int, n_out: int, n_in: int, dtype: torch.dtype, y_dtype: torch.dtype,
                    n_experts: Optional[int] = None) -> Tuple[int, int]:
    """The workgroup tile (rows of W, tokens) of the kernel that these sizes take (splr_linear_fp8_tile)."""
    rows, tokens = ctypes.c_int32(), ctypes.c_int32()
    _check("splr_linear_fp8_tile", lib().splr_linear_fp8_tile(M, n_experts or 0, n_out, n_in, _CODES[dtype], _CODES[y_dtype],
                                                              ctypes.byref(rows), ctypes.byref(tokens)))
    return rows.value, tokens.value


def dense_reconstruct(values: torch.Tensor, meta: torch.Tensor, U: Optional[torch.Tensor],
                      V: Optional[torch.Tensor], n_out: Optional[int] = None, n_in: Optional[int] = None,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """W_hat [n_out, n_in] float32 = S + U V (sizes default to U / V's, else to the tile grid)."""
    if not _is_device(values):
        raise ValueError("values must be a device tensor")
    if n_out is None:
        n_out = U.shape[0] if U is not None else values.shape[0] * 16
    if n_in is None:
        n_in = V.shape[1] if V is not None else values.shape[1] * 64
    _dtype_code(values)
    _check_packed_in(values, meta, n_out, n_in, values.dtype, values.device)
    r = _check_factors(U, V, n_out, n_in, values.dtype, values.device)
    if out is None:
        with torch.cuda.stream(_the_stream(stream)):
            out = torch.empty((n_out, n_in), dtype=torch.float32, device=values.device)
    _expect(out, "out", torch.float32, n_out * n_in, values.device, (n_out, n_in))
    _check("splr_dense_reconstruct",
           lib().splr_dense_reconstruct(_dev(values, "values"), _dev(meta, "meta"), _dev(U, "U"), _dev(V, "V"),
                                        n_out, n_in, r, _dtype_code(values), _dev(out, "out"), _stream(stream)))
    return out


MAX_CHOL_K = 192


def gram_f64(Y: torch.Tensor, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """G = Y^T Y in float64 for float32 Y [n, k] (k <= 192), on the device (splr_gram_f64)."""
    n, k = _matrix(Y, "Y")
    if not 1 <= k <= MAX_CHOL_K:
        raise ValueError(f"Y has {k} columns; splr_gram_f64 takes 1 .. {MAX_CHOL_K}")
    _expect(Y, "Y", torch.float32, n * k, Y.device)
    need = int(lib().splr_gram_workspace_bytes(n, k))
    if need == 0:
        raise ValueError(f"Y of shape {(n, k)} is out of range for splr_gram_f64")
    with torch.cuda.stream(_the_stream(stream)):
        if out is None:
            out = torch.empty((k, k), dtype=torch.float64, device=Y.device)
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=Y.device)
    _expect(out, "out", torch.float64, k * k, Y.device, (k, k))
    if not _is_device(workspace) or workspace.device != Y.device or workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor on Y's device")
    _check("splr_gram_f64", lib().splr_gram_f64(_dev(Y, "Y"), n, k, _dev(out, "out"), _dev(workspace, "workspace"),
                                                workspace.numel(), _stream(stream)))
    return out


def chol_rinv(G: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """R^-1 (float32, upper triangular) for the Cholesky factor of float64 G = R^T R [k, k]
    (splr_chol_rinv); NaN entries when G is not numerically positive definite."""
    k, k2 = _matrix(G, "G")
    if k != k2 or not 1 <= k <= MAX_CHOL_K:
        raise ValueError(f"G must be square with 1 .. {MAX_CHOL_K} rows, got {(k, k2)}")
    _expect(G, "G", torch.float64, k * k, G.device)
    if out is None:
        with torch.cuda.stream(_the_stream(stream)):
            out = torch.empty((k, k), dtype=torch.float32, device=G.device)
    _expect(out, "out", torch.float32, k * k, G.device, (k, k))
    _check("splr_chol_rinv", lib().splr_chol_rinv(_dev(G, "G"), k, _dev(out, "out"), _stream(stream)))
    return out


def version() -> str:
    return lib().splr_version().decode()
