"""Python binding of libsgmv.so, the MI355X SGMV library (C ABI in
``include/sgmv.h``).

Argument marshalling only: every function below checks tensor placement,
dtype and contiguity, passes raw device pointers, sizes and the current HIP
stream to the C function of the same name, and raises on a non-zero status
(the calls of the paged key/value cache, of drafted trees and of several
adapters per token through a small compiled module, ``_kv_binding.so``, the
others through ctypes).
All arithmetic runs in the library's gfx950 kernels. PyTorch supplies device
memory and streams.

If ``libsgmv.so`` has not been built, importing this package raises
``ImportError``: there is no fallback path.
"""
from __future__ import annotations

import ctypes
from pathlib import Path
from typing import Dict, Optional, Tuple

import numpy as np
import torch

_HERE = Path(__file__).resolve().parent
LIBRARY = _HERE / "libsgmv.so"

SGMV_F32 = 0
SGMV_BF16 = 1
SGMV_OK = 0

_DTYPES = {torch.float32: SGMV_F32, torch.bfloat16: SGMV_BF16}

# (name, restype, argtypes) for every symbol include/sgmv.h declares.
_i32, _i64, _vp, _f32, _f64, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double,
                                    ctypes.c_size_t)
EXPORTS = {
    "sgmv_shrink": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp,
                                   _sz, _vp]),
    "sgmv_expand": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _i32, _vp]),
    "sgmv_fused": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                  _f32, _i32, _vp, _sz, _vp]),
    "sgmv_fused_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                          _f32, _i32, _vp]),
    "sgmv_shrink_gather": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                          _vp, _sz, _vp]),
    "sgmv_expand_scatter": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _f32,
                                           _i32, _vp]),
    "sgmv_fused_gather": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32,
                                         _i32, _f32, _i32, _vp, _sz, _vp]),
    "sgmv_fused_layer": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _f32, _i32, _vp, _sz,
                                        _vp]),
    "sgmv_layer_workspace_bytes": (_sz, [_vp, _i32, _i32, _i32, _i32, _i32]),
    "sgmv_admit_adapter": (ctypes.c_int, [_vp, _vp, _vp, _vp, _sz, _sz, _vp, _vp, _i32, _i32, _vp]),
    "sgmv_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "sgmv_build_segments": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp]),
    "sgmv_pool_pointers": (ctypes.c_int, [_vp, _vp, _i32, _i64]),
    "sgmv_check_segments": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32]),
    "sgmv_stream_probe": (ctypes.c_int, [_vp, _sz, _vp, _i32, _vp]),
    "sgmv_workspace_status": (ctypes.c_int, [_vp, _vp, _vp]),
    "sgmv_set_wait_limit": (ctypes.c_uint32, [ctypes.c_uint32]),
    "sgmv_kv_tables": (ctypes.c_int, [_vp, _vp, _i32, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _i32, _vp]),
    "sgmv_rope_table": (ctypes.c_int, [_vp, _i32, _i32, _f64, _i32, _f64, _f64, _f64, _i32, _vp]),
    "sgmv_rope_append": (ctypes.c_int, [_vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _i32,
                                        _i32, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp]),
    "sgmv_paged_attention": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                                            _i32, _vp, _vp, _i32, _i32, _i32, _f32, _i32, _i32, _i32, _vp, _sz,
                                            _vp]),
    "sgmv_paged_attention_workspace_bytes": (_sz, [_i32, _i32]),
    "sgmv_tree_tables": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp]),
    "sgmv_tree_attention": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                                           _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _i32, _vp,
                                           _sz, _vp]),
    "sgmv_tree_accept": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _i32, _vp]),
    "sgmv_kv_commit": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32,
                                      _vp]),
    "sgmv_sort_tokens": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp]),
    "sgmv_sort_tokens_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "sgmv_spread_rows": (ctypes.c_int, [_vp, _i64, _i32, _vp, _i64, _vp, _i32, _i32, _i32, _i32, _vp]),
    "sgmv_combine_rows": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _vp]),
    "sgmv_combine_rows_grad": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32,
                                              _i32, _vp]),
    "sgmv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sgmv_version": (ctypes.c_int, []),
}


def _load() -> ctypes.CDLL:
    if not LIBRARY.exists():
        raise ImportError(f"{LIBRARY} is not built; run `python -m segmented_gather_gemm_sgmv_amd.build`")
    lib = ctypes.CDLL(str(LIBRARY))
    for name, (res, args) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class _NotBuilt:
    """In the place of the paged-cache calls' binding: the package's other calls do without it."""

    def __init__(self, error: ImportError):
        self._error = error

    def __getattr__(self, name):
        raise ImportError(f"{_HERE / '_kv_binding.so'} is not built or does not load; run "
                          "`python -m segmented_gather_gemm_sgmv_amd.build`") from self._error


try:
    from . import _kv_binding  # marshals the paged-cache calls; built with the library
except ImportError as e:
    _kv_binding = _NotBuilt(e)


SGMV_ERR_ALIGN = -5
_ROW_CALLS = ("sgmv_rope_table", "sgmv_rope_append", "sgmv_paged_attention", "sgmv_tree_attention", "sgmv_kv_commit",
              "sgmv_spread_rows", "sgmv_combine_rows", "sgmv_combine_rows_grad")  # their operands are not X, Y and V


class SGMVError(RuntimeError):
    def __init__(self, fn: str, status: int):
        if status == SGMV_ERR_ALIGN and fn in _ROW_CALLS:
            text = "an operand, or the rows of one, not 16-byte aligned"  # the library's text names the SGMV operands
        else:
            text = lib.sgmv_status_string(status).decode()
        super().__init__(f"{fn}: {text} (status {status})")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != SGMV_OK:
        raise SGMVError(fn, status)


def _dev(t: torch.Tensor, name: str, dtype=None, dim=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a stream object
_current_is_capturing = torch._C._cuda_isCurrentStreamCapturing


def _stream(t: torch.Tensor, stream) -> int:
    if stream is None:
        index = t.get_device()
        if index < 0:
            raise ValueError("every tensor must be on a GPU device")
        return _raw_stream(index)
    return _stream_handle(stream)


def _stream_handle(stream) -> int:
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return _DTYPES[t.dtype]


def _workspace_args(t: Optional[torch.Tensor], need: int, like: torch.Tensor, stream):
    if need == 0 and t is None:
        return None, 0
    if t is None:
        t = workspace(like.device, need, stream)
    return _dev(t, "workspace"), t.numel() * t.element_size()


def sgmv_shrink(V: torch.Tensor, X: torch.Tensor, A_ptrs: torch.Tensor, seg_start: torch.Tensor,
                seg_adapter: torch.Tensor, r: int, workspace_buf: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """V[M, r] (fp32, overwritten per segment row) = X[M, d_in] . A_k."""
    M, d_in = X.shape
    if V.shape != (M, r):
        raise ValueError("V must be M x r")
    need = sgmv_workspace_bytes(seg_adapter.numel(), M, d_in, d_in, r, X.dtype)
    ws, ws_bytes = _workspace_args(workspace_buf, need, X, stream)
    st = lib.sgmv_shrink(_dev(V, "V", torch.float32, 2), _dev(X, "X", dim=2),
                         _dev(A_ptrs, "A_ptrs", torch.int64, 1), A_ptrs.numel(),
                         _dev(seg_start, "seg_start", torch.int32, 1),
                         _dev(seg_adapter, "seg_adapter", torch.int32, 1), seg_adapter.numel(),
                         M, d_in, r, _dtype_code(X), ws, ws_bytes, _stream(X, stream))
    _check("sgmv_shrink", st)
    return V


def sgmv_expand(Y: torch.Tensor, V: torch.Tensor, B_ptrs: torch.Tensor, seg_start: torch.Tensor,
                seg_adapter: torch.Tensor, r: int, alpha: float, stream=None) -> torch.Tensor:
    """Y[M, d_out] += (alpha / r) * V . B_k per segment (in place)."""
    M, d_out = Y.shape
    if V.shape != (M, r):
        raise ValueError("V must be M x r")
    st = lib.sgmv_expand(_dev(Y, "Y", dim=2), _dev(V, "V", torch.float32, 2),
                         _dev(B_ptrs, "B_ptrs", torch.int64, 1), B_ptrs.numel(),
                         _dev(seg_start, "seg_start", torch.int32, 1),
                         _dev(seg_adapter, "seg_adapter", torch.int32, 1), seg_adapter.numel(),
                         M, d_out, r, float(alpha), _dtype_code(Y), _stream(Y, stream))
    _check("sgmv_expand", st)
    return Y


def sgmv_workspace_bytes(num_segments: int, M: int, d_in: int, d_out: int, r: int,
                         dtype: torch.dtype) -> int:
    return int(lib.sgmv_workspace_bytes(num_segments, M, d_in, d_out, r, _DTYPES[dtype]))


_workspaces: Dict[Tuple[int, int], torch.Tensor] = {}


def _torch_stream(device: torch.device, stream):
    """`stream` (None, a torch stream or a raw hipStream_t handle) as a torch
    stream object on `device`."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, (torch.cuda.Stream, torch.cuda.ExternalStream)):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


def workspace(device: torch.device, nbytes: int, stream=None) -> torch.Tensor:
    """A zero-filled workspace for sgmv_shrink and sgmv_fused, cached per
    (device, stream).

    Every call leaves the workspace zero again when its kernel completes, so
    one buffer serves every later call on the same stream. The buffer is
    allocated and zero-filled on that stream, so the fill is ordered before
    the calls that use it, and the caching allocator hands a replaced buffer
    to later work on the same stream only."""
    device = torch.device(device)
    if device.index is None:
        device = torch.device(device.type, torch.cuda.current_device())
    s = _torch_stream(device, stream)
    key = (device.index, s.cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        with torch.cuda.device(device), torch.cuda.stream(s):
            ws = torch.zeros(max(nbytes, 1 << 16), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def sgmv_workspace_status(ws: torch.Tensor, stream=None) -> int:
    """The workspace's sticky status word (0, or the OR of SGMV_WS_WAIT_TIMEOUT
    and SGMV_WS_BAD_OFFSETS), read after the work enqueued on `stream`
    (default: the current stream) has completed. A non-zero status stays
    until the workspace is zero-filled again; until then every call on it is
    a no-op."""
    word = ctypes.c_uint32(0)
    _check("sgmv_workspace_status", lib.sgmv_workspace_status(_dev(ws, "workspace"), ctypes.byref(word),
                                                              _stream(ws, stream)))
    return int(word.value)


def sgmv_set_wait_limit(polls: int) -> int:
    """Polls a waiting workgroup makes before it gives up, for calls launched
    from now on (process-wide); returns the previous value."""
    return int(lib.sgmv_set_wait_limit(int(polls)))


SGMV_WS_WAIT_TIMEOUT = 1
SGMV_WS_BAD_OFFSETS = 2


def sgmv_fused(Y: torch.Tensor, X: torch.Tensor, A_ptrs: torch.Tensor, B_ptrs: torch.Tensor,
               seg_start: torch.Tensor, seg_adapter: torch.Tensor, r: int, alpha: float,
               workspace_buf: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y += (alpha / r) * X . A_k . B_k per segment, in one launch (in place)."""
    M, d_in = X.shape
    M2, d_out = Y.shape
    if M2 != M:
        raise ValueError("X and Y must have the same number of rows")
    if A_ptrs.numel() != B_ptrs.numel():
        raise ValueError("A_ptrs and B_ptrs must have one entry per adapter")
    need = sgmv_workspace_bytes(seg_adapter.numel(), M, d_in, d_out, r, X.dtype)
    ws, ws_bytes = _workspace_args(workspace_buf, need, X, stream)
    st = lib.sgmv_fused(_dev(Y, "Y", dim=2), _dev(X, "X", dim=2),
                        _dev(A_ptrs, "A_ptrs", torch.int64, 1), _dev(B_ptrs, "B_ptrs", torch.int64, 1),
                        A_ptrs.numel(), _dev(seg_start, "seg_start", torch.int32, 1),
                        _dev(seg_adapter, "seg_adapter", torch.int32, 1), seg_adapter.numel(),
                        M, d_in, d_out, r, float(alpha), _dtype_code(X), ws, ws_bytes,
                        _stream(X, stream))
    _check("sgmv_fused", st)
    return Y


SGMV_NOALLOC_SCRATCH_BYTES = 16 << 20


def sgmv_fused_noalloc(Y: torch.Tensor, X: torch.Tensor, A_ptrs: torch.Tensor, B_ptrs: torch.Tensor,
                       seg_start: torch.Tensor, seg_adapter: torch.Tensor, r: int, alpha: float,
                       stream=None) -> torch.Tensor:
    """sgmv_fused on the library's static per-device scratch array instead of
    a workspace: nothing is allocated. Calls that overlap in time on one GPU
    must not be made (they share the array)."""
    M, d_in = X.shape
    M2, d_out = Y.shape
    if M2 != M:
        raise ValueError("X and Y must have the same number of rows")
    if A_ptrs.numel() != B_ptrs.numel():
        raise ValueError("A_ptrs and B_ptrs must have one entry per adapter")
    st = lib.sgmv_fused_noalloc(_dev(Y, "Y", dim=2), _dev(X, "X", dim=2),
                                _dev(A_ptrs, "A_ptrs", torch.int64, 1), _dev(B_ptrs, "B_ptrs", torch.int64, 1),
                                A_ptrs.numel(), _dev(seg_start, "seg_start", torch.int32, 1),
                                _dev(seg_adapter, "seg_adapter", torch.int32, 1), seg_adapter.numel(),
                                M, d_in, d_out, r, float(alpha), _dtype_code(X), _stream(X, stream))
    _check("sgmv_fused_noalloc", st)
    return Y


def _rows_arg(rows: torch.Tensor, M: int) -> int:
    if rows.numel() != M:
        raise ValueError("rows must hold one entry per row of the batch")
    return _dev(rows, "rows", torch.int32, 1)


def sgmv_shrink_gather(V: torch.Tensor, X: torch.Tensor, rows: torch.Tensor, A_ptrs: torch.Tensor,
                       seg_start: torch.Tensor, seg_adapter: torch.Tensor, r: int,
                       workspace_buf: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """V[p] (fp32, segment order) = X[rows[p]] . A_k, with X in token order."""
    M, d_in = X.shape
    if V.shape != (M, r):
        raise ValueError("V must be M x r")
    need = sgmv_workspace_bytes(seg_adapter.numel(), M, d_in, d_in, r, X.dtype)
    ws, ws_bytes = _workspace_args(workspace_buf, need, X, stream)
    st = lib.sgmv_shrink_gather(_dev(V, "V", torch.float32, 2), _dev(X, "X", dim=2), _rows_arg(rows, M),
                                _dev(A_ptrs, "A_ptrs", torch.int64, 1), A_ptrs.numel(),
                                _dev(seg_start, "seg_start", torch.int32, 1),
                                _dev(seg_adapter, "seg_adapter", torch.int32, 1), seg_adapter.numel(),
                                M, d_in, r, _dtype_code(X), ws, ws_bytes, _stream(X, stream))
    _check("sgmv_shrink_gather", st)
    return V


def sgmv_expand_scatter(Y: torch.Tensor, V: torch.Tensor, rows: torch.Tensor, B_ptrs: torch.Tensor,
                        seg_start: torch.Tensor, seg_adapter: torch.Tensor, r: int, alpha: float,
                        stream=None) -> torch.Tensor:
    """Y[rows[p]] += (alpha / r) * V[p] . B_k, with Y in token order (in place)."""
    M, d_out = Y.shape
    if V.shape != (M, r):
        raise ValueError("V must be M x r")
    st = lib.sgmv_expand_scatter(_dev(Y, "Y", dim=2), _dev(V, "V", torch.float32, 2), _rows_arg(rows, M),
                                 _dev(B_ptrs, "B_ptrs", torch.int64, 1), B_ptrs.numel(),
                                 _dev(seg_start, "seg_start", torch.int32, 1),
                                 _dev(seg_adapter, "seg_adapter", torch.int32, 1), seg_adapter.numel(),
                                 M, d_out, r, float(alpha), _dtype_code(Y), _stream(Y, stream))
    _check("sgmv_expand_scatter", st)
    return Y


def sgmv_fused_gather(Y: torch.Tensor, X: torch.Tensor, rows: torch.Tensor, A_ptrs: torch.Tensor,
                      B_ptrs: torch.Tensor, seg_start: torch.Tensor, seg_adapter: torch.Tensor, r: int,
                      alpha: float, workspace_buf: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Y[rows[p]] += (alpha / r) * X[rows[p]] . A_k . B_k in one launch, with X
    and Y in token order (in place)."""
    M, d_in = X.shape
    M2, d_out = Y.shape
    if M2 != M:
        raise ValueError("X and Y must have the same number of rows")
    if A_ptrs.numel() != B_ptrs.numel():
        raise ValueError("A_ptrs and B_ptrs must have one entry per adapter")
    need = sgmv_workspace_bytes(seg_adapter.numel(), M, d_in, d_out, r, X.dtype)
    ws, ws_bytes = _workspace_args(workspace_buf, need, X, stream)
    st = lib.sgmv_fused_gather(_dev(Y, "Y", dim=2), _dev(X, "X", dim=2), _rows_arg(rows, M),
                               _dev(A_ptrs, "A_ptrs", torch.int64, 1), _dev(B_ptrs, "B_ptrs", torch.int64, 1),
                               A_ptrs.numel(), _dev(seg_start, "seg_start", torch.int32, 1),
                               _dev(seg_adapter, "seg_adapter", torch.int32, 1), seg_adapter.numel(),
                               M, d_in, d_out, r, float(alpha), _dtype_code(X), ws, ws_bytes,
                               _stream(X, stream))
    _check("sgmv_fused_gather", st)
    return Y


SGMV_MAX_PROJECTIONS = 8


class SgmvProjection(ctypes.Structure):
    """``sgmv_projection`` of include/sgmv.h: one projection of a layer call."""
    _fields_ = [("Y", ctypes.c_void_p), ("X", ctypes.c_void_p), ("A_ptrs", ctypes.c_void_p),
                ("B_ptrs", ctypes.c_void_p), ("num_adapters", ctypes.c_int32), ("d_in", ctypes.c_int32),
                ("d_out", ctypes.c_int32)]


def _projection_array(projections, check=True):
    """(Y, X, A_ptrs, B_ptrs) tuples -> a ctypes array of SgmvProjection."""
    arr = (SgmvProjection * max(1, len(projections)))()
    for q, (Y, X, A_ptrs, B_ptrs) in enumerate(projections):
        if check:
            if X.shape[0] != Y.shape[0]:
                raise ValueError(f"projection {q}: X and Y must have the same number of rows")
            if A_ptrs.numel() != B_ptrs.numel():
                raise ValueError(f"projection {q}: A_ptrs and B_ptrs must have one entry per adapter")
        arr[q] = SgmvProjection(_dev(Y, "Y", dim=2), _dev(X, "X", dim=2),
                                _dev(A_ptrs, "A_ptrs", torch.int64, 1), _dev(B_ptrs, "B_ptrs", torch.int64, 1),
                                A_ptrs.numel(), X.shape[1], Y.shape[1])
    return arr


def sgmv_layer_workspace_bytes(projections, num_segments: int, M: int, r: int, dtype: torch.dtype) -> int:
    arr = _projection_array(projections)
    return int(lib.sgmv_layer_workspace_bytes(arr, len(projections), num_segments, M, r, _DTYPES[dtype]))


def sgmv_fused_layer(projections, seg_start: torch.Tensor, seg_adapter: torch.Tensor, r: int, alpha: float,
                     rows: Optional[torch.Tensor] = None, workspace_buf: Optional[torch.Tensor] = None,
                     stream=None):
    """Every projection (Y, X, A_ptrs, B_ptrs) of one batch in one launch:
    Y += (alpha / r) * X . A_k . B_k per projection (in place). ``rows``: None
    for a batch in segment order, else the token-order index."""
    if not projections:
        return
    Y0, X0 = projections[0][0], projections[0][1]
    M = X0.shape[0]
    for Y, X, _, _ in projections:
        if X.shape[0] != M or Y.shape[0] != M:
            raise ValueError("every projection must have the batch's M rows")
        if X.dtype != X0.dtype or Y.dtype != X0.dtype:
            raise TypeError("every projection must share one dtype")
    arr = _projection_array(projections)
    need = int(lib.sgmv_layer_workspace_bytes(arr, len(projections), seg_adapter.numel(), M, r,
                                              _dtype_code(X0)))
    ws, ws_bytes = _workspace_args(workspace_buf, need, X0, stream)
    rows_p = None if rows is None else _rows_arg(rows, M)
    st = lib.sgmv_fused_layer(arr, len(projections), rows_p, _dev(seg_start, "seg_start", torch.int32, 1),
                              _dev(seg_adapter, "seg_adapter", torch.int32, 1), seg_adapter.numel(), M, r,
                              float(alpha), _dtype_code(X0), ws, ws_bytes, _stream(X0, stream))
    _check("sgmv_fused_layer", st)


def sgmv_build_segments(token_adapter) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """Host: group tokens by adapter. Returns (perm, seg_start, seg_adapter)."""
    ids = np.ascontiguousarray(np.asarray(token_adapter, dtype=np.int32))
    M = int(ids.shape[0])
    perm = np.empty(M, np.int32)
    seg_start = np.empty(M + 1, np.int32)
    seg_adapter = np.empty(max(M, 1), np.int32)
    n = ctypes.c_int32(0)
    st = lib.sgmv_build_segments(ids.ctypes.data, M, perm.ctypes.data, seg_start.ctypes.data,
                                 seg_adapter.ctypes.data, ctypes.byref(n))
    _check("sgmv_build_segments", st)
    return perm, seg_start[: n.value + 1].copy(), seg_adapter[: n.value].copy()


def sgmv_pool_pointers(pool: torch.Tensor) -> torch.Tensor:
    """Device table (int64) of slot addresses of a packed pool tensor P x r x d.

    The table holds a reference to ``pool``, so the memory it points into
    cannot be freed while the table is alive."""
    if pool.dim() != 3 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous P x r x d tensor")
    P = pool.shape[0]
    table = np.empty(max(P, 1), np.uint64)
    slot_bytes = pool.shape[1] * pool.shape[2] * pool.element_size()
    st = lib.sgmv_pool_pointers(table.ctypes.data, ctypes.c_void_p(pool.data_ptr()), P, slot_bytes)
    _check("sgmv_pool_pointers", st)
    out = torch.from_numpy(table[:P].view(np.int64).copy()).to(pool.device)
    out._sgmv_pool = pool
    return out


def sgmv_admit_adapter(A_slot: torch.Tensor, B_slot: torch.Tensor, A_host: torch.Tensor, B_host: torch.Tensor,
                       A_ptrs: torch.Tensor, B_ptrs: torch.Tensor, slot: int, stream=None) -> None:
    """Copy an adapter from host memory into device slots A_slot (r x d_in)
    and B_slot (r x d_out), then point table entry `slot` at them, all in
    stream order. A_host / B_host: CPU tensors of the slots' shape and dtype
    (pinned for an asynchronous copy); keep them alive and unchanged until the
    stream reaches the copy."""
    for name, dev_t, host_t in (("A", A_slot, A_host), ("B", B_slot, B_host)):
        if host_t.device.type != "cpu" or not host_t.is_contiguous():
            raise ValueError(f"{name}_host must be a contiguous CPU tensor")
        if host_t.shape != dev_t.shape or host_t.dtype != dev_t.dtype:
            raise ValueError(f"{name}_host must match {name}_slot in shape and dtype")
    if A_ptrs.numel() != B_ptrs.numel():
        raise ValueError("A_ptrs and B_ptrs must have one entry per adapter")
    st = lib.sgmv_admit_adapter(_dev(A_slot, "A_slot"), _dev(B_slot, "B_slot"), A_host.data_ptr(),
                                B_host.data_ptr(), A_host.numel() * A_host.element_size(),
                                B_host.numel() * B_host.element_size(), _dev(A_ptrs, "A_ptrs", torch.int64, 1),
                                _dev(B_ptrs, "B_ptrs", torch.int64, 1), int(slot), A_ptrs.numel(),
                                _stream(A_slot, stream))
    _check("sgmv_admit_adapter", st)


def sgmv_check_segments(seg_start, seg_adapter, M: int, num_adapters: int) -> None:
    """Host check of segment metadata (numpy or CPU tensors): raises SGMVError
    unless the offsets start at 0, end at M and never decrease, and every
    adapter id lies in the pool."""
    ss = np.ascontiguousarray(np.asarray(seg_start, dtype=np.int32))
    sa = np.ascontiguousarray(np.asarray(seg_adapter, dtype=np.int32))
    if ss.ndim != 1 or sa.ndim != 1 or ss.shape[0] != sa.shape[0] + 1:
        raise ValueError("seg_start must hold one more entry than seg_adapter")
    _check("sgmv_check_segments",
           lib.sgmv_check_segments(ss.ctypes.data, sa.ctypes.data if sa.size else None, sa.shape[0], M,
                                   num_adapters))


class AdapterPool:
    """One projection's adapter pool in HBM: P slots of A (r x d_in) and B
    (r x d_out), packed back to back, with their device pointer tables.

    ``A_ptrs`` / ``B_ptrs`` are what the SGMV calls take. ``admit`` copies an
    adapter from host memory into a slot and points the slot's table entries
    at it, in stream order (sgmv_admit_adapter); the slot's memory is this
    pool's own."""

    def __init__(self, num_adapters: int, d_in: int, d_out: int, r: int, dtype=torch.bfloat16,
                 device="cuda"):
        self.num_adapters, self.d_in, self.d_out, self.r, self.dtype = num_adapters, d_in, d_out, r, dtype
        self.A = torch.zeros((num_adapters, r, d_in), dtype=dtype, device=device)
        self.B = torch.zeros((num_adapters, r, d_out), dtype=dtype, device=device)
        self.A_ptrs = sgmv_pool_pointers(self.A)
        self.B_ptrs = sgmv_pool_pointers(self.B)

    def admit(self, slot: int, A_host: torch.Tensor, B_host: torch.Tensor, stream=None) -> None:
        """Adapter `slot` := (A_host, B_host), CPU tensors of shape r x d_in and
        r x d_out (pinned for an asynchronous copy; keep them alive and
        unchanged until the stream reaches the copy)."""
        if not 0 <= slot < self.num_adapters:
            raise IndexError(f"slot {slot} outside the pool of {self.num_adapters}")
        sgmv_admit_adapter(self.A[slot], self.B[slot], A_host, B_host, self.A_ptrs, self.B_ptrs, slot, stream)


def sgmv_stream_probe(src: torch.Tensor, sink: torch.Tensor, nbytes: Optional[int] = None, stream=None) -> None:
    """Measurement helper: stream-read `nbytes` (default: all) of the device
    tensor `src` with sink.numel() workgroups; sink (int32) receives each
    workgroup's XOR of the words it read."""
    n = src.numel() * src.element_size() if nbytes is None else int(nbytes)
    if n > src.numel() * src.element_size():
        raise ValueError("nbytes exceeds the source tensor")
    st = lib.sgmv_stream_probe(_dev(src, "src"), n, _dev(sink, "sink", torch.int32, 1), sink.numel(),
                               _stream(src, stream))
    _check("sgmv_stream_probe", st)


# -- the paged key/value cache ---------------------------------------------------
SGMV_MAX_REQUESTS = 8192
SGMV_ROPE_PLAIN, SGMV_ROPE_LINEAR, SGMV_ROPE_BY_PARTS = 0, 1, 2


def sgmv_kv_tables(seq_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor, page_size: int,
                   free_pages: torch.Tensor, pool_in: torch.Tensor, pool_out: torch.Tensor, q_start: torch.Tensor,
                   kv_len: torch.Tensor, position: torch.Tensor, slot: torch.Tensor, stream=None) -> None:
    """One step's block tables and slots from the requests' lengths: requests
    that add new_len >= 0 tokens get pages from the ring of free pages, ended
    ones (new_len < 0) give theirs back; q_start, kv_len, position, slot and
    pool_out are written (see include/sgmv.h). Nothing is read on the host."""
    st = _kv_binding.kv_tables(seq_len, new_len, block_table, page_size, free_pages, pool_in, pool_out, q_start, kv_len,
                               position, slot, _stream(seq_len, stream))
    if st:
        raise SGMVError("sgmv_kv_tables", st)


def sgmv_rope_table(max_position: int, rot_dim: int, base: float = 10000.0, kind: int = SGMV_ROPE_PLAIN,
                    factor: float = 1.0, beta_fast: float = 32.0, beta_slow: float = 1.0, original_max: int = 0,
                    device="cuda", stream=None) -> torch.Tensor:
    """The rotary table [max_position, rot_dim / 2, 2] (cos, sin) that
    sgmv_rope_append takes; see include/sgmv.h for the scalings. Kept for as
    long as the model is served. Allocated and written on `stream` (the current
    one, if None): work on other streams waits for that before it reads it."""
    device = torch.device(device)
    with torch.cuda.device(device), torch.cuda.stream(_torch_stream(device, stream)):
        table = torch.empty((max_position, rot_dim // 2, 2), dtype=torch.float32, device=device)
        st = lib.sgmv_rope_table(_dev(table, "table"), max_position, rot_dim, base, kind, factor, beta_fast, beta_slow,
                                 original_max, _stream(table, stream))
    _check("sgmv_rope_table", st)
    return table


def sgmv_rope_append(q_out: Optional[torch.Tensor], q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                     v: Optional[torch.Tensor], K_cache: Optional[torch.Tensor], V_cache: Optional[torch.Tensor],
                     position: torch.Tensor, slot: Optional[torch.Tensor], table: Optional[torch.Tensor],
                     interleaved: bool = False, stream=None) -> None:
    """q_out = q rotated by each token's position; k, rotated, and v written to
    the paged cache at each token's slot. Rows [T, heads, head_dim] with any
    row stride; q_out may be q; q (with q_out) or k, v and the cache may be
    None. table: of sgmv_rope_table (its rot_dim elements of a head turn), or
    None to copy only."""
    st = _kv_binding.rope_append(q_out, q, k, v, K_cache, V_cache, position, slot, table, interleaved,
                                 _stream(position, stream))
    if st:
        raise SGMVError("sgmv_rope_append", st)


SGMV_ATTENTION_COUNTER_BYTES = 8192
_attention_workspaces: Dict[tuple, torch.Tensor] = {}


def _capturing(index: int, stream) -> bool:
    """Whether `stream` (None: device `index`'s current one) is being captured into a graph."""
    if index == torch.cuda.current_device() and (stream is None or _stream_handle(stream) == _raw_stream(index)):
        return _current_is_capturing()
    with torch.cuda.device(index), torch.cuda.stream(_torch_stream(torch.device("cuda", index), stream)):
        return _current_is_capturing()


def _new_attention_workspace(index: int, head_dim: int, dtype: torch.dtype, stream) -> torch.Tensor:
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    nbytes = int(lib.sgmv_paged_attention_workspace_bytes(head_dim, _DTYPES[dtype]))
    with torch.cuda.device(index), torch.cuda.stream(_torch_stream(torch.device("cuda", index), stream)):
        ws = torch.empty(max(nbytes, SGMV_ATTENTION_COUNTER_BYTES), dtype=torch.uint8, device=f"cuda:{index}")
        ws[:SGMV_ATTENTION_COUNTER_BYTES].zero_()
    return ws


def attention_workspace(device: torch.device, head_dim: int, dtype: torch.dtype, stream=None) -> torch.Tensor:
    """A workspace for sgmv_paged_attention with its counters cleared, cached
    per (device, stream, dtype, head width). It is not the SGMV calls'
    workspace. Not made while its stream is being captured into a graph: the
    clearing would then be a node of that graph, not done, and the memory the
    graph's."""
    device = torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    handle = _raw_stream(index) if stream is None else _torch_stream(device, stream).cuda_stream
    key = (index, handle, dtype, head_dim)
    ws = _attention_workspaces.get(key)
    if ws is None:
        if _capturing(index, stream):
            raise RuntimeError("attention_workspace: this stream has none yet and is being captured; make it before the capture")
        ws = _attention_workspaces[key] = _new_attention_workspace(index, head_dim, dtype, stream)
    return ws


def sgmv_paged_attention(out: torch.Tensor, q: torch.Tensor, K_cache: torch.Tensor, V_cache: torch.Tensor,
                         block_table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, scale: float,
                         max_q_len: int, window: int = 0, sinks: int = 0, lse: Optional[torch.Tensor] = None,
                         workspace_buf: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[T, q_heads, head_dim] = attention of each request's new tokens (rows
    q_start[b] .. of q) over its cached ones, themselves included: causal, with
    window > 0 only the last `window` keys and the first `sinks`. lse
    (optional, fp32 [T, q_heads]): log of the weights' sum. max_q_len: the
    largest number of new tokens of a request.

    Without workspace_buf a call uses its stream's cached workspace. One that
    is being captured into a graph uses memory of the graph instead (up to 77
    MB, which the graph's calls share), and clears the counters there (8 KB; a
    node of 1.5 us), so that graphs may be replayed in any order, on any stream
    and beside other calls; with a workspace_buf of the caller's there is no
    such node, and what uses that buffer must not overlap in time."""
    handle = _stream(q, stream)
    ws = _attention_workspace_of(q, handle, workspace_buf, stream)
    st = _kv_binding.paged_attention(out, q, K_cache, V_cache, block_table, q_start, kv_len, scale, max_q_len, window,
                                     sinks, lse, ws, handle)
    if st:
        raise SGMVError("sgmv_paged_attention", st)
    return out


def _attention_workspace_of(q: torch.Tensor, handle: int, workspace_buf: Optional[torch.Tensor], stream) -> torch.Tensor:
    """The workspace of an attention call on `stream` (raw: handle)."""
    if workspace_buf is not None:
        return workspace_buf
    if _capturing(q.get_device(), stream):
        return _new_attention_workspace(q.get_device(), q.shape[-1], q.dtype, stream)
    ws = _attention_workspaces.get((q.get_device(), handle, q.dtype, q.shape[-1]))
    return attention_workspace(q.device, q.shape[-1], q.dtype, stream) if ws is None else ws


# -- drafted trees -----------------------------------------------------------------
SGMV_MAX_TREE_WORDS = 32


def sgmv_tree_tables(parent: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, position: torch.Tensor,
                     mask: torch.Tensor, stream=None) -> None:
    """Positions and masks of a step that verifies a tree of drafted tokens per
    request: parent[T] holds each new token's parent among its request's new
    tokens (any value outside [0, its own index): none). position[T] and
    mask[T, words] (int32; bit m % 32 of word m / 32 is new token m) are
    written: a token is as far behind the cached ones as it is deep, and sees
    them, its ancestors and itself."""
    st = _kv_binding.tree_tables(parent, q_start, kv_len, position, mask, _stream(parent, stream))
    if st:
        raise SGMVError("sgmv_tree_tables", st)


def sgmv_tree_attention(out: torch.Tensor, q: torch.Tensor, K_cache: torch.Tensor, V_cache: torch.Tensor,
                        block_table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, mask: torch.Tensor,
                        scale: float, max_q_len: int, window: int = 0, sinks: int = 0,
                        lse: Optional[torch.Tensor] = None, workspace_buf: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """sgmv_paged_attention whose new tokens see, of each other, those of their
    mask (sgmv_tree_tables, or any bits), and the tokens cached before the step
    (with window > 0 the last `window` of what they see, and the first
    `sinks`; a window is at least max_q_len). Workspace as there."""
    handle = _stream(q, stream)
    ws = _attention_workspace_of(q, handle, workspace_buf, stream)
    st = _kv_binding.tree_attention(out, q, K_cache, V_cache, block_table, q_start, kv_len, scale, max_q_len, window,
                                    sinks, lse, ws, handle, mask)
    if st:
        raise SGMVError("sgmv_tree_attention", st)
    return out


def sgmv_tree_accept(parent: torch.Tensor, token: torch.Tensor, target: torch.Tensor, slot: torch.Tensor,
                     q_start: torch.Tensor, kv_len: torch.Tensor, page_size: int, block_table: torch.Tensor,
                     free_pages: torch.Tensor, pool_in: torch.Tensor, pool_out: torch.Tensor, path: torch.Tensor,
                     accepted: torch.Tensor, next_token: torch.Tensor, kept_len: torch.Tensor, stream=None) -> None:
    """The drafted tokens that the model agrees with: from a request's token 0
    on, the first child that holds target, the model's own token there. Writes
    path (row q_start[b] + d: index of the d-th accepted token, -1 past the
    last), accepted, next_token, kept_len and pool_out, and gives the pages past
    kept_len back to the ring (see include/sgmv.h). Nothing is read on the host."""
    st = _kv_binding.tree_accept(parent, token, target, slot, q_start, kv_len, page_size, block_table, free_pages, pool_in,
                                 pool_out, path, accepted, next_token, kept_len, _stream(parent, stream))
    if st:
        raise SGMVError("sgmv_tree_accept", st)


def sgmv_kv_commit(K_cache: torch.Tensor, V_cache: torch.Tensor, slot: torch.Tensor, q_start: torch.Tensor,
                   path: torch.Tensor, stream=None) -> None:
    """Accepted tokens' keys and values to the slots of a plain step: row
    slot[q_start[b] + d] becomes row slot[q_start[b] + path[q_start[b] + d]].
    One layer's caches [pages, kv_heads, page_size, head_dim], or all layers'
    with a leading dimension. Once per sgmv_tree_accept."""
    st = _kv_binding.kv_commit(K_cache, V_cache, slot, q_start, path, _stream(slot, stream))
    if st:
        raise SGMVError("sgmv_kv_commit", st)


# -- several adapters per token ------------------------------------------------------
SGMV_MAX_CHOICES, SGMV_MAX_SORTED_ADAPTERS = 64, 4096


def sgmv_sort_tokens(choice: torch.Tensor, num_adapters: int, seg_start: torch.Tensor, seg_adapter: torch.Tensor,
                     order: torch.Tensor, place: torch.Tensor, workspace_buf: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Sorts the choices [T, choices] (adapters; outside [0, num_adapters): none)
    by adapter, on the GPU: order[i] is the choice (token * choices + which) in
    row i, place[T, choices] each choice's row (-1: none), and seg_start,
    seg_adapter are the segments that the SGMV calls take, the empty ones last
    (seg_adapter holds at least min(num_adapters, T * choices) entries). With
    one choice per token order is their `rows`."""
    ws = workspace_buf
    if ws is None and choice.dim() == 2:
        need = int(lib.sgmv_sort_tokens_workspace_bytes(choice.shape[0], choice.shape[1], int(num_adapters)))
        if need and choice.is_cuda:  # the call's own, so that calls on other streams and replays have nothing to do with it
            with torch.cuda.stream(None if stream is None else _torch_stream(choice.device, stream)):
                ws = torch.empty(need, dtype=torch.uint8, device=choice.device)
    st = _kv_binding.sort_tokens(choice, num_adapters, seg_start, seg_adapter, order, place, ws, _stream(choice, stream))
    if st:
        raise SGMVError("sgmv_sort_tokens", st)


def sgmv_spread_rows(Xs: torch.Tensor, X: torch.Tensor, place: torch.Tensor, stream=None) -> torch.Tensor:
    """Xs[place[t, j]] = X[t]: the tokens' rows in segment order. Rows that no
    choice has are left as they were. The gradient is sgmv_combine_rows of dXs,
    without weights."""
    st = _kv_binding.spread_rows(Xs, X, place, _stream(X, stream))
    if st:
        raise SGMVError("sgmv_spread_rows", st)
    return Xs


def sgmv_combine_rows(Y: torch.Tensor, Ys: torch.Tensor, place: torch.Tensor, weight: Optional[torch.Tensor] = None,
                      base: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y[t] = base[t] + sum_j weight[t, j] * Ys[place[t, j]], summed in fp32 and
    rounded once. weight: fp32 [T, choices], None for ones; base: None for
    zeros, Y itself, or rows of its own."""
    st = _kv_binding.combine_rows(Y, Ys, place, weight, base, _stream(Y, stream))
    if st:
        raise SGMVError("sgmv_combine_rows", st)
    return Y


def sgmv_combine_rows_grad(dYs: Optional[torch.Tensor], dweight: Optional[torch.Tensor], dY: torch.Tensor,
                           Ys: Optional[torch.Tensor], place: torch.Tensor, weight: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """Gradients of sgmv_combine_rows: dYs[place[t, j]] = weight[t, j] * dY[t] and
    dweight[t, j] = dY[t] . Ys[place[t, j]] (fp32). Either may be None. Each
    choice has a row of its own, as sgmv_sort_tokens gives it. The gradient of
    base is dY."""
    st = _kv_binding.combine_rows_grad(dYs, dweight, dY, Ys, place, weight, _stream(dY, stream))
    if st:
        raise SGMVError("sgmv_combine_rows_grad", st)


class PagedKVCache:
    """Paged K and V of one or more layers, with the one block table, the ring
    of free pages and the lengths that their requests share; all of it on
    `device`, which need not be the current one, carried from step to step
    without the host reading it. Made on that device's current stream: work on
    other streams waits for it.

    A step: ``step`` (slots for the step's new tokens, ended requests' pages
    back), then per layer ``append`` and ``attend``. Requests are the rows
    0 .. max_requests - 1; one that ended is free for another at once, its
    pages from the next step on.

    A step that verifies trees of drafted tokens: ``step``, then ``draft`` (positions
    and masks), per layer ``append`` and ``attend`` with the mask, then ``accept``
    (lengths and pages of the tokens that the model agrees with) and ``commit``.

    Graphs: lengths and pool are kept twice and change places at every step and
    every accept, so steps are captured two at a time (or another even number;
    a drafted step with its accept is two), and an even number of other changes
    lies between replays. The position and slot that a
    captured call uses stay where they are for as long as the cache lives, and
    serve the other steps of that many tokens too."""

    def __init__(self, num_pages: int, page_size: int, kv_heads: int, head_dim: int, max_requests: int,
                 max_blocks: int, num_layers: int = 1, dtype=torch.bfloat16, device="cuda"):
        self.page_size = page_size
        shape = (num_layers, num_pages, kv_heads, page_size, head_dim)
        self.K, self.V = torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device)

        def ints(*size):
            return torch.zeros(size, dtype=torch.int32, device=device)

        self.block_table = ints(max_requests, max_blocks).fill_(-1)
        self.free_pages = torch.arange(num_pages, dtype=torch.int32, device=device)
        self._len, self._pool = [ints(max_requests), ints(max_requests)], [ints(4), ints(4)]
        self._pool[0][1] = num_pages
        self.q_start = ints(max_requests + 1)
        self.position = self.slot = ints(0)
        self._slot_stream = _stream(self.slot, None)
        self._held = {}  # by number of tokens: (position, slot, their stream) that graphs refer to

    def _use_slots(self, stream) -> None:
        """Keeps position and slot, which a later step may replace, until `stream`'s work on them is done; for good
        if that work is being captured."""
        if _capturing(self.slot.get_device(), stream):
            self._held[self.slot.numel()] = (self.position, self.slot, self._slot_stream)
        if _stream(self.slot, stream) != self._slot_stream:
            s = _torch_stream(self.slot.device, stream)
            self.position.record_stream(s)
            self.slot.record_stream(s)

    @property
    def kv_len(self) -> torch.Tensor:
        """Tokens each request has in the cache, the last step's included."""
        return self._len[0]

    @property
    def pool(self) -> torch.Tensor:
        """[ring's first entry, free pages, requests the last step refused, its tokens]."""
        return self._pool[0]

    def step(self, new_len: torch.Tensor, num_tokens: int, stream=None) -> None:
        """The next step: request b adds new_len[b] tokens (num_tokens in all),
        or has ended (new_len[b] < 0). Sets q_start, kv_len, position, slot.

        A request that does not fit is refused: pool[2] counts them, its kv_len
        stays, its tokens' slots are -1, and their rows of this step's append
        and attend mean nothing. They are to be offered again."""
        if num_tokens in self._held:
            self.position, self.slot, self._slot_stream = self._held[num_tokens]
        elif self.slot.numel() != num_tokens:
            with torch.cuda.stream(_torch_stream(self.slot.device, stream)):
                self.position = torch.empty(num_tokens, dtype=torch.int32, device=self.slot.device)
                self.slot = torch.empty_like(self.position)
            self._slot_stream = _stream(self.slot, stream)
        self._use_slots(stream)
        sgmv_kv_tables(self._len[0], new_len, self.block_table, self.page_size, self.free_pages, self._pool[0],
                       self._pool[1], self.q_start, self._len[1], self.position, self.slot, stream)
        self._len.reverse()
        self._pool.reverse()

    def append(self, q_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
               table: Optional[torch.Tensor], interleaved: bool = False, layer: int = 0, stream=None) -> None:
        """q_out = q rotated; k (rotated) and v of the step's tokens to the cache."""
        self._use_slots(stream)
        sgmv_rope_append(q_out, q, k, v, self.K[layer], self.V[layer], self.position, self.slot, table, interleaved,
                         stream)

    def attend(self, out: torch.Tensor, q: torch.Tensor, scale: float, max_q_len: int, window: int = 0,
               sinks: int = 0, lse: Optional[torch.Tensor] = None, layer: int = 0, stream=None,
               workspace_buf: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        """out = attention of the step's tokens over what their requests have cached; with the mask of ``draft`` a
        drafted token sees its ancestors only, of the step's tokens."""
        if mask is not None:
            return sgmv_tree_attention(out, q, self.K[layer], self.V[layer], self.block_table, self.q_start, self.kv_len,
                                       mask, scale, max_q_len, window, sinks, lse, workspace_buf, stream)
        return sgmv_paged_attention(out, q, self.K[layer], self.V[layer], self.block_table, self.q_start, self.kv_len,
                                    scale, max_q_len, window, sinks, lse, workspace_buf, stream)

    def draft(self, parent: torch.Tensor, mask: torch.Tensor, stream=None) -> None:
        """The step's tokens are trees: parent[T] as for sgmv_tree_tables. Sets position (what ``append`` rotates by) and
        writes mask [T, words]."""
        self._use_slots(stream)
        sgmv_tree_tables(parent, self.q_start, self.kv_len, self.position, mask, stream)

    def accept(self, parent: torch.Tensor, token: torch.Tensor, target: torch.Tensor, path: torch.Tensor,
               accepted: torch.Tensor, next_token: torch.Tensor, stream=None) -> None:
        """Keeps, of the step's trees, what the model agrees with: target[T] is its own token after each of the step's
        tokens. Writes path [T], accepted and next_token [max_requests] (sgmv_tree_accept); kv_len and the pool are those
        without the other tokens from here on. Once per step, after its last ``attend``.

        All requests are verified: a prompt in a drafted step is a chain (parent[i] = i - 1) of at most 32 * words tokens,
        and is kept whole where target[i] is its own token i + 1 (the model's at its last one only)."""
        self._use_slots(stream)
        sgmv_tree_accept(parent, token, target, self.slot, self.q_start, self._len[0], self.page_size, self.block_table,
                         self.free_pages, self._pool[0], self._pool[1], path, accepted, next_token, self._len[1], stream)
        self._len.reverse()
        self._pool.reverse()

    def commit(self, path: torch.Tensor, stream=None) -> None:
        """The accepted tokens' keys and values, of every layer, to their places. Once per ``accept``, before the next
        ``step``."""
        self._use_slots(stream)
        sgmv_kv_commit(self.K, self.V, self.slot, self.q_start, path, stream)


def sgmv_version() -> int:
    return int(lib.sgmv_version())


__all__ = ["sgmv_shrink", "sgmv_expand", "sgmv_fused", "sgmv_shrink_gather", "sgmv_expand_scatter",
           "sgmv_fused_gather", "sgmv_fused_layer", "sgmv_layer_workspace_bytes", "SgmvProjection",
           "SGMV_MAX_PROJECTIONS", "sgmv_admit_adapter", "sgmv_check_segments", "AdapterPool", "sgmv_stream_probe",
           "sgmv_workspace_bytes", "sgmv_build_segments",
           "sgmv_pool_pointers", "sgmv_version", "workspace", "SGMVError", "lib", "EXPORTS",
           "LIBRARY", "SGMV_F32", "SGMV_BF16", "sgmv_workspace_status", "sgmv_set_wait_limit",
           "sgmv_kv_tables", "sgmv_rope_table", "sgmv_rope_append", "sgmv_paged_attention", "attention_workspace", "PagedKVCache",
           "SGMV_MAX_REQUESTS", "SGMV_ATTENTION_COUNTER_BYTES", "SGMV_ROPE_PLAIN", "SGMV_ROPE_LINEAR", "SGMV_ROPE_BY_PARTS",
           "sgmv_tree_tables", "sgmv_tree_attention", "sgmv_tree_accept", "sgmv_kv_commit", "SGMV_MAX_TREE_WORDS",
           "sgmv_sort_tokens", "sgmv_spread_rows", "sgmv_combine_rows", "sgmv_combine_rows_grad", "SGMV_MAX_CHOICES",
           "SGMV_MAX_SORTED_ADAPTERS",
           "SGMV_WS_WAIT_TIMEOUT", "SGMV_WS_BAD_OFFSETS", "sgmv_fused_noalloc", "SGMV_NOALLOC_SCRATCH_BYTES"]
