"""Thin Python binding of libtb.so (ctypes).

Argument marshalling only: every step of the projection runs in the HIP
kernels behind the C ABI declared in ``include/tb.h``.  PyTorch supplies
device memory and the current HIP stream.  There is no fallback: if the
library is missing or fails to load, the import raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtb.so")

TB_OK, TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP = 0, 1, 2, 3
TB_F32, TB_BF16, TB_E4M3, TB_INT8 = 0, 1, 2, 3
TB_SCALE_F32, TB_SCALE_E8M0 = 0, 1
FP8_BLOCK = 128
FP8_MAX_IN_DIM = 1 << 22
FP8_MAX_TOKENS = 1 << 24
INT8_MAX_IN_DIM = 65536
MAX_NORM_DIM = 32768
MAX_AXES = 4
TB_PAIRS_HALF, TB_PAIRS_INTERLEAVED, TB_PAIRS_AXIS = 0, 1, 2
MAX_HEAD_DIM = 1024
MAX_HEADS = 65535
MAX_HEAD_TOKENS = 1 << 25
MAX_GROUP = 8
WORKSPACE_CONTROL_BYTES = MAX_GROUP * 65536
FROBENIUS_WORKSPACE_BYTES = 65536

EXPORTED = (
    "tb_band_index", "tb_linear_forward_workspace_size", "tb_linear_forward", "tb_dense_forward",
    "tb_linear_forward_group_workspace_size", "tb_linear_forward_group",
    "tb_reconstruct_weight", "tb_rel_frobenius_error", "tb_reconstruction_error",
    "tb_shared_block", "tb_row_scale", "tb_lowrank_factors_workspace_size", "tb_lowrank_factors",
    "tb_lowrank_factors_batch", "tb_refine_shared_block_workspace_size", "tb_refine_shared_block",
    "tb_debug_set_wait_polls", "tb_status_string", "tb_last_error", "tb_linear_forward_no_alloc",
    "tb_quantize_activations", "tb_reconstruct_weight_fp8", "tb_dense_forward_fp8_workspace_size",
    "tb_dense_forward_fp8", "tb_head_norm_rotate", "tb_head_norm_rotate_axes",
    "tb_quantize_rows_int8", "tb_dense_forward_int8_workspace_size", "tb_dense_forward_int8", "tb_residual_norm",
)
NO_ALLOC_SCRATCH_BYTES = 96 << 20
DEFAULT_WAIT_POLLS = 1 << 20
MAX_BAND_LAYERS = 128
MAX_PROBE = 512


class Projection(ctypes.Structure):
    """tb_projection: one member of a grouped forward call."""
    _fields_ = [("x", ctypes.c_void_p), ("s", ctypes.c_void_p), ("w0", ctypes.c_void_p), ("u", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("y", ctypes.c_void_p), ("out_dim", ctypes.c_int64),
                ("in_dim", ctypes.c_int64), ("rank", ctypes.c_int64)]


class HeadPart(ctypes.Structure):
    """tb_head_part: one tensor of heads in tb_head_norm_rotate."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("x_token_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("y_token_stride", ctypes.c_int64), ("y_head_stride", ctypes.c_int64)]


class Residual(ctypes.Structure):
    """tb_residual: the tensors of tb_residual_norm."""
    _fields_ = [("h", ctypes.c_void_p), ("y", ctypes.c_void_p), ("post_weight", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("h_out", ctypes.c_void_p),
                ("z", ctypes.c_void_p), ("z_scale", ctypes.c_void_p), ("h_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("h_out_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("gate_rows", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("gate_channels", ctypes.c_int64)]


class TBError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libtb status {status}: {message}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m rank_factored_linear_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    c_i32, c_i64, c_p, c_sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    lib.tb_band_index.argtypes = [c_i32, c_i32, c_i32, ctypes.POINTER(c_i32)]
    lib.tb_linear_forward_workspace_size.argtypes = [c_i64, c_i64, c_i64, c_i64, ctypes.c_int, ctypes.POINTER(c_sz)]
    lib.tb_linear_forward.argtypes = [c_p, c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i64, c_i64, ctypes.c_int, c_p, c_sz, c_p]
    lib.tb_dense_forward.argtypes = [c_p, c_p, c_p, c_i64, c_i64, c_i64, ctypes.c_int, c_p, c_sz, c_p]
    lib.tb_linear_forward_group_workspace_size.argtypes = [c_i32, ctypes.POINTER(Projection), c_i64, ctypes.c_int,
                                                           ctypes.POINTER(c_sz)]
    lib.tb_linear_forward_group.argtypes = [c_i32, ctypes.POINTER(Projection), c_i64, ctypes.c_int, c_p, c_sz, c_p]
    lib.tb_reconstruct_weight.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int, c_p]
    lib.tb_rel_frobenius_error.argtypes = [c_p, c_p, c_i64, c_i64, ctypes.c_int, c_p, c_p, c_sz, c_p]
    lib.tb_reconstruction_error.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int,
                                            c_p, c_p, c_sz, c_p]
    lib.tb_shared_block.argtypes = [ctypes.POINTER(c_p), c_i32, c_i64, c_i64, ctypes.c_int, c_p, c_p]
    lib.tb_row_scale.argtypes = [c_p, c_p, c_i64, c_i64, ctypes.c_int, c_p, c_p]
    lib.tb_lowrank_factors_workspace_size.argtypes = [c_i64, c_i64, c_i64, c_i64, ctypes.POINTER(c_sz)]
    lib.tb_lowrank_factors.argtypes = [c_p, c_p, c_p, c_i64, c_i64, c_i64, ctypes.c_int, c_p, c_i64, c_i32, c_p, c_p,
                                       c_p, c_sz, c_p]
    lib.tb_lowrank_factors_batch.argtypes = [ctypes.POINTER(c_p), c_i32, ctypes.POINTER(c_p), c_p, c_i64, c_i64, c_i64,
                                             ctypes.c_int, c_p,
                                             c_i64, c_i32, c_p, c_p, c_p, c_sz, c_p]
    lib.tb_refine_shared_block_workspace_size.argtypes = [c_i64, c_i64, c_i32, c_i64, ctypes.POINTER(c_sz)]
    lib.tb_refine_shared_block.argtypes = [ctypes.POINTER(c_p), ctypes.POINTER(c_p), ctypes.POINTER(c_p),
                                           ctypes.POINTER(c_p), c_i32, c_i64, c_i64, c_i64, ctypes.c_int, c_p, c_p,
                                           c_p, c_sz, c_p]
    lib.tb_debug_set_wait_polls.argtypes = [c_i32]
    lib.tb_linear_forward_no_alloc.argtypes = [c_p, c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i64, c_i64, ctypes.c_int,
                                               c_p]
    lib.tb_quantize_activations.argtypes = [c_p, c_p, c_p, c_i64, c_i64, ctypes.c_int, ctypes.c_int, c_p]
    lib.tb_reconstruct_weight_fp8.argtypes = [c_p, c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i64, ctypes.c_int,
                                              ctypes.c_int, c_p]
    lib.tb_dense_forward_fp8_workspace_size.argtypes = [c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                        ctypes.POINTER(c_sz)]
    lib.tb_dense_forward_fp8.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_int, c_p, c_sz, c_p]
    lib.tb_head_norm_rotate.argtypes = [c_i32, c_p, c_i64, c_i64, c_i64, c_i32, c_p, c_p,
                                        ctypes.c_float, ctypes.c_float, ctypes.c_int, c_p]
    lib.tb_head_norm_rotate_axes.argtypes = [c_i32, c_p, c_i64, c_i64, c_i64, ctypes.c_int, c_i32, c_p, c_p, c_p, c_i32,
                                             ctypes.c_float, ctypes.c_float, ctypes.c_int, c_p]
    lib.tb_quantize_rows_int8.argtypes = [c_p, c_p, c_p, c_i64, c_i64, ctypes.c_int, c_p]
    lib.tb_dense_forward_int8_workspace_size.argtypes = [c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int,
                                                         ctypes.POINTER(c_sz)]
    lib.tb_dense_forward_int8.argtypes = [c_p, c_p, c_p, c_p, c_p, c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int, c_p,
                                          c_sz, c_p]
    lib.tb_residual_norm.argtypes = [c_p, c_i64, c_i64, ctypes.c_float, ctypes.c_float, ctypes.c_float, c_i32,
                                     ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, c_p]
    lib.tb_status_string.argtypes = [ctypes.c_int]
    lib.tb_status_string.restype = ctypes.c_char_p
    lib.tb_last_error.argtypes = []
    lib.tb_last_error.restype = ctypes.c_char_p
    for name in ("tb_band_index", "tb_linear_forward_workspace_size", "tb_linear_forward",
                 "tb_linear_forward_group_workspace_size", "tb_linear_forward_group",
                 "tb_reconstruct_weight", "tb_rel_frobenius_error", "tb_reconstruction_error"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()


def _check(status: int) -> None:
    if status != TB_OK:
        raise TBError(status, lib.tb_last_error().decode())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return TB_BF16
    if dt == torch.float32:
        return TB_F32
    raise TBError(TB_ERR_UNSUPPORTED, f"dtype {dt} is not supported (bfloat16 or float32)")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    # The raw handle, without building a torch.cuda.Stream around it on every call.
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _need_device(*ts):
    """Every tensor lives on the current GPU (the device the library launches on)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        d = t.get_device()   # -1 on the CPU
        if dev is None and d >= 0:
            dev = torch.cuda.current_device()
        if d != dev or d < 0:
            if d < 0:
                raise TBError(TB_ERR_INVALID_ARGUMENT, "tensors must live on the GPU")
            raise TBError(TB_ERR_INVALID_ARGUMENT, f"tensor on {t.device}, but the current device is cuda:{dev}")


def _need_cuda(*ts):
    """Every tensor is contiguous and lives on the current GPU."""
    _need_device(*ts)
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise TBError(TB_ERR_UNSUPPORTED, "tensors must be contiguous")


def _here(ts: list) -> int:
    """The device of tensors that are contiguous and live on the current GPU (else _need_cuda says what is wrong)."""
    dev = ts[0].get_device()
    fine = dev >= 0 and dev == torch.cuda.current_device()
    for t in ts:
        fine = fine and t.get_device() == dev and t.is_contiguous()
    if not fine:
        _need_cuda(*ts)
    return dev


# Shape and dtype checks run before the device checks and before anything
# crosses the C ABI: the library sees raw pointers only, so a mis-sized
# tensor would otherwise become out-of-bounds device reads or writes.


def _expect(name: str, t: torch.Tensor, shape, dtype: torch.dtype | None = None) -> None:
    if t.shape != shape:   # (torch.Size compares as a tuple)
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"{name} must be {list(shape)}, got {list(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"{name} must be {dtype}, got {t.dtype}")


def _expect_out(out: torch.Tensor | None, shape, dtype: torch.dtype | None = None) -> None:
    if out is not None:
        _expect("out", out, shape, dtype)


def _output(out: torch.Tensor | None, shape, dtype: torch.dtype, like: torch.Tensor) -> torch.Tensor:
    """A new output of this shape and dtype on like's device, or the caller's `out` after checking it."""
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _expect("out", out, shape, dtype)
    if out.device != like.device:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"out is on {out.device}, the inputs on {like.device}")
    return out


def _projection_dims(x, s, W0, U, V):
    """(m, out_dim, in_dim, rank, U, V) of one projection after checking every operand against x and W0:
    x [m, in], W0 [out, in], s [out] or None, U [out, rank] and V [in, rank] or both None; one dtype.
    A rank-0 U/V pair becomes None."""
    if x.dim() != 2 or W0.dim() != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "x must be [m, in] and W0 [out, in]")
    _dtype_code(x.dtype)
    m, in_dim = x.shape
    out_dim = W0.shape[0]
    _expect("W0", W0, (out_dim, in_dim), x.dtype)
    if s is not None:
        _expect("s", s, (out_dim,), x.dtype)
    if (U is None) != (V is None):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "U and V are given together or not at all")
    rank = 0
    if U is not None:
        if U.dim() != 2:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "U must be [out, rank]")
        rank = U.shape[1]
        _expect("U", U, (out_dim, rank), x.dtype)
        _expect("V", V, (in_dim, rank), x.dtype)
        if rank == 0:
            U = V = None
    return m, out_dim, in_dim, rank, U, V


def _workspace_bytes(ws: torch.Tensor) -> int:
    _need_cuda(ws)
    return ws.numel() * ws.element_size()


# ---------------------------------------------------------------------------
# Workspace: one zero-initialised buffer per (device, stream), grown on
# demand.  Its control words are zero when created and the library keeps
# them consistent from call to call.
# ---------------------------------------------------------------------------
_ws_lock = threading.Lock()
_ws: dict = {}


def workspace_for(nbytes: int) -> torch.Tensor:
    dev = torch.cuda.current_device()
    key = (dev, torch.cuda.current_stream().cuda_stream)
    with _ws_lock:
        buf = _ws.get(key)
        if buf is None or buf.numel() < nbytes:
            size = max(nbytes, WORKSPACE_CONTROL_BYTES)
            size = (size + (1 << 20) - 1) >> 20 << 20
            buf = torch.zeros(size, dtype=torch.uint8, device=f"cuda:{dev}")
            _ws[key] = buf
        return buf


def set_wait_polls(polls: int = DEFAULT_WAIT_POLLS) -> None:
    """Bound of the decode kernels' wait for x . V (tb_debug_set_wait_polls); 0 forces the timeout path."""
    _check(lib.tb_debug_set_wait_polls(polls))


def workspace_error_word() -> int:
    """Sticky error word of the current stream's workspace (nonzero if a bounded wait timed out)."""
    key = (torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream)
    buf = _ws.get(key)
    if buf is None:
        return 0
    return int(buf[:32].view(torch.int32)[2].item())


# ---------------------------------------------------------------------------
# Entry points
# ---------------------------------------------------------------------------


def band_index(num_layers: int, num_bands: int, layer: int) -> int:
    out = ctypes.c_int32(-1)
    _check(lib.tb_band_index(num_layers, num_bands, layer, ctypes.byref(out)))
    return out.value


def linear_forward_workspace_size(m: int, out_dim: int, in_dim: int, rank: int, dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.tb_linear_forward_workspace_size(m, out_dim, in_dim, rank, _dtype_code(dtype), ctypes.byref(out)))
    return out.value


def linear_forward(x: torch.Tensor, s: torch.Tensor | None, W0: torch.Tensor, U: torch.Tensor | None,
                   V: torch.Tensor | None, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = s * (x @ W0.T) + (x @ V) @ U.T on the GPU, via tb_linear_forward (s None: unit scale)."""
    m, out_dim, in_dim, rank, U, V = _projection_dims(x, s, W0, U, V)
    _expect_out(out, (m, out_dim), x.dtype)
    _need_cuda(x, s, W0, U, V, out)
    out = _output(out, (m, out_dim), x.dtype, x)
    need = linear_forward_workspace_size(m, out_dim, in_dim, rank, x.dtype)
    ws = workspace if workspace is not None else workspace_for(need)
    _check(lib.tb_linear_forward(_ptr(x), _ptr(s), _ptr(W0), _ptr(U), _ptr(V), _ptr(out), m, out_dim, in_dim, rank,
                                 _dtype_code(x.dtype), _ptr(ws), _workspace_bytes(ws), _stream()))
    return out


def linear_forward_no_alloc(x: torch.Tensor, s: torch.Tensor | None, W0: torch.Tensor, U: torch.Tensor | None,
                            V: torch.Tensor | None, out: torch.Tensor | None = None) -> torch.Tensor:
    """linear_forward with the library's static device scratch as its workspace (tb_linear_forward_no_alloc):
    with `out` given, nothing is allocated."""
    m, out_dim, in_dim, rank, U, V = _projection_dims(x, s, W0, U, V)
    _expect_out(out, (m, out_dim), x.dtype)
    _need_cuda(x, s, W0, U, V, out)
    out = _output(out, (m, out_dim), x.dtype, x)
    _check(lib.tb_linear_forward_no_alloc(_ptr(x), _ptr(s), _ptr(W0), _ptr(U), _ptr(V), _ptr(out), m, out_dim, in_dim,
                                          rank, _dtype_code(x.dtype), _stream()))
    return out


def dense_forward(x: torch.Tensor, W: torch.Tensor, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = x @ W.T on the GPU, via tb_dense_forward (a weight materialised once, e.g. by reconstruct_weight)."""
    m, out_dim, in_dim, _, _, _ = _projection_dims(x, None, W, None, None)
    _expect_out(out, (m, out_dim), x.dtype)
    _need_cuda(x, W, out)
    out = _output(out, (m, out_dim), x.dtype, x)
    need = linear_forward_workspace_size(m, out_dim, in_dim, 0, x.dtype)
    ws = workspace if workspace is not None else workspace_for(need)
    _check(lib.tb_dense_forward(_ptr(x), _ptr(W), _ptr(out), m, out_dim, in_dim, _dtype_code(x.dtype), _ptr(ws),
                                _workspace_bytes(ws), _stream()))
    return out


def projection_array(members) -> ctypes.Array:
    """tb_projection array for (x, s, W0, U, V, y) tuples (U, V may be None)."""
    arr = (Projection * len(members))()
    for j, (x, s, W0, U, V, y) in enumerate(members):
        rank = 0 if U is None else U.shape[1]
        arr[j] = Projection(_ptr(x), _ptr(s), _ptr(W0), _ptr(U) if rank else None, _ptr(V) if rank else None, _ptr(y),
                            W0.shape[0], W0.shape[1], rank)
    return arr


def linear_forward_group(members, workspace: torch.Tensor | None = None, outs=None) -> list:
    """Several independent projections [(x, s, W0, U, V), ...] of one token count and dtype in one call
    (tb_linear_forward_group); returns their outputs (written into `outs` when given)."""
    if not 1 <= len(members) <= MAX_GROUP:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"a group holds 1..{MAX_GROUP} projections")
    if outs is not None and len(outs) != len(members):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "one output per member")
    dims = []
    for j, (x, s, W0, U, V) in enumerate(members):
        m, out_dim, in_dim, rank, U, V = _projection_dims(x, s, W0, U, V)
        if m != members[0][0].shape[0] or x.dtype != members[0][0].dtype:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "group members must share the token count and dtype")
        if outs is not None:
            _expect_out(outs[j], (m, out_dim), x.dtype)
        dims.append((x, s, W0, U, V))
    full = []
    for j, (x, s, W0, U, V) in enumerate(dims):
        _need_cuda(x, s, W0, U, V)
        y = _output(None if outs is None else outs[j], (x.shape[0], W0.shape[0]), x.dtype, x)
        _need_cuda(y)
        full.append((x, s, W0, U, V, y))
    m, dtype = members[0][0].shape[0], members[0][0].dtype
    arr = projection_array(full)
    need = ctypes.c_size_t(0)
    _check(lib.tb_linear_forward_group_workspace_size(len(full), arr, m, _dtype_code(dtype), ctypes.byref(need)))
    ws = workspace if workspace is not None else workspace_for(need.value)
    _check(lib.tb_linear_forward_group(len(full), arr, m, _dtype_code(dtype), _ptr(ws), _workspace_bytes(ws),
                                       _stream()))
    return [f[5] for f in full]


def _bundle_dims(s, W0, U, V):
    """(out_dim, in_dim, rank, U, V) of a bundle after checking s [out] (where there is one), U [out, rank], V [in, rank]
    against W0 (one dtype); a rank-0 U/V pair becomes None."""
    if W0.dim() != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "W0 must be [out, in]")
    _dtype_code(W0.dtype)
    out_dim, in_dim = W0.shape
    if s is not None:
        _expect("s", s, (out_dim,), W0.dtype)
    if (U is None) != (V is None):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "U and V are given together or not at all")
    rank = 0
    if U is not None:
        if U.dim() != 2:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "U must be [out, rank]")
        rank = U.shape[1]
        _expect("U", U, (out_dim, rank), W0.dtype)
        _expect("V", V, (in_dim, rank), W0.dtype)
        if rank == 0:
            U = V = None
    return out_dim, in_dim, rank, U, V


def reconstruct_weight(s: torch.Tensor, W0: torch.Tensor, U: torch.Tensor | None, V: torch.Tensor | None,
                       out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """diag(s) @ W0 + U @ V.T on the GPU, via tb_reconstruct_weight (into `out` when given; its dtype wins)."""
    out_dim, in_dim, rank, U, V = _bundle_dims(s, W0, U, V)
    _expect_out(out, (out_dim, in_dim))
    _need_cuda(s, W0, U, V, out)
    out = _output(out, (out_dim, in_dim), out_dtype if out is None else out.dtype, W0)
    _check(lib.tb_reconstruct_weight(_ptr(s), _ptr(W0), _ptr(U), _ptr(V), _ptr(out), out_dim, in_dim, rank,
                                     _dtype_code(W0.dtype), _dtype_code(out.dtype), _stream()))
    return out


def _expect_error_out(out: torch.Tensor | None) -> None:
    """The error lands in one device double."""
    if out is not None and (out.dtype != torch.float64 or out.numel() != 1):
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"out must hold one float64, got {out.dtype} {list(out.shape)}")


def _error_output(out: torch.Tensor | None, like: torch.Tensor) -> torch.Tensor:
    if out is None:
        return torch.empty((), dtype=torch.float64, device=like.device)
    _need_cuda(out)
    return out


_frob_ws: dict = {}


def _error_workspace() -> torch.Tensor:
    key = (torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream)
    ws = _frob_ws.get(key)
    if ws is None:
        ws = torch.zeros(FROBENIUS_WORKSPACE_BYTES, dtype=torch.uint8, device=f"cuda:{key[0]}")
        _frob_ws[key] = ws
    return ws


def rel_frobenius_error(original: torch.Tensor, reconstructed: torch.Tensor,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """||original - reconstructed||_F / ||original||_F as a 0-d float64 GPU tensor (no sync)."""
    if original.dim() != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "original must be 2-D")
    _dtype_code(original.dtype)
    _expect("reconstructed", reconstructed, original.shape, original.dtype)
    _expect_error_out(out)
    _need_cuda(original, reconstructed)
    rows, cols = original.shape
    out = _error_output(out, original)
    ws = _error_workspace()
    _check(lib.tb_rel_frobenius_error(_ptr(original), _ptr(reconstructed), rows, cols, _dtype_code(original.dtype),
                                      _ptr(out), _ptr(ws), ws.numel(), _stream()))
    return out


def reconstruction_error(original: torch.Tensor, s: torch.Tensor, W0: torch.Tensor, U: torch.Tensor | None,
                         V: torch.Tensor | None, out: torch.Tensor | None = None) -> torch.Tensor:
    """relative_frobenius_error(original, diag(s) @ W0 + U @ V.T) without forming the rebuilt weight, as a 0-d
    float64 GPU tensor (no sync), via tb_reconstruction_error."""
    out_dim, in_dim, rank, U, V = _bundle_dims(s, W0, U, V)
    _expect("original", original, (out_dim, in_dim))
    _dtype_code(original.dtype)
    _expect_error_out(out)
    _need_cuda(original, s, W0, U, V)
    out = _error_output(out, W0)
    ws = _error_workspace()
    _check(lib.tb_reconstruction_error(_ptr(s), _ptr(W0), _ptr(U), _ptr(V), _ptr(original), out_dim, in_dim, rank,
                                       _dtype_code(W0.dtype), _dtype_code(original.dtype), _ptr(out), _ptr(ws),
                                       ws.numel(), _stream()))
    return out


# ---------------------------------------------------------------------------
# 8-bit blocks: e4m3 numbers with a scale per 128 columns of a token and per
# 128 x 128 block of a weight
# ---------------------------------------------------------------------------
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _scale_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return TB_SCALE_F32
    if dt == E8M0:
        return TB_SCALE_E8M0
    raise TBError(TB_ERR_UNSUPPORTED, f"scales are float32 or float8_e8m0fnu, not {dt}")


def _fp8_blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def quantize_activations(x: torch.Tensor, scale_dtype: torch.dtype = torch.float32) -> tuple:
    """(e4m3 [m, in], scales [m, ceil(in / 128)]) of x [m, in], via tb_quantize_activations."""
    if x.dim() != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "x must be [m, in]")
    code, sc = _dtype_code(x.dtype), _scale_code(scale_dtype)
    m, in_dim = x.shape
    _need_cuda(x)
    q = x.new_empty((m, in_dim), dtype=E4M3)
    scale = x.new_empty((m, _fp8_blocks(in_dim)), dtype=scale_dtype)
    _check(lib.tb_quantize_activations(_ptr(x), _ptr(q), _ptr(scale), m, in_dim, code, sc, _stream()))
    return q, scale


# The checks below look at shapes and dtypes only, and a serving loop repeats its shapes: their results are kept by
# those (a refusal is raised, not kept).


def _kind(t: torch.Tensor | None):
    return None if t is None else (t.shape, t.dtype)


def _expect_kind(name: str, kind, shape, dtype: torch.dtype | None = None) -> None:
    if kind[0] != shape:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"{name} must be {list(shape)}, got {list(kind[0])}")
    if dtype is not None and kind[1] != dtype:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"{name} must be {dtype}, got {kind[1]}")


@functools.lru_cache(maxsize=4096)
def _rebuild_fp8_dims(s, W0, U, V, q, scale, scale_dtype):
    """(out_dim, in_dim, rank, dtype code, scale code, scale shape) of reconstruct_weight_fp8's operands by kind."""
    shape, dtype = W0
    if len(shape) != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "W0 must be [out, in]")
    code = _dtype_code(dtype)
    out_dim, in_dim = shape
    if s is not None:
        _expect_kind("s", s, (out_dim,), dtype)
    if (U is None) != (V is None):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "U and V are given together or not at all")
    rank = 0
    if U is not None:
        if len(U[0]) != 2:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "U must be [out, rank]")
        rank = U[0][1]
        _expect_kind("U", U, (out_dim, rank), dtype)
        _expect_kind("V", V, (in_dim, rank), dtype)
    sc = _scale_code(scale_dtype)
    blocks = _fp8_blocks(out_dim), _fp8_blocks(in_dim)
    if q is not None:
        _expect_kind("out", q, (out_dim, in_dim), E4M3)
        _expect_kind("out", scale, blocks, scale_dtype)
    return out_dim, in_dim, rank, code, sc, blocks


def reconstruct_weight_fp8(s: torch.Tensor | None, W0: torch.Tensor, U: torch.Tensor | None, V: torch.Tensor | None,
                           scale_dtype: torch.dtype = torch.float32, out=None) -> tuple:
    """diag(s) @ W0 + U @ V.T as (e4m3 [out, in], scales [ceil(out / 128), ceil(in / 128)]) without forming it wide,
    via tb_reconstruct_weight_fp8 (s None: unit scale; into the pair `out` when given, whose scale dtype wins)."""
    q = scale = None
    if out is not None:
        q, scale = out
        scale_dtype = scale.dtype
    out_dim, in_dim, rank, code, sc, blocks = _rebuild_fp8_dims(_kind(s), _kind(W0), _kind(U), _kind(V), _kind(q),
                                                                _kind(scale), scale_dtype)
    dev = _here([t for t in (W0, s, U, V, q, scale) if t is not None])
    if q is None:
        q = W0.new_empty((out_dim, in_dim), dtype=E4M3)
        scale = W0.new_empty(blocks, dtype=scale_dtype)
    _check(lib.tb_reconstruct_weight_fp8(_ptr(s), W0.data_ptr(), _ptr(U) if rank else None, _ptr(V) if rank else None,
                                         q.data_ptr(), scale.data_ptr(), out_dim, in_dim, rank, code, sc,
                                         torch._C._cuda_getCurrentRawStream(dev)))
    return q, scale


def quantize_weight(W: torch.Tensor, scale_dtype: torch.dtype = torch.float32, out=None) -> tuple:
    """A dense weight [out, in] as (e4m3, block scales): reconstruct_weight_fp8 with unit scale and rank 0."""
    return reconstruct_weight_fp8(None, W, None, None, scale_dtype, out)


@functools.lru_cache(maxsize=4096)
def _fp8_workspace_size(device: int, m: int, out_dim: int, in_dim: int, x_code: int, y_code: int, scale: int) -> int:
    """By sizes and types (and the device, whose compute units the plan counts): a serving loop asks once per shape."""
    out = ctypes.c_size_t(0)
    _check(lib.tb_dense_forward_fp8_workspace_size(m, out_dim, in_dim, x_code, y_code, scale, ctypes.byref(out)))
    return out.value


def dense_forward_fp8_workspace_size(m: int, out_dim: int, in_dim: int, x_dtype: torch.dtype, out_dtype: torch.dtype,
                                     scale_dtype: torch.dtype) -> int:
    """Bytes of workspace that dense_forward_fp8 takes on the current device for these sizes."""
    code = TB_E4M3 if x_dtype == E4M3 else _dtype_code(x_dtype)
    return _fp8_workspace_size(torch.cuda.current_device(), m, out_dim, in_dim, code, _dtype_code(out_dtype),
                               _scale_code(scale_dtype))


@functools.lru_cache(maxsize=4096)
def _dense_fp8_dims(x, Wq, w_scale, x_scale, out, out_dtype):
    """(m, out_dim, in_dim, x code, y code, scale code, y dtype) of dense_forward_fp8's operands by kind."""
    (x_shape, x_dtype), (w_shape, _) = x, Wq
    if len(x_shape) != 2 or len(w_shape) != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "x must be [m, in] and Wq [out, in]")
    quantised = x_dtype == E4M3
    x_code = TB_E4M3 if quantised else _dtype_code(x_dtype)
    m, in_dim = x_shape
    out_dim = w_shape[0]
    _expect_kind("Wq", Wq, (out_dim, in_dim), E4M3)
    sc = _scale_code(w_scale[1])
    _expect_kind("w_scale", w_scale, (_fp8_blocks(out_dim), _fp8_blocks(in_dim)))
    if quantised != (x_scale is not None):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "x_scale goes with an x in float8_e4m3fn, and only with one")
    if quantised:
        _expect_kind("x_scale", x_scale, (m, _fp8_blocks(in_dim)), w_scale[1])
    if out_dtype is None:
        out_dtype = out[1] if out is not None else torch.bfloat16 if quantised else x_dtype
    y_code = _dtype_code(out_dtype)
    if out is not None:
        _expect_kind("out", out, (m, out_dim), out_dtype)
    return m, out_dim, in_dim, x_code, y_code, sc, out_dtype


def dense_forward_fp8(x: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, x_scale: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = Q(x) @ Wq.T with the block scales applied, via tb_dense_forward_fp8.

    x [m, in] in bfloat16 or float32 is quantised within the call (scales of w_scale's dtype); in float8_e4m3fn it
    comes with x_scale (quantize_activations).  y has out's dtype, out_dtype, x's dtype, or bfloat16 for an e4m3 x.
    In bfloat16 y is off by up to 7 x 2^-13 of its terms' magnitudes beside its rounding (much, where outliers cancel);
    float32 sums without that, at half the matrix rate."""
    m, out_dim, in_dim, x_code, y_code, sc, y_dtype = _dense_fp8_dims(_kind(x), _kind(Wq), _kind(w_scale),
                                                                      _kind(x_scale), _kind(out), out_dtype)
    dev = _here([t for t in (x, Wq, w_scale, x_scale, out, workspace) if t is not None])
    if out is None:
        out = x.new_empty((m, out_dim), dtype=y_dtype)
    if workspace is None:
        nbytes = _fp8_workspace_size(dev, m, out_dim, in_dim, x_code, y_code, sc)
        # From torch's allocator, per call: it follows the stream and, under graph capture, the graph's own pool,
        # so no two graphs share it.
        workspace = x.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _check(lib.tb_dense_forward_fp8(x.data_ptr(), _ptr(x_scale), Wq.data_ptr(), w_scale.data_ptr(), out.data_ptr(), m,
                                    out_dim, in_dim, x_code, y_code, sc, _ptr(workspace), nbytes,
                                    torch._C._cuda_getCurrentRawStream(dev)))
    return out


# ---------------------------------------------------------------------------
# 8-bit integers: whole numbers with a scale per token of an activation and per
# output channel of a weight
# ---------------------------------------------------------------------------
INT8 = torch.int8


@functools.lru_cache(maxsize=4096)
def _rows_int8_dims(x, q, scale):
    """(m, in_dim, dtype code) of quantize_rows_int8's operands by kind."""
    if len(x[0]) != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "x must be [m, in]")
    code = _dtype_code(x[1])
    m, in_dim = x[0]
    if q is not None:
        _expect_kind("out", q, (m, in_dim), INT8)
        _expect_kind("out", scale, (m,), torch.float32)
    return m, in_dim, code


def quantize_rows_int8(x: torch.Tensor, out=None) -> tuple:
    """(int8 [m, in], float32 scales [m]) of x [m, in], each row scaled by its largest value, via tb_quantize_rows_int8
    (into the pair `out` when given)."""
    q, scale = (None, None) if out is None else out
    m, in_dim, code = _rows_int8_dims(_kind(x), _kind(q), _kind(scale))
    dev = _here([t for t in (x, q, scale) if t is not None])
    if q is None:
        q, scale = x.new_empty((m, in_dim), dtype=INT8), x.new_empty((m,), dtype=torch.float32)
    _check(lib.tb_quantize_rows_int8(x.data_ptr(), q.data_ptr(), scale.data_ptr(), m, in_dim, code,
                                     torch._C._cuda_getCurrentRawStream(dev)))
    return q, scale


def quantize_weight_int8(W: torch.Tensor, out=None) -> tuple:
    """A dense weight [out, in] as (int8, a scale per output channel): quantize_rows_int8 of its rows."""
    return quantize_rows_int8(W, out)


def reconstruct_weight_int8(s: torch.Tensor, W0: torch.Tensor, U: torch.Tensor | None, V: torch.Tensor | None,
                            out=None) -> tuple:
    """diag(s) @ W0 + U @ V.T as (int8 [out, in], float32 scales [out]): rebuilt in float32, then quantised by rows.  The
    rebuilt weight is a temporary of 4 x out x in bytes."""
    if out is not None:
        _rows_int8_dims((W0.shape, torch.float32), _kind(out[0]), _kind(out[1]))
    return quantize_rows_int8(reconstruct_weight(s, W0, U, V), out)


@functools.lru_cache(maxsize=4096)
def _int8_workspace_size(device: int, m: int, out_dim: int, in_dim: int, x_code: int, y_code: int) -> int:
    """By sizes and types (and the device, whose compute units the plan counts): a serving loop asks once per shape."""
    out = ctypes.c_size_t(0)
    _check(lib.tb_dense_forward_int8_workspace_size(m, out_dim, in_dim, x_code, y_code, ctypes.byref(out)))
    return out.value


def dense_forward_int8_workspace_size(m: int, out_dim: int, in_dim: int, x_dtype: torch.dtype,
                                      out_dtype: torch.dtype) -> int:
    """Bytes of workspace that dense_forward_int8 takes on the current device for these sizes."""
    code = TB_INT8 if x_dtype == INT8 else _dtype_code(x_dtype)
    return _int8_workspace_size(torch.cuda.current_device(), m, out_dim, in_dim, code, _dtype_code(out_dtype))


@functools.lru_cache(maxsize=4096)
def _dense_int8_dims(x, Wq, w_scale, x_scale, out, out_dtype):
    """(m, out_dim, in_dim, x code, y code, y dtype) of dense_forward_int8's operands by kind."""
    (x_shape, x_dtype), (w_shape, _) = x, Wq
    if len(x_shape) != 2 or len(w_shape) != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "x must be [m, in] and Wq [out, in]")
    quantised = x_dtype == INT8
    x_code = TB_INT8 if quantised else _dtype_code(x_dtype)
    m, in_dim = x_shape
    out_dim = w_shape[0]
    _expect_kind("Wq", Wq, (out_dim, in_dim), INT8)
    _expect_kind("w_scale", w_scale, (out_dim,), torch.float32)
    if quantised != (x_scale is not None):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "x_scale goes with an x in int8, and only with one")
    if quantised:
        _expect_kind("x_scale", x_scale, (m,), torch.float32)
    if out_dtype is None:
        out_dtype = out[1] if out is not None else torch.bfloat16 if quantised else x_dtype
    y_code = _dtype_code(out_dtype)
    if out is not None:
        _expect_kind("out", out, (m, out_dim), out_dtype)
    return m, out_dim, in_dim, x_code, y_code, out_dtype


def dense_forward_int8(x: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, x_scale: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                       workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = Q(x) @ Wq.T with the scales of tokens and channels applied, via tb_dense_forward_int8.

    x [m, in] in bfloat16 or float32 is quantised within the call (quantize_rows_int8); in int8 it comes with x_scale.
    y has out's dtype, out_dtype, x's dtype, or bfloat16 for an int8 x.  Sums are exact: a token's row is the same bits
    in a batch and alone."""
    m, out_dim, in_dim, x_code, y_code, y_dtype = _dense_int8_dims(_kind(x), _kind(Wq), _kind(w_scale), _kind(x_scale),
                                                                   _kind(out), out_dtype)
    dev = _here([t for t in (x, Wq, w_scale, x_scale, out, workspace) if t is not None])
    if out is None:
        out = x.new_empty((m, out_dim), dtype=y_dtype)
    if workspace is None:
        nbytes = _int8_workspace_size(dev, m, out_dim, in_dim, x_code, y_code)
        # From torch's allocator, per call: it follows the stream and, under graph capture, the graph's own pool,
        # so no two graphs share it.
        workspace = x.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _check(lib.tb_dense_forward_int8(x.data_ptr(), _ptr(x_scale), Wq.data_ptr(), w_scale.data_ptr(), out.data_ptr(), m,
                                     out_dim, in_dim, x_code, y_code, _ptr(workspace), nbytes,
                                     torch._C._cuda_getCurrentRawStream(dev)))
    return out


# ---------------------------------------------------------------------------
# The norms before and after a block, with its gate and residual scale
# ---------------------------------------------------------------------------


_RESIDUAL = ctypes.c_int64 * 15


@functools.lru_cache(maxsize=4096)
def _residual_dims(h, y, weight, post_weight, gate, out_dtype, scale_dtype, norm, dtype, h_out, z, z_scale):
    """(m, n, dtype code, h code, z code, scale code, z shape and dtype, its scales' shape and dtype, rows per gate row)
    of residual_norm's operands by kind."""
    shape, h_dtype = h
    if len(shape) != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "h must be [m, n]")
    m, n = shape
    h_code, code = _dtype_code(h_dtype), _dtype_code(dtype)
    if y is not None:
        _expect_kind("y", y, (m, n), dtype)
    for name, w in (("weight", weight), ("post_weight", post_weight)):
        if w is not None:
            _expect_kind(name, w, (n,), dtype)
    rows = 1
    if gate is not None:
        g, _ = gate
        if g == (n,):
            rows = max(m, 1)
        elif len(g) == 2 and g[1] in (n, 1) and (g[0] > 0 and m % g[0] == 0 or g[0] == m):
            rows = max(m // max(g[0], 1), 1)
        else:
            raise TBError(TB_ERR_INVALID_ARGUMENT, f"gate must be [n], or [g, n] or [g, 1] with g dividing {m} rows of {n}, "
                                                   f"got {list(g)}")
        _expect_kind("gate", gate, g, dtype)
    z_code, sc, scales = code, TB_SCALE_F32, None
    if out_dtype == INT8:
        z_code, scales = TB_INT8, ((m,), torch.float32)
    elif out_dtype == E4M3:
        z_code, sc, scales = TB_E4M3, _scale_code(scale_dtype), ((m, _fp8_blocks(n)), scale_dtype)
    elif out_dtype is not None and out_dtype != dtype:
        raise TBError(TB_ERR_UNSUPPORTED, f"z is in {dtype}, int8 or float8_e4m3fn, not {out_dtype}")
    if not norm and (weight is not None or out_dtype is not None):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "weight and out_dtype go with the norm")
    z_kind = ((m, n), out_dtype or dtype) if norm else None
    if h_out is not None:
        _expect_kind("out", h_out, (m, n), h_dtype)
    if z is not None:
        if not norm:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "an output for z goes with the norm")
        _expect_kind("out", z, *z_kind)
        if (z_scale is None) != (scales is None):
            raise TBError(TB_ERR_INVALID_ARGUMENT, "an 8-bit z comes with its scales, and only an 8-bit one")
        if scales is not None:
            _expect_kind("out", z_scale, *scales)
    return m, n, code, h_code, z_code, sc, z_kind, scales, rows


def residual_norm(h: torch.Tensor, y: torch.Tensor | None = None, weight: torch.Tensor | None = None, *,
                  post_norm: bool = False, post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                  residual_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0, norm: bool = True,
                  out_dtype: torch.dtype | None = None, scale_dtype: torch.dtype = torch.float32, outs=None) -> tuple:
    """(h', z): the norms before and after a block with its gate and residual scale in one pass, via tb_residual_norm.

    h' = residual_scale * h + gate * a with a = y, or y normed and weighted by post_weight (post_norm); z is h' normed and
    weighted by weight, for the next projection.  h [m, n] may be float32 beside bfloat16 blocks.  gate: [n], or [g, n] or
    [g, 1] whose rows serve m / g rows each.  Weights count as weight + weight_offset.  z is in y's dtype (without a y in
    the weight's, else out_dtype's or h's), or with out_dtype int8 or float8_e4m3fn a pair (numbers, scales) that the 8-bit
    projections take.  Without y h' is h itself; with norm=False z is None.  outs: (h', z or None), h' may be h and z y; h,
    y and the outputs may be strided with adjacent elements (an 8-bit z is dense)."""
    ho = zo = so = None
    if outs is not None:
        ho, zo = outs
        if isinstance(zo, (tuple, list)):
            if len(zo) != 2 or zo[0] is None or zo[1] is None:
                raise TBError(TB_ERR_INVALID_ARGUMENT, "an 8-bit z comes with its scales")
            zo, so = zo
            scale_dtype = so.dtype
            if out_dtype is None:
                out_dtype = zo.dtype
    if y is not None:
        dtype = y.dtype
    elif weight is not None:
        dtype = weight.dtype
    else:
        dtype = out_dtype if out_dtype in (torch.bfloat16, torch.float32) else h.dtype
    if out_dtype is dtype:
        out_dtype = None
    m, n, code, h_code, z_code, sc, z_kind, scales, gate_rows = _residual_dims(
        (h.shape, h.dtype), _kind(y), _kind(weight), _kind(post_weight), _kind(gate), out_dtype, scale_dtype, norm, dtype,
        _kind(ho), _kind(zo), _kind(so))
    if y is None and ho is not None:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "without a y there is no h' to write")
    dev = h.get_device()
    fine = dev >= 0 and dev == torch.cuda.current_device()
    hs, he = h.stride()
    # tb_residual, every field eight bytes
    yp = pp = gp = wp = hop = zp = sp = ys = hos = zs = gs = 0
    adjacent = he == 1
    if y is not None:
        ys, e = y.stride()
        yp = y.data_ptr()
        if ho is None:
            ho = h if not fine else torch.empty_like(h) if hs == n and adjacent else h.new_empty((m, n))
        hos, oe = ho.stride()
        hop = ho.data_ptr()
        fine = fine and y.get_device() == dev and ho.get_device() == dev
        adjacent = adjacent and e == 1 and oe == 1
    if weight is not None:
        wp = weight.data_ptr()
        fine = fine and weight.get_device() == dev and weight.is_contiguous()
    if post_weight is not None:
        pp = post_weight.data_ptr()
        fine = fine and post_weight.get_device() == dev and post_weight.is_contiguous()
    channels = False
    if gate is not None:
        gp = gate.data_ptr()
        gs = gate.stride(0) if gate.dim() == 2 else 0
        fine = fine and gate.get_device() == dev
        channels = gate.shape[-1] == n
        adjacent = adjacent and (not channels or gate.stride(-1) == 1)
    if z_kind is not None:
        if zo is None and fine:
            zo = torch.empty(z_kind[0], dtype=z_kind[1], device=h.device)
            if scales is not None:
                so = torch.empty(scales[0], dtype=scales[1], device=h.device)
        if zo is not None:
            zs, e = zo.stride()
            zp = zo.data_ptr()
            fine = fine and zo.get_device() == dev
            adjacent = adjacent and e == 1
            if so is not None:
                sp = so.data_ptr()
                fine = fine and so.get_device() == dev and so.is_contiguous() and zo.is_contiguous()
    if not fine:
        _need_device(h, y, gate, ho, zo)
        _need_cuda(weight, post_weight, so, zo if scales is not None else None)
    if not adjacent and n > 1:
        raise TBError(TB_ERR_UNSUPPORTED, "the elements of a row must be adjacent")
    _check(lib.tb_residual_norm(_RESIDUAL(h.data_ptr(), yp, pp, gp, wp, hop, zp, sp, hs, ys, hos, zs, gate_rows, gs, channels), m, n,
                                residual_scale, eps, weight_offset, post_norm, code, h_code, z_code, sc,
                                torch._C._cuda_getCurrentRawStream(dev)))
    return ho if y is not None else h, (zo, so) if scales is not None else zo


# ---------------------------------------------------------------------------
# Head norms with the position rotation, and the path that ends in them
# ---------------------------------------------------------------------------


def _rotated_dims(positions, freqs, tokens: int, dim: int, axes=None) -> int:
    """rot_dim after checking the kinds of positions [tokens] ([axes, tokens] where the pairs have axes) and freqs
    [rot_dim / 2] (both None: 0) against heads of dim."""
    if (positions is None) != (freqs is None):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "positions and freqs are given together or not at all")
    if freqs is None:
        if axes is not None:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "axes go with positions and freqs")
        return 0
    if len(freqs[0]) != 1:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "freqs must be [rot_dim / 2]")
    rot = 2 * freqs[0][0]
    if rot > dim:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"{rot} rotated dimensions, but heads of {dim}")
    _expect_kind("freqs", freqs, (rot // 2,), torch.float64)
    if axes is None:
        _expect_kind("positions", positions, (tokens,), torch.int64)
        return rot
    if len(axes) != rot // 2 or rot == 0:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"axes names the axis of each of {rot // 2} pairs, got {len(axes)}")
    if len(positions[0]) != 2 or not 1 <= positions[0][0] <= MAX_AXES:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"positions must be [1..{MAX_AXES} axes, tokens], got {list(positions[0])}")
    _expect_kind("positions", positions, (positions[0][0], tokens), torch.int64)
    if not all(isinstance(a, int) and 0 <= a < positions[0][0] for a in axes):
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"an axis lies outside 0..{positions[0][0] - 1}")
    return rot


def _axis_layout(axes, axis_halves: bool, interleaved: bool, norm: bool) -> None:
    if axes is None and (axis_halves or not norm):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "axis_halves and norm=False go with axes")
    if axis_halves:
        if interleaved:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "pairs are interleaved or in halves of their axis's span, not both")
        if sum(a != b for a, b in zip(axes, axes[1:])) != len(set(axes)) - 1:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "with axis_halves the pairs of each axis are consecutive")


@functools.lru_cache(maxsize=4096)
def _heads_dims(parts, positions, freqs, outs, axes=None):
    """(tokens, head_dim, rot_dim, dtype code, the axes as bytes) of head_norm_rotate's operands by kind."""
    if not 1 <= len(parts) <= MAX_GROUP:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"a call takes 1..{MAX_GROUP} parts")
    if outs is not None and len(outs) != len(parts):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "one output per part")
    for (shape, _), _ in parts:
        if len(shape) != 3:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "x must be [tokens, heads, head_dim]")
    (tokens, _, dim), dtype = parts[0][0]
    code = _dtype_code(dtype)
    rot = _rotated_dims(positions, freqs, tokens, dim, axes)
    for j, (x, w) in enumerate(parts):
        _expect_kind(f"part {j}", x, (tokens, x[0][1], dim), dtype)
        if w is not None:
            _expect_kind("weight", w, (dim,), dtype)
        if outs is not None:
            _expect_kind("out", outs[j], x[0], dtype)
    return tokens, dim, rot, code, None if axes is None else bytes(axes)


def head_norm_rotate(parts, positions: torch.Tensor | None, freqs: torch.Tensor | None, eps: float = 1e-6,
                     weight_offset: float = 0.0, interleaved: bool = False, outs=None, axes=None,
                     axis_halves: bool = False, norm: bool = True) -> list:
    """Per-head norm and position rotation of several tensors of heads in one pass, via tb_head_norm_rotate.

    parts: (x [tokens, heads, head_dim], weight [head_dim] or None) pairs of one dtype, e.g. queries and keys; x may
    be strided (a view of packed rows) with adjacent elements.  positions int64 [tokens], freqs float64 [rot_dim / 2]
    (radians per position; both None: no rotation).  Returns new tensors, or writes `outs` (x itself for in place, or
    a view of a cache).

    With several axes (time, height, width; via tb_head_norm_rotate_axes) positions are [axes, tokens] and `axes` names
    the axis of each of the rot_dim / 2 pairs (a tuple of ints); with axis_halves a pair's elements lie in the two halves
    of its axis's own span instead of the head's.  With norm=False (and axes) the heads are rotated only."""
    if axes is not None:
        axes = tuple(axes)
    tokens, dim, rot, code, pair_axis = _heads_dims(
        tuple([(_kind(x), _kind(w)) for x, w in parts]), _kind(positions), _kind(freqs),
        None if outs is None else tuple([_kind(y) for y in outs]), axes)
    _axis_layout(axes, axis_halves, interleaved, norm)
    dev = parts[0][0].get_device()
    fine = dev >= 0 and dev == torch.cuda.current_device()
    ys, fields = [], []
    for j, (x, w) in enumerate(parts):
        heads = x.shape[1]
        xt, xh, xe = x.stride()
        fine = fine and x.get_device() == dev
        if outs is not None:
            y = outs[j]
            yt, yh, ye = y.stride()
            fine = fine and y.get_device() == dev
        else:
            y = x if not fine else torch.empty_like(x) if x.is_contiguous() else x.new_empty((tokens, heads, dim))
            yt, yh, ye = heads * dim, dim, 1
        if (xe != 1 or ye != 1) and dim > 1:
            raise TBError(TB_ERR_UNSUPPORTED, "the elements of a head must be adjacent")
        wp = 0
        if w is not None:
            wp = w.data_ptr()
            fine = fine and w.get_device() == dev and w.is_contiguous()
        # tb_head_part, every field eight bytes
        fields += (x.data_ptr(), y.data_ptr(), wp, heads, xt, xh, yt, yh)
        ys.append(y)
    if rot:
        fine = (fine and positions.get_device() == dev and freqs.get_device() == dev and positions.is_contiguous()
                and freqs.is_contiguous())
    if not fine:
        _need_device(*[x for x, _ in parts], *ys)
        _need_cuda(positions, freqs, *[w for _, w in parts])
    if axes is None:
        _check(lib.tb_head_norm_rotate(len(parts), (ctypes.c_int64 * len(fields))(*fields), tokens, dim, rot, interleaved,
                                       _ptr(positions), _ptr(freqs), eps, weight_offset, code,
                                       torch._C._cuda_getCurrentRawStream(dev)))
    else:
        pairs = TB_PAIRS_AXIS if axis_halves else TB_PAIRS_INTERLEAVED if interleaved else TB_PAIRS_HALF
        _check(lib.tb_head_norm_rotate_axes(len(parts), (ctypes.c_int64 * len(fields))(*fields), tokens, dim, rot, pairs,
                                            positions.shape[0], positions.data_ptr(), pair_axis, freqs.data_ptr(), norm,
                                            eps, weight_offset, code, torch._C._cuda_getCurrentRawStream(dev)))
    return ys


def qkv_forward(x, q, k, v, head_dim: int, positions: torch.Tensor | None, freqs: torch.Tensor | None,
                q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                weight_offset: float = 0.0, interleaved: bool = False, axes=None, axis_halves: bool = False,
                out_dtype: torch.dtype | None = None) -> tuple:
    """The input half of an attention layer: (queries, keys, values), each [m, heads, head_dim], of x [m, in].

    q, k, v are the layer's projections, all as bundles (s, W0, U, V) in one grouped launch, or all in 8 bits (Wq,
    w_scale), e4m3 blocks or int8 channels, with x quantised once; for these x may be the pair (numbers, scales) that
    residual_norm made, and out_dtype (bfloat16) is the type of the heads.  Queries and keys then get their head norms and
    rotation in place (axes, axis_halves: as in head_norm_rotate)."""
    kinds = {len(p) for p in (q, k, v)}
    if kinds not in ({4}, {2}):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "q, k and v are all (s, W0, U, V) or all (Wq, w_scale)")
    at = 1 if kinds == {4} else 0
    x_scale = None
    if isinstance(x, (tuple, list)):
        if kinds == {4} or len(x) != 2:
            raise TBError(TB_ERR_INVALID_ARGUMENT, "an x of (numbers, scales) goes with projections in 8 bits")
        x, x_scale = x
    if x.dim() != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "x must be [m, in]")
    if x_scale is None and out_dtype not in (None, x.dtype):
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"the heads of an x in {x.dtype} are in {x.dtype}")
    dtype = (out_dtype or torch.bfloat16) if x_scale is not None else x.dtype
    for name, p in zip("qkv", (q, k, v)):
        if head_dim < 1 or p[at].dim() != 2 or p[at].shape[0] % head_dim:
            raise TBError(TB_ERR_INVALID_ARGUMENT, f"{name}: {list(p[at].shape)} is not rows of heads of {head_dim}")
    # What the later calls would refuse is refused before the first one is made.
    if head_dim > MAX_HEAD_DIM:
        raise TBError(TB_ERR_UNSUPPORTED, f"head_dim {head_dim} exceeds {MAX_HEAD_DIM}")
    if (q[at].shape[0] + k[at].shape[0]) // head_dim > MAX_HEADS:
        raise TBError(TB_ERR_UNSUPPORTED, f"more than {MAX_HEADS} heads of queries and keys")
    if not eps >= 0:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "eps must be >= 0")
    if axes is not None:
        axes = tuple(axes)
    _rotated_dims(_kind(positions), _kind(freqs), x.shape[0], head_dim, axes)
    _axis_layout(axes, axis_halves, interleaved, True)
    for w in (q_weight, k_weight):
        if w is not None:
            _expect("head weight", w, (head_dim,), dtype)
    int8 = kinds == {2} and q[0].dtype == INT8
    if kinds == {2}:
        _dtype_code(dtype)
        m, in_dim = x.shape
        sizes = []
        for name, (Wq, scale) in zip("qkv", (q, k, v)):
            if int8:
                xs = _kind(x_scale) if x_scale is not None else ((m,), torch.float32)
                x_kind = _kind(x) if x_scale is not None else (x.shape, INT8)
                sizes.append(_dense_int8_dims(x_kind, _kind(Wq), _kind(scale), xs, None, dtype)[:5])
                continue
            if scale.dtype != q[1].dtype:
                raise TBError(TB_ERR_INVALID_ARGUMENT, f"{name}: scales are {scale.dtype}, those of q {q[1].dtype}")
            xs = _kind(x_scale) if x_scale is not None else ((m, _fp8_blocks(in_dim)), scale.dtype)
            x_kind = _kind(x) if x_scale is not None else (x.shape, E4M3)
            sizes.append(_dense_fp8_dims(x_kind, _kind(Wq), _kind(scale), xs, None, dtype)[:6])
        if in_dim % 16:
            raise TBError(TB_ERR_UNSUPPORTED, f"in_dim {in_dim} is not a multiple of 16")
        if x_scale is None:
            _dtype_code(x.dtype)
    _need_cuda(positions, freqs, q_weight, k_weight)
    if kinds == {4}:
        ys = linear_forward_group([(x, *p) for p in (q, k, v)])
    else:
        dev = _here([t for t in (x, x_scale, *q, *k, *v) if t is not None])
        for name, (Wq, _), size in zip("qkv", (q, k, v), sizes):
            if Wq.data_ptr() % 16:
                raise TBError(TB_ERR_UNSUPPORTED, f"{name}: Wq must be 16-byte aligned")
            (_int8_workspace_size if int8 else _fp8_workspace_size)(dev, *size)   # (raises where a size is too large)
        if x_scale is None:
            x, x_scale = quantize_rows_int8(x) if int8 else quantize_activations(x, q[1].dtype)
        dense = dense_forward_int8 if int8 else dense_forward_fp8
        ys = [dense(x, *p, x_scale=x_scale, out_dtype=dtype) for p in (q, k, v)]
    yq, yk, yv = (y.view(y.shape[0], y.shape[1] // head_dim, head_dim) for y in ys)
    head_norm_rotate([(yq, q_weight), (yk, k_weight)], positions, freqs, eps, weight_offset, interleaved, [yq, yk], axes,
                     axis_halves)
    return yq, yk, yv


# ---------------------------------------------------------------------------
# Analytic decomposition
# ---------------------------------------------------------------------------


def shared_block(weights, out: torch.Tensor | None = None) -> torch.Tensor:
    """Mean of a band's weight matrices (fp32), via tb_shared_block."""
    n = len(weights)
    if not 1 <= n <= MAX_BAND_LAYERS:
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"a band holds 1..{MAX_BAND_LAYERS} layers")
    if weights[0].dim() != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "weights must be [out, in]")
    out_dim, in_dim = weights[0].shape
    for j, w in enumerate(weights):
        _expect(f"weights[{j}]", w, (out_dim, in_dim), weights[0].dtype)
    _expect_out(out, (out_dim, in_dim), torch.float32)
    _need_cuda(*weights, out)
    out = _output(out, (out_dim, in_dim), torch.float32, weights[0])
    ptrs = (ctypes.c_void_p * n)(*[w.data_ptr() for w in weights])
    _check(lib.tb_shared_block(ptrs, n, out_dim, in_dim, _dtype_code(weights[0].dtype), _ptr(out), _stream()))
    return out


def row_scale(weight: torch.Tensor, W0: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Per-row least-squares scale of weight against W0 (fp32 [out]), via tb_row_scale."""
    if weight.dim() != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "weight must be [out, in]")
    _expect("W0", W0, weight.shape, torch.float32)
    _expect_out(out, (weight.shape[0],), torch.float32)
    _need_cuda(weight, W0, out)
    out = _output(out, (weight.shape[0],), torch.float32, weight)
    _check(lib.tb_row_scale(_ptr(weight), _ptr(W0), weight.shape[0], weight.shape[1], _dtype_code(weight.dtype),
                            _ptr(out), _stream()))
    return out


def lowrank_factors_workspace_size(out_dim: int, in_dim: int, rank: int, k: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.tb_lowrank_factors_workspace_size(out_dim, in_dim, rank, k, ctypes.byref(out)))
    return out.value


def lowrank_factors(weight: torch.Tensor, W0: torch.Tensor, s: torch.Tensor, rank: int, omega: torch.Tensor,
                    power_iters: int, workspace: torch.Tensor | None = None):
    """U [out, rank], V [in, rank] (fp32) of weight - diag(s) W0 by the randomized SVD with probe omega [in, k],
    via tb_lowrank_factors."""
    if weight.dim() != 2 or omega.dim() != 2:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "weight must be [out, in] and omega [in, k]")
    out_dim, in_dim = weight.shape
    k = omega.shape[1]
    _expect("W0", W0, (out_dim, in_dim), torch.float32)
    _expect("s", s, (out_dim,), torch.float32)
    _expect("omega", omega, (in_dim, k), torch.float32)
    _need_cuda(weight, W0, s, omega)
    U = torch.zeros((out_dim, rank), dtype=torch.float32, device=weight.device)
    V = torch.zeros((in_dim, rank), dtype=torch.float32, device=weight.device)
    need = lowrank_factors_workspace_size(out_dim, in_dim, rank, k)
    ws = workspace if workspace is not None and workspace.numel() >= need else \
        torch.empty(need, dtype=torch.uint8, device=weight.device)
    _check(lib.tb_lowrank_factors(_ptr(weight), _ptr(W0), _ptr(s), out_dim, in_dim, rank, _dtype_code(weight.dtype),
                                  _ptr(omega), k, power_iters, _ptr(U) if rank else None, _ptr(V) if rank else None,
                                  _ptr(ws), ws.numel(), _stream()))
    return U, V


def lowrank_factors_batch(weights, W0s, S: torch.Tensor, rank: int, omega: torch.Tensor,
                          power_iters: int, workspace: torch.Tensor | None = None):
    """U [n, out, rank], V [n, in, rank] (fp32) for n weights of one shape, each with its shared block (W0s: one
    fp32 tensor for all, or a list of n), S [n, out], omega [n, in, k], via tb_lowrank_factors_batch."""
    n = len(weights)
    if weights[0].dim() != 2 or omega.dim() != 3:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "weights must be [out, in] and omega [n, in, k]")
    out_dim, in_dim = weights[0].shape
    k = omega.shape[2]
    W0s = list(W0s) if isinstance(W0s, (list, tuple)) else [W0s] * n
    if len(W0s) != n:
        raise TBError(TB_ERR_INVALID_ARGUMENT, "one shared block per weight")
    for j in range(n):
        _expect(f"weights[{j}]", weights[j], (out_dim, in_dim), weights[0].dtype)
        _expect(f"W0s[{j}]", W0s[j], (out_dim, in_dim), torch.float32)
    _expect("S", S, (n, out_dim), torch.float32)
    _expect("omega", omega, (n, in_dim, k), torch.float32)
    _need_cuda(S, omega, *weights, *W0s)
    U = torch.zeros((n, out_dim, rank), dtype=torch.float32, device=S.device)
    V = torch.zeros((n, in_dim, rank), dtype=torch.float32, device=S.device)
    need = n * lowrank_factors_workspace_size(out_dim, in_dim, rank, k)
    ws = workspace if workspace is not None and workspace.numel() >= need else \
        torch.empty(need, dtype=torch.uint8, device=S.device)
    ptrs = (ctypes.c_void_p * n)(*[w.data_ptr() for w in weights])
    w0p = (ctypes.c_void_p * n)(*[w.data_ptr() for w in W0s])
    _check(lib.tb_lowrank_factors_batch(ptrs, n, w0p, _ptr(S), out_dim, in_dim, rank,
                                        _dtype_code(weights[0].dtype), _ptr(omega), k, power_iters,
                                        _ptr(U) if rank else None, _ptr(V) if rank else None, _ptr(ws), ws.numel(),
                                        _stream()))
    return U, V


def decompose(weights, num_bands: int, rank: int, oversampling: int = 16, power_iters: int = 2, seed: int = 0,
              batch_bytes: int = 24 << 30) -> dict:
    """One family's theta bundle on the GPU: per band the shared block, per layer the row scale, and the low-rank
    factors of all layers batched (tb_lowrank_factors_batch, at most `batch_bytes` of workspace per call).  The
    randomized SVD uses k = min(rank + oversampling, out, in) and one probe per layer, drawn from a seeded normal
    generator in layer order.  Returns {"W0": [per band], "band": [per layer], "s", "U", "V": [per layer]} of
    fp32 device tensors."""
    L = len(weights)
    bands = [band_index(L, num_bands, l) for l in range(L)]
    out_dim, in_dim = weights[0].shape
    dev = weights[0].device
    W0 = [shared_block([weights[l] for l in range(L) if bands[l] == b]) for b in range(num_bands)]
    res = {"W0": W0, "band": bands, "s": [row_scale(weights[l], W0[bands[l]]) for l in range(L)],
           "U": [None] * L, "V": [None] * L}
    if rank == 0:
        res["U"] = [torch.zeros((out_dim, 0), dtype=torch.float32, device=dev) for _ in range(L)]
        res["V"] = [torch.zeros((in_dim, 0), dtype=torch.float32, device=dev) for _ in range(L)]
        return res
    k = min(rank + oversampling, out_dim, in_dim, MAX_PROBE)
    gen = torch.Generator(device="cpu").manual_seed(seed)
    omegas = [torch.randn((in_dim, k), generator=gen, dtype=torch.float32) for _ in range(L)]
    per = lowrank_factors_workspace_size(out_dim, in_dim, rank, k)
    chunk = max(1, min(MAX_BAND_LAYERS, batch_bytes // per))
    for c0 in range(0, L, chunk):
        part = list(range(c0, min(L, c0 + chunk)))
        S = torch.stack([res["s"][l] for l in part])
        om = torch.stack([omegas[l] for l in part]).to(dev)
        U, V = lowrank_factors_batch([weights[l] for l in part], [W0[bands[l]] for l in part], S, rank, om,
                                     power_iters)
        for j, l in enumerate(part):
            res["U"][l], res["V"][l] = U[j], V[j]
    return res


def refine_shared_block(weights, s_list, U_list, V_list, W0_prev: torch.Tensor,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """Least-squares refit of a band's shared block with every layer's s, U, V fixed (fp32), via
    tb_refine_shared_block; `out` may be W0_prev itself."""
    n = len(weights)
    if W0_prev.dim() != 2 or not (len(s_list) == len(U_list) == len(V_list) == n):
        raise TBError(TB_ERR_INVALID_ARGUMENT, "W0_prev must be [out, in], with s, U, V lists as long as weights")
    out_dim, in_dim = W0_prev.shape
    _expect("W0_prev", W0_prev, (out_dim, in_dim), torch.float32)
    rank = 0 if U_list[0] is None else U_list[0].shape[1]
    for j in range(n):
        _expect(f"weights[{j}]", weights[j], (out_dim, in_dim), weights[0].dtype)
        _expect(f"s[{j}]", s_list[j], (out_dim,), torch.float32)
        if rank:
            _expect(f"U[{j}]", U_list[j], (out_dim, rank), torch.float32)
            _expect(f"V[{j}]", V_list[j], (in_dim, rank), torch.float32)
    _expect_out(out, (out_dim, in_dim), torch.float32)
    _need_cuda(W0_prev, out, *weights, *s_list, *(U_list if rank else []), *(V_list if rank else []))
    out = _output(out, (out_dim, in_dim), torch.float32, W0_prev)
    arr = lambda ts: (ctypes.c_void_p * n)(*[t.data_ptr() for t in ts])
    need = ctypes.c_size_t(0)
    _check(lib.tb_refine_shared_block_workspace_size(out_dim, in_dim, n, rank, ctypes.byref(need)))
    ws = torch.empty(need.value, dtype=torch.uint8, device=W0_prev.device)
    _check(lib.tb_refine_shared_block(arr(weights), arr(s_list), arr(U_list) if rank else None,
                                      arr(V_list) if rank else None, n, out_dim, in_dim, rank,
                                      _dtype_code(weights[0].dtype), _ptr(W0_prev), _ptr(out), _ptr(ws), ws.numel(),
                                      _stream()))
    return out


def als_decompose(weights, num_bands: int, rank: int, iters: int, oversampling: int = 16, power_iters: int = 2,
                  seed: int = 0) -> dict:
    """decompose() followed by `iters` rounds of alternating least squares: every band's W0 refitted with s, U, V
    fixed (refine_shared_block), then every layer's s and U, V against the new W0 (new probes per round)."""
    bun = decompose(weights, num_bands, rank, oversampling, power_iters, seed)
    L = len(weights)
    bands = bun["band"]
    out_dim, in_dim = weights[0].shape
    dev = weights[0].device
    k = min(rank + oversampling, out_dim, in_dim, MAX_PROBE)
    for it in range(iters):
        for b in range(num_bands):
            mem = [l for l in range(L) if bands[l] == b]
            refine_shared_block([weights[l] for l in mem], [bun["s"][l] for l in mem],
                                [bun["U"][l] if rank else None for l in mem],
                                [bun["V"][l] if rank else None for l in mem], bun["W0"][b], out=bun["W0"][b])
        bun["s"] = [row_scale(weights[l], bun["W0"][bands[l]]) for l in range(L)]
        if rank:
            gen = torch.Generator(device="cpu").manual_seed(seed + 1 + it)
            om = torch.stack([torch.randn((in_dim, k), generator=gen, dtype=torch.float32) for _ in range(L)]).to(dev)
            U, V = lowrank_factors_batch(weights, [bun["W0"][bands[l]] for l in range(L)], torch.stack(bun["s"]), rank,
                                         om, power_iters)
            bun["U"] = [U[l] for l in range(L)]
            bun["V"] = [V[l] for l in range(L)]
    return bun



# The seven projection families of a decoder layer ("The theta bundle", section "Projection families").
ATTENTION_FAMILIES = ("q_proj", "k_proj", "v_proj", "o_proj")
MLP_FAMILIES = ("gate_proj", "up_proj", "down_proj")


def decompose_model(weights_by_family: dict, num_bands: int, rank: int, tie_families: str = "all",
                    oversampling: int = 16, power_iters: int = 2, seed: int = 0) -> dict:
    """Theta bundles for the projection families of a model ("The theta bundle", section "Projection families").

    weights_by_family maps a family name to its per-layer weights.  tie_families="all": every family goes through
    decompose() (family j of the dict order uses seed + j).  tie_families="attn": only q/k/v/o do; each MLP layer
    stays a plain dense layer, returned as the bundle whose W0 is the layer's own weight (the caller's tensor, not a
    copy; every layer its own band), with s = None (unit scale) and U = V = None, which linear_forward,
    linear_forward_group and dense_forward take as they are."""
    if tie_families not in ("all", "attn"):
        raise TBError(TB_ERR_INVALID_ARGUMENT, f"tie_families must be 'all' or 'attn', not {tie_families!r}")
    for fam in weights_by_family:
        if fam not in ATTENTION_FAMILIES + MLP_FAMILIES:
            raise TBError(TB_ERR_INVALID_ARGUMENT, f"unknown projection family {fam!r}")
    out = {}
    for j, (fam, weights) in enumerate(weights_by_family.items()):
        if tie_families == "attn" and fam in MLP_FAMILIES:
            L = len(weights)
            out[fam] = {"W0": list(weights), "band": list(range(L)), "s": [None] * L, "U": [None] * L,
                        "V": [None] * L}
        else:
            out[fam] = decompose(weights, num_bands, rank, oversampling, power_iters, seed + j)
    return out
