"""Binding of libdsix_prep (include/dsix_prep.h): what an indexer step needs
before its logits -- block tables and slot maps from request lengths, rotary
positions, layer norm with its gradient, and the indexer key's fused norm +
rotary + fp8 write.

As in the package itself: argument marshalling only, shapes checked before any
pointer is taken, outputs allocated by the caller, every call asynchronous on
``stream`` and capturable, no fallback without the library.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Sequence

import torch

from . import BLOCK_SIZE, HEAD_DIM, DsixError, _need

__all__ = [
    "PREP_LIB_PATH", "load_prep", "ix_prep_device_status", "ix_plan_step", "ix_rope_frequencies", "ix_rope_table",
    "ix_rope", "ix_layer_norm", "ix_layer_norm_bwd", "ix_layer_norm_bwd_workspace_size", "ix_norm_rope_write_k",
]

PREP_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdsix_prep.so")

_P, _I64, _I32, _F64, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_float


class _RopeTensor(ctypes.Structure):
    _fields_ = [("x", _P), ("out", _P), ("heads", _I32), ("x_token_stride", _I64), ("x_head_stride", _I64),
                ("out_token_stride", _I64), ("out_head_stride", _I64)]


_RP = ctypes.POINTER(_RopeTensor)
_DP = ctypes.POINTER(_F64)
_SIGNATURES = {
    "ix_prep_device_status": ([_P], _I32),
    "ix_plan_step": ([_P, _P, _I32, _I32, _P, _I64, _P, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64,
                      _P], _I32),
    "ix_rope_frequencies": ([_I32, _I32, _F64, _F64, _F64, _F64, _F64, _DP], _I32),
    "ix_rope_table": ([_DP, _I32, _I64, _I64, _F64, _P, _P], _I32),
    "ix_rope": ([_RP, _RP, _I32, _I64, _I32, _I32, _P, _P, _I64, _I32, _I32, _P], _I32),
    "ix_layer_norm": ([_P, _I64, _P, _P, _I32, _F32, _I64, _I32, _P, _I64, _P, _P, _I32, _P], _I32),
    "ix_layer_norm_bwd_workspace_size": ([_I64, _I32], ctypes.c_size_t),
    "ix_layer_norm_bwd": ([_P, _I64, _P, _I64, _P, _I32, _P, _P, _I64, _I32, _P, _I64, _P, _P, _I32, _P,
                           ctypes.c_size_t, _P], _I32),
    "ix_norm_rope_write_k": ([_P, _I64, _I32, _I64, _P, _P, _F32, _P, _P, _I64, _I32, _I32, _I32, _P, _P, _I64,
                              _I32, _P], _I32),
}

_lib = None
_lock = threading.Lock()


def load_prep(path: Optional[str] = None):
    """Load libdsix_prep.so (built by ``deepseek_v3_sparse_gb300.build``); raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        p = path or PREP_LIB_PATH
        if not os.path.exists(p):
            raise DsixError(f"{p} is missing: build it with `python -m deepseek_v3_sparse_gb300.build` "
                            "(there is no non-CUDA fallback)")
        lib = ctypes.CDLL(p)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        if path is None:
            _lib = lib
        return lib


def _check(rc: int, name: str):
    if rc != 0:
        from . import ix_status_string
        raise DsixError(f"{name}: {ix_status_string(rc)} ({rc})")


def ix_prep_device_status() -> int:
    """Synchronously read and clear this library's device status word (IX_DEV_* bits)."""
    v = ctypes.c_int(0)
    rc = load_prep().ix_prep_device_status(ctypes.byref(v))
    if rc not in (0, -7):
        _check(rc, "ix_prep_device_status")
    return int(v.value)


_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _device(t: torch.Tensor, name: str) -> int:
    """The current device's index, on which every tensor of a call has to be: the
    library launches there."""
    dev = t.get_device()
    if dev < 0:
        raise DsixError(f"{name}: must be a CUDA tensor")
    if dev != torch.cuda.current_device():
        raise DsixError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _ptr(t: torch.Tensor, name: str, dtype: torch.dtype, dev: int) -> int:
    """The pointer of a contiguous tensor of a type on device `dev`."""
    if t.get_device() != dev:
        _device(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise DsixError(f"{name}: must be contiguous")
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, dev: int):
    return None if t is None else _ptr(t, name, dtype, dev)


def _tensor(t, name: str, dim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dim() != dim:
        raise DsixError(f"{name}: shape {tuple(t.shape)}, expected {dim} dimensions")


def _flat(t, n: int, name: str):
    """A tensor of at least n elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.numel() < n:
        raise DsixError(f"{name}: {t.numel()} elements, expected >= {n}")


def _strided(t: torch.Tensor, name: str, shape, dtype=None):
    """An activation: the shape given, its last dimension contiguous."""
    _tensor(t, name, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise DsixError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise DsixError(f"{name}: the last dimension must be contiguous")
    if t.dtype not in _TYPES if dtype is None else t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype or tuple(_TYPES)}")


def _stream(stream, dev: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def ix_plan_step(cached_lens: torch.Tensor, new_lens: torch.Tensor, free_blocks: torch.Tensor,
                 block_table: torch.Tensor, context_lens: torch.Tensor, cu_new: torch.Tensor, cu_ctx: torch.Tensor,
                 cu_blocks: torch.Tensor, slot_mapping: torch.Tensor, positions: torch.Tensor, row_req: torch.Tensor,
                 row_len: torch.Tensor, ks: torch.Tensor, ke: torch.Tensor, block_size: int = BLOCK_SIZE,
                 stream=None) -> None:
    """cached_lens, new_lens [B] int32; free_blocks [F] int32; block_table [B, width] int32 (its new entries
    are written).  Written: context_lens [B], cu_new, cu_ctx, cu_blocks [B + 1] int32; for the step's rows (as
    many as slot_mapping has, the ones past the new tokens empty) slot_mapping, positions int64 and row_req,
    row_len, ks, ke int32."""
    _tensor(cached_lens, "cached_lens", 1)
    batch = cached_lens.shape[0]
    _flat(new_lens, batch, "new_lens")
    _tensor(free_blocks, "free_blocks", 1)
    _tensor(block_table, "block_table", 2)
    _need(block_table.shape[0] >= batch, f"block_table: {block_table.shape[0]} rows, expected >= {batch}")
    _flat(context_lens, batch, "context_lens")
    _flat(cu_new, batch + 1, "cu_new")
    _flat(cu_ctx, batch + 1, "cu_ctx")
    _flat(cu_blocks, batch + 1, "cu_blocks")
    _tensor(slot_mapping, "slot_mapping", 1)
    rows = slot_mapping.shape[0]
    _flat(positions, rows, "positions")
    _flat(row_req, rows, "row_req")
    _flat(row_len, rows, "row_len")
    _flat(ks, rows, "ks")
    _flat(ke, rows, "ke")
    dev = _device(cached_lens, "cached_lens")
    i32, i64, width = torch.int32, torch.int64, block_table.shape[1]
    rc = load_prep().ix_plan_step(
        _ptr(cached_lens, "cached_lens", i32, dev), _ptr(new_lens, "new_lens", i32, dev), batch, block_size,
        _ptr(free_blocks, "free_blocks", i32, dev), free_blocks.shape[0], _ptr(block_table, "block_table", i32, dev),
        width, width, _ptr(context_lens, "context_lens", i32, dev), _ptr(cu_new, "cu_new", i32, dev),
        _ptr(cu_ctx, "cu_ctx", i32, dev), _ptr(cu_blocks, "cu_blocks", i32, dev),
        _ptr(slot_mapping, "slot_mapping", i64, dev), _ptr(positions, "positions", i64, dev),
        _ptr(row_req, "row_req", i32, dev), _ptr(row_len, "row_len", i32, dev), _ptr(ks, "ks", i32, dev),
        _ptr(ke, "ke", i32, dev), rows, _stream(stream, dev))
    _check(rc, "ix_plan_step")


_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}


def ix_rope_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                        original: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """The rot / 2 rotary frequencies (radians per position) as a list, computed on the host; scaling: None,
    "linear", "ntk" or "yarn" (see ix_rope_frequencies in dsix_prep.h)."""
    _need(scaling in _SCALINGS, f"scaling: {scaling!r} is none of {tuple(_SCALINGS)}")
    out = (_F64 * max(1, int(rot) // 2))()
    rc = load_prep().ix_rope_frequencies(_SCALINGS[scaling], int(rot), float(base), float(factor), float(original),
                                         float(beta_fast), float(beta_slow), out)
    _check(rc, "ix_rope_frequencies")
    return list(out)


def ix_rope_table(cos_sin: torch.Tensor, inv_freq: Sequence[float], first_position: int = 0, amplitude: float = 1.0,
                  stream=None) -> None:
    """cos_sin [n, rot] f32 (written): amplitude * (rot / 2 cosines, then rot / 2 sines) of the positions
    first_position .. first_position + n - 1; inv_freq: rot / 2 numbers."""
    _tensor(cos_sin, "cos_sin", 2)
    n, rot = cos_sin.shape
    _need(rot == 2 * len(inv_freq), f"inv_freq: {len(inv_freq)} values, cos_sin has {rot} columns")
    dev = _device(cos_sin, "cos_sin")
    rc = load_prep().ix_rope_table((_F64 * len(inv_freq))(*inv_freq), rot, int(first_position), n, float(amplitude),
                                   _ptr(cos_sin, "cos_sin", torch.float32, dev), _stream(stream, dev))
    _check(rc, "ix_rope_table")


def _rope_side(x, out, names, tokens, dim, dtype):
    _tensor(x, names[0], 3)
    _need(x.shape[0] == tokens and x.shape[2] == dim,
          f"{names[0]}: shape {tuple(x.shape)}, expected ({tokens}, heads, {dim})")
    _strided(x, names[0], x.shape, dtype)
    _strided(out, names[1], x.shape, x.dtype)


def ix_rope(x: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor, out: torch.Tensor, offset: int = 0,
            interleaved: bool = False, inverse: bool = False, x2: Optional[torch.Tensor] = None,
            out2: Optional[torch.Tensor] = None, stream=None) -> None:
    """x, out [T, H, D] bf16, fp16 or f32 (strided; out may be x); positions [T] int64; cos_sin [max_pos, rot]
    f32: the values offset .. offset + rot - 1 of every head are turned, the others copied.  inverse: the
    transposed rotation (the gradient).  x2, out2 [T, H2, D]: a second tensor turned in the same launch."""
    _tensor(x, "x", 3)
    tokens, heads, dim = x.shape
    _rope_side(x, out, ("x", "out"), tokens, dim, None)
    if x2 is not None:
        _rope_side(x2, out2, ("x2", "out2"), tokens, dim, x.dtype)
    _flat(positions, tokens, "positions")
    _tensor(cos_sin, "cos_sin", 2)
    max_pos, rot = cos_sin.shape
    dev = _device(x, "x")
    for t, name in ((out, "out"), (x2, "x2"), (out2, "out2")):
        if t is not None and t.get_device() != dev:
            _device(t, name)
    xs, os = x.stride(), out.stride()
    side = _RopeTensor(x.data_ptr(), out.data_ptr(), heads, xs[0], xs[1], os[0], os[1])
    side2 = None
    if x2 is not None:
        xs, os = x2.stride(), out2.stride()
        side2 = ctypes.byref(_RopeTensor(x2.data_ptr(), out2.data_ptr(), x2.shape[1], xs[0], xs[1], os[0], os[1]))
    rc = load_prep().ix_rope(ctypes.byref(side), side2, _TYPES[x.dtype], tokens, dim, offset,
                             _ptr(positions, "positions", torch.int64, dev),
                             _ptr(cos_sin, "cos_sin", torch.float32, dev), max_pos, rot,
                             (1 if interleaved else 0) | (2 if inverse else 0), _stream(stream, dev))
    _check(rc, "ix_rope")


def _weights(cols: int, dtype: torch.dtype, **weights):
    """The C type of the weights (f32, or the activations'), which those given share."""
    kind = None
    for name, w in weights.items():
        if w is None:
            continue
        _tensor(w, name, 1)
        _need(w.shape[0] == cols, f"{name}: {w.shape[0]} elements, expected {cols}")
        if w.dtype is not torch.float32 and w.dtype is not dtype:
            raise TypeError(f"{name}: dtype {w.dtype}, expected {torch.float32} or {dtype}")
        _need(kind is None or w.dtype is kind, f"{name}: dtype {w.dtype}, the other weights have {kind}")
        kind = w.dtype
    return torch.float32 if kind is None else kind


def ix_layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], eps: float,
                  out: torch.Tensor, mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """x, out [rows, cols] bf16, fp16 or f32 (rows strided; out may be x); gamma, beta [cols] f32 or of x's type,
    or None; mean, rstd [rows] f32 (written, for ix_layer_norm_bwd) or None."""
    _tensor(x, "x", 2)
    rows, cols = x.shape
    _strided(x, "x", x.shape)
    _strided(out, "out", x.shape, x.dtype)
    wt = _weights(cols, x.dtype, gamma=gamma, beta=beta)
    _need((mean is None) == (rstd is None), "mean and rstd: both or neither")
    if mean is not None:
        _flat(mean, rows, "mean")
        _flat(rstd, rows, "rstd")
    dev = _device(x, "x")
    if out.get_device() != dev:
        _device(out, "out")
    rc = load_prep().ix_layer_norm(x.data_ptr(), x.stride(0), _opt(gamma, "gamma", wt, dev),
                                   _opt(beta, "beta", wt, dev), _TYPES[wt], eps, rows, cols, out.data_ptr(),
                                   out.stride(0), _opt(mean, "mean", torch.float32, dev),
                                   _opt(rstd, "rstd", torch.float32, dev), _TYPES[x.dtype], _stream(stream, dev))
    _check(rc, "ix_layer_norm")


def ix_layer_norm_bwd_workspace_size(rows: int, cols: int) -> int:
    """Bytes of scratch that ix_layer_norm_bwd needs for the weights' gradients."""
    return int(load_prep().ix_layer_norm_bwd_workspace_size(int(rows), int(cols)))


def ix_layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor], mean: torch.Tensor,
                      rstd: torch.Tensor, dx: torch.Tensor, dgamma: Optional[torch.Tensor] = None,
                      dbeta: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """dy, x, dx [rows, cols] of one type (rows strided; dx may be dy); gamma, mean, rstd as in ix_layer_norm;
    dgamma, dbeta [cols] f32 (written) or None; workspace uint8 of at least
    ix_layer_norm_bwd_workspace_size(rows, cols) bytes (with dgamma)."""
    _tensor(x, "x", 2)
    rows, cols = x.shape
    _strided(x, "x", x.shape)
    _strided(dy, "dy", x.shape, x.dtype)
    _strided(dx, "dx", x.shape, x.dtype)
    wt = _weights(cols, x.dtype, gamma=gamma)
    _flat(mean, rows, "mean")
    _flat(rstd, rows, "rstd")
    _need((dgamma is None) == (dbeta is None), "dgamma and dbeta: both or neither")
    if dgamma is not None:
        _flat(dgamma, cols, "dgamma")
        _flat(dbeta, cols, "dbeta")
    dev = _device(x, "x")
    for t, name in ((dy, "dy"), (dx, "dx")):
        if t.get_device() != dev:
            _device(t, name)
    f32 = torch.float32
    rc = load_prep().ix_layer_norm_bwd(
        dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), _opt(gamma, "gamma", wt, dev), _TYPES[wt],
        _ptr(mean, "mean", f32, dev), _ptr(rstd, "rstd", f32, dev), rows, cols, dx.data_ptr(), dx.stride(0),
        _opt(dgamma, "dgamma", f32, dev), _opt(dbeta, "dbeta", f32, dev), _TYPES[x.dtype],
        _opt(workspace, "workspace", torch.uint8, dev), 0 if workspace is None else workspace.numel(),
        _stream(stream, dev))
    _check(rc, "ix_layer_norm_bwd")


def ix_norm_rope_write_k(k: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float,
                         positions: torch.Tensor, cos_sin: torch.Tensor, slot_mapping: torch.Tensor,
                         cache: torch.Tensor, rope_offset: int = 0, interleaved: bool = False,
                         block_size: int = BLOCK_SIZE, stream=None) -> None:
    """k [n, 128] bf16, fp16 or f32 (rows strided, 16-byte aligned); gamma, beta [128] f32; positions,
    slot_mapping [n] int64; cos_sin [max_pos, rot] f32; cache uint8 [num_blocks, 8448] (written)."""
    _tensor(k, "k", 2)
    n = k.shape[0]
    _strided(k, "k", (n, HEAD_DIM))
    _flat(gamma, HEAD_DIM, "gamma")
    _flat(beta, HEAD_DIM, "beta")
    _flat(positions, n, "positions")
    _flat(slot_mapping, n, "slot_mapping")
    _tensor(cos_sin, "cos_sin", 2)
    _tensor(cache, "cache", 2)
    _need(cache.shape[1] == block_size * (HEAD_DIM + 4),
          f"cache: {cache.shape[1]} bytes a block, expected {block_size * (HEAD_DIM + 4)}")
    max_pos, rot = cos_sin.shape
    dev = _device(k, "k")
    f32, i64 = torch.float32, torch.int64
    rc = load_prep().ix_norm_rope_write_k(
        k.data_ptr(), k.stride(0), _TYPES[k.dtype], n, _ptr(gamma, "gamma", f32, dev), _ptr(beta, "beta", f32, dev),
        eps, _ptr(positions, "positions", i64, dev), _ptr(cos_sin, "cos_sin", f32, dev), max_pos, rot, rope_offset,
        1 if interleaved else 0, _ptr(slot_mapping, "slot_mapping", i64, dev),
        _ptr(cache, "cache", torch.uint8, dev), cache.shape[0], block_size, _stream(stream, dev))
    _check(rc, "ix_norm_rope_write_k")
