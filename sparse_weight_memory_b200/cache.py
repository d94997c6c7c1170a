"""Thin ctypes binding of the paged key-value cache (include/fwpkm_cache.h).

Argument checks and marshalling only: the work runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from .fwpkm import FWPKM_BF16, FWPKM_EINVAL, FWPKM_ESHAPE, FWPKM_F32, FwpkmError, load_library

E4M3 = 2                       # FWPKM_E4M3
ROTATE = {"halves": 0, "pairs": 1}
BAD_PAGE, BAD_LENGTH = 32, 64  # bits of an `errors` word

_DTYPES = {torch.float32: FWPKM_F32, torch.bfloat16: FWPKM_BF16, torch.float8_e4m3fn: E4M3}
_vp = ctypes.c_void_p


class _Cache(ctypes.Structure):  # fwpkm_cache
    _fields_ = [("keys", _vp), ("values", _vp), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("key_scale", _vp), ("value_scale", _vp)]


class _Batch(ctypes.Structure):  # fwpkm_cache_batch
    _fields_ = [("B", ctypes.c_int), ("table_width", ctypes.c_int),
                ("table_stride", ctypes.c_int64), ("table", _vp), ("lengths", _vp)]


_lib = None


def _library():
    global _lib
    if _lib is None:
        L = load_library()
        i32, i64, f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_float
        pc, pb = ctypes.POINTER(_Cache), ctypes.POINTER(_Batch)
        L.fwpkm_cache_append.argtypes = [pc, pb, i32, i32, _vp, i64, _vp, i64, _vp, i64, _vp, i64,
                                         i32, _vp, i32, i32, _vp, _vp, _vp]
        L.fwpkm_cache_append.restype = i32
        L.fwpkm_cache_attend.argtypes = [pc, pb, i32, i32, _vp, i64, f32, i32, _vp, _vp, _vp, i64,
                                         _vp, _vp]
        L.fwpkm_cache_attend.restype = i32
        L.fwpkm_cache_attend_workspace.argtypes = [pc, i32, i32]
        L.fwpkm_cache_attend_workspace.restype = i64
        _lib = L
    return _lib


def _check(rc: int):
    if rc < 0:
        raise FwpkmError(rc, _library().fwpkm_last_error().decode())
    return rc


def _shape(ok: bool, message: str):
    if not ok:
        raise FwpkmError(FWPKM_ESHAPE, message)


class KVCache:
    """A paged cache of keys and values, written by ``append`` and read by ``attend``.

    ``keys`` and ``values`` are the pools, [pages][kv_heads][page_size][dim] in
    fp32, bf16 or float8_e4m3fn (one the transpose of another layout will do:
    only the last dimension has to be contiguous, and both need the same
    strides).  Without them the sizes are given, and both start at zero.
    ``key_scale`` and ``value_scale``, fp32 [kv_heads], are what an element of
    an 8-bit pool is multiplied by (default 1).

    Row b of ``table`` (int32 [B][width]) lists the pages of sequence b in
    order; ``lengths`` (int32 [B]) are the sequences' tokens, the new ones
    included.  Both lie on the device, so a captured graph follows them.
    """

    def __init__(self, pages: Optional[int] = None, page_size: Optional[int] = None,
                 kv_heads: Optional[int] = None, dim: Optional[int] = None,
                 dtype=torch.bfloat16, device="cuda", keys=None, values=None, key_scale=None,
                 value_scale=None):
        if (keys is None) != (values is None):
            raise FwpkmError(FWPKM_EINVAL, "keys and values must both be given, or neither")
        if keys is None:
            if None in (pages, page_size, kv_heads, dim):
                raise FwpkmError(FWPKM_EINVAL, "pages, page_size, kv_heads and dim, or the pools")
            _shape(min(pages, page_size, kv_heads, dim) >= 1, "the cache's sizes must be >= 1")
            if dtype not in _DTYPES:
                raise TypeError(f"unsupported dtype {dtype}")
            keys = torch.zeros((pages, kv_heads, page_size, dim), dtype=dtype, device=device)
            values = torch.zeros_like(keys)
        if keys.dtype not in _DTYPES or values.dtype != keys.dtype:
            raise TypeError(f"unsupported dtypes {keys.dtype}, {values.dtype}")
        _shape(keys.dim() == 4 and keys.shape == values.shape and min(keys.shape) >= 1,
               "keys and values must be [pages][kv_heads][page_size][dim]")
        _shape(keys.stride(3) == 1 and keys.stride() == values.stride(),
               "keys and values need a contiguous last dimension and the same strides")
        self._keys, self._values = keys, values
        self._scales = (key_scale, value_scale)
        self.device, self.dtype = keys.device, keys.dtype
        self.pages, self.kv_heads, self.page_size, self.dim = keys.shape
        if values.device != self.device:
            raise FwpkmError(FWPKM_EINVAL, "keys and values must be on one device")
        for s in self._scales:
            if s is not None:
                self._on_device(s, torch.float32, "scale")
                _shape(s.shape == (self.kv_heads,), "a scale must be [kv_heads]")
        ps, hs, rs, _ = keys.stride()
        self._c = _Cache(keys.data_ptr(), values.data_ptr(), ps, hs, rs, self.pages,
                         self.page_size, self.kv_heads, self.dim, _DTYPES[self.dtype],
                         *(None if s is None else s.data_ptr() for s in self._scales))
        self._ref = ctypes.byref(self._c)
        # what the sizes alone decide is refused here
        _check(_library().fwpkm_cache_attend_workspace(self._ref, 1, self.kv_heads))

    @property
    def keys(self):
        return self._keys

    @property
    def values(self):
        return self._values

    # -- checks --------------------------------------------------------------
    def _on_device(self, t, dtype, name, contiguous=True):
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
        if t.device != self.device:
            raise FwpkmError(FWPKM_EINVAL, f"{name} is on {t.device}, the cache on {self.device}")
        if contiguous and not t.is_contiguous():
            raise FwpkmError(FWPKM_ESHAPE, f"{name} must be contiguous")

    def _batch(self, table, lengths):
        self._on_device(table, torch.int32, "table", contiguous=False)
        self._on_device(lengths, torch.int32, "lengths")
        _shape(table.dim() == 2 and lengths.dim() == 1 and table.shape[0] == lengths.shape[0],
               "table must be [B][width] and lengths [B]")
        B, width = table.shape
        _shape(B >= 1 and width >= 1, "B and the table's width must be >= 1")
        _shape((width == 1 or table.stride(1) == 1) and (B == 1 or table.stride(0) >= width),
               "table rows must be contiguous")
        return _Batch(B, width, table.stride(0) if B > 1 else width, table.data_ptr(),
                      lengths.data_ptr())

    def _rows(self, t, name, dtype, heads=None):
        """[rows][heads][dim] with contiguous rows; the stride between rows."""
        self._on_device(t, dtype, name, contiguous=False)
        _shape(t.dim() == 3 and t.shape[2] == self.dim and (heads is None or t.shape[1] == heads),
               f"{name} must be [rows][{'heads' if heads is None else heads}][{self.dim}]")
        _shape(t.stride(2) == 1 and (t.shape[1] == 1 or t.stride(1) == self.dim),
               f"the rows of {name} must be contiguous")
        return t.stride(0) if t.shape[0] > 1 else t.shape[1] * self.dim

    def _errors(self, errors):
        if errors is None:
            return None
        self._on_device(errors, torch.int32, "errors")
        _shape(errors.numel() >= 1, "errors must hold a word")
        return errors.data_ptr()

    def _elsewhere(self):
        return self.device.type == "cuda" and torch.cuda.current_device() != self.device.index

    def _current_stream(self):
        if self.device.type != "cuda":
            raise FwpkmError(FWPKM_EINVAL, f"the cache is on {self.device}, not on a CUDA device")
        return torch.cuda.current_stream().cuda_stream

    @contextlib.contextmanager
    def _other(self, stream):
        """The cache's device, and `stream` where one is given, made current."""
        with torch.cuda.device(self.device):
            if stream is None:
                yield
            else:
                if not isinstance(stream, torch.cuda.Stream):
                    stream = torch.cuda.ExternalStream(stream or 0, device=self.device)
                with torch.cuda.stream(stream):
                    yield

    # -- the calls -----------------------------------------------------------
    def append(self, k, v, table, lengths, starts=None, q=None, freqs=None,
               style: str = "halves", q_out=None, errors=None, stream=None):
        """Write new tokens: k, v [rows][kv_heads][dim] (fp32 or bf16; rows may
        be strided, as parts of one projection are).  Rows starts[b] ..
        starts[b+1]-1 (int32 [B+1]) are sequence b's last tokens; without
        ``starts`` each sequence has one row, or none where its length is 0.
        ``freqs`` (fp32 [rotary/2], radians per token): the first ``rotary``
        elements of keys and queries turn by position, ``style`` "halves" or
        "pairs".  Returns the rotated ``q`` [rows][heads][dim] (in ``q_out``,
        which may be ``q``), or None without ``q``."""
        if stream is not None or self._elsewhere():
            with self._other(stream):
                return self._append(k, v, table, lengths, starts, q, freqs, style, q_out, errors)
        return self._append(k, v, table, lengths, starts, q, freqs, style, q_out, errors)

    def _append(self, k, v, table, lengths, starts, q, freqs, style, q_out, errors):
        batch = self._batch(table, lengths)
        if k.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"unsupported dtype {k.dtype}")
        if style not in ROTATE:
            raise FwpkmError(FWPKM_EINVAL, f"style must be one of {sorted(ROTATE)}")
        k_stride = self._rows(k, "k", k.dtype, self.kv_heads)
        v_stride = self._rows(v, "v", k.dtype, self.kv_heads)
        rows = k.shape[0]
        _shape(v.shape[0] == rows, "k and v must have the same rows")
        heads = q_stride = out_stride = 0
        if q is not None:
            q_stride, heads = self._rows(q, "q", k.dtype), q.shape[1]
            _shape(q.shape[0] == rows, "k and q must have the same rows")
            if q_out is None:
                q_out = torch.empty((rows, heads, self.dim), dtype=q.dtype, device=q.device)
            out_stride = self._rows(q_out, "q_out", q.dtype, heads)
            _shape(q_out.shape[0] == rows, "q and q_out must have the same rows")
        elif q_out is not None:
            raise FwpkmError(FWPKM_EINVAL, "q_out without q")
        rotary = 0
        if freqs is not None:
            self._on_device(freqs, torch.float32, "freqs")
            rotary = 2 * freqs.numel()
        if starts is not None:
            self._on_device(starts, torch.int32, "starts")
            _shape(starts.shape == (batch.B + 1,), "starts must be [B+1]")
        _check(_library().fwpkm_cache_append(
            self._ref, ctypes.byref(batch), rows, _DTYPES[k.dtype], k.data_ptr(), k_stride,
            v.data_ptr(), v_stride, None if q is None else q.data_ptr(), q_stride,
            None if q is None else q_out.data_ptr(), out_stride, heads,
            None if starts is None else starts.data_ptr(), rotary, ROTATE[style],
            freqs.data_ptr() if rotary else None, self._errors(errors),
            self._current_stream()))
        return q_out

    def attend(self, q, table, lengths, scale: Optional[float] = None, window: int = 0, out=None,
               lse=None, errors=None, stream=None, workspace=None):
        """Attention of one token of each sequence, q [B][heads][dim], over its
        cached tokens (the last ``window`` of them, or all): returns ``out``
        [B][heads][dim]; ``lse`` (fp32 [B][heads], optional) receives the log
        of the softmax's denominator.  ``scale`` defaults to 1/sqrt(dim).
        ``workspace``: see ``attend_workspace``; allocated per call without."""
        if stream is not None or self._elsewhere():
            with self._other(stream):
                return self._attend(q, table, lengths, scale, window, out, lse, errors, workspace)
        return self._attend(q, table, lengths, scale, window, out, lse, errors, workspace)

    def _attend(self, q, table, lengths, scale, window, out, lse, errors, workspace):
        batch = self._batch(table, lengths)
        if q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"unsupported dtype {q.dtype}")
        q_stride = self._rows(q, "q", q.dtype)
        B, heads, _ = q.shape
        _shape(B == batch.B, "q must have a row for each sequence")
        if out is None:
            out = torch.empty((B, heads, self.dim), dtype=q.dtype, device=q.device)
        else:
            self._on_device(out, q.dtype, "out")
            _shape(out.shape == q.shape, "out must be [B][heads][dim]")
        if lse is not None:
            self._on_device(lse, torch.float32, "lse")
            _shape(lse.shape == (B, heads), "lse must be [B][heads]")
        if workspace is None:
            workspace = torch.empty(self.attend_workspace(B, heads), dtype=torch.uint8,
                                    device=q.device)
        else:
            self._on_device(workspace, torch.uint8, "workspace")
        _check(_library().fwpkm_cache_attend(
            self._ref, ctypes.byref(batch), heads, _DTYPES[q.dtype], q.data_ptr(), q_stride,
            1.0 / math.sqrt(self.dim) if scale is None else scale, window, out.data_ptr(),
            None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
            self._errors(errors), self._current_stream()))
        return out

    def attend_workspace(self, B: int, heads: int) -> int:
        """Bytes of device memory that one running ``attend`` of these sizes needs."""
        return _check(_library().fwpkm_cache_attend_workspace(self._ref, B, heads))
