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

from .fwpkm import (FWPKM_BF16, FWPKM_EINVAL, FWPKM_ESHAPE, FWPKM_EUNSUPPORTED, FWPKM_F32,
                    FwpkmError, load_library)

E4M3 = 2                       # FWPKM_E4M3
ROTATE = {"halves": 0, "pairs": 1}
BAD_PAGE, BAD_LENGTH = 32, 64  # bits of an `errors` word

_DTYPES = {torch.float32: FWPKM_F32, torch.bfloat16: FWPKM_BF16, torch.float8_e4m3fn: E4M3}
_INPUTS = {torch.float32: FWPKM_F32, torch.bfloat16: FWPKM_BF16}
_vp = ctypes.c_void_p
# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Cache(ctypes.Structure):  # fwpkm_cache
    _fields_ = [("keys", _vp), ("values", _vp), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("key_scale", _vp), ("value_scale", _vp)]


class _Batch(ctypes.Structure):  # fwpkm_cache_batch
    _fields_ = [("B", ctypes.c_int), ("table_width", ctypes.c_int),
                ("table_stride", ctypes.c_int64), ("table", _vp), ("lengths", _vp)]


_INT = 2 ** 31  # sizes from here on do not fit the library's ints
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


def _refuse_gradients():
    raise FwpkmError(FWPKM_EUNSUPPORTED, "no gradients pass through the cache: call it under "
                     "torch.no_grad(), or detach its inputs")


class KVCache:
    """A paged cache of keys and values, written by ``append`` and read by ``attend``.

    ``keys`` and ``values`` are the pools, [pages][kv_heads][page_size][dim] in
    fp32, bf16 or float8_e4m3fn (one the transpose of another layout will do:
    only the last dimension has to be contiguous, and both need the same
    strides).  Without them the sizes are given, and both start at zero.
    ``key_scale`` and ``value_scale``, fp32 [kv_heads], are what an element of
    an 8-bit pool is multiplied by (default 1).

    Row b of ``table`` (int32 [B][width]) lists the pages of sequence b in
    order (rows may overlap or be one row expanded: sequences may share pages);
    ``lengths`` (int32 [B]) are the sequences' tokens, the new ones included.
    Both lie on the device, so a captured graph follows them.

    ``stream`` (a torch stream or a handle) is where a call runs, the current
    one by default.  Tensors that the caller gives back before it has run there
    need ``record_stream``, as for any work on a second stream.  No gradients
    pass through either call, so neither takes a tensor that requires them
    while gradients are recorded (``torch.no_grad()`` or ``detach()`` says that
    none are wanted).
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
        _shape(max(keys.shape) < _INT, "a cache's sizes must be under 2^31")
        self._keys, self._values = keys, values
        self._scales = (key_scale, value_scale)
        self.device, self.dtype = keys.device, keys.dtype
        self._index = keys.get_device()  # -1: not on a CUDA device
        self._bytes_of = torch.empty(0, dtype=torch.uint8, device=self.device)
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
        self._ref, self._lib = self._c, _library()
        self._scale = 1.0 / math.sqrt(self.dim)
        # what the sizes alone decide is refused here
        self._bytes = {}  # workspace bytes by (B, heads)
        self.attend_workspace(1, self.kv_heads)

    @property
    def keys(self):
        return self._keys

    @property
    def values(self):
        return self._values

    # -- checks --------------------------------------------------------------
    # Each call checks every tensor it hands on; the common case is kept short,
    # since a small call takes less time on the GPU than in here.
    def _on_device(self, t, dtype, name, contiguous=True):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
        if t.get_device() != self._index:
            raise FwpkmError(FWPKM_EINVAL, f"{name} is on {t.device}, the cache on {self.device}")
        if contiguous and not t.is_contiguous():
            raise FwpkmError(FWPKM_ESHAPE, f"{name} must be contiguous")

    def _batch(self, table, lengths):
        if table.dtype is not torch.int32 or table.get_device() != self._index:
            self._on_device(table, torch.int32, "table", contiguous=False)
        if lengths.dtype is not torch.int32 or lengths.get_device() != self._index or \
                not lengths.is_contiguous():
            self._on_device(lengths, torch.int32, "lengths")
        shape = table.shape
        if len(shape) != 2 or lengths.shape != shape[:1] or 0 in shape:
            raise FwpkmError(FWPKM_ESHAPE, "table must be [B][width] and lengths [B], B and width "
                             ">= 1")
        B, width = shape
        if B >= _INT or width >= _INT:
            raise FwpkmError(FWPKM_ESHAPE, "table's sizes must be under 2^31")
        rows, cols = table.stride()
        if cols != 1 and width > 1:
            raise FwpkmError(FWPKM_ESHAPE, "table rows must be contiguous")
        return _Batch(B, width, rows if B > 1 else width, table.data_ptr(), lengths.data_ptr())

    def _rows(self, t, name, dtype, rows, heads=None):
        """The element stride between the rows of t [rows][heads][dim], each contiguous."""
        if t.dtype is not dtype or t.get_device() != self._index:
            self._on_device(t, dtype, name, contiguous=False)
        shape, dim = t.shape, self.dim
        if len(shape) != 3 or shape[0] != rows or shape[2] != dim or \
                (heads is not None and shape[1] != heads):
            raise FwpkmError(FWPKM_ESHAPE, f"{name} must be [{rows}]"
                             f"[{'heads' if heads is None else heads}][{dim}]")
        if rows >= _INT or shape[1] >= _INT:
            raise FwpkmError(FWPKM_ESHAPE, f"{name}'s sizes must be under 2^31")
        step, head, one = t.stride()
        if one != 1 or (head != dim and shape[1] > 1):
            raise FwpkmError(FWPKM_ESHAPE, f"the rows of {name} must be contiguous")
        return step if rows > 1 else shape[1] * dim

    def _errors(self, errors):
        self._on_device(errors, torch.int32, "errors")
        _shape(errors.numel() >= 1, "errors must hold a word")
        return errors.data_ptr()

    def _elsewhere(self):
        return self._index >= 0 and _current_device() != self._index

    def _current_stream(self):
        if self._index < 0:
            raise FwpkmError(FWPKM_EINVAL, f"the cache is on {self.device}, not on a CUDA device")
        return _raw_stream(self._index)

    @contextlib.contextmanager
    def _other(self, stream):
        """The cache's device, and `stream` where one is given, made current."""
        with torch.cuda.device(self.device):
            if stream is None:
                yield
            else:
                if not isinstance(stream, torch.cuda.Stream):
                    stream = torch.cuda.ExternalStream(stream or 0, device=self.device)
                elif stream.device != self.device:
                    raise FwpkmError(FWPKM_EINVAL, f"a stream of {stream.device}, a cache on "
                                     f"{self.device}")
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
        which may be ``q``), or None without ``q``.  Rows of no token (behind
        the last sequence's, or of an empty one) are not written there."""
        if stream is not None or self._elsewhere():
            with self._other(stream):
                return self._append(k, v, table, lengths, starts, q, freqs, style, q_out, errors)
        return self._append(k, v, table, lengths, starts, q, freqs, style, q_out, errors)

    def _append(self, k, v, table, lengths, starts, q, freqs, style, q_out, errors):
        batch = self._batch(table, lengths)
        dtype = k.dtype
        if dtype not in _INPUTS:
            raise TypeError(f"unsupported dtype {dtype}")
        if style not in ROTATE:
            raise FwpkmError(FWPKM_EINVAL, f"style must be one of {sorted(ROTATE)}")
        if torch.is_grad_enabled() and (
                k.requires_grad or v.requires_grad or (q is not None and q.requires_grad) or
                (freqs is not None and freqs.requires_grad)):
            _refuse_gradients()
        rows = k.shape[0] if k.dim() else 0
        k_stride = self._rows(k, "k", dtype, rows, self.kv_heads)
        v_stride = self._rows(v, "v", dtype, rows, self.kv_heads)
        heads = q_stride = out_stride = rotary = 0
        q_at = out_at = starts_at = freqs_at = None
        if q is not None:
            q_stride = self._rows(q, "q", dtype, rows)
            heads = q.shape[1]
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
                out_stride = heads * self.dim
            else:
                out_stride = self._rows(q_out, "q_out", dtype, rows, heads)
            q_at, out_at = q.data_ptr(), q_out.data_ptr()
        elif q_out is not None:
            raise FwpkmError(FWPKM_EINVAL, "q_out without q")
        if freqs is not None:
            self._on_device(freqs, torch.float32, "freqs")
            rotary = 2 * freqs.numel()
            freqs_at = freqs.data_ptr() if rotary else None
        if starts is not None:
            self._on_device(starts, torch.int32, "starts")
            _shape(starts.shape == (batch.B + 1,), "starts must be [B+1]")
            starts_at = starts.data_ptr()
        if errors is not None:
            errors = self._errors(errors)
        rc = self._lib.fwpkm_cache_append(
            self._ref, batch, rows, _INPUTS[dtype], k.data_ptr(), k_stride, v.data_ptr(), v_stride,
            q_at, q_stride, out_at, out_stride, heads, starts_at, rotary, ROTATE[style], freqs_at,
            errors, self._current_stream())
        if rc:
            _check(rc)
        return q_out

    def attend(self, q, table, lengths, scale: Optional[float] = None, window: int = 0, out=None,
               lse=None, errors=None, stream=None, workspace=None):
        """Attention of one token of each sequence, q [B][heads][dim], over its
        cached tokens (the last ``window`` of them, or all): returns ``out``
        [B][heads][dim]; ``lse`` (fp32 [B][heads], optional) receives the log
        of the softmax's denominator.  ``scale`` defaults to 1/sqrt(dim).
        ``workspace`` (uint8, ``attend_workspace`` bytes) is this call's alone
        until it has run; without one it is allocated per call."""
        if stream is not None or self._elsewhere():
            with self._other(stream):
                return self._attend(q, table, lengths, scale, window, out, lse, errors, workspace)
        return self._attend(q, table, lengths, scale, window, out, lse, errors, workspace)

    def _attend(self, q, table, lengths, scale, window, out, lse, errors, workspace):
        batch = self._batch(table, lengths)
        if not 0 <= window < _INT:
            raise FwpkmError(FWPKM_EINVAL, f"window={window} must be 0 .. 2^31 - 1")
        dtype, B = q.dtype, batch.B
        if dtype not in _INPUTS:
            raise TypeError(f"unsupported dtype {dtype}")
        if q.requires_grad and torch.is_grad_enabled():
            _refuse_gradients()
        q_stride = self._rows(q, "q", dtype, B)
        heads = q.shape[1]
        need = self.attend_workspace(B, heads)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            self._on_device(out, dtype, "out")
            _shape(out.shape == q.shape, "out must be [B][heads][dim]")
        lse_at = None
        if lse is not None:
            self._on_device(lse, torch.float32, "lse")
            _shape(lse.shape == (B, heads), "lse must be [B][heads]")
            lse_at = lse.data_ptr()
        if workspace is None:
            workspace, size = self._bytes_of.new_empty(need), need
        else:
            self._on_device(workspace, torch.uint8, "workspace")
            size = workspace.numel()
        if errors is not None:
            errors = self._errors(errors)
        rc = self._lib.fwpkm_cache_attend(
            self._ref, batch, heads, _INPUTS[dtype], q.data_ptr(), q_stride,
            self._scale if scale is None else scale, window, out.data_ptr(), lse_at,
            workspace.data_ptr(), size, errors, self._current_stream())
        if rc:
            _check(rc)
        return out

    def attend_workspace(self, B: int, heads: int) -> int:
        """Bytes of device memory that one running ``attend`` of these sizes needs."""
        need = self._bytes.get((B, heads))
        if need is None:
            need = _check(self._lib.fwpkm_cache_attend_workspace(self._ref, B, heads))
            self._bytes[B, heads] = need
        return need
