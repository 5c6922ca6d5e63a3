"""ctypes binding of the pages' assignment of libibp.so (include/ibp_kv_pages.h).

As `kv`: argument marshalling only, on torch tensors (whose sizes, dtype and device are checked:
ValueError) or addresses with explicit sizes; a non-zero status raises IbpError.
"""
from __future__ import annotations

import ctypes

import torch

from . import ibp
from .ibp import IbpError  # noqa: F401  (what the functions raise)
from .kv import _device, _on_device, _plain, _strides, _stream, _workspace

_vp = ctypes.c_void_p
_u32 = ctypes.c_uint32
_u64 = ctypes.c_uint64


class _CPool(ctypes.Structure):
    _fields_ = [("page_table", _vp), ("free_pages", _vp), ("table_stride", _u64), ("n_pages", _u64),
                ("max_pages", _u32), ("page_tokens", _u32)]


class _CStep(ctypes.Structure):
    _fields_ = [("had", _vp), ("keep", _vp), ("add", _vp), ("free_count", _vp), ("n_rows", _u64),
                ("n_seqs", _u32)]


class _CAssigned(ctypes.Structure):
    _fields_ = [("q_start", _vp), ("kv_len", _vp), ("length", _vp), ("free_count", _vp),
                ("unserved", _vp), ("slots", _vp), ("positions", _vp)]


# name -> argument types (all return int status)
_SIGS = {
    "ibp_kv_assign": [ctypes.POINTER(_CPool), ctypes.POINTER(_CStep), ctypes.POINTER(_CAssigned), _vp,
                      _u64, _vp],
    "ibp_kv_assign_workspace": [_u32, _u64, ctypes.POINTER(_u64)],
}
for _name, _args in _SIGS.items():
    _fn = getattr(ibp._lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int

EXPORTED = tuple(_SIGS)


class Pool:
    """The pages of a cache and who holds them: page_table (n_seqs, max_pages) and free_pages
    (n_pages,), int32."""

    def __init__(self, page_table, free_pages, n_pages, page_tokens):
        self.device = _device()
        _on_device("page_table", page_table, torch.int32, self.device)
        if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be (n_seqs, max_pages) with contiguous rows")
        self.n_seqs = page_table.shape[0]
        self._set(page_table.data_ptr(), _plain("free_pages", free_pages, torch.int32, n_pages, self.device),
                  _strides(page_table)[0], n_pages, page_table.shape[1], page_tokens)
        self.page_table, self.free_pages = page_table, free_pages

    @classmethod
    def from_pointers(cls, page_table, free_pages, n_pages, page_tokens, max_pages, table_stride=None):
        self = cls.__new__(cls)
        self.device = self.n_seqs = None
        self.page_table, self.free_pages = page_table, free_pages
        self._set(ibp._ptr(page_table), ibp._ptr(free_pages), max_pages if table_stride is None else table_stride,
                  n_pages, max_pages, page_tokens)
        return self

    def _set(self, table, free, stride, n_pages, max_pages, page_tokens):
        if min(stride, n_pages, max_pages, page_tokens) < 0 or max(max_pages, page_tokens) >= 1 << 32:
            raise ValueError("strides, pages and tokens must not be negative, and fit their types")
        self._c = _CPool(table, free, stride, n_pages, max_pages, page_tokens)


def _sizes(n_seqs, n_rows):
    if min(n_seqs, n_rows) < 0 or n_seqs >= 1 << 32 or n_rows >= 1 << 64:
        raise ValueError("n_seqs and n_rows must not be negative, and fit their types")


def assign_workspace(n_seqs, n_rows) -> int:
    """Workspace bytes of assign."""
    _sizes(n_seqs, n_rows)
    n = _u64()
    ibp._check(ibp._lib.ibp_kv_assign_workspace(n_seqs, n_rows, n))
    return n.value


def assign(pool, had, add, free_count, q_start, kv_len, length, free_count_out, slots, positions=None,
           keep=None, unserved=None, workspace=None, n_seqs=None, n_rows=None, stream=None):
    """had, add, keep, kv_len, length: int32 (n_seqs,); q_start: int32 (n_seqs + 1,); free_count,
    free_count_out, unserved: int32 (1,); slots, positions: int64 (n_rows,).  length may be had, and
    free_count_out free_count.  n_seqs and n_rows are needed where had and slots are addresses."""
    dev = _device()
    if pool.device is not None and pool.device != dev:
        raise ValueError(f"pool: on device {pool.device}, not on the current one")
    if isinstance(had, torch.Tensor):
        n_seqs = had.numel()
    elif n_seqs is None:
        raise ValueError("n_seqs is needed with a pointer")
    if isinstance(slots, torch.Tensor):
        n_rows = slots.numel()
    elif n_rows is None:
        raise ValueError("n_rows is needed with a pointer")
    _sizes(n_seqs, n_rows)
    if pool.n_seqs is not None and pool.n_seqs < n_seqs:
        raise ValueError(f"page_table: {n_seqs} rows needed, got {pool.n_seqs}")
    i32, i64 = torch.int32, torch.int64
    step = _CStep(_plain("had", had, i32, n_seqs, dev), _plain("keep", keep, i32, n_seqs, dev),
                  _plain("add", add, i32, n_seqs, dev), _plain("free_count", free_count, i32, 1, dev), n_rows, n_seqs)
    out = _CAssigned(_plain("q_start", q_start, i32, n_seqs + 1, dev), _plain("kv_len", kv_len, i32, n_seqs, dev),
                     _plain("length", length, i32, n_seqs, dev),
                     _plain("free_count_out", free_count_out, i32, 1, dev),
                     _plain("unserved", unserved, i32, 1, dev), _plain("slots", slots, i64, n_rows, dev),
                     _plain("positions", positions, i64, n_rows, dev))
    ws, ws_bytes = _workspace(workspace, dev)
    ibp._check(ibp._lib.ibp_kv_assign(pool._c, step, out, ws, ws_bytes, _stream(stream, dev)))
