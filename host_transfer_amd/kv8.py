"""ctypes binding of the 8-bit paged K/V cache of libibp.so (include/ibp_kv8.h).

As `kv`, whose Batch and Rows it takes: argument marshalling only, on torch tensors (whose sizes,
strides, dtype and device are checked: ValueError) or addresses with explicit sizes; a non-zero
status raises IbpError.
"""
from __future__ import annotations

import ctypes

import torch

from . import ibp
from .ibp import IbpError  # noqa: F401  (what the functions raise)
from .kv import (BF16, CAUSAL, F16, ROPE_INTERLEAVED, _DTYPES, Batch, Rows, _CBatch,  # noqa: F401
                 _CRows, _current, _device, _of_dtype, _on_device, _plain, _rows, _stream, _strides, _workspace)

_vp = ctypes.c_void_p
_u32 = ctypes.c_uint32
_u64 = ctypes.c_uint64


class _CCache8(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_exp", _vp), ("v_exp", _vp), ("n_pages", _u64),
                ("page_stride", _u64), ("token_stride", _u64), ("head_stride", _u64), ("page_tokens", _u32),
                ("block_tokens", _u32), ("n_heads", _u32), ("head_dim", _u32)]


_f = ctypes.c_float
_u = ctypes.c_uint
_pc, _pr, _pb = (ctypes.POINTER(x) for x in (_CCache8, _CRows, _CBatch))

# name -> argument types (all return int status)
_SIGS = {
    "ibp_kv8_append": [_pc, _pb, _u32, _pr, _pr, _pr, _pr, _vp, _vp, _u64, _u32, _vp, _vp, _f, _u, _vp],
    "ibp_kv8_attend": [_pc, _pb, _u32, _pr, _pr, _f, _u32, _u, _vp, _vp, _u64, _vp],
    "ibp_kv8_attend_workspace": [_pc, _pb, _u32, ctypes.POINTER(_u64)],
}
for _name, _args in _SIGS.items():
    _fn = getattr(ibp._lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int

EXPORTED = tuple(_SIGS)


class Cache:
    """A paged cache of one layer in 8 bits: k and v of (n_pages, page_tokens, n_heads, head_dim),
    float8_e4m3fn, the same strides, channels contiguous; k_exp and v_exp of (n_pages, blocks, n_heads),
    uint8, contiguous, blocks a divisor of page_tokens."""

    def __init__(self, k, v, k_exp, v_exp):
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must both be (n_pages, page_tokens, n_heads, head_dim)")
        dev = _device()
        _on_device("k", k, torch.float8_e4m3fn, dev)
        _on_device("v", v, torch.float8_e4m3fn, dev)
        s = _strides(k)
        if s != _strides(v):
            raise ValueError("k and v must have the same strides")
        if s[3] != 1:
            raise ValueError("the channels of k and v must be contiguous")
        n_pages, page_tokens, n_heads, head_dim = k.shape
        for name, e in (("k_exp", k_exp), ("v_exp", v_exp)):
            _on_device(name, e, torch.uint8, dev)
            if e.dim() != 3 or e.shape != k_exp.shape or e.shape[0] != n_pages or e.shape[2] != n_heads or \
                    not e.is_contiguous() or not e.shape[1] or page_tokens % e.shape[1]:
                raise ValueError(f"{name}: ({n_pages}, a divisor of {page_tokens}, {n_heads}) and contiguous "
                                 f"needed, got {tuple(e.shape)}")
        self._set(k.data_ptr(), v.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), n_pages, page_tokens,
                  page_tokens // k_exp.shape[1], n_heads, head_dim, *s[:3])
        self.k, self.v, self.k_exp, self.v_exp, self.device = k, v, k_exp, v_exp, dev

    @classmethod
    def from_pointers(cls, k, v, k_exp, v_exp, n_pages, page_tokens, block_tokens, n_heads, head_dim,
                      page_stride=None, token_stride=None, head_stride=None):
        """k, v, k_exp, v_exp: addresses; strides in bytes, packed where they are not given."""
        self = cls.__new__(cls)
        head_stride = head_dim if head_stride is None else head_stride
        token_stride = n_heads * head_stride if token_stride is None else token_stride
        page_stride = page_tokens * token_stride if page_stride is None else page_stride
        self._set(*(ibp._ptr(x) for x in (k, v, k_exp, v_exp)), n_pages, page_tokens, block_tokens, n_heads,
                  head_dim, page_stride, token_stride, head_stride)
        self.k, self.v, self.k_exp, self.v_exp, self.device = k, v, k_exp, v_exp, None
        return self

    def _set(self, k, v, k_exp, v_exp, n_pages, page_tokens, block_tokens, n_heads, head_dim, *strides):
        self.n_pages, self.page_tokens, self.block_tokens = n_pages, page_tokens, block_tokens
        self.n_heads, self.head_dim = n_heads, head_dim
        self._c = _CCache8(k, v, k_exp, v_exp, n_pages, *strides, page_tokens, block_tokens, n_heads, head_dim)


class _Of:
    """A cache with the dtype of a call's rows: what the checks of rows ask."""

    def __init__(self, cache, dtype):
        self.n_heads, self.head_dim, self.torch_dtype = cache.n_heads, cache.head_dim, dtype


def _dtype(name, t, dtype):
    """(the C value, the torch dtype) of a call's rows: of tensor t, or given with Rows."""
    if isinstance(t, Rows):
        if dtype is None:
            raise ValueError(f"{name}: the dtype is needed with Rows")
    elif dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} needed, got {t.dtype}")
    else:
        dtype = t.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"{name}: float16 or bfloat16 needed, got {dtype}")
    return _DTYPES[dtype], dtype


def append(cache, batch, k, v, q=None, q_out=None, positions=None, rope=None, flags=0, q_norm=None,
           k_norm=None, eps=1e-6, n_rows=None, n_positions=None, rope_dim=None, dtype=None, stream=None):
    """k, v, q, q_out: (rows, heads, head_dim) tensors or Rows (n_rows and dtype, float16 or bfloat16, are
    then needed); rope: float32 (n_positions, rope_dim), cosines then sines; positions: int64 (rows,)."""
    dev = _current(cache, batch)
    c_dtype, dtype = _dtype("k", k, dtype)
    of = _Of(cache, dtype)
    kr, n = _rows("k", of, k, n_rows, dev)
    vr, _ = _rows("v", of, v, n, dev)
    qr = None if q is None else _rows("q", of, q, n, dev)[0]
    qo = None if q_out is None else _rows("q_out", of, q_out, n, dev)[0]
    if isinstance(rope, torch.Tensor):
        if rope.dim() != 2:
            raise ValueError("rope must be (n_positions, rope_dim)")
        n_positions, rope_dim = rope.shape
    elif ibp._ptr(rope) and (n_positions is None or rope_dim is None):
        raise ValueError("n_positions and rope_dim are needed with a pointer")
    ibp._check(ibp._lib.ibp_kv8_append(
        cache._c, batch._c(cache, n), c_dtype, kr, vr, qr, qo, _plain("positions", positions, torch.int64, n, dev),
        _plain("rope", rope, torch.float32, 0, dev), n_positions or 0, rope_dim or 0,
        _of_dtype("q_norm", of, q_norm, cache.head_dim, dev),
        _of_dtype("k_norm", of, k_norm, cache.head_dim, dev), eps, flags, _stream(stream, dev)))


def attend_workspace(cache, batch, n_rows, n_q_heads) -> int:
    """Workspace bytes of attend."""
    n = _u64()
    ibp._check(ibp._lib.ibp_kv8_attend_workspace(cache._c, batch._c(cache, n_rows), n_q_heads, n))
    return n.value


def attend(cache, batch, q, out, scale, window=0, flags=CAUSAL, lse=None, workspace=None, n_rows=None,
           dtype=None, stream=None):
    """q, out: (rows, heads, head_dim) tensors or Rows (n_rows and dtype are then needed); lse: float32
    (rows, heads); workspace: a device tensor of at least attend_workspace() bytes."""
    dev = _current(cache, batch)
    c_dtype, dtype = _dtype("q", q, dtype)
    of = _Of(cache, dtype)
    qr, n = _rows("q", of, q, n_rows, dev)
    orow, _ = _rows("out", of, out, n, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    ibp._check(ibp._lib.ibp_kv8_attend(
        cache._c, batch._c(cache, n), c_dtype, qr, orow, scale, window, flags,
        _plain("lse", lse, torch.float32, n * qr.n_heads, dev), ws, ws_bytes, _stream(stream, dev)))
