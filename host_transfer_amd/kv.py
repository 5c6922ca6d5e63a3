"""ctypes binding of the paged K/V calls of libibp.so (include/ibp_kv.h).

As `ibp`, argument marshalling only: the functions forward to the C entry
points of the same names (ibp_kv_append, ...), all work runs in the library's
HIP kernels, `stream` defaults to torch's current HIP stream and a non-zero
status raises IbpError.  A cache, a batch and rows of tokens are given as torch
tensors, whose sizes and strides are then taken (and whose dtype and device
are checked: ValueError), or with explicit pointers and sizes through
`Cache.from_pointers`, `Batch.from_pointers` and `Rows`.
"""
from __future__ import annotations

import ctypes

import torch

from . import ibp
from .ibp import IbpError  # noqa: F401  (what the functions raise)

F16, BF16 = 0, 1
MAX_HEAD_DIM = 256
MAX_SELECT = 4096
CAUSAL = 1
ROPE_INTERLEAVED = 1

_DTYPES = {torch.float16: F16, torch.bfloat16: BF16}

_vp = ctypes.c_void_p
_u32 = ctypes.c_uint32
_u64 = ctypes.c_uint64


class _CCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("n_pages", _u64), ("page_stride", _u64),
                ("token_stride", _u64), ("head_stride", _u64), ("page_tokens", _u32),
                ("n_heads", _u32), ("head_dim", _u32), ("dtype", _u32)]


class _CRows(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _u64), ("head_stride", _u64), ("n_heads", _u32)]


class _CBatch(ctypes.Structure):
    _fields_ = [("q_start", _vp), ("kv_len", _vp), ("page_table", _vp), ("table_stride", _u64),
                ("n_rows", _u64), ("n_seqs", _u32), ("max_q", _u32), ("max_kv", _u32)]


_f = ctypes.c_float
_u = ctypes.c_uint
_pc, _pr, _pb = (ctypes.POINTER(x) for x in (_CCache, _CRows, _CBatch))
_pu64 = ctypes.POINTER(_u64)

# name -> argument types (all return int status)
_SIGS = {
    "ibp_kv_append": [_pc, _pr, _pr, _pr, _pr, _vp, _vp, _u64, _vp, _u64, _u32, _vp, _vp, _f, _u,
                      _vp],
    "ibp_kv_page_bounds": [_pc, _pb, _vp, _vp],
    "ibp_kv_attend": [_pc, _pb, _pr, _pr, _f, _u32, _u, _vp, _vp, _u64, _vp],
    "ibp_kv_attend_workspace": [_pc, _pb, _u32, _pu64],
    "ibp_kv_select": [_pc, _pb, _vp, _u64, _pr, _u32, _u32, _u32, _vp, _vp, _u64, _vp],
    "ibp_kv_select_workspace": [_pc, _pb, _u32, _pu64],
    "ibp_kv_attend_selected": [_pc, _pb, _pr, _pr, _vp, _u32, _f, _vp, _vp, _u64, _vp],
    "ibp_kv_attend_selected_workspace": [_pc, _pb, _u32, _u32, _pu64],
}
for _name, _args in _SIGS.items():
    _fn = getattr(ibp._lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int

EXPORTED = tuple(_SIGS)


# the current stream's handle without building a torch Stream around it (some microseconds)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _device():
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


def _stream(s, dev):
    if s is None and _raw_stream is not None and dev >= 0:
        return _raw_stream(dev)
    return ibp._stream(s)


def _on_device(name, t, dtype, dev):
    """Checks that t is of this dtype and on the current device `dev`."""
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} needed, got {t.dtype}")
    d = t.get_device()
    if d != dev:
        raise ValueError(f"{name}: a GPU tensor is needed" if d < 0 else
                         f"{name}: on device {d}, not on the current one")


def _current(cache, batch=None):
    """The current device; the tensors of the cache and of the batch must be on it."""
    dev = _device()
    for name, x in (("cache", cache), ("batch", batch)):
        if x is not None and x.device is not None and x.device != dev:
            raise ValueError(f"{name}: on device {x.device}, not on the current one")
    return dev


def _strides(t):
    """Strides, those of axes of size 1 as if packed (they address nothing)."""
    if 1 not in t.shape:
        return t.stride()
    out, inner = [], 1
    for n, s in zip(reversed(t.shape), reversed(t.stride())):
        out.append(s if n > 1 else inner)
        inner = max(inner, out[-1] * n)
    return tuple(reversed(out))


def _plain(name, t, dtype, numel, dev):
    """Pointer of a contiguous device array with at least numel elements; other
    pointers as they are."""
    if not isinstance(t, torch.Tensor):
        return ibp._ptr(t)
    _on_device(name, t, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is needed")
    if t.numel() < numel:
        raise ValueError(f"{name}: {numel} elements needed, got {t.numel()}")
    return t.data_ptr()


class Cache:
    """A paged cache of one layer: k and v of (n_pages, page_tokens, n_heads, head_dim),
    float16 or bfloat16, the same strides, channels contiguous."""

    def __init__(self, k, v):
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must both be (n_pages, page_tokens, n_heads, head_dim)")
        if k.dtype not in _DTYPES:
            raise ValueError(f"k: float16 or bfloat16 needed, got {k.dtype}")
        dev = _device()
        _on_device("k", k, k.dtype, dev)
        _on_device("v", v, k.dtype, dev)
        s = _strides(k)
        if s != _strides(v):
            raise ValueError("k and v must have the same strides")
        if s[3] != 1:
            raise ValueError("the channels of k and v must be contiguous")
        n_pages, page_tokens, n_heads, head_dim = k.shape
        self._set(k.data_ptr(), v.data_ptr(), n_pages, page_tokens, n_heads, head_dim,
                  _DTYPES[k.dtype], *s[:3])
        self.k, self.v, self.torch_dtype, self.device = k, v, k.dtype, dev

    @classmethod
    def from_pointers(cls, k, v, n_pages, page_tokens, n_heads, head_dim, dtype, page_stride=None,
                      token_stride=None, head_stride=None):
        """k, v: addresses; strides in elements, packed where they are not given."""
        self = cls.__new__(cls)
        head_stride = head_dim if head_stride is None else head_stride
        token_stride = n_heads * head_stride if token_stride is None else token_stride
        page_stride = page_tokens * token_stride if page_stride is None else page_stride
        self._set(ibp._ptr(k), ibp._ptr(v), n_pages, page_tokens, n_heads, head_dim, dtype,
                  page_stride, token_stride, head_stride)
        self.k, self.v, self.device = k, v, None
        self.torch_dtype = next((t for t, x in _DTYPES.items() if x == dtype), None)
        return self

    def _set(self, k, v, n_pages, page_tokens, n_heads, head_dim, dtype, *strides):
        self.n_pages, self.page_tokens, self.n_heads, self.head_dim = (n_pages, page_tokens, n_heads,
                                                                       head_dim)
        self.dtype = dtype
        self._c = _CCache(k, v, n_pages, *strides, page_tokens, n_heads, head_dim, dtype)


class Rows:
    """Rows of tokens given by address: token t, head h at data + t*token_stride + h*head_stride
    (elements)."""

    def __init__(self, data, token_stride, head_stride, n_heads):
        self.n_heads = n_heads
        self._keep = data
        self._c = _CRows(ibp._ptr(data), token_stride, head_stride, n_heads)


class Batch:
    """Sequences of a call: q_start (n_seqs + 1,), kv_len (n_seqs,), page_table (n_seqs, pages),
    int32; max_q and max_kv as in include/ibp_kv.h."""

    def __init__(self, q_start, kv_len, page_table, max_q, max_kv):
        n = kv_len.numel()
        self.device = _device()
        for name, t in (("q_start", q_start), ("kv_len", kv_len), ("page_table", page_table)):
            _on_device(name, t, torch.int32, self.device)
        if q_start.dim() != 1 or kv_len.dim() != 1 or q_start.numel() != n + 1 or \
                not q_start.is_contiguous() or not kv_len.is_contiguous():
            raise ValueError("q_start must be (n_seqs + 1,), kv_len (n_seqs,), both contiguous")
        if page_table.dim() != 2 or page_table.shape[0] != n or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be (n_seqs, pages) with contiguous rows")
        self.pages = page_table.shape[1]
        self._set(q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(),
                  _strides(page_table)[0], n, max_q, max_kv)
        self._keep = (q_start, kv_len, page_table)

    @classmethod
    def from_pointers(cls, q_start, kv_len, page_table, table_stride, n_seqs, max_q, max_kv):
        self = cls.__new__(cls)
        self.pages = self.device = None
        self._keep = (q_start, kv_len, page_table)
        self._set(ibp._ptr(q_start), ibp._ptr(kv_len), ibp._ptr(page_table), table_stride, n_seqs,
                  max_q, max_kv)
        return self

    def _set(self, q_start, kv_len, table, table_stride, n_seqs, max_q, max_kv):
        if min(max_q, max_kv, n_seqs) < 0 or max(max_q, max_kv, n_seqs) >= 1 << 31:
            raise ValueError("max_q, max_kv and n_seqs must be in [0, 2^31)")
        self.n_seqs, self.max_q, self.max_kv = n_seqs, max_q, max_kv
        self._args = (q_start, kv_len, table, table_stride)

    def _c(self, cache, n_rows):
        if self.pages is not None and self.pages * cache.page_tokens < self.max_kv:
            raise ValueError(f"page_table: {self.pages} pages of {cache.page_tokens} tokens do not "
                             f"cover max_kv = {self.max_kv}")
        return _CBatch(*self._args, n_rows, self.n_seqs, self.max_q, self.max_kv)


def _rows(name, cache, t, n_tokens, dev):
    """(struct, tokens) of a (tokens, heads, head_dim) tensor or a Rows."""
    if isinstance(t, Rows):
        if n_tokens is None:
            raise ValueError(f"{name}: the number of tokens is needed with Rows")
        return t._c, n_tokens
    shape = t.shape
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError(f"{name}: (tokens, heads, {cache.head_dim}) needed, got {tuple(shape)}")
    _on_device(name, t, cache.torch_dtype, dev)
    n = shape[0]
    if n_tokens is not None and n != n_tokens:
        raise ValueError(f"{name}: {n_tokens} tokens needed, got {n}")
    s0, s1, s2 = t.stride()
    heads, head_dim = shape[1], shape[2]
    if s2 != 1 and head_dim > 1:
        raise ValueError(f"{name}: channels must be contiguous")
    if heads == 1:  # the stride of an axis of size 1 addresses nothing
        s1 = head_dim
    if n == 1:
        s0 = heads * s1
    return _CRows(t.data_ptr(), s0, s1, heads), n


def _of_dtype(name, cache, t, numel, dev):
    return _plain(name, t, cache.torch_dtype, numel, dev)


def _workspace(ws, dev):
    if ws is None:
        return None, 0
    _on_device("workspace", ws, ws.dtype, dev)
    if not ws.is_contiguous():
        raise ValueError("workspace: a contiguous tensor is needed")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _sel(sel, cache, n, n_select, dev):
    if isinstance(sel, torch.Tensor):
        if sel.dim() != 3 or tuple(sel.shape[:2]) != (n, cache.n_heads):
            raise ValueError(f"sel: ({n}, {cache.n_heads}, n_select) needed, got {tuple(sel.shape)}")
        n_select = sel.shape[2]
    elif n_select is None:
        raise ValueError("n_select is needed with a pointer")
    return _plain("sel", sel, torch.int32, 0, dev), n_select


def append(cache, k, v, slots, q=None, q_out=None, positions=None, rope=None, flags=0, q_norm=None,
           k_norm=None, eps=1e-6, n_tokens=None, n_positions=None, rope_dim=None, stream=None):
    """k, v, q, q_out: (tokens, heads, head_dim) tensors or Rows (n_tokens is then needed); rope:
    float32 (n_positions, rope_dim), cosines then sines; slots, positions: int64 (tokens,)."""
    dev = _current(cache)
    kr, n = _rows("k", cache, k, n_tokens, dev)
    vr, _ = _rows("v", cache, v, n, dev)
    qr = None if q is None else _rows("q", cache, q, n, dev)[0]
    qo = None if q_out is None else _rows("q_out", cache, q_out, n, dev)[0]
    if isinstance(rope, torch.Tensor):
        if rope.dim() != 2:
            raise ValueError("rope must be (n_positions, rope_dim)")
        n_positions, rope_dim = rope.shape
    elif ibp._ptr(rope) and (n_positions is None or rope_dim is None):
        raise ValueError("n_positions and rope_dim are needed with a pointer")
    ibp._check(ibp._lib.ibp_kv_append(
        cache._c, kr, vr, qr, qo, _plain("slots", slots, torch.int64, n, dev),
        _plain("positions", positions, torch.int64, n, dev), n,
        _plain("rope", rope, torch.float32, 0, dev), n_positions or 0, rope_dim or 0,
        _of_dtype("q_norm", cache, q_norm, cache.head_dim, dev),
        _of_dtype("k_norm", cache, k_norm, cache.head_dim, dev), eps, flags, _stream(stream, dev)))


def page_bounds(cache, batch, bounds, stream=None):
    """bounds: (n_pages, n_heads, 2, head_dim) of the cache's dtype."""
    dev = _current(cache, batch)
    ibp._check(ibp._lib.ibp_kv_page_bounds(
        cache._c, batch._c(cache, 0),
        _of_dtype("bounds", cache, bounds, cache.n_pages * cache.n_heads * 2 * cache.head_dim, dev),
        _stream(stream, dev)))


def attend_workspace(cache, batch, n_rows, n_q_heads) -> int:
    """Workspace bytes of attend."""
    n = _u64()
    ibp._check(ibp._lib.ibp_kv_attend_workspace(cache._c, batch._c(cache, n_rows), n_q_heads, n))
    return n.value


def attend(cache, batch, q, out, scale, window=0, flags=CAUSAL, lse=None, workspace=None,
           n_rows=None, stream=None):
    """q, out: (rows, heads, head_dim) tensors or Rows (n_rows is then needed); lse: float32
    (rows, heads); workspace: a device tensor of at least attend_workspace() bytes."""
    dev = _current(cache, batch)
    qr, n = _rows("q", cache, q, n_rows, dev)
    orow, _ = _rows("out", cache, out, n, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    ibp._check(ibp._lib.ibp_kv_attend(
        cache._c, batch._c(cache, n), qr, orow, scale, window, flags,
        _plain("lse", lse, torch.float32, n * qr.n_heads, dev), ws, ws_bytes, _stream(stream, dev)))


def select_workspace(cache, batch, n_rows, n_select) -> int:
    """Workspace bytes of select."""
    n = _u64()
    ibp._check(ibp._lib.ibp_kv_select_workspace(cache._c, batch._c(cache, n_rows), n_select, n))
    return n.value


def select(cache, batch, bounds, q, sel, n_first=1, n_last=1, n_select=None, n_bounds=None,
           workspace=None, n_rows=None, stream=None):
    """bounds: (n_bounds, n_heads, 2, head_dim) of the cache's dtype; sel: int32 (rows, n_heads,
    n_select)."""
    dev = _current(cache, batch)
    qr, n = _rows("q", cache, q, n_rows, dev)
    sel_p, n_select = _sel(sel, cache, n, n_select, dev)
    if isinstance(bounds, torch.Tensor):
        if bounds.dim() != 4 or tuple(bounds.shape[1:]) != (cache.n_heads, 2, cache.head_dim):
            raise ValueError(f"bounds: (pages, {cache.n_heads}, 2, {cache.head_dim}) needed, got "
                             f"{tuple(bounds.shape)}")
        n_bounds = bounds.shape[0]
    elif n_bounds is None:
        raise ValueError("n_bounds is needed with a pointer")
    ws, ws_bytes = _workspace(workspace, dev)
    ibp._check(ibp._lib.ibp_kv_select(
        cache._c, batch._c(cache, n), _of_dtype("bounds", cache, bounds, 0, dev), n_bounds, qr, n_first,
        n_last, n_select, sel_p, ws, ws_bytes, _stream(stream, dev)))


def attend_selected_workspace(cache, batch, n_rows, n_q_heads, n_select) -> int:
    """Workspace bytes of attend_selected."""
    n = _u64()
    ibp._check(ibp._lib.ibp_kv_attend_selected_workspace(cache._c, batch._c(cache, n_rows),
                                                         n_q_heads, n_select, n))
    return n.value


def attend_selected(cache, batch, q, sel, out, scale, lse=None, n_select=None, workspace=None,
                    n_rows=None, stream=None):
    """As attend (causal), over the pages that sel lists for each row and key head."""
    dev = _current(cache, batch)
    qr, n = _rows("q", cache, q, n_rows, dev)
    orow, _ = _rows("out", cache, out, n, dev)
    sel_p, n_select = _sel(sel, cache, n, n_select, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    ibp._check(ibp._lib.ibp_kv_attend_selected(
        cache._c, batch._c(cache, n), qr, orow, sel_p, n_select, scale,
        _plain("lse", lse, torch.float32, n * qr.n_heads, dev), ws, ws_bytes, _stream(stream, dev)))
