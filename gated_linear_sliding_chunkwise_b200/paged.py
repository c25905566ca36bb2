"""Paged key/value cache (lizard_paged_attn, lizard_pages_*; see include/lizard.h).

Argument marshalling only, like :mod:`.lizard`.  The cache is the caller's
tensors: k_pages, v_pages [layers, num_pages, Hkv, page, d], refs [num_pages],
table [rows, max_pages] and lens [rows] (int32).  A serving loop calls
``reserve`` for the tokens to come, ``attn`` once per layer, ``fork`` and
``free`` as sequences branch and end, ``compact`` when the pool is to shrink.

Every call returns (or, for ``attn``, includes) its workspace;
``lizard.workspace_status(workspace)`` reads the call's device status.
"""

from __future__ import annotations

import ctypes

import torch

from . import lizard as lz
from .lizard import _check, _dtype_code, _i32, _lib, _ptr, _stream, _vp, _workspace, _f32


class PagedArgs(ctypes.Structure):
    _fields_ = [("layers", _i32), ("num_pages", _i32), ("Hkv", _i32), ("page", _i32), ("d", _i32),
                ("rows", _i32), ("max_pages", _i32), ("B", _i32), ("T", _i32), ("H", _i32),
                ("layer", _i32), ("max_q", _i32), ("window", _i32), ("sinks", _i32), ("dtype", _i32),
                ("impl", _i32), ("softmax_scale", _f32), ("q", _vp), ("k", _vp), ("v", _vp),
                ("k_pages", _vp), ("v_pages", _vp), ("table", _vp), ("lens", _vp), ("cu_q", _vp),
                ("row", _vp), ("o", _vp), ("lse", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t)]


class PagesArgs(ctypes.Structure):
    _fields_ = [("layers", _i32), ("num_pages", _i32), ("Hkv", _i32), ("page", _i32), ("d", _i32),
                ("rows", _i32), ("max_pages", _i32), ("dtype", _i32), ("n", _i32),
                ("k_pages", _vp), ("v_pages", _vp), ("refs", _vp), ("table", _vp), ("lens", _vp),
                ("row", _vp), ("src", _vp), ("grow", _vp), ("table_out", _vp), ("refs_out", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


_lib.lizard_paged_attn_workspace_size.argtypes = [ctypes.POINTER(PagedArgs)]
_lib.lizard_paged_attn_workspace_size.restype = ctypes.c_size_t
_lib.lizard_paged_attn.argtypes = [ctypes.POINTER(PagedArgs), _vp]
_lib.lizard_paged_attn.restype = ctypes.c_int
_lib.lizard_pages_workspace_size.argtypes = [ctypes.POINTER(PagesArgs)]
_lib.lizard_pages_workspace_size.restype = ctypes.c_size_t
for _name in ("reserve", "free", "fork", "compact"):
    _fn = getattr(_lib, "lizard_pages_" + _name)
    _fn.argtypes = [ctypes.POINTER(PagesArgs), _vp]
    _fn.restype = ctypes.c_int


def _call(fn, where, a, device, stream):
    """The C call on the cache's device (its current stream unless one is given)."""
    if device.index == torch.cuda.current_device():
        _check(fn(ctypes.byref(a), _stream(stream)), where)
        return
    with torch.cuda.device(device):
        _check(fn(ctypes.byref(a), _stream(stream)), where)


def _int32(name, t, shape, device):
    """Device arrays of indices: int32, contiguous, of this shape, on the cache's device."""
    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: int32 of shape {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    _placed(name, t, device)


def _placed(name, t, device):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")


def _pool(a, k_pages, v_pages):
    """The pool's sizes, checked against each other."""
    if k_pages.dim() != 5 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype:
        raise ValueError("k_pages and v_pages: [layers, num_pages, Hkv, page, d], alike")
    _placed("k_pages", k_pages, k_pages.device)
    _placed("v_pages", v_pages, k_pages.device)
    a.layers, a.num_pages, a.Hkv, a.page, a.d = k_pages.shape
    a.dtype = _dtype_code(k_pages)
    a.k_pages, a.v_pages = k_pages.data_ptr(), v_pages.data_ptr()


def attn(q, k, v, k_pages, v_pages, table, lens, cu_q, *, max_q, row=None, layer=0, window=0, sinks=0,
         softmax_scale=0.0, want_lse=False, impl=lz.IMPL_AUTO, out=None, workspace=None, stream=None):
    """Attention of new tokens over one layer's pages (lizard_paged_attn).

    q [T, H, d]; k, v [T, Hkv, d], written into their pages first, or both
    None when they are there already.  Sequence b's new tokens are rows
    cu_q[b] .. cu_q[b + 1] - 1 and the last ones of the lens[r] tokens of
    table row r = row[b] (b without row); max_q bounds their number.  window
    > 0: a token sees its last `window` tokens and the sequence's first
    `sinks` ones.  Returns a dict with o [T, H, d], lse [T, H] (or None) and
    the workspace."""
    dev = k_pages.device
    a = PagedArgs()
    _pool(a, k_pages, v_pages)
    if q.dim() != 3 or q.shape[2] != a.d:
        raise ValueError(f"q: [T, H, {a.d}] expected, got {tuple(q.shape)}")
    T, H, d = q.shape
    for name, t, shape in (("q", q, (T, H, d)), ("k", k, (T, a.Hkv, d)), ("v", v, (T, a.Hkv, d)),
                           ("out", out, (T, H, d))):
        if t is None:
            continue
        if tuple(t.shape) != shape or t.dtype != k_pages.dtype:
            raise ValueError(f"{name}: {k_pages.dtype} of shape {shape} expected, got {t.dtype} {tuple(t.shape)}")
        _placed(name, t, dev)
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    B = cu_q.shape[0] - 1 if cu_q.dim() == 1 else -1
    if table.dim() != 2:
        raise ValueError("table: [rows, max_pages]")
    a.rows, a.max_pages = table.shape
    _int32("table", table, table.shape, dev)
    _int32("lens", lens, (a.rows,), dev)
    _int32("cu_q", cu_q, (max(B, 0) + 1,), dev)
    if row is not None:
        _int32("row", row, (B,), dev)
    elif B > a.rows:
        raise ValueError(f"{B} sequences, but the table has {a.rows} rows")
    a.B, a.T, a.H, a.layer, a.max_q = B, T, H, layer, max_q
    a.window, a.sinks, a.impl, a.softmax_scale = window, sinks, impl, softmax_scale
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty(T, H, dtype=torch.float32, device=dev) if want_lse else None
    a.q, a.k, a.v, a.o, a.lse = _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse)
    a.table, a.lens, a.cu_q, a.row = table.data_ptr(), lens.data_ptr(), cu_q.data_ptr(), _ptr(row)
    ws = _workspace(int(_lib.lizard_paged_attn_workspace_size(ctypes.byref(a))), dev, workspace)
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _call(_lib.lizard_paged_attn, "lizard_paged_attn", a, dev, stream)
    return {"o": o, "lse": lse, "workspace": ws}


def _pages_call(name, refs, table, *, page, lens=None, row=None, src=None, grow=None, k_pages=None, v_pages=None,
                table_out=None, refs_out=None, workspace=None, stream=None):
    dev = refs.device
    a = PagesArgs()
    if k_pages is not None:
        _pool(a, k_pages, v_pages)
        _placed("k_pages", k_pages, dev)
    a.num_pages, a.page = refs.shape[0], page
    if k_pages is not None and k_pages.shape[1] != refs.shape[0]:
        raise ValueError(f"refs counts {refs.shape[0]} pages, the pool has {k_pages.shape[1]}")
    if table.dim() != 2:
        raise ValueError("table: [rows, max_pages]")
    a.rows, a.max_pages = table.shape
    _int32("refs", refs, (a.num_pages,), dev)
    _int32("table", table, table.shape, dev)
    if lens is not None:
        _int32("lens", lens, (a.rows,), dev)
    a.n = 0 if row is None else row.shape[0]
    for what, t in (("row", row), ("src", src), ("grow", grow)):
        if t is not None:
            _int32(what, t, (a.n,), dev)
    if table_out is not None:
        _int32("table_out", table_out, table.shape, dev)
    if refs_out is not None:
        _int32("refs_out", refs_out, refs.shape, dev)
    a.refs, a.table, a.lens = refs.data_ptr(), table.data_ptr(), _ptr(lens)
    a.row, a.src, a.grow = _ptr(row), _ptr(src), _ptr(grow)
    a.table_out, a.refs_out = _ptr(table_out), _ptr(refs_out)
    ws = _workspace(int(_lib.lizard_pages_workspace_size(ctypes.byref(a))), dev, workspace)
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    where = "lizard_pages_" + name
    _call(getattr(_lib, where), where, a, dev, stream)
    return ws


def reserve(refs, table, lens, row, grow, *, page, workspace=None, stream=None):
    """Row row[i] grows by grow[i] tokens (lizard_pages_reserve); refs, table
    and lens are updated in place.  Returns the workspace."""
    return _pages_call("reserve", refs, table, page=page, lens=lens, row=row, grow=grow, workspace=workspace,
                       stream=stream)


def free(refs, table, lens, row, *, page, workspace=None, stream=None):
    """The listed rows give up their tokens (lizard_pages_free), in place.
    Returns the workspace."""
    return _pages_call("free", refs, table, page=page, lens=lens, row=row, workspace=workspace, stream=stream)


def fork(k_pages, v_pages, refs, table, lens, src, row, *, workspace=None, stream=None):
    """Row row[i] continues from row src[i] (lizard_pages_fork): whole pages
    shared, a part-filled last page copied; in place.  Returns the workspace."""
    return _pages_call("fork", refs, table, page=k_pages.shape[3], lens=lens, row=row, src=src, k_pages=k_pages,
                       v_pages=v_pages, workspace=workspace, stream=stream)


def compact(k_pages, v_pages, refs, table, *, table_out=None, refs_out=None, workspace=None, stream=None):
    """The live pages move to the lowest numbers (lizard_pages_compact).
    Returns (table, refs) with the new numbers: table_out and refs_out, which
    may be table and refs themselves, or new tensors."""
    table_out = torch.empty_like(table) if table_out is None else table_out
    refs_out = torch.empty_like(refs) if refs_out is None else refs_out
    _pages_call("compact", refs, table, page=k_pages.shape[3], k_pages=k_pages, v_pages=v_pages,
                table_out=table_out, refs_out=refs_out, workspace=workspace, stream=stream)
    return table_out, refs_out
