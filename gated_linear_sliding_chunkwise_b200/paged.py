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
import struct

import torch

from . import lizard as lz
from .lizard import _check, _f32, _i32, _lib, _stream, _vp


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


# A serving step makes these calls for every layer and token, and the smallest
# of them run for about 10 us on the GPU.  So the arguments are packed in one
# go (the C layouts above), tensors are looked at in one expression each, and
# what is wrong with one is found out only when something is.
_ATTN = struct.Struct("16if4x13Q")
_PAGES = struct.Struct("9i4x12Q")
_TAIL = struct.Struct("2Q")
assert _ATTN.size == ctypes.sizeof(PagedArgs) and _PAGES.size == ctypes.sizeof(PagesArgs)


def _packed(name):
    """The C function, taking its struct as bytes."""
    fn = _lib[name]
    fn.argtypes = [ctypes.c_char_p, _vp]
    fn.restype = ctypes.c_int
    return fn


def _sizer(name):
    fn = _lib[name]
    fn.argtypes = [ctypes.c_char_p]
    fn.restype = ctypes.c_size_t
    return fn


_attn = _packed("lizard_paged_attn")
_attn_size = _sizer("lizard_paged_attn_workspace_size")
_pages = {name: _packed("lizard_pages_" + name) for name in ("reserve", "free", "fork", "compact")}
_pages_size = _sizer("lizard_pages_workspace_size")
_I32 = torch.int32
_CODES = {torch.bfloat16: lz.BF16, torch.float32: lz.FP32}


def _fits(t, shape, dtype, index):
    """A contiguous tensor of this shape and type on the cache's device."""
    return t.shape == shape and t.dtype is dtype and t.get_device() == index and t.is_contiguous()


def _refuse(index, *wants):
    """Says which of the (name, tensor, shape, dtype) does not fit."""
    for name, t, shape, dtype in wants:
        if t is None or _fits(t, shape, dtype, index):
            continue
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{name}: {dtype} of shape {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, the cache on another device")
        raise ValueError(f"{name} must be contiguous")
    raise ValueError("arguments do not fit together")


def _code(dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"activations must be bf16 or fp32, got {dtype}")
    return code


def _space(nbytes, device, workspace, stream):
    """The caller's workspace, or one from torch's allocator for this call,
    and the last two fields of the C structs (its address and bytes)."""
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        if stream is not None:     # not handed out again before that stream has done with it
            workspace.record_stream(stream if isinstance(stream, torch.cuda.Stream)
                                    else torch.cuda.ExternalStream(int(stream), device=device))
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace, _TAIL.pack(workspace.data_ptr(), workspace.numel() * workspace.element_size())


def _call(fn, where, args, index, stream):
    """The C call on the cache's device (its current stream unless one is given)."""
    if stream is None:
        if index != torch.cuda.current_device():
            with torch.cuda.device(index):
                return _check(fn(args, torch._C._cuda_getCurrentRawStream(index)), where)
        code = fn(args, torch._C._cuda_getCurrentRawStream(index))
    else:
        code = fn(args, _stream(stream))
    if code:
        _check(code, where)


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
    pool, dtype, index = k_pages.shape, k_pages.dtype, k_pages.get_device()
    code = _code(dtype)
    if len(pool) != 5 or q.dim() != 3 or table.dim() != 2 or cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("k_pages, v_pages: [layers, num_pages, Hkv, page, d]; q: [T, H, d]; table: [rows, max_pages]; "
                         "cu_q: [B + 1]")
    layers, num_pages, Hkv, page, d = pool
    T, H, _ = q.shape
    rows, max_pages = table.shape
    B = cu_q.shape[0] - 1
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    if row is None and B > rows:
        raise ValueError(f"{B} sequences, but the table has {rows} rows")
    new, like = (T, Hkv, d), (T, H, d)
    if not (_fits(q, like, dtype, index) and (k is None or (_fits(k, new, dtype, index) and _fits(v, new, dtype, index)))
            and k_pages.is_contiguous() and _fits(v_pages, pool, dtype, index)
            and _fits(table, (rows, max_pages), _I32, index) and _fits(lens, (rows,), _I32, index)
            and _fits(cu_q, (B + 1,), _I32, index) and (row is None or _fits(row, (B,), _I32, index))
            and (out is None or _fits(out, like, dtype, index))):
        _refuse(index, ("q", q, like, dtype), ("k", k, new, dtype), ("v", v, new, dtype), ("k_pages", k_pages, pool, dtype),
                ("v_pages", v_pages, pool, dtype), ("table", table, (rows, max_pages), _I32), ("lens", lens, (rows,), _I32),
                ("cu_q", cu_q, (B + 1,), _I32), ("row", row, (B,), _I32), ("out", out, like, dtype))
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    o = torch.empty_like(q) if out is None else out
    lse = q.new_empty((T, H), dtype=torch.float32) if want_lse else None
    args = _ATTN.pack(layers, num_pages, Hkv, page, d, rows, max_pages, B, T, H, layer, max_q, window, sinks, code, impl,
                      softmax_scale, q.data_ptr(), 0 if k is None else k.data_ptr(), 0 if v is None else v.data_ptr(),
                      k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(), cu_q.data_ptr(),
                      0 if row is None else row.data_ptr(), o.data_ptr(), 0 if lse is None else lse.data_ptr(), 0, 0)
    ws, tail = _space(_attn_size(args), q.device, workspace, stream)
    _call(_attn, "lizard_paged_attn", args[:-16] + tail, index, stream)
    return {"o": o, "lse": lse, "workspace": ws}


def _bookkeep(name, refs, table, lens, row, src, grow, page, pool, table_out, refs_out, workspace, stream):
    """One of the four calls; pool: (k_pages, v_pages) or None."""
    index = refs.get_device()
    if refs.dim() != 1 or table.dim() != 2 or (row is not None and row.dim() != 1):
        raise ValueError("refs: [num_pages]; table: [rows, max_pages]; row: [n]")
    num_pages, (rows, max_pages) = refs.shape[0], table.shape
    n = 0 if row is None else row.shape[0]
    layers = Hkv = d = code = kp = vp = 0
    if pool is not None:
        k_pages, v_pages = pool
        shape, dtype = k_pages.shape, k_pages.dtype
        code = _code(dtype)
        if len(shape) != 5 or shape[1] != num_pages:
            raise ValueError(f"k_pages: [layers, {num_pages}, Hkv, page, d] expected, got {tuple(shape)}")
        if not (_fits(k_pages, shape, dtype, index) and _fits(v_pages, shape, dtype, index)):
            _refuse(index, ("k_pages", k_pages, shape, dtype), ("v_pages", v_pages, shape, dtype))
        layers, _, Hkv, page, d = shape
        kp, vp = k_pages.data_ptr(), v_pages.data_ptr()
    if not (_fits(refs, (num_pages,), _I32, index) and _fits(table, (rows, max_pages), _I32, index)
            and (lens is None or _fits(lens, (rows,), _I32, index)) and (row is None or _fits(row, (n,), _I32, index))
            and (src is None or _fits(src, (n,), _I32, index)) and (grow is None or _fits(grow, (n,), _I32, index))
            and (table_out is None or _fits(table_out, (rows, max_pages), _I32, index))
            and (refs_out is None or _fits(refs_out, (num_pages,), _I32, index))):
        _refuse(index, ("refs", refs, (num_pages,), _I32), ("table", table, (rows, max_pages), _I32),
                ("lens", lens, (rows,), _I32), ("row", row, (n,), _I32), ("src", src, (n,), _I32),
                ("grow", grow, (n,), _I32), ("table_out", table_out, (rows, max_pages), _I32),
                ("refs_out", refs_out, (num_pages,), _I32))
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    args = _PAGES.pack(layers, num_pages, Hkv, page, d, rows, max_pages, code, n, kp, vp, refs.data_ptr(),
                       table.data_ptr(), 0 if lens is None else lens.data_ptr(), 0 if row is None else row.data_ptr(),
                       0 if src is None else src.data_ptr(), 0 if grow is None else grow.data_ptr(),
                       0 if table_out is None else table_out.data_ptr(),
                       0 if refs_out is None else refs_out.data_ptr(), 0, 0)
    ws, tail = _space(_pages_size(args), refs.device, workspace, stream)
    _call(_pages[name], "lizard_pages_" + name, args[:-16] + tail, index, stream)
    return ws


def reserve(refs, table, lens, row, grow, *, page, workspace=None, stream=None):
    """Row row[i] grows by grow[i] tokens (lizard_pages_reserve); refs, table
    and lens are updated in place.  Returns the workspace."""
    return _bookkeep("reserve", refs, table, lens, row, None, grow, page, None, None, None, workspace, stream)


def free(refs, table, lens, row, *, page, workspace=None, stream=None):
    """The listed rows give up their tokens (lizard_pages_free), in place.
    Returns the workspace."""
    return _bookkeep("free", refs, table, lens, row, None, None, page, None, None, None, workspace, stream)


def fork(k_pages, v_pages, refs, table, lens, src, row, *, workspace=None, stream=None):
    """Row row[i] continues from row src[i] (lizard_pages_fork): whole pages
    shared, a part-filled last page copied; in place.  Returns the workspace."""
    return _bookkeep("fork", refs, table, lens, row, src, None, 0, (k_pages, v_pages), None, None, workspace, stream)


def compact(k_pages, v_pages, refs, table, *, table_out=None, refs_out=None, workspace=None, stream=None):
    """The live pages move to the lowest numbers (lizard_pages_compact).
    Returns (table, refs) with the new numbers: table_out and refs_out, which
    may be table and refs themselves, or new tensors."""
    table_out = torch.empty_like(table) if table_out is None else table_out
    refs_out = torch.empty_like(refs) if refs_out is None else refs_out
    _bookkeep("compact", refs, table, None, None, None, None, 0, (k_pages, v_pages), table_out, refs_out, workspace,
              stream)
    return table_out, refs_out
