"""Paged key/value cache (lizard_paged_attn, lizard_pages_*; see include/lizard.h).

Argument marshalling only, like :mod:`.lizard`, but in a small extension module
(``_paged_call``, ``csrc/paged_binding.cpp``): the smallest of these calls run
for 10 us on the GPU.  The cache is the caller's tensors: k_pages, v_pages
[layers, num_pages, Hkv, page, d], refs [num_pages], table [rows, max_pages]
and lens [rows] (int32), contiguous and on 16-byte boundaries, as all tensors
here.  A serving loop calls ``reserve`` for the tokens to come, ``attn`` once
per layer, ``fork`` and ``free`` as sequences branch and end, ``compact`` when
the pool is to shrink.

Every call returns its workspace, or a result that includes it (``attn``,
``compact``); ``lizard.workspace_status(workspace)`` reads the call's device status.

A call runs on ``stream`` (a torch stream or a handle), or on the current one.
What it allocates, outputs and workspace, belongs to that stream, as it does
under ``torch.cuda.stream(stream)``: to use it on another stream, order the two
and call ``record_stream``.
"""

from __future__ import annotations

import ctypes
import os

from . import lizard as lz
from .lizard import _check, _f32, _i32, _lib, _vp

if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_paged_call.so")):
    raise ImportError("_paged_call.so is missing: build it with "
                      "`python -m gated_linear_sliding_chunkwise_b200.build`")
from . import _paged_call


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


def _handle(stream):
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


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
    code, o, lse, ws = _paged_call.attn(q, k, v, k_pages, v_pages, table, lens, cu_q, row, out, workspace, max_q,
                                        layer, window, sinks, softmax_scale, want_lse, impl, _handle(stream))
    if code:
        _check(code, "lizard_paged_attn")
    return {"o": o, "lse": lse, "workspace": ws}


_OPS = ("reserve", "free", "fork", "compact")


def _bookkeep(op, *args):
    code, table_out, refs_out, ws = _paged_call.bookkeep(op, *args)
    if code:
        _check(code, "lizard_pages_" + _OPS[op])
    return table_out, refs_out, ws


def reserve(refs, table, lens, row, grow, *, page, workspace=None, stream=None):
    """Row row[i] grows by grow[i] tokens (lizard_pages_reserve); refs, table
    and lens are updated in place.  Returns the workspace."""
    return _bookkeep(0, refs, table, lens, row, None, grow, page, None, None, None, None, workspace, _handle(stream))[2]


def free(refs, table, lens, row, *, page, workspace=None, stream=None):
    """The listed rows give up their tokens (lizard_pages_free), in place.
    Returns the workspace."""
    return _bookkeep(1, refs, table, lens, row, None, None, page, None, None, None, None, workspace, _handle(stream))[2]


def fork(k_pages, v_pages, refs, table, lens, src, row, *, workspace=None, stream=None):
    """Row row[i] continues from row src[i] (lizard_pages_fork): whole pages
    shared, a part-filled last page copied; in place.  Returns the workspace."""
    return _bookkeep(2, refs, table, lens, row, src, None, 0, k_pages, v_pages, None, None, workspace,
                     _handle(stream))[2]


class Compacted(tuple):
    """(table, refs) with the new numbers, and the call's `workspace`."""
    workspace = None


def compact(k_pages, v_pages, refs, table, *, table_out=None, refs_out=None, workspace=None, stream=None):
    """The live pages move to the lowest numbers (lizard_pages_compact).
    Returns (table, refs) with the new numbers: table_out and refs_out, which
    may be table and refs themselves, or new tensors.  The result's attribute
    `workspace` holds the call's status (an entry of the table that is not a
    live page)."""
    table, refs, ws = _bookkeep(3, refs, table, None, None, None, None, 0, k_pages, v_pages, table_out, refs_out,
                                workspace, _handle(stream))
    out = Compacted((table, refs))
    out.workspace = ws
    return out
