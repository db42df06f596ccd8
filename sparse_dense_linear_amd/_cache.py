"""ctypes binding of appending rows to a paged cache (include/cache.h):
argument marshalling only."""
from __future__ import annotations

import ctypes
from struct import Struct

from . import _attn
from ._attn import (_PACK_ROWS, CACHE_AS_IS, _codes, _dtype, _first, _index, _is_tensor, _On, _paging, _rows, _scales,
                    _with)
from ._binding import _check


class _Append(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "S", "T", "Hq", "Hkv", "D", "page", "pages", "page_stride", "row_stride", "head_stride", "table_stride",
        "rotated", "angles")] + [("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_PACK_APPEND = Struct("13q2i")


def _tables(cos, sin, device):
    """Addresses of the tables of the rotation, their rows and twice their columns."""
    if cos is None and sin is None:
        return None, None, 0, 0
    _is_tensor(cos, "cos")
    shape = tuple(cos.shape)
    if len(shape) != 2:
        raise ValueError("cos must have two dimensions: positions, pairs")
    f32 = _attn.torch.float32
    return _index(cos, "cos", device, f32, shape), _index(sin, "sin", device, f32, shape), shape[0], 2 * shape[1]


def append_pages(k, v, k_pages, v_pages, table, ctx, rowptr, q=None, cos=None, sin=None, tree=None,
                 interleaved: bool = False, k_scale=None, v_scale=None, q_out=None, stream=None):
    """New rows go into the pages of a cache behind the context of their
    sequence, k and q rotated by their position on the way (cache_append).

    Sequence s has ctx[s] cached positions, and its new rows are rows rowptr[s]
    .. rowptr[s+1]-1 of k and v [T, Hkv, D]: row t becomes position ctx[s] + t,
    where tree_attention reads it (row p % page of page table[s, p // page] of
    the pools [pages, page, Hkv, D]).  Rows whose table entry is out of range are
    passed over.

    cos and sin [positions, R / 2] float32 rotate the first R elements of each
    head of k, and of q [T, Hq, D] if it is given, by the position where a row
    stands: ctx + t, or with `tree` (masks, as tree_attention takes them) where
    the draft stands.  Pairs are elements i and i + R / 2, or interleaved 2 i and
    2 i + 1; R is a multiple of 8.  Positions past the tables give NaN.

    The pools hold rows of k's type, or, with k_scale and v_scale [pages, page /
    block, Hkv] float32, codes of 8 bits (float8_e4m3fn or int8).  A block's
    scale is the smallest power of two that holds its values; where new rows
    need a larger one than the rows before them, these are rounded to it.  A value
    that is not finite is a code of its own in float8_e4m3fn; in int8 it makes all
    rows of its block and head NaN, those before it too, even if it is a draft's
    that is not kept.

    Returns the rotated q (q_out, which may be q itself; None: allocated, on
    `stream` if given), or None without q.  Records no autograd graph."""
    device = _first(k, "k", 3, "three dimensions: rows, heads, D")
    torch = _attn.torch
    dt = _dtype(k, "k")
    _with(k_pages, "k_pages", device)
    _with(v_pages, "v_pages", device)
    _is_tensor(table, "table")
    _is_tensor(ctx, "ctx")
    if k_pages.dim() != 4:
        raise ValueError("the pools must have four dimensions: pages, page, heads, D")
    if table.dim() != 2:
        raise ValueError("table must have two dimensions: sequences, pages")
    S = ctx.numel()
    T, Hkv, D = k.shape
    i32 = torch.int32
    cp = _index(ctx, "ctx", device, i32, (S,))
    rp = _index(rowptr, "rowptr", device, i32, (S + 1,))
    bp = _index(table, "table", device, i32, (S, table.shape[1]))
    tp = None
    if tree is not None:
        _is_tensor(tree, "tree")
        if tree.dtype not in (torch.int64, torch.uint64):
            raise TypeError("tree must hold 64-bit masks (int64 or uint64)")
        tp = _index(tree, "tree", device, tree.dtype, (T,))
    held, scales = CACHE_AS_IS, None
    pages, page, heads, ps, rs, hs = _paging(k_pages, v_pages, D)
    if heads != Hkv:
        raise ValueError("the pools must have the heads of k")
    if v_pages.dtype is not k_pages.dtype:
        raise TypeError("the pools must have one element type")
    if k_scale is not None or v_scale is not None:
        held = _codes(k_pages, "k_pages")
        scales = _scales(k_scale, v_scale, device, pages, page, Hkv)
        if k_scale.data_ptr() == v_scale.data_ptr() and pages:
            raise ValueError("the scales must not overlap")
    elif k_pages.dtype is not k.dtype:
        raise TypeError("the pools (without scales) must have the element type of k")
    kpp, vpp = k_pages.data_ptr() or None, v_pages.data_ptr() or None
    if kpp == vpp and kpp is not None:
        raise ValueError("the pools must not overlap")
    cosp, sinp, angles, rotated = _tables(cos, sin, device)
    r = []
    _rows(r, k, "k", device, k.dtype, k.shape)
    _rows(r, v, "v", device, k.dtype, k.shape)
    Hq = 0
    with _On(device, stream) as handle:
        if q is not None:
            _with(q, "q", device)
            if q.dim() != 3 or q.shape[0] != T or q.shape[2] != D:
                raise ValueError("q must have three dimensions: the rows and the D of k, and heads between them")
            Hq = q.shape[1]
            if Hq < 1:
                raise ValueError("q must have heads")
            _rows(r, q, "q", device, k.dtype, q.shape)
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
                r += (q_out.data_ptr(), Hq * D, D)
            else:
                _rows(r, q_out, "q_out", device, k.dtype, q.shape)
            if r[9] and (r[9] in (r[0], r[3]) or (r[9] == r[6] and r[10:] != r[7:9])):
                raise ValueError("q_out must not overlap k or v, and be q itself or apart from it")
        elif q_out is not None:
            raise ValueError("q_out goes with q")
        pack = _PACK_ROWS.pack
        w = _PACK_APPEND.pack(S, T, Hq, Hkv, D, page, pages, ps, rs, hs, table.shape[1], rotated, angles,
                              bool(interleaved), 0)
        st = _attn._ready.cache_append(
            dt, held, w, pack(*r[6:9]) if Hq else None, pack(*r[:3]), pack(*r[3:6]), cosp, sinp, bp, cp, rp, tp,
            kpp, vpp, scales, pack(*r[9:]) if Hq else None, handle)
    if st:
        _check(st, "cache_append")
    return q_out
