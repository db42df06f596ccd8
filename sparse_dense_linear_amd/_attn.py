"""ctypes binding of the attention operators and the cache's page moves
(include/attn.h): argument marshalling only."""
from __future__ import annotations

import ctypes
import math
from array import array
from operator import index

from ._binding import DTYPE_BF16, DTYPE_F32, _check, _torch, lib

#: A window that no sequence reaches past.
NO_WINDOW = (1 << 30) - 1


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _Window(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("S", "Tq", "Tk", "Hq", "Hkv", "D", "window", "sinks")] + \
               [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class _Tree(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "S", "Tq", "Hq", "Hkv", "D", "page", "page_stride", "row_stride", "head_stride",
        "table_stride", "window", "sinks")] + \
        [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class _Pool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + \
               [(n, ctypes.c_int64) for n in ("layers", "pages", "page", "row_bytes")]


#: Bytes of one operand's description (attn_rows_t): descriptions of a call
#: are laid out one after another in an array of 64-bit numbers.
_ROWS = ctypes.sizeof(_Rows)

_ready = None
torch = None


def _lib():
    global _ready, torch
    if _ready is None:
        torch = _torch()
        L = lib()
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.window_attn_fwd.argtypes = [I32] + [P] * 9 + [I64, P]
        L.window_attn_fwd_scratch.argtypes = [I32, P, P]
        L.window_attn_bwd.argtypes = [I32] + [P] * 13 + [I64, P]
        L.window_attn_bwd_scratch.argtypes = [P, P]
        L.tree_attn_paged.argtypes = [I32] + [P] * 11 + [I64, P]
        L.tree_attn_scratch.argtypes = [I32, P, P]
        L.pages_copy.argtypes = [P, P, P, I64, P]
        L.pages_compact.argtypes = [P, P, I64, P, P, I64, I64, P]
        for name in ("window_attn_fwd", "window_attn_fwd_scratch", "window_attn_bwd", "window_attn_bwd_scratch",
                     "tree_attn_paged", "tree_attn_scratch", "pages_copy", "pages_compact"):
            getattr(L, name).restype = I32
        _ready = L
    return _ready


# ------------------------------------------------------------ marshalling

class _On:
    """The device of the operands and the stream of a call (default: the
    device's current stream): launches inside go there, and what is allocated
    inside belongs to that stream.  Entering gives the stream's handle."""

    def __init__(self, device, stream):
        cuda = torch.cuda
        self.guards = []
        if cuda.current_device() != device.index:
            self.guards.append(cuda.device(device))
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)
        else:
            if stream.device != device:
                raise ValueError("stream is on another device than the operands")
            self.guards.append(cuda.stream(stream))
            self.handle = stream.cuda_stream

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _is_tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")


def _first(t, name, dims, what):
    """The operand that the others are held against."""
    _lib()
    _is_tensor(t, name)
    if t.device.type != "cuda":
        raise ValueError("operands must live on a GPU")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {what}")
    return t.device


def _dtype(t, name) -> int:
    if t.dtype is torch.float32:
        return DTYPE_F32
    if t.dtype is torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"{name} must be float32 or bfloat16")


def _with(t, name, device):
    _is_tensor(t, name)
    if t.device != device:
        raise ValueError(f"{name} must live on the same GPU as the other operands")


def _index(t, name, device, dtype, shape):
    """The address of a contiguous array."""
    _with(t, name, device)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _rows(out, t, name, device, dtype, shape):
    """Adds the description of t [rows, heads, D], with any row and head
    strides and D contiguous, to the list `out`."""
    _with(t, name, device)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have the element type of q")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    n, h, d = shape
    rs, hs, ds = t.stride()
    if n == 0 or h == 0 or d == 0:
        out += (0, h * d, d)
        return
    if ds != 1 and d > 1:
        raise ValueError(f"{name} must be contiguous along D")
    # the stride of a dimension that holds one element says nothing
    out += (t.data_ptr(), rs if n > 1 else h * d, hs if h > 1 else d)


def _apart(r, outs, names):
    """Refuses an output that begins where another operand of the call does:
    results would be written over what is still to be read."""
    at = r[::3]
    for i in outs:
        if at[i] and at.count(at[i]) > 1:
            j = next(j for j in range(len(at)) if j != i and at[j] == at[i])
            raise ValueError(f"{names[i]} must not overlap {names[j]}")


def _scale(scale, d) -> float:
    return 1.0 / math.sqrt(d or 1) if scale is None else float(scale)


def _window_size(window) -> int:
    if window is None:
        return NO_WINDOW
    window = index(window)
    return window if -1 <= window <= NO_WINDOW else _cut(window, NO_WINDOW)


def _sinks(sinks) -> int:
    sinks = index(sinks)
    return sinks if -1 <= sinks <= NO_WINDOW else _cut(sinks, NO_WINDOW)


def _cut(x, most) -> int:
    """A number past 64 bits would lose its upper ones on its way into a
    structure; those below 0 and above `most` are all alike."""
    return most if x > most else -1


def _window_shape(q, k, v, q_rowptr, window, sinks, scale, device):
    """attn_window_t of a call, and the number of sequences."""
    _with(k, "k", device)
    _with(q_rowptr, "q_rowptr", device)
    if k.dim() != 3:
        raise ValueError("k must have three dimensions: rows, heads, D")
    if k.shape[2] != q.shape[2]:
        raise ValueError("q and k must have the same D")
    S = q_rowptr.numel() - 1
    if S < 0:
        raise ValueError("q_rowptr must hold S+1 entries")
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    return _Window(S, Tq, Tk, Hq, Hkv, D, _window_size(window), _sinks(sinks), _scale(scale, D), 0), S


# ----------------------------------------------------------------- window
# (fresh: the outputs were just allocated)

def _fwd(q, k, v, q_rowptr, k_rowptr, o, lse, window, sinks, scale, device, handle, fresh=False):
    dt = _dtype(q, "q")
    w, S = _window_shape(q, k, v, q_rowptr, window, sinks, scale, device)
    i32 = torch.int32
    qp = _index(q_rowptr, "q_rowptr", device, i32, (S + 1,))
    kp = qp if k_rowptr is q_rowptr else _index(k_rowptr, "k_rowptr", device, i32, (S + 1,))
    lp = _index(lse, "lse", device, torch.float32, (w.Hq, w.Tq))
    r = []
    e = q.dtype
    _rows(r, q, "q", device, e, q.shape)
    _rows(r, k, "k", device, e, k.shape)
    _rows(r, v, "v", device, e, k.shape)
    _rows(r, o, "o", device, e, q.shape)
    if not fresh:
        _apart(r, (3,), ("q", "k", "v", "o"))
    r = array("q", r)
    at, shape = r.buffer_info()[0], ctypes.addressof(w)
    need = ctypes.c_int64()
    st = _ready.window_attn_fwd_scratch(dt, shape, ctypes.addressof(need))
    if st:
        _check(st, "window_attn_fwd_scratch")
    scratch = torch.empty(need.value, dtype=torch.uint8, device=device) if need.value else None
    st = _ready.window_attn_fwd(dt, shape, at, at + _ROWS, at + 2 * _ROWS, qp, kp, at + 3 * _ROWS, lp,
                                scratch.data_ptr() if need.value else None, need.value, handle)
    if st:
        _check(st, "window_attn_fwd")


def _bwd(dout, q, k, v, o, lse, q_rowptr, k_rowptr, dq, dk, dv, window, sinks, scale, device, handle,
         fresh=False):
    dt = _dtype(q, "q")
    w, S = _window_shape(q, k, v, q_rowptr, window, sinks, scale, device)
    i32 = torch.int32
    qp = _index(q_rowptr, "q_rowptr", device, i32, (S + 1,))
    kp = qp if k_rowptr is q_rowptr else _index(k_rowptr, "k_rowptr", device, i32, (S + 1,))
    lp = _index(lse, "lse", device, torch.float32, (w.Hq, w.Tq))
    r = []
    e, qs, ks = q.dtype, q.shape, k.shape
    _rows(r, dout, "dout", device, e, qs)
    _rows(r, q, "q", device, e, qs)
    _rows(r, k, "k", device, e, ks)
    _rows(r, v, "v", device, e, ks)
    _rows(r, o, "o", device, e, qs)
    _rows(r, dq, "dq", device, e, qs)
    _rows(r, dk, "dk", device, e, ks)
    _rows(r, dv, "dv", device, e, ks)
    if not fresh:
        _apart(r, (5, 6, 7), ("dout", "q", "k", "v", "o", "dq", "dk", "dv"))
    r = array("q", r)
    at, shape = r.buffer_info()[0], ctypes.addressof(w)
    need = ctypes.c_int64()
    st = _ready.window_attn_bwd_scratch(shape, ctypes.addressof(need))
    if st:
        _check(st, "window_attn_bwd_scratch")
    scratch = torch.empty(need.value, dtype=torch.uint8, device=device)
    st = _ready.window_attn_bwd(dt, shape, at, at + _ROWS, at + 2 * _ROWS, at + 3 * _ROWS, at + 4 * _ROWS,
                                lp, qp, kp, at + 5 * _ROWS, at + 6 * _ROWS, at + 7 * _ROWS,
                                scratch.data_ptr() or None, need.value, handle)
    if st:
        _check(st, "window_attn_bwd")


def window_attn_fwd(q, k, v, q_rowptr, k_rowptr, o, lse, window=None, sinks: int = 0,
                    scale: float | None = None, stream=None) -> None:
    """o and lse of window attention (window_attn_fwd); enqueued on `stream`
    (default: torch's current stream of q's device).  q and o [Tq, Hq, D], k
    and v [Tk, Hkv, D] with any row and head strides, lse [Hq, Tq] float32; o
    and lse overlap nothing that the call reads.
    window None: no window; scale None: 1 / sqrt(D).  The scratch memory, if
    the call needs any, is taken from torch for this call alone."""
    device = _first(q, "q", 3, "three dimensions: rows, heads, D")
    with _On(device, stream) as handle:
        _fwd(q, k, v, q_rowptr, k_rowptr, o, lse, window, sinks, scale, device, handle)


def window_attn_bwd(dout, q, k, v, o, lse, q_rowptr, k_rowptr, dq, dk, dv, window=None,
                    sinks: int = 0, scale: float | None = None, stream=None) -> None:
    """Gradients of window_attn_fwd into dq, dk and dv (window_attn_bwd), which
    overlap neither each other nor anything that the call reads.  The scratch
    memory is taken from torch for this call alone."""
    device = _first(q, "q", 3, "three dimensions: rows, heads, D")
    with _On(device, stream) as handle:
        _bwd(dout, q, k, v, o, lse, q_rowptr, k_rowptr, dq, dk, dv, window, sinks, scale, device, handle)


def window_attention(q, k, v, q_rowptr, k_rowptr=None, window=None, sinks: int = 0,
                     scale: float | None = None, stream=None):
    """(o, lse) of attention over a window with first keys that stay visible.

    Sequences are packed: s owns rows rowptr[s] .. rowptr[s+1]-1 of q (and
    of k and v; k_rowptr None: the same).  Its queries are its last
    positions: query i of Lq has position i + Lk - Lq and sees key j when
    j <= position and (position - j < window or j < sinks).  Allocates o
    [Tq, Hq, D] in q's type and lse [Hq, Tq] float32, on `stream` if given;
    rows of no sequence are left as they were allocated.

    As all operators of this library it records no autograd graph, also for
    operands that require gradients: window_attention_backward gives them."""
    device = _first(q, "q", 3, "three dimensions: rows, heads, D")
    with _On(device, stream) as handle:
        o = torch.empty(q.shape, dtype=q.dtype, device=device)
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=device)
        _fwd(q, k, v, q_rowptr, q_rowptr if k_rowptr is None else k_rowptr, o, lse, window, sinks, scale,
             device, handle, fresh=True)
    return o, lse


def window_attention_backward(dout, q, k, v, o, lse, q_rowptr, k_rowptr=None, window=None,
                              sinks: int = 0, scale: float | None = None, stream=None):
    """(dq, dk, dv) of window_attention for the gradient dout of its o; o and
    lse as it returned them, the other arguments as it took them."""
    device = _first(q, "q", 3, "three dimensions: rows, heads, D")
    _is_tensor(k, "k")
    _is_tensor(v, "v")
    with _On(device, stream) as handle:
        dq, dk, dv = (torch.empty(t.shape, dtype=q.dtype, device=device) for t in (q, k, v))
        _bwd(dout, q, k, v, o, lse, q_rowptr, q_rowptr if k_rowptr is None else k_rowptr, dq, dk, dv, window,
             sinks, scale, device, handle, fresh=True)
    return dq, dk, dv


# ------------------------------------------------------------------- tree

def _tree(q, k_pages, v_pages, table, ctx, q_rowptr, tree, o, lse, window, sinks, scale, device, handle):
    dt = _dtype(q, "q")
    _with(k_pages, "k_pages", device)
    _with(v_pages, "v_pages", device)
    _with(table, "table", device)
    _with(ctx, "ctx", device)
    _with(o, "o", device)
    if k_pages.dim() != 4:
        raise ValueError("the pools must have four dimensions: pages, page, heads, D")
    if table.dim() != 2:
        raise ValueError("table must have two dimensions: sequences, pages")
    S = ctx.numel()
    Tq, Hq, D = q.shape
    pages, page, Hkv, Dk = k_pages.shape
    i32 = torch.int32
    cp = _index(ctx, "ctx", device, i32, (S,))
    qp = _index(q_rowptr, "q_rowptr", device, i32, (S + 1,))
    bp = _index(table, "table", device, i32, (S, table.shape[1]))
    tp = None
    if tree is not None:
        _is_tensor(tree, "tree")
        if tree.dtype not in (torch.int64, torch.uint64):
            raise TypeError("tree must hold 64-bit masks (int64 or uint64)")
        tp = _index(tree, "tree", device, tree.dtype, (Tq,))
    lp = _index(lse, "lse", device, torch.float32, (Hq, Tq))
    if k_pages.dtype is not q.dtype or v_pages.dtype is not q.dtype or o.dtype is not q.dtype:
        raise TypeError("the pools and o must have the element type of q")
    if v_pages.shape != k_pages.shape or Dk != D:
        raise ValueError("the pools must have one shape, with the D of q")
    if o.shape != q.shape or not o.is_contiguous():
        raise ValueError("o must be contiguous, with the shape of q")
    if page < 1:
        raise ValueError("a page must hold at least one position")
    ps, rs, hs, ds = k_pages.stride()
    if pages and Hkv and D and (v_pages.stride() != (ps, rs, hs, ds) or (D > 1 and ds != 1)):
        raise ValueError("the pools must have the same strides and be contiguous along D")
    # the stride of a dimension that holds one element says nothing
    hs = hs if Hkv > 1 else D
    rs = rs if page > 1 else Hkv * D
    ps = ps if pages > 1 else page * Hkv * D
    w = _Tree(S, Tq, Hq, Hkv, D, page, ps, rs, hs, table.shape[1], _window_size(window), _sinks(sinks),
              _scale(scale, D), 0)
    r = []
    _rows(r, q, "q", device, q.dtype, q.shape)
    op = o.data_ptr()
    if op and op == r[0]:
        raise ValueError("o must not overlap q")
    r = array("q", r)
    need, shape = ctypes.c_int64(), ctypes.addressof(w)
    st = _ready.tree_attn_scratch(dt, shape, ctypes.addressof(need))
    if st:
        _check(st, "tree_attn_scratch")
    scratch = torch.empty(need.value, dtype=torch.uint8, device=device)
    st = _ready.tree_attn_paged(dt, shape, r.buffer_info()[0], k_pages.data_ptr() or None,
                                v_pages.data_ptr() or None, bp, cp, qp, tp, op or None, lp,
                                scratch.data_ptr() or None, need.value, handle)
    if st:
        _check(st, "tree_attn_paged")


def tree_attn_paged(q, k_pages, v_pages, table, ctx, q_rowptr, tree, o, lse, window=None,
                    sinks: int = 0, scale: float | None = None, stream=None) -> None:
    """Attention of drafted tokens over a paged cache into o [Tq, Hq, D] and
    lse [Hq, Tq] (tree_attn_paged); see tree_attention.  o and lse overlap
    nothing that the call reads.  The scratch memory is taken from torch for
    this call alone."""
    device = _first(q, "q", 3, "three dimensions: rows, heads, D")
    with _On(device, stream) as handle:
        _tree(q, k_pages, v_pages, table, ctx, q_rowptr, tree, o, lse, window, sinks, scale, device, handle)


def tree_attention(q, k_pages, v_pages, table, ctx, q_rowptr, tree=None, window=None, sinks: int = 0,
                   scale: float | None = None, stream=None):
    """(o, lse) of drafted tokens over a paged cache.

    Sequence s has ctx[s] cached positions, and its drafts are rows
    q_rowptr[s] .. q_rowptr[s+1]-1 of q; the drafts' keys and values lie in
    the cache behind the context.  Position j is row j % page of page
    table[s, j // page] of the pools [pages, page, Hkv, D].  Bit a of
    tree[row] says that the draft sees draft a of its sequence (tree None: a
    chain; one token is a chain of one).  A draft stands at position ctx +
    (drafts it sees) - 1, and the window and the sinks are those of
    window_attention.  Allocates o [Tq, Hq, D] and lse [Hq, Tq] float32, on
    `stream` if given; records no autograd graph."""
    device = _first(q, "q", 3, "three dimensions: rows, heads, D")
    with _On(device, stream) as handle:
        o = torch.empty(q.shape, dtype=q.dtype, device=device)
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=device)
        _tree(q, k_pages, v_pages, table, ctx, q_rowptr, tree, o, lse, window, sinks, scale, device, handle)
    return o, lse


# ------------------------------------------------------------------ pages

def _pool(k_pool, v_pool, one=False):
    """attn_pool_t of pools [layers, pages, page, ...], contiguous, of one
    shape and type, that do not overlap (one: or are one), and their device."""
    _lib()
    _is_tensor(k_pool, "k_pool")
    device = k_pool.device
    if device.type != "cuda":
        raise ValueError("operands must live on a GPU")
    _with(v_pool, "v_pool", device)
    shape = k_pool.shape
    if len(shape) < 4:
        raise ValueError("a pool must have at least four dimensions: layers, pages, page, row")
    if shape != v_pool.shape or k_pool.dtype is not v_pool.dtype:
        raise ValueError("the pools must have one shape and element type")
    if not k_pool.is_contiguous() or not v_pool.is_contiguous():
        raise ValueError("the pools must be contiguous")
    layers, pages, page = shape[:3]
    row = math.prod(shape[3:]) * k_pool.element_size()
    kp, vp = k_pool.data_ptr(), v_pool.data_ptr()
    if abs(kp - vp) < layers * pages * page * row and not (one and kp == vp):
        raise ValueError("the pools must not overlap")
    return _Pool(kp or None, vp or None, layers, pages, page, row), device


def copy_pages(k_pool, v_pool, src, dst, stream=None) -> None:
    """Page dst[i] becomes a copy of page src[i] in every layer of both pools
    [layers, pages, page, ...] (pages_copy), which may be one.  Pairs with a
    number outside the pool are passed over; dst numbers must differ from each
    other and from the src of other pairs."""
    pool, device = _pool(k_pool, v_pool, one=True)
    _is_tensor(src, "src")
    n = src.numel()
    sp = _index(src, "src", device, torch.int32, (n,))
    dp = _index(dst, "dst", device, torch.int32, (n,))
    with _On(device, stream) as handle:
        st = _ready.pages_copy(ctypes.addressof(pool), sp, dp, n, handle)
    if st:
        _check(st, "pages_copy")


def compact_pages(k_pool, v_pool, table, ctx, keep, stream=None) -> None:
    """The kept drafts of each sequence move to the front of its drafts, in
    every layer of both pools (pages_compact): position ctx[s] + keep[s, t]
    to ctx[s] + t, up to the first negative entry of keep [S, kept]; the
    entries before it are strictly ascending."""
    pool, device = _pool(k_pool, v_pool)
    _is_tensor(table, "table")
    _is_tensor(ctx, "ctx")
    _is_tensor(keep, "keep")
    S = ctx.numel()
    if table.dim() != 2 or keep.dim() != 2:
        raise ValueError("table and keep must have two dimensions, sequences first")
    wide, kept = table.shape[1], keep.shape[1]
    cp = _index(ctx, "ctx", device, torch.int32, (S,))
    bp = _index(table, "table", device, torch.int32, (S, wide))
    kp = _index(keep, "keep", device, torch.int32, (S, kept))
    with _On(device, stream) as handle:
        st = _ready.pages_compact(ctypes.addressof(pool), bp, wide, cp, kp, S, kept, handle)
    if st:
        _check(st, "pages_compact")
