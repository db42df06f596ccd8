"""ctypes binding of the attention operators and the cache's page moves
(include/attn.h): argument marshalling only."""
from __future__ import annotations

import ctypes
import math

from ._binding import DTYPE_BF16, DTYPE_F32, _check, _ptr, _torch, lib

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


_ready = None


def _lib():
    global _ready
    if _ready is None:
        L = lib()
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        R, W, T, O = (ctypes.POINTER(x) for x in (_Rows, _Window, _Tree, _Pool))
        B = ctypes.POINTER(I64)
        L.window_attn_fwd.argtypes = [I32, W, R, R, R, P, P, R, P, P]
        L.window_attn_bwd.argtypes = [I32, W, R, R, R, R, R, P, P, P, R, R, R, P, I64, P]
        L.window_attn_bwd_scratch.argtypes = [W, B]
        L.tree_attn_paged.argtypes = [I32, T, R, P, P, P, P, P, P, P, P, P, I64, P]
        L.tree_attn_scratch.argtypes = [I32, T, B]
        L.pages_copy.argtypes = [O, P, P, I64, P]
        L.pages_compact.argtypes = [O, P, I64, P, P, I64, I64, P]
        for name in ("window_attn_fwd", "window_attn_bwd", "window_attn_bwd_scratch",
                     "tree_attn_paged", "tree_attn_scratch", "pages_copy", "pages_compact"):
            getattr(L, name).restype = I32
        _ready = L
    return _ready


# ------------------------------------------------------------ marshalling

class _On:
    """The device of `t` and `stream` (default: its current stream) for the
    calls inside: launches go to that device, and what is allocated inside
    belongs to that stream."""

    def __init__(self, t, stream):
        cuda = _torch().cuda
        self.device = t.device
        self.guards = []
        if cuda.current_device() != t.device.index:
            self.guards.append(cuda.device(t.device))
        if stream is not None:
            if stream.device != t.device:
                raise ValueError("stream is on another device than the operands")
            self.guards.append(cuda.stream(stream))
        self.stream = stream

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        if self.stream is None:
            return _torch().cuda.current_stream(self.device).cuda_stream
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _dtype(t, name) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"{name} must be float32 or bfloat16")


def _tensors(dev, **tensors):
    torch = _torch()
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if dev.type != "cuda":
        raise ValueError("operands must live on a GPU")
    for name, t in tensors.items():
        if t.device != dev:
            raise ValueError(f"{name} must live on the same GPU as the other operands")


def _index(t, name, shape, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, like=None, shape=None) -> _Rows:
    """[rows, heads, D] with any row and head strides and contiguous D."""
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions: rows, heads, D")
    if like is not None and t.dtype != like.dtype:
        raise TypeError(f"{name} must have the element type of q")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    n, h, d = t.shape
    if d > 1 and t.stride(2) != 1 and t.numel() > 0:
        raise ValueError(f"{name} must be contiguous along D")
    # the stride of a dimension that holds one element says nothing
    hs = t.stride(1) if h > 1 else d
    rs = t.stride(0) if n > 1 else h * d
    return _Rows(_ptr(t), rs, hs)


def _scale(scale, d) -> float:
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _window_size(window) -> int:
    return NO_WINDOW if window is None else int(window)


def _window_shape(q, k, v, q_rowptr, k_rowptr, window, sinks, scale):
    torch = _torch()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    _tensors(q.device, k=k, v=v, q_rowptr=q_rowptr, k_rowptr=k_rowptr)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must have three dimensions: rows, heads, D")
    S = q_rowptr.numel() - 1
    if S < 0:
        raise ValueError("q_rowptr must hold S+1 entries")
    _index(q_rowptr, "q_rowptr", (S + 1,), torch.int32)
    _index(k_rowptr, "k_rowptr", (S + 1,), torch.int32)
    if k.shape[2] != q.shape[2]:
        raise ValueError("q and k must have the same D")
    return _Window(S, q.shape[0], k.shape[0], q.shape[1], k.shape[1], q.shape[2],
                   _window_size(window), int(sinks), _scale(scale, q.shape[2] or 1), 0)


# ----------------------------------------------------------------- window

def window_attn_fwd(q, k, v, q_rowptr, k_rowptr, o, lse, window=None, sinks: int = 0,
                    scale: float | None = None, stream=None) -> None:
    """o and lse of window attention (window_attn_fwd); enqueued on `stream`
    (default: torch's current stream of q's device).  q and o [Tq, Hq, D], k
    and v [Tk, Hkv, D] with any row and head strides, lse [Hq, Tq] float32.
    window None: no window; scale None: 1 / sqrt(D)."""
    torch = _torch()
    w = _window_shape(q, k, v, q_rowptr, k_rowptr, window, sinks, scale)
    _tensors(q.device, o=o, lse=lse)
    _index(lse, "lse", (w.Hq, w.Tq), torch.float32)
    dt = _dtype(q, "q")
    rq, rk = _rows(q, "q"), _rows(k, "k", q)
    rv, ro = _rows(v, "v", q, k.shape), _rows(o, "o", q, q.shape)
    with _On(q, stream) as s:
        _check(_lib().window_attn_fwd(dt, w, rq, rk, rv, _ptr(q_rowptr), _ptr(k_rowptr), ro,
                                      _ptr(lse), s), "window_attn_fwd")


def window_attn_bwd(dout, q, k, v, o, lse, q_rowptr, k_rowptr, dq, dk, dv, window=None,
                    sinks: int = 0, scale: float | None = None, stream=None) -> None:
    """Gradients of window_attn_fwd into dq, dk and dv (window_attn_bwd).
    The scratch memory is taken from torch for this call alone."""
    torch = _torch()
    w = _window_shape(q, k, v, q_rowptr, k_rowptr, window, sinks, scale)
    _tensors(q.device, dout=dout, o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    _index(lse, "lse", (w.Hq, w.Tq), torch.float32)
    dt = _dtype(q, "q")
    rows = [_rows(t, n, q, like.shape) for n, t, like in (
        ("dout", dout, q), ("q", q, q), ("k", k, k), ("v", v, k), ("o", o, q))]
    outs = [_rows(t, n, q, like.shape) for n, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, k))]
    need = ctypes.c_int64()
    _check(_lib().window_attn_bwd_scratch(w, ctypes.byref(need)), "window_attn_bwd_scratch")
    with _On(q, stream) as s:
        scratch = torch.empty(need.value, dtype=torch.uint8, device=q.device)
        _check(_lib().window_attn_bwd(dt, w, *rows, _ptr(lse), _ptr(q_rowptr), _ptr(k_rowptr), *outs,
                                      _ptr(scratch), need.value, s), "window_attn_bwd")


def window_attention(q, k, v, q_rowptr, k_rowptr=None, window=None, sinks: int = 0,
                     scale: float | None = None, stream=None):
    """(o, lse) of attention over a window with first keys that stay visible.

    Sequences are packed: s owns rows rowptr[s] .. rowptr[s+1]-1 of q (and
    of k and v; k_rowptr None: the same).  Its queries are its last
    positions: query i of Lq has position i + Lk - Lq and sees key j when
    j <= position and (position - j < window or j < sinks).  Allocates o
    [Tq, Hq, D] in q's type and lse [Hq, Tq] float32, on `stream` if given;
    rows of no sequence are left as they were allocated."""
    torch = _torch()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    _tensors(q.device, q=q)
    if q.dim() != 3:
        raise ValueError("q must have three dimensions: rows, heads, D")
    with _On(q, stream):
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    window_attn_fwd(q, k, v, q_rowptr, q_rowptr if k_rowptr is None else k_rowptr, o, lse, window,
                    sinks, scale, stream)
    return o, lse


def window_attention_backward(dout, q, k, v, o, lse, q_rowptr, k_rowptr=None, window=None,
                              sinks: int = 0, scale: float | None = None, stream=None):
    """(dq, dk, dv) of window_attention for the gradient dout of its o; o and
    lse as it returned them, the other arguments as it took them."""
    torch = _torch()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    _tensors(q.device, q=q, k=k, v=v)
    with _On(q, stream):
        dq, dk, dv = (torch.empty(t.shape, dtype=q.dtype, device=q.device) for t in (q, k, v))
    window_attn_bwd(dout, q, k, v, o, lse, q_rowptr, q_rowptr if k_rowptr is None else k_rowptr, dq,
                    dk, dv, window, sinks, scale, stream)
    return dq, dk, dv


# ------------------------------------------------------------------- tree

def tree_attn_paged(q, k_pages, v_pages, table, ctx, q_rowptr, tree, o, lse, window=None,
                    sinks: int = 0, scale: float | None = None, stream=None) -> None:
    """Attention of drafted tokens over a paged cache into o [Tq, Hq, D] and
    lse [Hq, Tq] (tree_attn_paged); see tree_attention.  The scratch memory is
    taken from torch for this call alone."""
    torch = _torch()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    _tensors(q.device, k_pages=k_pages, v_pages=v_pages, table=table, ctx=ctx, q_rowptr=q_rowptr, o=o,
             lse=lse)
    if q.dim() != 3 or k_pages.dim() != 4:
        raise ValueError("q must have three dimensions (rows, heads, D) and the pools four "
                         "(pages, page, heads, D)")
    S = ctx.numel()
    Tq, Hq, D = q.shape
    pages, page, Hkv, Dk = k_pages.shape
    _index(ctx, "ctx", (S,), torch.int32)
    _index(q_rowptr, "q_rowptr", (S + 1,), torch.int32)
    if table.dim() != 2:
        raise ValueError("table must have two dimensions: sequences, pages")
    _index(table, "table", (S, table.shape[1]), torch.int32)
    if tree is not None:
        _tensors(q.device, tree=tree)
        if tree.dtype not in (torch.int64, torch.uint64):
            raise TypeError("tree must hold 64-bit masks (int64 or uint64)")
        _index(tree, "tree", (Tq,), tree.dtype)
    _index(lse, "lse", (Hq, Tq), torch.float32)
    dt = _dtype(q, "q")
    if k_pages.dtype != q.dtype or v_pages.dtype != q.dtype or o.dtype != q.dtype:
        raise TypeError("the pools and o must have the element type of q")
    if v_pages.shape != k_pages.shape or Dk != D:
        raise ValueError("the pools must have one shape, with the D of q")
    if tuple(o.shape) != (Tq, Hq, D) or not o.is_contiguous():
        raise ValueError("o must be contiguous, with the shape of q")
    if page < 1:
        raise ValueError("a page must hold at least one position")
    if k_pages.numel() > 0 and (k_pages.stride() != v_pages.stride() or
                                (D > 1 and k_pages.stride(3) != 1)):
        raise ValueError("the pools must have the same strides and be contiguous along D")
    # the stride of a dimension that holds one element says nothing
    hs = k_pages.stride(2) if Hkv > 1 else D
    rs = k_pages.stride(1) if page > 1 else Hkv * D
    ps = k_pages.stride(0) if pages > 1 else page * Hkv * D
    w = _Tree(S, Tq, Hq, Hkv, D, page, ps, rs, hs, table.shape[1], _window_size(window), int(sinks),
              _scale(scale, D or 1), 0)
    rq = _rows(q, "q")
    need = ctypes.c_int64()
    _check(_lib().tree_attn_scratch(dt, w, ctypes.byref(need)), "tree_attn_scratch")
    with _On(q, stream) as s:
        scratch = torch.empty(need.value, dtype=torch.uint8, device=q.device)
        _check(_lib().tree_attn_paged(dt, w, rq, _ptr(k_pages), _ptr(v_pages), _ptr(table), _ptr(ctx),
                                      _ptr(q_rowptr), None if tree is None else _ptr(tree), _ptr(o),
                                      _ptr(lse), _ptr(scratch), need.value, s), "tree_attn_paged")


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
    `stream` if given."""
    torch = _torch()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    _tensors(q.device, q=q)
    if q.dim() != 3:
        raise ValueError("q must have three dimensions: rows, heads, D")
    with _On(q, stream):
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    tree_attn_paged(q, k_pages, v_pages, table, ctx, q_rowptr, tree, o, lse, window, sinks, scale, stream)
    return o, lse


# ------------------------------------------------------------------ pages

def _pool(k_pool, v_pool) -> _Pool:
    """Pools [layers, pages, page, ...], contiguous, of one shape and type."""
    torch = _torch()
    if not isinstance(k_pool, torch.Tensor):
        raise TypeError("k_pool must be a torch.Tensor")
    _tensors(k_pool.device, v_pool=v_pool)
    if k_pool.dim() < 4:
        raise ValueError("a pool must have at least four dimensions: layers, pages, page, row")
    if k_pool.shape != v_pool.shape or k_pool.dtype != v_pool.dtype:
        raise ValueError("the pools must have one shape and element type")
    if not k_pool.is_contiguous() or not v_pool.is_contiguous():
        raise ValueError("the pools must be contiguous")
    layers, pages, page = k_pool.shape[:3]
    row = math.prod(k_pool.shape[3:]) * k_pool.element_size()
    return _Pool(_ptr(k_pool), _ptr(v_pool), layers, pages, page, row)


def copy_pages(k_pool, v_pool, src, dst, stream=None) -> None:
    """Page dst[i] becomes a copy of page src[i] in every layer of both pools
    [layers, pages, page, ...] (pages_copy).  Pairs with a number outside the
    pool are passed over; dst numbers must differ from each other and from
    the src of other pairs."""
    torch = _torch()
    pool = _pool(k_pool, v_pool)
    _tensors(k_pool.device, src=src, dst=dst)
    _index(src, "src", (src.numel(),), torch.int32)
    _index(dst, "dst", (src.numel(),), torch.int32)
    with _On(k_pool, stream) as s:
        _check(_lib().pages_copy(pool, _ptr(src), _ptr(dst), src.numel(), s), "pages_copy")


def compact_pages(k_pool, v_pool, table, ctx, keep, stream=None) -> None:
    """The kept drafts of each sequence move to the front of its drafts, in
    every layer of both pools (pages_compact): position ctx[s] + keep[s, t]
    to ctx[s] + t, up to the first negative entry of keep [S, kept]; the
    entries before it are strictly ascending."""
    torch = _torch()
    pool = _pool(k_pool, v_pool)
    _tensors(k_pool.device, table=table, ctx=ctx, keep=keep)
    S = ctx.numel()
    _index(ctx, "ctx", (S,), torch.int32)
    if table.dim() != 2 or keep.dim() != 2:
        raise ValueError("table and keep must have two dimensions, sequences first")
    _index(table, "table", (S, table.shape[1]), torch.int32)
    _index(keep, "keep", (S, keep.shape[1]), torch.int32)
    with _On(k_pool, stream) as s:
        _check(_lib().pages_compact(pool, _ptr(table), table.shape[1], _ptr(ctx), _ptr(keep), S,
                                    keep.shape[1], s), "pages_compact")
