"""The C ABI of include/attn.h and its binding without a GPU: exports, and
every refusal, which is found on the host before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

import sparse_dense_linear_amd as sdl
from sparse_dense_linear_amd import _attn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000          # never dereferenced: every call below returns first
INVALID, HIP, UNSUPPORTED = 1, 2, 4
F32, BF16 = 0, 1


class _Library:
    """The library's functions, taking structures and numbers alike."""

    def __getattr__(self, name):
        f = getattr(_attn._lib(), name)
        return lambda *a: f(*(ctypes.addressof(x) if isinstance(x, (ctypes.Structure, ctypes.c_int64)) else x
                              for x in a))


LIB = _Library()


def header_functions():
    text = open(os.path.join(ROOT, "include", "attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*spmm_status_t\s*(\w+)\s*\(", text, re.M)))


def test_library_exports_every_declared_symbol():
    names = header_functions()
    assert names == ["pages_compact", "pages_copy", "tree_attn_paged", "tree_attn_scratch",
                     "window_attn_bwd", "window_attn_bwd_scratch", "window_attn_fwd",
                     "window_attn_fwd_scratch"]
    lib = ctypes.CDLL(sdl.lib_path())
    assert not [n for n in names if not hasattr(lib, n)]


def test_structures_match_the_header():
    """Sizes of the structures as a C compiler lays them out."""
    assert ctypes.sizeof(_attn._Rows) == 24
    assert ctypes.sizeof(_attn._Window) == 72
    assert ctypes.sizeof(_attn._Tree) == 104
    assert ctypes.sizeof(_attn._Pool) == 48


def window(**change):
    a = dict(S=2, Tq=10, Tk=10, Hq=4, Hkv=2, D=64, window=8, sinks=1, scale=0.1, reserved=0)
    a.update(change)
    return _attn._Window(**a)


def rows(heads=4, D=64, data=FAKE, **change):
    a = dict(data=data, row_stride=heads * D, head_stride=D)
    a.update(change)
    return _attn._Rows(**a)


def fwd(w=None, dtype=F32, q=None, k=None, v=None, o=None, qp=FAKE, kp=FAKE, lse=FAKE, scratch=FAKE, size=1 << 40):
    return LIB.window_attn_fwd(dtype, w or window(), q or rows(), k or rows(2), v or rows(2), qp, kp,
                               o or rows(), lse, scratch, size, None)


def bwd(w=None, dtype=F32, scratch=FAKE, size=1 << 30, lse=FAKE, **r):
    d = {n: rows() for n in ("dout", "q", "o", "dq")} | {n: rows(2) for n in ("k", "v", "dk", "dv")}
    d.update(r)
    return LIB.window_attn_bwd(dtype, w or window(), d["dout"], d["q"], d["k"], d["v"], d["o"], lse,
                                        FAKE, FAKE, d["dq"], d["dk"], d["dv"], scratch, size, None)


BAD_HEADS = [(dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=3), INVALID), (dict(Hq=-4), INVALID),
             (dict(Hq=1 << 20), UNSUPPORTED), (dict(D=0), INVALID), (dict(D=-8), INVALID),
             (dict(D=12), UNSUPPORTED), (dict(D=136), UNSUPPORTED), (dict(window=0), INVALID),
             (dict(window=-5), INVALID), (dict(sinks=-1), INVALID), (dict(sinks=129), UNSUPPORTED),
             (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
             (dict(scale=float("inf")), INVALID), (dict(reserved=1), INVALID), (dict(S=-1), INVALID),
             (dict(Tq=-1), INVALID), (dict(S=1 << 30), INVALID), (dict(Tq=1 << 30), INVALID)]


@pytest.mark.parametrize("change,expect", BAD_HEADS + [
    (dict(Tk=-1), INVALID), (dict(Tk=1 << 40), INVALID), (dict(S=(1 << 30) - 1, Hq=64), UNSUPPORTED)])
def test_window_refuses_shapes(change, expect):
    assert fwd(window(**change)) == expect
    assert bwd(window(**change)) == expect
    assert sdl.lib().spmm_last_error() != b""
    need = ctypes.c_int64(-1)
    assert LIB.window_attn_bwd_scratch(window(**change), need) == expect
    assert LIB.window_attn_fwd_scratch(F32, window(**change), need) == expect
    assert need.value == -1


@pytest.mark.parametrize("bad", [
    dict(data=None), dict(data=FAKE + 8), dict(row_stride=-256), dict(row_stride=258), dict(head_stride=2),
    dict(head_stride=-64), dict(row_stride=(1 << 32) + 4)])
def test_window_refuses_operands(bad):
    for n in ("q", "k", "v", "o"):
        assert fwd(**{n: rows(**bad)}) == INVALID, n
    for n in ("dout", "q", "k", "v", "o", "dq", "dk", "dv"):
        assert bwd(**{n: rows(**bad)}) == INVALID, n


def test_window_refuses_the_rest():
    assert fwd(dtype=2) == INVALID and bwd(dtype=-1) == INVALID
    # strides in units of 16 bytes: 8 elements of bf16
    assert fwd(dtype=BF16, q=rows(row_stride=260)) == INVALID
    # an output whose rows or heads overlap
    assert fwd(o=rows(row_stride=0)) == INVALID
    assert fwd(o=rows(head_stride=32)) == INVALID
    assert bwd(dk=rows(2, row_stride=64)) == INVALID
    assert fwd(qp=None) == INVALID and fwd(kp=None) == INVALID and fwd(qp=FAKE + 2) == INVALID
    assert fwd(lse=None) == INVALID and fwd(lse=FAKE + 1) == INVALID and bwd(lse=None) == INVALID
    need = ctypes.c_int64()
    assert LIB.window_attn_bwd_scratch(window(), need) == 0
    assert need.value > 0
    assert bwd(size=need.value - 1) == INVALID and bwd(scratch=None) == INVALID
    assert bwd(scratch=FAKE + 4) == INVALID
    assert LIB.window_attn_bwd_scratch(window(), None) == INVALID
    assert LIB.window_attn_fwd_scratch(F32, window(), None) == INVALID
    assert LIB.window_attn_fwd(F32, None, rows(), rows(), rows(), FAKE, FAKE, rows(), FAKE, FAKE, 1, None) == INVALID
    assert LIB.window_attn_fwd(F32, window(), None, rows(), rows(), FAKE, FAKE, rows(), FAKE, FAKE, 1,
                               None) == INVALID
    # few queries behind many keys: the walks are split, and need room
    long = window(Tk=1 << 20, window=1 << 20)
    assert LIB.window_attn_fwd_scratch(F32, long, need) == 0 and need.value > 0
    assert fwd(long, size=need.value - 1) == INVALID and fwd(long, scratch=None) == INVALID
    assert fwd(long, scratch=FAKE + 8) == INVALID
    assert LIB.window_attn_fwd_scratch(F32, window(), need) == 0 and need.value == 0


def test_nothing_to_do():
    empty = rows(data=None)
    assert fwd(window(S=0), qp=None, kp=None, lse=None) == 0
    assert fwd(window(Tq=0), q=empty, o=empty, qp=None, kp=None, lse=None) == 0
    assert bwd(window(S=0), scratch=None, size=0, lse=None) == 0
    assert bwd(window(Tq=0, Tk=0), scratch=None, size=0, lse=None, **{
        n: empty for n in ("dout", "q", "k", "v", "o", "dq", "dk", "dv")}) == 0
    assert tree(tshape(S=0)) == 0 and tree(tshape(Tq=0), q=empty) == 0
    assert copy(count=0, src=None, dst=None) == 0
    for n in ("layers", "pages", "page", "row_bytes"):
        assert copy(pool(k=None, v=None, **{n: 0})) == 0
        assert compact(pool(k=None, v=None, **{n: 0})) == 0
    assert compact(S=0) == 0 and compact(kept=0) == 0 and compact(table_stride=0) == 0


def tshape(**change):
    a = dict(S=2, Tq=10, Hq=4, Hkv=2, D=64, page=16, page_stride=2048, row_stride=128, head_stride=64,
             table_stride=5, window=8, sinks=1, scale=0.1, reserved=0)
    a.update(change)
    return _attn._Tree(**a)


def tree(w=None, dtype=F32, q=None, scratch=FAKE, size=1 << 30, **p):
    a = dict(k=FAKE, v=FAKE, table=FAKE, ctx=FAKE, rp=FAKE, tree=None, o=FAKE, lse=FAKE)
    a.update(p)
    return LIB.tree_attn_paged(dtype, w or tshape(), q or rows(), a["k"], a["v"], a["table"], a["ctx"],
                                        a["rp"], a["tree"], a["o"], a["lse"], scratch, size, None)


@pytest.mark.parametrize("change,expect", BAD_HEADS + [
    (dict(page=0), INVALID), (dict(page=-1), INVALID), (dict(page=1 << 30), INVALID),
    (dict(table_stride=-1), INVALID), (dict(page_stride=-4), INVALID), (dict(row_stride=2), INVALID),
    (dict(head_stride=65), INVALID), (dict(page_stride=1 << 40), INVALID),
    (dict(Tq=(1 << 30) - 1, Hq=8), UNSUPPORTED)])
def test_tree_refuses_shapes(change, expect):
    assert tree(tshape(**change)) == expect
    assert sdl.lib().spmm_last_error() != b""
    need = ctypes.c_int64(-1)
    assert LIB.tree_attn_scratch(F32, tshape(**change), need) == expect
    assert need.value == -1


def test_tree_refuses_the_rest():
    for n in ("k", "v", "table", "ctx", "rp", "o", "lse"):
        assert tree(**{n: None}) == INVALID, n
        assert tree(**{n: FAKE + 2}) == INVALID, n
    assert tree(tree=FAKE + 4) == INVALID and tree(k=FAKE + 8) == INVALID and tree(dtype=7) == INVALID
    assert tree(q=rows(data=FAKE + 8)) == INVALID and tree(q=rows(row_stride=3)) == INVALID
    need = ctypes.c_int64()
    assert LIB.tree_attn_scratch(F32, tshape(), need) == 0
    assert tree(size=need.value - 1) == INVALID and tree(scratch=None) == INVALID
    assert tree(scratch=FAKE + 8) == INVALID
    assert LIB.tree_attn_scratch(9, tshape(), need) == INVALID


def pool(**change):
    a = dict(k=FAKE, v=FAKE, layers=2, pages=8, page=16, row_bytes=256)
    a.update(change)
    return _attn._Pool(**a)


def copy(p=None, src=FAKE, dst=FAKE, count=3):
    return LIB.pages_copy(p or pool(), src, dst, count, None)


def compact(p=None, table=FAKE, table_stride=4, ctx=FAKE, keep=FAKE, S=2, kept=3):
    return LIB.pages_compact(p or pool(), table, table_stride, ctx, keep, S, kept, None)


@pytest.mark.parametrize("change,expect", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(layers=-1), INVALID),
    (dict(pages=-1), INVALID), (dict(page=-1), INVALID), (dict(row_bytes=-16), INVALID),
    (dict(row_bytes=24), UNSUPPORTED), (dict(layers=1 << 30), INVALID),
    (dict(layers=(1 << 30) - 1), UNSUPPORTED), (dict(row_bytes=(1 << 30) - 16, layers=1 << 20), UNSUPPORTED)])
def test_pages_refuse_pools(change, expect):
    assert copy(pool(**change)) == expect and compact(pool(**change)) == expect


def test_pages_refuse_the_rest():
    assert copy(src=None) == INVALID and copy(dst=FAKE + 1) == INVALID and copy(count=-1) == INVALID
    assert copy(count=1 << 30) == UNSUPPORTED
    assert compact(table=None) == INVALID and compact(ctx=None) == INVALID and compact(keep=FAKE + 2) == INVALID
    assert compact(S=-1) == INVALID and compact(kept=-1) == INVALID and compact(table_stride=-1) == INVALID
    assert compact(S=1 << 30) == INVALID and compact(kept=1 << 30) == INVALID
    assert LIB.pages_copy(None, FAKE, FAKE, 1, None) == INVALID


#: calls at the edge of what a launch holds (2^32 - 1 threads along x): below it,
#: they get as far as a HIP call
EDGE = 1 << 24
WIDE = {n: rows(32) for n in ("dout", "q", "o", "dq")} | {n: rows(8) for n in ("k", "v", "dk", "dv")}
AT_THE_LIMIT = [
    # 128 queries of a head to a workgroup, and one more for each sequence
    (lambda n: fwd(window(S=n, Hq=1, Hkv=1)), EDGE - 1),
    (lambda n: fwd(window(S=524000, Tq=128 * n, Hq=32), q=rows(32), o=rows(32)), EDGE // 32 - 524000 - 1),
    # the backward pass: queries, keys in tiles of 64, the far runs of first keys and their joining
    (lambda n: bwd(window(S=n, Tk=0, Hq=1, Hkv=1), size=1 << 50), EDGE - 1),
    (lambda n: bwd(window(S=8, Tk=64 * n, Hq=32, Hkv=8, sinks=0), size=1 << 50, **WIDE), EDGE // 8 - 9),
    (lambda n: bwd(window(S=n, Hq=1, Hkv=1, window=10), size=1 << 50), EDGE - 1),
    (lambda n: bwd(window(S=n, Tq=512 * 9, Tk=64 * 1000, Hq=1, Hkv=1), size=1 << 50), (EDGE - 1 - 1009) // 2),
    (lambda n: bwd(window(S=n, Hq=1, Hkv=1, sinks=128), size=1 << 50), EDGE * 4 // 128 - 1),
    # blocks of 16 queries
    (lambda n: tree(tshape(S=n, Hq=1, Hkv=1)), EDGE - 1),
    # 16 KB of a page, in a layer of a pool
    (lambda n: copy(pool(layers=64), count=n), EDGE // 128 - 1),
    (lambda n: copy(pool(layers=64, row_bytes=1024), count=n), EDGE // 128 - 1),
    (lambda n: copy(pool(layers=64, row_bytes=1040), count=n), EDGE // 256 - 1),
    (lambda n: compact(S=n), EDGE - 1),
]


@pytest.mark.parametrize("case", range(len(AT_THE_LIMIT)))
def test_calls_that_no_launch_holds_are_refused(case):
    call, most = AT_THE_LIMIT[case]
    assert call(most + 1) == UNSUPPORTED
    assert sdl.lib().spmm_last_error() != b""
    if not torch.cuda.is_available():
        assert call(most) == HIP


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_report_hip_errors():
    assert fwd() == HIP and bwd() == HIP and tree() == HIP and copy() == HIP and compact() == HIP
    assert sdl.lib().spmm_last_error() != b""


def test_binding_refuses_cpu_tensors_and_non_tensors():
    q = torch.zeros(4, 2, 64)
    rp = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        sdl.window_attention(q, q, q, rp)
    with pytest.raises(ValueError):
        sdl.window_attention_backward(q, q, q, q, q, q, rp)
    with pytest.raises(ValueError):
        sdl.tree_attention(q, q[None], q[None], rp[None], rp, rp)
    with pytest.raises(ValueError):
        sdl.copy_pages(q[None], q[None], rp, rp)
    with pytest.raises(ValueError):
        sdl.compact_pages(q[None], q[None], rp[None], rp, rp[None])
    for call in (lambda: sdl.window_attention([1], q, q, rp), lambda: sdl.tree_attention(1, q, q, rp, rp, rp),
                 lambda: sdl.window_attention_backward(q, 1, q, q, q, q, rp),
                 lambda: sdl.copy_pages(1, q, rp, rp), lambda: sdl.compact_pages(1, q, rp, rp, rp)):
        with pytest.raises(TypeError):
            call()
