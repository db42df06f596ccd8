"""The C ABI of include/cache.h and its binding without a GPU: exports, and every
refusal, which is found on the host before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

import sparse_dense_linear_amd as sdl
from sparse_dense_linear_amd import _attn, _cache
from test_attn_host import BAD_HEADS, BF16, F32, FAKE, HIP, INVALID, LIB, ROOT, UNSUPPORTED, rows, tshape

AS_IS, E4M3, INT8 = 0, 1, 2


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "cache.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"^\s*spmm_status_t\s*(\w+)\s*\(", text, re.M)))
    assert names == ["cache_append", "cache_compact", "cache_copy", "cache_tree_attn", "cache_tree_attn_scratch"]
    lib = ctypes.CDLL(sdl.lib_path())
    assert not [n for n in names if not hasattr(lib, n)]


def test_structures_match_the_header():
    assert ctypes.sizeof(_attn._Scales) == 48
    assert ctypes.sizeof(_attn._CodePool) == 80
    assert ctypes.sizeof(_cache._Append) == 112


def scales(**change):
    a = dict(k=FAKE, v=FAKE, block=8, page_stride=4, block_stride=2, head_stride=1)
    a.update(change)
    return _attn._Scales(**a)


BAD_SCALES = [dict(k=None), dict(v=None), dict(k=FAKE + 2), dict(block=0), dict(block=-8), dict(block=3),
              dict(block=32), dict(page_stride=-1), dict(block_stride=-1), dict(head_stride=-1),
              dict(page_stride=(1 << 32) + 1)]


# ------------------------------------------------------------- attention

def tree(w=None, dtype=F32, held=E4M3, q=None, sc=None, scratch=FAKE, size=1 << 30, **p):
    a = dict(k=FAKE, v=FAKE, table=FAKE, ctx=FAKE, rp=FAKE, tree=None, o=FAKE, lse=FAKE)
    a.update(p)
    return LIB.cache_tree_attn(dtype, held, w or tshape(), q or rows(), a["k"], a["v"], sc or scales(), a["table"],
                               a["ctx"], a["rp"], a["tree"], a["o"], a["lse"], scratch, size, None)


@pytest.mark.parametrize("change,expect", BAD_HEADS + [
    (dict(D=8), UNSUPPORTED), (dict(D=24), UNSUPPORTED), (dict(D=120), UNSUPPORTED),
    (dict(page=0), INVALID), (dict(page=-1), INVALID), (dict(page=1 << 30), INVALID),
    (dict(table_stride=-1), INVALID), (dict(page_stride=-16), INVALID), (dict(row_stride=8), INVALID),
    (dict(head_stride=72), INVALID), (dict(page_stride=1 << 40), INVALID),
    (dict(Tq=(1 << 30) - 1, Hq=8), UNSUPPORTED)])
def test_tree_refuses_shapes(change, expect):
    for held in (E4M3, INT8):
        assert tree(tshape(**change), held=held) == expect
        assert sdl.lib().spmm_last_error() != b""
        need = ctypes.c_int64(-1)
        assert LIB.cache_tree_attn_scratch(F32, held, tshape(**change), need) == expect
        assert need.value == -1


def test_tree_refuses_the_rest():
    for n in ("k", "v", "table", "ctx", "rp", "o", "lse"):
        assert tree(**{n: None}) == INVALID, n
        assert tree(**{n: FAKE + 2}) == INVALID, n
    assert tree(tree=FAKE + 4) == INVALID and tree(k=FAKE + 8) == INVALID and tree(dtype=7) == INVALID
    assert tree(held=AS_IS) == INVALID and tree(held=3) == INVALID and tree(held=-1) == INVALID
    assert tree(q=rows(data=FAKE + 8)) == INVALID and tree(q=rows(row_stride=3)) == INVALID
    for bad in BAD_SCALES:
        assert tree(sc=scales(**bad)) == INVALID, bad
    assert LIB.cache_tree_attn(F32, E4M3, tshape(), rows(), FAKE, FAKE, None, FAKE, FAKE, FAKE, None, FAKE, FAKE,
                               FAKE, 1 << 30, None) == INVALID
    need = ctypes.c_int64()
    assert LIB.cache_tree_attn_scratch(F32, E4M3, tshape(), need) == 0
    assert tree(size=need.value - 1) == INVALID and tree(scratch=None) == INVALID
    assert tree(scratch=FAKE + 8) == INVALID
    assert LIB.cache_tree_attn_scratch(9, E4M3, tshape(), need) == INVALID
    assert LIB.cache_tree_attn_scratch(F32, AS_IS, tshape(), need) == INVALID
    assert LIB.cache_tree_attn_scratch(F32, E4M3, tshape(), None) == INVALID
    assert LIB.cache_tree_attn_scratch(F32, E4M3, None, need) == INVALID


# ------------------------------------------------------------- appending

def ashape(**change):
    a = dict(S=2, T=10, Hq=4, Hkv=2, D=64, page=16, pages=8, page_stride=2048, row_stride=128, head_stride=64,
             table_stride=5, rotated=64, angles=100, interleaved=0, reserved=0)
    a.update(change)
    return _cache._Append(**a)


def append(w=None, dtype=F32, held=AS_IS, q=None, k=None, v=None, q_out=None, sc="default", **p):
    a = dict(cos=FAKE, sin=FAKE, table=FAKE, ctx=FAKE, rp=FAKE, tree=None, kp=FAKE, vp=FAKE)
    a.update(p)
    sc = (None if held == AS_IS else scales()) if sc == "default" else sc
    return LIB.cache_append(dtype, held, w or ashape(), q or rows(), k or rows(2), v or rows(2), a["cos"], a["sin"],
                            a["table"], a["ctx"], a["rp"], a["tree"], a["kp"], a["vp"], sc, q_out or rows(), None)


@pytest.mark.parametrize("change,expect", [
    (dict(Hq=3), INVALID), (dict(Hq=-4), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=0, Hkv=0), INVALID),
    (dict(Hq=0, Hkv=-1), INVALID), (dict(Hq=1 << 20), UNSUPPORTED), (dict(D=0), INVALID), (dict(D=-8), INVALID),
    (dict(D=12), UNSUPPORTED), (dict(D=136), UNSUPPORTED), (dict(reserved=1), INVALID), (dict(S=-1), INVALID),
    (dict(T=-1), INVALID), (dict(S=1 << 30), INVALID), (dict(T=1 << 30), INVALID), (dict(pages=-1), INVALID),
    (dict(pages=1 << 30), INVALID), (dict(table_stride=-1), INVALID), (dict(table_stride=1 << 30), INVALID),
    (dict(page=0), INVALID), (dict(page=1 << 30), INVALID), (dict(page_stride=-16), INVALID),
    (dict(row_stride=2), INVALID), (dict(head_stride=1 << 40), INVALID), (dict(rotated=-8), INVALID),
    (dict(rotated=72), INVALID), (dict(rotated=12), UNSUPPORTED), (dict(angles=-1), INVALID),
    (dict(interleaved=2), INVALID), (dict(interleaved=-1), INVALID)])
def test_append_refuses_shapes(change, expect):
    for held in (AS_IS, E4M3, INT8):
        assert append(ashape(**change), held=held) == expect
        assert sdl.lib().spmm_last_error() != b""


def test_append_refuses_the_rest():
    assert append(dtype=2) == INVALID and append(held=3) == INVALID and append(held=-1) == INVALID
    for n in ("table", "ctx", "rp", "kp", "vp", "cos", "sin"):
        assert append(**{n: None}) == INVALID, n
        assert append(**{n: FAKE + 2}) == INVALID, n
    assert append(cos=FAKE + 8) == INVALID and append(tree=FAKE + 4) == INVALID and append(kp=FAKE + 8) == INVALID
    for bad in (dict(data=None), dict(data=FAKE + 8), dict(row_stride=-256), dict(row_stride=258),
                dict(head_stride=2), dict(row_stride=(1 << 32) + 4)):
        for n in ("q", "k", "v", "q_out"):
            assert append(**{n: rows(**bad)}) == INVALID, n
    assert append(dtype=BF16, k=rows(2, row_stride=132)) == INVALID
    # rows or heads of q_out that overlap
    assert append(q_out=rows(row_stride=0)) == INVALID and append(q_out=rows(head_stride=32)) == INVALID
    # scales with pools of 8 bits, and only there; D a multiple of 16 and strides of 16 bytes
    assert append(held=E4M3, sc=None) == INVALID and append(sc=scales()) == INVALID
    for bad in BAD_SCALES:
        assert append(held=INT8, sc=scales(**bad)) == INVALID, bad
    assert append(ashape(D=40, rotated=40, head_stride=48), held=E4M3) == UNSUPPORTED
    assert append(ashape(head_stride=72), held=E4M3) == INVALID
    assert LIB.cache_append(F32, AS_IS, None, rows(), rows(2), rows(2), FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE,
                            None, rows(), None) == INVALID
    assert LIB.cache_append(F32, AS_IS, ashape(), None, rows(2), rows(2), FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE,
                            FAKE, None, rows(), None) == INVALID


@pytest.mark.parametrize("change,fine", [
    (dict(page_stride=0), False), (dict(row_stride=0), False), (dict(head_stride=0), False),
    (dict(page_stride=2032), False), (dict(row_stride=112), False), (dict(head_stride=48), False),
    (dict(page_stride=0, pages=1), True), (dict(row_stride=0, page=1, page_stride=128), True),
    (dict(head_stride=0, Hkv=1, Hq=0), True),
    # heads outside the rows, pages inside them
    (dict(row_stride=64, head_stride=1024, page_stride=2048), True),
    (dict(row_stride=64, head_stride=1008, page_stride=2048), False),
    (dict(page_stride=64, head_stride=8 * 64, row_stride=16 * 64), True),
    (dict(page_stride=64, head_stride=8 * 64, row_stride=15 * 64), False),
    (dict(page_stride=1 << 32, row_stride=1 << 32, head_stride=1 << 32, page=(1 << 30) - 1, pages=(1 << 30) - 1), False),
    (dict(page_stride=1 << 32), True)])
def test_append_refuses_pools_that_overlap_themselves(change, fine):
    for held in (AS_IS, E4M3, INT8):
        block = scales(block=1, page_stride=64, block_stride=2) if held != AS_IS else None
        st = append(ashape(T=0, **change), held=held, sc=block)
        assert st == (0 if fine else INVALID)


@pytest.mark.parametrize("change", [dict(page_stride=0), dict(block_stride=0), dict(head_stride=0),
                                    dict(page_stride=3), dict(block_stride=1), dict(head_stride=2)])
def test_append_refuses_scales_that_overlap(change):
    assert append(held=INT8, sc=scales(**change)) == INVALID
    assert b"overlap" in sdl.lib().spmm_last_error()


def test_nothing_to_do():
    empty = rows(data=None)
    assert append(ashape(S=0), table=None, ctx=None, rp=None, kp=None, vp=None) == 0
    assert append(ashape(T=0), q=empty, k=empty, v=empty, q_out=empty, kp=None, vp=None) == 0
    assert tree(tshape(S=0)) == 0 and tree(tshape(Tq=0), q=empty) == 0
    assert copy(count=0, src=None, dst=None) == 0
    for n in ("layers", "pages", "page", "row_bytes"):
        assert copy(pool(k=None, v=None, **{n: 0})) == 0
        assert compact(pool(k=None, v=None, **{n: 0})) == 0
    assert compact(S=0) == 0 and compact(kept=0) == 0 and compact(table_stride=0) == 0


# ------------------------------------------------------------------ moves

def pool(**change):
    a = dict(k=FAKE, v=FAKE, layers=2, pages=8, page=16, row_bytes=256)
    b = dict(k_scale=FAKE, v_scale=FAKE, block=8, heads=4)
    for n, x in change.items():
        (a if n in a else b)[n] = x
    return _attn._CodePool(_attn._Pool(**a), **b)


def copy(p=None, src=FAKE, dst=FAKE, count=3):
    return LIB.cache_copy(p or pool(), src, dst, count, None)


def compact(p=None, held=E4M3, table=FAKE, table_stride=4, ctx=FAKE, keep=FAKE, S=2, kept=3):
    return LIB.cache_compact(held, p or pool(), table, table_stride, ctx, keep, S, kept, None)


@pytest.mark.parametrize("change,expect", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(layers=-1), INVALID),
    (dict(pages=-1), INVALID), (dict(page=-1), INVALID), (dict(row_bytes=-16), INVALID),
    (dict(row_bytes=24), UNSUPPORTED), (dict(layers=1 << 30), INVALID), (dict(heads=0), INVALID),
    (dict(heads=3), INVALID), (dict(heads=1 << 20), INVALID), (dict(heads=32), UNSUPPORTED), (dict(block=0), INVALID),
    (dict(block=5), INVALID), (dict(block=-8), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=FAKE + 2), INVALID),
    (dict(layers=(1 << 30) - 1), UNSUPPORTED), (dict(row_bytes=(1 << 30) - 64, layers=1 << 20), UNSUPPORTED)])
def test_moves_refuse_pools(change, expect):
    assert copy(pool(**change)) == expect and compact(pool(**change)) == expect


@pytest.mark.parametrize("heads,row", [(1, 144), (1, 4096), (1, 8192), (1, 1 << 20), (2, 1 << 16)])
def test_moves_refuse_heads_that_no_turn_of_threads_holds(heads, row):
    """Past 256 threads of 16 bytes to a head a workgroup would make no headway."""
    assert copy(pool(heads=heads, row_bytes=row)) == UNSUPPORTED
    for kept in (3, 100):
        assert compact(pool(heads=heads, row_bytes=row), kept=kept) == UNSUPPORTED


def test_moves_refuse_the_rest():
    assert copy(src=None) == INVALID and copy(dst=FAKE + 1) == INVALID and copy(count=-1) == INVALID
    assert copy(count=1 << 30) == UNSUPPORTED
    assert compact(table=None) == INVALID and compact(ctx=None) == INVALID and compact(keep=FAKE + 2) == INVALID
    assert compact(S=-1) == INVALID and compact(kept=-1) == INVALID and compact(table_stride=-1) == INVALID
    assert compact(S=1 << 30) == INVALID and compact(kept=1 << 30) == INVALID
    assert compact(held=AS_IS) == INVALID and compact(held=4) == INVALID
    assert LIB.cache_copy(None, FAKE, FAKE, 1, None) == INVALID
    assert LIB.cache_compact(E4M3, None, FAKE, 4, FAKE, FAKE, 2, 3, None) == INVALID


@pytest.mark.parametrize("call,held", [(c, h) for c in range(3) for h in (E4M3, INT8)])
def test_calls_that_no_launch_holds_are_refused(call, held):
    edge = 1 << 24
    # blocks of eight queries: ten queries have one number more than there are sequences
    calls = [(lambda n: tree(tshape(S=n, Hq=1, Hkv=1), held=held), edge - 2),
             (lambda n: copy(pool(layers=64), count=n), edge // 128 - 1),
             (lambda n: compact(S=n, held=held), edge - 1)]
    run, most = calls[call]
    assert run(most + 1) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert run(most) == HIP


def test_appends_that_no_launch_holds_are_refused():
    big = (1 << 30) - 1
    for held in (AS_IS, E4M3, INT8):
        w = ashape(T=big, Hq=64, Hkv=64, row_stride=64 * 64, page_stride=16 * 64 * 64)
        sc = None if held == AS_IS else scales(block_stride=64, page_stride=128)
        assert append(w, held=held, q=rows(64), q_out=rows(64), k=rows(64), v=rows(64), sc=sc) == UNSUPPORTED
    # two blocks of each sequence, head and pool, four to a workgroup
    assert append(ashape(S=big, Hq=0), held=E4M3) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert append(ashape(T=1 << 20)) == HIP and append(ashape(S=1 << 20, Hq=0), held=INT8) == HIP


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_report_hip_errors():
    assert append() == HIP and append(ashape(Hq=0)) == HIP and append(held=E4M3) == HIP and append(held=INT8) == HIP
    assert append(ashape(rotated=0), cos=None, sin=None) == HIP
    assert tree() == HIP and tree(held=INT8) == HIP and copy() == HIP and compact() == HIP and compact(held=INT8) == HIP
    assert sdl.lib().spmm_last_error() != b""


def test_binding_refuses_cpu_tensors_and_non_tensors():
    k = torch.zeros(4, 2, 64)
    rp = torch.tensor([0, 4], dtype=torch.int32)
    pages = torch.zeros(3, 16, 2, 64).to(torch.int8)
    sc = torch.ones(3, 2, 2)
    with pytest.raises(ValueError):
        sdl.append_pages(k, k, k[None], k[None], rp[None], rp[:1], rp)
    with pytest.raises(ValueError):
        sdl.tree_attention(k, pages, pages, rp[None], rp, rp, k_scale=sc, v_scale=sc)
    with pytest.raises(ValueError):
        sdl.copy_pages(pages[None], pages[None], rp, rp, k_scale=sc[None], v_scale=sc[None])
    with pytest.raises(ValueError):
        sdl.compact_pages(pages[None], pages[None], rp[None], rp, rp[None], k_scale=sc[None], v_scale=sc[None])
    with pytest.raises(TypeError):
        sdl.append_pages(1, k, k[None], k[None], rp[None], rp[:1], rp)


def test_scales_go_by_powers_of_two():
    """The reference's scale against its definition."""
    import math
    from cache_ref import MOST, scale_of_top
    for held, most in MOST.items():
        for top in [most * 2.0 ** e * f for e in range(-150, 119) for f in (0.51, 0.999, 1.0, 1.0001, 1.9)]:
            s = scale_of_top(top, held)
            assert math.frexp(s)[0] == 0.5 and top <= most * s and (s == 2.0 ** -126 or top > most * s / 2)
        assert scale_of_top(0.0, held) == 2.0 ** -126
