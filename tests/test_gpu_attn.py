"""Window attention, forward and backward, against its definition in 64 bits
(tests/attn_ref.py states the bounds)."""
import math
import random

import pytest
import torch

import sparse_dense_linear_amd as sdl
from attn_ref import assert_close, window_ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32 = torch.bfloat16, torch.float32


def starts(lengths, first=0):
    out = [first]
    for x in lengths:
        out.append(out[-1] + x)
    return out


def i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def operands(ql, kl, Hq, Hkv, D, dtype, seed=0, first=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    qs, ks = starts(ql, first), starts(kl, first)

    def normal(rows, heads):
        return torch.randn(rows + behind, heads, D, generator=g).to(dtype)

    return normal(qs[-1], Hq), normal(ks[-1], Hkv), normal(ks[-1], Hkv), normal(qs[-1], Hq), qs, ks


def check(ql, kl, Hq, Hkv, D, dtype, window, sinks, seed=0, scale=None, grad=True):
    q, k, v, do, qs, ks = operands(ql, kl, Hq, Hkv, D, dtype, seed)
    w = sdl.NO_WINDOW if window is None else window
    want = window_ref(q, k, v, qs, ks, w, sinks, scale, do if grad else None)
    a = dict(window=window, sinks=sinks, scale=scale)
    qc, kc, vc, dc = q.cuda(), k.cuda(), v.cuda(), do.cuda()
    o, lse = sdl.window_attention(qc, kc, vc, i32(qs), i32(ks), **a)
    torch.cuda.synchronize()
    assert o.dtype == dtype and lse.dtype == F32
    assert_close(o, want["o"], want["o_tol"], "o")
    assert_close(lse, want["lse"], want["lse_tol"], "lse")
    if not grad:
        return
    got = sdl.window_attention_backward(dc, qc, kc, vc, o, lse, i32(qs), i32(ks), **a)
    torch.cuda.synchronize()
    for n, x in zip(("dq", "dk", "dv"), got):
        assert x.dtype == dtype
        assert_close(x, want[n], want[n + "_tol"], n)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [8, 40, 64, 72, 128])
def test_head_sizes(dtype, D):
    check([150, 1, 33], [150, 1, 33], 4, 2, D, dtype, 40, 3, seed=D)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (31, 0), (32, 4), (33, 32), (64, 64),
                                          (100, 128), (None, 0), (None, 7), (300, 0), (200, 65)])
def test_windows(dtype, window, sinks):
    check([290, 70], [290, 70], 2, 1, 64, dtype, window, sinks, seed=1)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
def test_lengths(dtype, n):
    check([n], [n], 2, 2, 128, dtype, 50, 2, seed=n)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (3, 1), (8, 2), (12, 4)])
def test_shared_heads(dtype, Hq, Hkv):
    check([100, 41], [100, 41], Hq, Hkv, 64, dtype, 37, 2, seed=Hq)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("ql,kl", [
    ([1, 60, 129], [500, 60, 700]),          # queries are the last positions
    ([5, 0, 7], [5, 9, 0]),                  # no queries; no keys
    ([200, 3], [130, 2]),                    # more queries than keys: some see nothing
    ([0, 0], [3, 0]),                        # nothing at all
    ([40], [1500]),                          # every query past the window of the first keys
])
def test_pieces_and_empty_sequences(dtype, ql, kl):
    check(ql, kl, 4, 2, 64, dtype, 48, 3, seed=5)
    check(ql, kl, 4, 2, 128, dtype, None, 0, seed=6)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_many_far_runs(dtype):
    """First keys that several runs of queries past the window see."""
    check([1700, 600, 513], [1700, 600, 513], 2, 1, 64, dtype, 20, 33, seed=8)
    check([1100], [2100], 2, 2, 128, dtype, 100, 128, seed=9)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("window,sinks", [(None, 0), (300, 70), (100, 4)])
def test_few_key_tiles_are_taken_in_parts(dtype, D, window, sinks):
    """Many queries on few keys: what parts of the queries add to dk and dv is
    joined, with the far runs of first keys; a query that is no number reaches
    the keys it sees alone."""
    check([500, 130, 0, 1], [500, 130, 5, 1], 16, 2, D, dtype, window, sinks, seed=25)
    check([300, 20], [64, 700], 16, 1, D, dtype, window, sinks, seed=26)
    ql, at = [500, 130], 400
    q, k, v, do, qs, ks = operands(ql, ql, 16, 2, D, dtype, seed=27)
    w = sdl.NO_WINDOW if window is None else window
    do[at] = 0
    want = window_ref(q, k, v, qs, ks, w, sinks, None, do)
    q[at], do[at] = float("nan"), float("nan")
    a = dict(window=window, sinks=sinks)
    t = [x.cuda() for x in (q, k, v, do)]
    o, lse = sdl.window_attention(*t[:3], i32(qs), **a)
    first = sdl.window_attention_backward(t[3], *t[:3], o, lse, i32(qs), **a)
    again = sdl.window_attention_backward(t[3], *t[:3], o, lse, i32(qs), **a)
    for x, y in zip(first, again):
        assert torch.equal(torch.nan_to_num(x, nan=9.0), torch.nan_to_num(y, nan=9.0))
    sees = torch.tensor([j <= at and (at - j < w or j < sinks) for j in range(qs[-1])])
    for n, x in zip(("dk", "dv"), first[1:]):
        assert bool(torch.isnan(x.cpu()[sees]).all()), n
        assert_close(x.cpu()[~sees], want[n][~sees], want[n + "_tol"][~sees], n)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_parts_in_a_graph_into_slices(dtype):
    """The joined gradients as slices of one fused tensor with rows of no
    sequence around them, in a captured call whose lengths change between
    replays."""
    Hq, Hkv, D, ql = 16, 2, 72, [400, 150]
    q, k, v, do, qs, ks = operands(ql, ql, Hq, Hkv, D, dtype, seed=28, first=6, behind=9)
    a = dict(window=250, sinks=5)
    t = [x.cuda() for x in (q, k, v, do)]
    rp = i32(qs)
    fused = torch.full((q.shape[0], Hq + 2 * Hkv, D), 7.0, dtype=dtype, device="cuda")
    grads = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    o = torch.full_like(t[0], 7.0)
    lse = torch.zeros((Hq, q.shape[0]), device="cuda")

    def run():
        sdl.window_attn_fwd(*t[:3], rp, rp, o, lse, **a)
        sdl.window_attn_bwd(t[3], *t[:3], o, lse, rp, rp, *grads, **a)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lengths in (ql, [120, 430], [550, 0], ql):
        rows = starts(lengths, 6)
        want = window_ref(q, k, v, rows, rows, 250, 5, None, do)
        rp.copy_(i32(rows))
        fused.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for n, x in zip(("dq", "dk", "dv"), grads):
            assert_close(x[6:rows[-1]], want[n][6:rows[-1]], want[n + "_tol"][6:rows[-1]], n)
        assert bool((fused[:6] == 7.0).all()) and bool((fused[rows[-1]:] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(None, 0), (3000, 70), (700, 4)])
def test_long_walks_are_split_and_joined(dtype, window, sinks):
    """Few queries behind many keys, beside short sequences; what a masked
    place holds stays out of the joined results too."""
    check([300, 60], [5000, 60], 2, 1, 64, dtype, window, sinks, seed=24, grad=False)   # 128 to a workgroup
    ql, kl = [70, 1, 5, 0], [5000, 3000, 40, 7]                                         # 64
    check(ql, kl, 2, 1, 72, dtype, window, sinks, seed=22)
    q, k, v, do, qs, ks = operands(ql, kl, 2, 1, 128, dtype, seed=23)
    w = sdl.NO_WINDOW if window is None else window
    want = window_ref(q, k, v, qs, ks, w, sinks)
    k2, v2 = k.clone(), v.clone()
    k2[4990], v2[4990] = float("nan"), float("inf")    # queries 60 and later of the first sequence see it
    o, lse = sdl.window_attention(q.cuda(), k2.cuda(), v2.cuda(), i32(qs), i32(ks), window=window, sinks=sinks)
    keep = torch.tensor([i for i in range(qs[-1]) if not 60 <= i < 70])
    assert_close(o.cpu()[keep], want["o"][keep], want["o_tol"][keep], "o")
    assert_close(lse.cpu()[:, keep], want["lse"][:, keep], want["lse_tol"][:, keep], "lse")
    assert bool(torch.isnan(o[60:70]).all()) and bool(torch.isnan(lse[:, 60:70]).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D,window,sinks", [(64, 100, 70), (72, 33, 4), (128, None, 0), (128, 100, 70)])
def test_batches_that_fill_the_gpu(dtype, D, window, sinks):
    """Enough workgroups that walks stay whole, dq takes 128 queries at a time,
    and far runs are of 512: (Tq / 128 + S) Hq is at least 1024 and (Tk / 64 + S)
    Hkv at least 512."""
    r = random.Random(D)
    ql = [1300, 0, 570] + [r.choice([1, 2, 31, 33, 64, 65, 100, 130]) for _ in range(60)]
    kl = [n + r.choice([0, 0, 1, 50]) for n in ql]
    Hq, Hkv = 16, 8
    assert (sum(ql) // 128 + len(ql)) * Hq >= 1024 and (sum(kl) // 64 + len(kl)) * Hkv >= 512
    check(ql, kl, Hq, Hkv, D, dtype, window, sinks, seed=50)
    # a query that is no number, among those of the far runs: the first keys
    # it sees, and those of its window, and nothing else
    q, k, v, do, qs, ks = operands(ql, kl, Hq, Hkv, D, dtype, seed=51)
    at, w = 1250, sdl.NO_WINDOW if window is None else window
    do[at] = 0
    want = window_ref(q, k, v, qs, ks, w, sinks, None, do)
    q[at], do[at] = math.nan, math.nan
    t = [x.cuda() for x in (q, k, v, do)]
    a = dict(window=window, sinks=sinks)
    o, lse = sdl.window_attention(*t[:3], i32(qs), i32(ks), **a)
    got = [x.cpu() for x in sdl.window_attention_backward(t[3], *t[:3], o, lse, i32(qs), i32(ks), **a)]
    p = at + kl[0] - ql[0]
    sees = torch.tensor([j <= p and (p - j < w or j < sinks) for j in range(ks[-1])])
    others = torch.arange(qs[-1]) != at
    assert_close(o.cpu()[others], want["o"][others], want["o_tol"][others], "o")
    assert_close(got[0][others], want["dq"][others], want["dq_tol"][others], "dq")
    for n, x in zip(("dk", "dv"), got[1:]):
        assert bool(torch.isnan(x[sees]).all()), n
        assert_close(x[~sees], want[n][~sees], want[n + "_tol"][~sees], n)


def test_scale():
    check([90], [90], 2, 1, 64, F32, 33, 1, seed=2, scale=0.7)
    check([90], [90], 2, 1, 64, BF16, 33, 1, seed=2, scale=0.05)


def test_rows_of_no_sequence_are_left():
    """Rows before rowptr[0] and behind rowptr[S] are not written, and what
    they hold is not read."""
    ql = [50, 130]
    q, k, v, do, qs, ks = operands(ql, ql, 4, 2, 64, BF16, seed=3, first=9, behind=11)
    for t in (q, k, v, do):
        t[:9] = float("nan")
        t[qs[-1]:] = float("nan")
    want = window_ref(q, k, v, qs, ks, 40, 2, None, do)
    qc, kc, vc, dc = (t.cuda() for t in (q, k, v, do))
    o = torch.full_like(qc, 7.0)
    lse = torch.full((4, q.shape[0]), 7.0, device="cuda")
    a = dict(window=40, sinks=2)
    sdl.window_attn_fwd(qc, kc, vc, i32(qs), i32(ks), o, lse, **a)
    grads = [torch.full_like(t, 7.0) for t in (qc, kc, vc)]
    sdl.window_attn_bwd(dc, qc, kc, vc, o, lse, i32(qs), i32(ks), *grads, **a)
    torch.cuda.synchronize()
    inside = slice(9, qs[-1])
    for n, x in zip(("o", "dq", "dk", "dv"), [o] + grads):
        assert_close(x[inside], want[n][inside], want[n + "_tol"][inside], n)
        assert bool((x[:9] == 7.0).all()) and bool((x[qs[-1]:] == 7.0).all()), n
    assert_close(lse[:, inside], want["lse"][:, inside], want["lse_tol"][:, inside], "lse")
    assert bool((lse[:, :9] == 7.0).all()) and bool((lse[:, qs[-1]:] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_strides(dtype):
    """Slices of one fused tensor, heads-first layouts, a key head shared by a
    stride of zero, and strided outputs."""
    n, Hq, Hkv, D = 140, 4, 2, 64
    q, k, v, do, qs, ks = operands([n], [n], Hq, Hkv, D, dtype, seed=4)
    want = window_ref(q, k, v, qs, ks, 50, 3, None, do)
    fused = torch.cat([q, k, v], 1).cuda()
    qf, kf, vf = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    heads_first = do.permute(1, 0, 2).contiguous().cuda().permute(1, 0, 2)
    o = torch.empty((Hq, n, D), dtype=dtype, device="cuda").permute(1, 0, 2)
    lse = torch.empty((Hq, n), device="cuda")
    a = dict(window=50, sinks=3)
    sdl.window_attn_fwd(qf, kf, vf, i32(qs), i32(ks), o, lse, **a)
    dfused = torch.empty_like(fused)
    grads = dfused[:, :Hq], dfused[:, Hq:Hq + Hkv], dfused[:, Hq + Hkv:]
    sdl.window_attn_bwd(heads_first, qf, kf, vf, o, lse, i32(qs), i32(ks), *grads, **a)
    torch.cuda.synchronize()
    for name, x in zip(("o", "dq", "dk", "dv"), (o,) + grads):
        assert_close(x, want[name], want[name + "_tol"], name)

    one = k[:, :1].expand(n, Hkv, D)                   # one key head under two names
    want = window_ref(q, one, v, qs, ks, 50, 3)
    shared = k[:, :1].contiguous().cuda().expand(n, Hkv, D)
    o, lse = sdl.window_attention(q.cuda(), shared, v.cuda(), i32(qs), **a)
    assert_close(o, want["o"], want["o_tol"], "o")
    same = do[:1, :1].expand(n, Hq, D)                 # a broadcast gradient
    want = window_ref(q, k, v, qs, ks, 50, 3, None, same)
    o, lse = sdl.window_attention(q.cuda(), k.cuda(), v.cuda(), i32(qs), **a)
    got = sdl.window_attention_backward(do[:1, :1].cuda().expand(n, Hq, D), q.cuda(), k.cuda(), v.cuda(),
                                        o, lse, i32(qs), **a)
    for name, x in zip(("dq", "dk", "dv"), got):
        assert_close(x, want[name], want[name + "_tol"], name)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_masked_places_may_hold_anything(dtype, value):
    """Key 90's row of k and v is out of the window of queries 130 and later;
    queries before 90 do not reach it either.  What it holds changes no result
    of a query that does not see it, and no gradient of a pair without it."""
    n, w, s, at = 260, 40, 2, 90
    q, k, v, do, qs, ks = operands([n], [n], 2, 1, 64, dtype, seed=6)
    k[at], v[at] = value, value
    a = dict(window=w, sinks=s)
    blind = torch.tensor([i for i in range(n) if i < at or i - at >= w])
    clean_k, clean_v = k.clone(), v.clone()
    clean_k[at], clean_v[at] = 0, 0
    o, lse = sdl.window_attention(q.cuda(), k.cuda(), v.cuda(), i32(qs), **a)
    want = window_ref(q, clean_k, clean_v, qs, ks, w, s)
    assert_close(o.cpu()[blind], want["o"][blind], want["o_tol"][blind], "o")
    assert_close(lse.cpu()[:, blind], want["lse"][:, blind], want["lse_tol"][:, blind], "lse")

    # a query row whose q and do hold it: keys that it does not see keep
    # their gradients (their sums do not contain it)
    q, k, v, do, qs, ks = operands([n], [n], 2, 1, 64, dtype, seed=7)
    want = window_ref(q, k, v, qs, ks, w, s, None, do)
    row = 150
    q2, do2 = q.clone(), do.clone()
    q2[row], do2[row] = value, value
    o, lse = sdl.window_attention(q2.cuda(), k.cuda(), v.cuda(), i32(qs), **a)
    dq, dk, dv = sdl.window_attention_backward(do2.cuda(), q2.cuda(), k.cuda(), v.cuda(), o, lse, i32(qs), **a)
    unseen = torch.tensor([j for j in range(s, n) if j > row or row - j >= w])
    others = torch.tensor([i for i in range(n) if i != row])
    for name, x, keep in (("o", o, others), ("dq", dq, others), ("dk", dk, unseen), ("dv", dv, unseen)):
        assert_close(x.cpu()[keep], want[name][keep], want[name + "_tol"][keep], name)
    # and the far runs of the first keys: a row past the window sees key 0,
    # a row of another sequence does not
    q, k, v, do, qs, ks = operands([700, 300], [700, 300], 2, 1, 64, dtype, seed=8)
    want = window_ref(q, k, v, qs, ks, w, s, None, do)
    k2 = k.clone()
    k2[300] = value
    o, lse = sdl.window_attention(q.cuda(), k2.cuda(), v.cuda(), i32(qs), **a)
    got = sdl.window_attention_backward(do.cuda(), q.cuda(), k2.cuda(), v.cuda(), o, lse, i32(qs), **a)
    hit = set(range(300, 300 + w))
    keep = torch.tensor([i for i in range(1000) if i not in hit])
    assert_close(got[0].cpu()[keep], want["dq"][keep], want["dq_tol"][keep], "dq")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_seen_infinities_and_nan_go_where_arithmetic_sends_them(dtype):
    """An infinity or a NaN in a value reaches exactly the queries that see
    it; a key of -infinity scores nothing or everything by the query's sign."""
    n, w, s = 200, 40, 2
    q, k, v, do, qs, ks = operands([n], [n], 2, 1, 64, dtype, seed=9)
    v[50, 0, 3], v[60, 0, 5] = float("inf"), float("nan")
    o, _ = sdl.window_attention(q.cuda(), k.cuda(), v.cuda(), i32(qs), window=w, sinks=s)
    o = o.cpu()
    i = torch.arange(n)
    sees = lambda j: (i >= j) & (i - j < w)  # noqa: E731
    assert bool((torch.isposinf(o[:, 0, 3]) == sees(50)).all())
    assert bool((torch.isnan(o[:, 1, 5]) == sees(60)).all())
    assert bool(torch.isfinite(o[:, :, :3]).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [40, 64, 128])
def test_infinite_keys(dtype, D):
    """One element of a key is infinite: scores of the queries that see it are
    -infinity (weight 0) or infinity (no number), by the sign of the query;
    sizes of D that fill a tile and that do not."""
    n, w, s = 150, 40, 2
    for at in (60, 0):
        q, k, v, do, qs, ks = operands([n], [n], 2, 1, D, dtype, seed=20)
        k[at, 0, D - 1] = float("-inf")
        want = window_ref(q, k, v, qs, ks, w, s)
        o, lse = sdl.window_attention(q.cuda(), k.cuda(), v.cuda(), i32(qs), window=w, sinks=s)
        assert_close(o, want["o"], want["o_tol"], "o")
        assert_close(lse, want["lse"], want["lse_tol"], "lse")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [40, 128])
def test_a_lost_training_step(dtype, D):
    """Everything NaN, or one infinite value that every later query sees:
    the gradients say so, in ordinary time."""
    n = 3000
    q, k, v, do, qs, ks = operands([n], [n], 4, 2, D, dtype, seed=21)
    t = [x.cuda() for x in (q, k, v, do)]
    nan = [torch.full_like(x, float("nan")) for x in t]
    o, lse = sdl.window_attention(*nan[:3], i32(qs))
    out = (o, lse) + sdl.window_attention_backward(nan[3], *nan[:3], o, lse, i32(qs))
    assert all(bool(torch.isnan(x).all()) for x in out)
    t[2][0, 0, 1] = float("inf")
    o, lse = sdl.window_attention(*t[:3], i32(qs))
    assert bool(torch.isposinf(o[:, :2, 1]).all())
    assert bool(torch.isfinite(o[:, :2, 2:]).all()) and bool(torch.isfinite(o[:, 2:]).all())
    assert bool(torch.isfinite(lse).all())
    dq, dk, dv = sdl.window_attention_backward(t[3], *t[:3], o, lse, i32(qs))
    assert not bool(torch.isfinite(dq[:, :2]).all(dim=2).any()) and bool(torch.isfinite(dq[:, 2:]).all())
    assert bool(torch.isfinite(dv).all()) and bool(torch.isfinite(dk[:, 1]).all())


SIZES = pytest.mark.parametrize("D", [40, 64, 96, 128])
#: query heads on one key head: dk and dv of a key tile in one piece, and in parts
PARTS = pytest.mark.parametrize("Hq", [2, 16], ids=["whole", "parts"])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@SIZES
@PARTS
def test_scores_that_are_all_minus_infinity(dtype, D, Hq):
    """Queries 0 .. 30 see only keys whose scores are -infinity: their weights
    are no numbers, and so is all that takes part in them.  For the others
    those keys have weight 0, which leaves attention of queries 31 .. 63 over
    keys 95 .. 127."""
    c = 7
    q, k, v, do, qs, ks = operands([64], [128], Hq, 1, D, dtype, seed=40)
    q[:, :, c] = q[:, :, c].abs() + 0.5
    want = window_ref(q[31:], k[95:], v[95:], [0, 33], [0, 33], sdl.NO_WINDOW, 0, None, do[31:])
    k[:95, :, c] = -math.inf
    t = [x.cuda() for x in (q, k, v, do)]
    o, lse = sdl.window_attention(*t[:3], i32(qs), i32(ks))
    dq, dk, dv = (x.cpu() for x in sdl.window_attention_backward(t[3], *t[:3], o, lse, i32(qs), i32(ks)))
    o, lse = o.cpu(), lse.cpu()
    assert bool(torch.isneginf(lse[:, :31]).all())
    for name, x in (("o", o[:31]), ("dq", dq[:31]), ("dk", dk[:95]), ("dv", dv[:95])):
        assert bool(torch.isnan(x).all()), name
    assert bool(torch.isnan(dq[31:, :, c]).all())            # 0 times the infinite element
    assert_close(o[31:], want["o"], want["o_tol"], "o")
    assert_close(lse[:, 31:], want["lse"], want["lse_tol"], "lse")
    rest = [d for d in range(D) if d != c]
    assert_close(dq[31:][:, :, rest], want["dq"][:, :, rest], want["dq_tol"][:, :, rest], "dq")
    assert_close(dk[95:], want["dk"], want["dk_tol"], "dk")
    assert_close(dv[95:], want["dv"], want["dv_tol"], "dv")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@SIZES
@PARTS
@pytest.mark.parametrize("value", [math.nan, math.inf, 3e38])
def test_a_key_that_no_query_sees_has_no_gradient(dtype, D, Hq, value):
    """Key 352 is just behind the window of the first query, in the tiles of
    keys that are seen: whatever it holds, its gradients are zero and the others
    do not change.  (3e38: finite, but its products are not.)"""
    at, a = 352, dict(window=48, sinks=2)
    q, k, v, do, qs, ks = operands([100], [500], Hq, 1, D, dtype, seed=41)
    want = window_ref(q, k, v, qs, ks, 48, 2, None, do)
    k[at], v[at] = value, value
    t = [x.cuda() for x in (q, k, v, do)]
    o, lse = sdl.window_attention(*t[:3], i32(qs), i32(ks), **a)
    got = sdl.window_attention_backward(t[3], *t[:3], o, lse, i32(qs), i32(ks), **a)
    assert_close(o, want["o"], want["o_tol"], "o")
    assert_close(lse, want["lse"], want["lse_tol"], "lse")
    for name, x in zip(("dq", "dk", "dv"), got):
        assert_close(x, want[name], want[name + "_tol"], name)
    assert not bool(got[1][at].any()) and not bool(got[2][at].any())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@SIZES
@PARTS
def test_an_infinite_gradient_in_the_last_query(dtype, D, Hq):
    """The last query of a sequence whose length fills no tile has one
    infinite element of the incoming gradient: it reaches that element of dv of
    the keys that the query sees, the first keys among them, as an infinity, and
    no other element."""
    n, w, s, d = 300, 40, 3, 5
    q, k, v, do, qs, ks = operands([n, 20], [n, 20], Hq, 1, D, dtype, seed=42)
    do[n - 1, 0, d] = 0
    want = window_ref(q, k, v, qs, ks, w, s, None, do)
    do[n - 1, 0, d] = math.inf
    want["dv"][[j for j in range(n) if n - 1 - j < w or j < s], 0, d] = math.inf
    t = [x.cuda() for x in (q, k, v, do)]
    o, lse = sdl.window_attention(*t[:3], i32(qs), window=w, sinks=s)
    dv = sdl.window_attention_backward(t[3], *t[:3], o, lse, i32(qs), window=w, sinks=s)[2]
    assert_close(dv, want["dv"], want["dv_tol"], "dv")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@SIZES
@pytest.mark.parametrize("ql,kl", [([300, 40], [300, 40]), ([40, 3], [5000, 700])], ids=["whole", "split"])
def test_values_near_the_end_of_the_range(dtype, D, ql, kl):
    """Values of up to 2^126: their weighted mean is finite, their sum with
    weights that are not yet divided is not."""
    q, k, v, do, qs, ks = operands(ql, kl, 2, 1, D, dtype, seed=43)
    v[:, :, 3] = (v[:, :, 3].abs() + 1).clamp(max=3) * 2.0 ** 124
    want = window_ref(q, k, v, qs, ks, 2000, 2)
    o, lse = sdl.window_attention(q.cuda(), k.cuda(), v.cuda(), i32(qs), i32(ks), window=2000, sinks=2)
    assert_close(o, want["o"], want["o_tol"], "o")
    assert_close(lse, want["lse"], want["lse_tol"], "lse")


def test_large_scores():
    """Scores far apart: weights of exactly 0 and 1, no overflow."""
    n = 100
    for dtype in (F32, BF16):
        q, k, v, do, qs, ks = operands([n], [n], 1, 1, 64, dtype, seed=10)
        want = window_ref(q * 64, k * 64, v, qs, ks, 30, 2, None, do)
        q, k = (q * 64).cuda(), (k * 64).cuda()
        o, lse = sdl.window_attention(q, k, v.cuda(), i32(qs), window=30, sinks=2)
        assert_close(o, want["o"], want["o_tol"], "o")
        assert_close(lse, want["lse"], want["lse_tol"], "lse")


@pytest.mark.parametrize("which", [0, 1, 2])
def test_gradients_against_differences(which):
    """<gradient, direction> against central differences of the definition in
    64 bits.  The differences are off by h^2 / 6 times a third derivative,
    which for unit-scale operands and h = 1e-3 stays below 1e-4 of the sum of
    magnitudes; the gradient is off by its bound."""
    q, k, v, do, qs, ks = operands([70, 33], [70, 40], 4, 2, 64, F32, seed=11)
    a = dict(window=30, sinks=3)
    o, lse = sdl.window_attention(q.cuda(), k.cuda(), v.cuda(), i32(qs), i32(ks), **a)
    got = sdl.window_attention_backward(do.cuda(), q.cuda(), k.cuda(), v.cuda(), o, lse, i32(qs), i32(ks), **a)
    want = window_ref(q, k, v, qs, ks, 30, 3, None, do)
    name = ("dq", "dk", "dv")[which]
    x = [t.double() for t in (q, k, v)]
    u = torch.randn(x[which].shape, generator=torch.Generator().manual_seed(12), dtype=torch.float64)
    h = 1e-3

    def loss(sign):
        y = list(x)
        y[which] = y[which] + sign * h * u
        return (window_ref(*y, qs, ks, 30, 3)["o"] * do.double()).sum()

    slope = float(loss(1) - loss(-1)) / (2 * h)
    along = float((got[which].cpu().double() * u).sum())
    bound = float((want[name + "_tol"] * u.abs()).sum()) + 1e-4 * float((want[name] * u).abs().sum())
    assert abs(along - slope) <= bound


def test_same_as_the_products_on_the_pattern():
    """The library's own SDDMM and SpMM on the window's CSR pattern, with a
    softmax between them."""
    n, w, s, D = 300, 25, 2, 64
    q, k, v, _, qs, ks = operands([n], [n], 1, 1, D, F32, seed=13)
    rows = [[j for j in range(i + 1) if i - j < w or j < s] for i in range(n)]
    rowptr = i32(starts([len(r) for r in rows]))
    colind = i32([j for r in rows for j in r])
    qc, kc, vc = (t[:, 0].contiguous().cuda() for t in (q, k, v))
    x = sdl.sddmm(rowptr, colind, qc, kc) / math.sqrt(D)
    of = torch.repeat_interleave(torch.arange(n), torch.tensor([len(r) for r in rows])).cuda()
    top = torch.full((n,), -math.inf, device="cuda").scatter_reduce(0, of, x, "amax")
    e = torch.exp(x - top[of])
    p = e / torch.zeros(n, device="cuda").index_add_(0, of, e)[of]
    o, _ = sdl.window_attention(q.cuda(), k.cuda(), v.cuda(), i32(qs), window=w, sinks=s)
    want = window_ref(q, k, v, qs, ks, w, s)
    assert_close(sdl.spmm(rowptr, colind, p, vc), want["o"][:, 0], 2 * want["o_tol"][:, 0], "products")
    assert_close(o, want["o"], want["o_tol"], "o")


def test_repeats_bit_for_bit():
    q, k, v, do, qs, ks = operands([900, 300], [900, 300], 8, 2, 128, BF16, seed=14)
    a = dict(window=100, sinks=4)
    t = [x.cuda() for x in (q, k, v, do)]
    first = None
    for _ in range(3):
        o, lse = sdl.window_attention(*t[:3], i32(qs), **a)
        out = (o, lse) + sdl.window_attention_backward(t[3], *t[:3], o, lse, i32(qs), **a)
        if first is not None:
            assert all(torch.equal(x, y) for x, y in zip(first, out))
        first = out


def test_streams_and_graphs():
    """Calls on two streams at once, and two captured steps replayed several
    times with eager work between, all equal to the eager results."""
    a = dict(window=60, sinks=3)
    sets = []
    for seed, n in ((15, 400), (16, 333)):
        q, k, v, do, qs, ks = operands([n, 50], [n, 50], 4, 2, 64, BF16, seed=seed)
        sets.append([x.cuda() for x in (q, k, v, do)] + [i32(qs)])

    def step(q, k, v, do, rp, stream=None):
        o, lse = sdl.window_attention(q, k, v, rp, stream=stream, **a)
        return (o, lse) + sdl.window_attention_backward(do, q, k, v, o, lse, rp, stream=stream, **a)

    eager = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            got[i].append(step(*sets[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(out, eager[i]))

    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*s))
        graphs.append(g)
    for _ in range(4):
        for out in outs:
            for x in out:
                x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graphs[0].replay()
        with torch.cuda.stream(streams[1]):
            graphs[1].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(x, y) for x, y in zip(outs[i], eager[i]))
        again = step(*sets[0])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(again, eager[0]))


def test_offsets_past_32_bits():
    """A token stride that puts the second sequence's rows more than 2^32
    elements behind the first's."""
    n, D = 40, 64
    stride = (1 << 32) // 60 + 8 & ~7
    rows = 2 * n
    if torch.cuda.mem_get_info()[0] < 3 * rows * stride * 2:
        pytest.skip("needs 35 GB")
    q, k, v, do, qs, ks = operands([n, n], [n, n], 1, 1, D, BF16, seed=17)
    big = torch.empty(rows * stride, dtype=BF16, device="cuda")
    views = []
    for i, t in enumerate((q, k, v, do)):
        x = torch.as_strided(big, (rows, 1, D), (stride, D, 1), i * D)
        x.copy_(t.cuda())
        views.append(x)
    a = dict(window=20, sinks=2)
    want = window_ref(q, k, v, qs, ks, 20, 2, None, do)
    o, lse = sdl.window_attention(*views[:3], i32(qs), **a)
    dq, dk, dv = sdl.window_attention_backward(views[3], *views[:3], o, lse, i32(qs), **a)
    for name, x in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert_close(x, want[name], want[name + "_tol"], name)


def test_binding_refusals():
    """Arguments that the binding turns away before the library sees them."""
    q = torch.zeros(10, 4, 64, device="cuda")
    k = torch.zeros(10, 2, 64, device="cuda")
    rp = i32([0, 10])
    ok = dict(q=q, k=k, v=k, q_rowptr=rp)

    def bad(error, **change):
        with pytest.raises(error):
            sdl.window_attention(**(ok | change))

    bad(TypeError, q=q.half(), k=k.half(), v=k.half())
    bad(TypeError, k=k.bfloat16())
    bad(TypeError, q_rowptr=rp.long())
    bad(ValueError, q=q[0])
    bad(ValueError, k=k[:, :, :32], v=k[:, :, :32])
    bad(ValueError, v=k[:5])
    bad(ValueError, k=k.cpu())
    bad(ValueError, q_rowptr=rp[:0])
    bad(ValueError, q=torch.zeros(10, 64, 4, device="cuda").transpose(1, 2))
    bad(ValueError, k_rowptr=i32([0, 5, 10]))
    bad(sdl.SpmmError, q=q[:, :3])                       # 3 heads on 2
    bad(sdl.SpmmError, q=q[:, :, :60], k=k[:, :, :60], v=k[:, :, :60])
    bad(sdl.SpmmError, q=torch.zeros(10, 4, 66, device="cuda")[:, :, :64])   # strides
    bad(sdl.SpmmError, window=0)
    bad(TypeError, window=2.5)
    bad(TypeError, sinks=1.0)
    bad(sdl.SpmmError, sinks=200)
    bad(sdl.SpmmError, scale=-1.0)
    o, lse = sdl.window_attention(**ok)
    with pytest.raises(ValueError):
        sdl.window_attention_backward(q, q, k, k, o, lse.t(), rp)
    with pytest.raises(TypeError):
        sdl.window_attention_backward(q, q, k, k, o.bfloat16(), lse, rp)
    with pytest.raises(ValueError):
        sdl.window_attention_backward(q[:, :2], q, k, k, o, lse, rp)


def test_outputs_over_inputs_are_refused():
    """Results written over what is still to be read."""
    q, k, v, do = (torch.randn(40, h, 64, device="cuda") for h in (4, 2, 2, 4))
    rp = i32([0, 40])
    o, lse = sdl.window_attention(q, k, v, rp)
    for t in (q, torch.cat([q, k], 1)[:, :4]):
        with pytest.raises(ValueError, match="o must not overlap q"):
            sdl.window_attn_fwd(t, k, v, rp, rp, t, lse)
    grads = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
    for name, over in (("dq", q), ("dq", do), ("dq", o), ("dk", k), ("dk", v), ("dv", v), ("dk", grads["dv"])):
        with pytest.raises(ValueError, match="must not overlap"):
            sdl.window_attn_bwd(do, q, k, v, o, lse, rp, rp, **(grads | {name: over}))
    same = sdl.window_attention(q, k, k, rp)[0]          # inputs may be one tensor
    assert torch.equal(same, sdl.window_attention(q, k, k.clone(), rp)[0])
    pool, table, ctx = k[:32].view(2, 16, 2, 64), i32([[0, 1]]), i32([20])
    with pytest.raises(ValueError, match="o must not overlap q"):
        sdl.tree_attn_paged(q[:1], pool, pool, table, ctx, i32([0, 1]), None, q[:1], lse[:, :1].contiguous())


def test_numbers_past_64_bits():
    """A window of any size is taken for what it is, and so is a count of first
    keys: refused."""
    q, k = torch.randn(40, 2, 64, device="cuda"), torch.randn(40, 2, 64, device="cuda")
    rp = i32([0, 40])
    want = sdl.window_attention(q, k, k, rp)[0]
    pool, table, ctx = k[:32].view(2, 16, 2, 64), i32([[0, 1]]), i32([20])
    answer = sdl.tree_attention(q[:1], pool, pool, table, ctx, i32([0, 1]))[0]
    for window in ((1 << 62) + 1, (1 << 63) + 5, (1 << 64) + 1, 1 << 100):
        assert torch.equal(sdl.window_attention(q, k, k, rp, window=window)[0], want)
        assert torch.equal(sdl.tree_attention(q[:1], pool, pool, table, ctx, i32([0, 1]), window=window)[0], answer)
    for bad in (dict(window=-(1 << 64) + 1), dict(sinks=1 << 64), dict(sinks=(1 << 64) + 3), dict(sinks=-(1 << 64))):
        with pytest.raises(sdl.SpmmError):
            sdl.window_attention(q, k, k, rp, **bad)
        with pytest.raises(sdl.SpmmError):
            sdl.tree_attention(q[:1], pool, pool, table, ctx, i32([0, 1]), **bad)
