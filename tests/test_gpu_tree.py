"""Attention of drafted tokens over a paged cache, and the moves of its
pages, against their definitions in 64 bits (tests/attn_ref.py states the
bounds)."""
import math
import random

import pytest
import torch

import sparse_dense_linear_amd as sdl
from attn_ref import assert_close, chain_seen, head_forward, tree_seen, window_ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32 = torch.bfloat16, torch.float32
BOTH = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def i64(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64).cuda()


def starts(lengths, first=0):
    out = [first]
    for x in lengths:
        out.append(out[-1] + x)
    return out


def random_tree(T, r):
    m = []
    for a in range(T):
        parent = r.randint(max(-1, a - 7), a - 1) if a else -1
        m.append((m[parent] if parent >= 0 else 0) | 1 << a)
    return m


class Cache:
    """A paged cache whose unused rows and pages hold NaN, with page numbers
    in random order; table entries of pages that nothing sees are nonsense."""

    def __init__(self, lengths, page, Hkv, D, dtype, seed, dead=()):
        r, g = random.Random(seed), torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        pool = sum(need) + 2
        order = list(range(pool))
        r.shuffle(order)
        self.k = torch.full((pool, page, Hkv, D), float("nan")).to(dtype)
        self.v = self.k.clone()
        self.rows_k = [torch.randn(n, Hkv, D, generator=g).to(dtype) for n in lengths]
        self.rows_v = [torch.randn(n, Hkv, D, generator=g).to(dtype) for n in lengths]
        self.table, at = [], 0
        wide = max(need + [1])
        for s, n in enumerate(lengths):
            mine = order[at:at + need[s]]
            at += need[s]
            for p, number in enumerate(mine):
                rows = slice(p * page, min(n, (p + 1) * page))
                self.k[number, :rows.stop - rows.start] = self.rows_k[s][rows]
                self.v[number, :rows.stop - rows.start] = self.rows_v[s][rows]
            self.table.append(mine + [-1000000] * (wide - need[s]))
        for s, p in dead:
            number = self.table[s][p]
            self.k[number] = self.v[number] = float("nan")
            self.table[s][p] = -1000000

    def on_gpu(self):
        return self.k.cuda(), self.v.cuda(), i32(self.table)


def check(ctx, drafts, Hq, Hkv, D, dtype, page, window, sinks, masks="tree", seed=0, dead=(), scale=None):
    r = random.Random(seed)
    cache = Cache([c + t for c, t in zip(ctx, drafts)], page, Hkv, D, dtype, seed, dead)
    q = torch.randn(sum(drafts), Hq, D, generator=torch.Generator().manual_seed(seed + 1)).to(dtype)
    qs = starts(drafts)
    if masks == "tree":
        masks = [random_tree(t, r) for t in drafts]
    w = sdl.NO_WINDOW if window is None else window
    k, v, table = cache.on_gpu()
    tree = None if masks is None else i64([m for x in masks for m in x])
    o, lse = sdl.tree_attention(q.cuda(), k, v, table, i32(ctx), i32(qs), tree, window=window, sinks=sinks,
                                scale=scale)
    torch.cuda.synchronize()
    assert o.dtype == dtype and lse.dtype == F32
    sc = 1 / math.sqrt(D) if scale is None else scale
    want = {n: torch.zeros(q.shape, dtype=torch.float64) for n in ("o", "o_tol")}
    want |= {n: torch.zeros((Hq, q.shape[0]), dtype=torch.float64) for n in ("lse", "lse_tol")}
    for s in range(len(ctx)):
        a = slice(qs[s], qs[s + 1])
        seen = chain_seen(ctx[s], drafts[s], w, sinks) if masks is None else tree_seen(ctx[s], masks[s], w, sinks)
        for h in range(Hq):
            f = head_forward(q[a, h].double(), cache.rows_k[s][:, h * Hkv // Hq].double(),
                             cache.rows_v[s][:, h * Hkv // Hq].double(), seen, sc, dtype)
            want["o"][a, h], want["o_tol"][a, h] = f["o"], f["o_tol"]
            want["lse"][h, a], want["lse_tol"][h, a] = f["lse"], f["lse_tol"]
    # the joining of partial results rounds once more for each of them: a
    # factor 2 on the fp32 part covers up to as many parts as keys
    assert_close(o, want["o"], 2 * want["o_tol"], "o")
    assert_close(lse, want["lse"], 2 * want["lse_tol"], "lse")


@BOTH
@pytest.mark.parametrize("page", [1, 7, 16, 24, 64, 128, 300])
def test_pages(dtype, page):
    check([0, 1, 200, 515], [3, 1, 9, 2], 4, 2, 64, dtype, page, None, 0, seed=page)


@BOTH
@pytest.mark.parametrize("D", [8, 40, 64, 96, 128])
def test_head_sizes(dtype, D):
    check([130, 0, 33], [5, 2, 1], 4, 4, D, dtype, 16, 60, 3, seed=D)


@BOTH
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (40, 4), (129, 128), (500, 17), (None, 5)])
def test_windows(dtype, window, sinks):
    check([700, 260, 20], [12, 33, 4], 2, 1, 64, dtype, 16, window, sinks, seed=3)


@BOTH
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (6, 2), (8, 1), (16, 1), (40, 1)])
@pytest.mark.parametrize("drafts", [[1, 1], [3, 17], [64, 40]])
def test_shared_heads(dtype, Hq, Hkv, drafts):
    """From one column of a matrix to many blocks of them."""
    check([300, 77], drafts, Hq, Hkv, 64, dtype, 32, 200, 2, seed=Hq)


@BOTH
def test_chains(dtype):
    """No masks: causal pieces, of any length."""
    check([300, 0, 64], [1, 130, 65], 4, 2, 64, dtype, 16, None, 0, masks=None, seed=4)
    check([300, 0, 640], [1, 130, 65], 4, 1, 128, dtype, 16, 70, 3, masks=None, seed=5)


@BOTH
def test_masks_that_see_nothing_or_anything(dtype):
    """Rows that see no draft, and none of the cache; drafts that see later
    ones; bits past the drafts; drafts past the 64th."""
    check([0, 0, 9], [2, 3, 2], 2, 1, 64, dtype, 8, None, 0, seed=6,
          masks=[[0, 2], [0, 0, 0], [0, (1 << 64) - 1]])
    check([5, 300], [3, 70], 2, 1, 64, dtype, 8, 4, 0, seed=7,
          masks=[[0b111, 0b100, 0], [(0x9E3779B97F4A7C15 * (i + 1)) & (1 << 64) - 1 for i in range(70)]])
    check([50], [4], 2, 1, 64, dtype, 8, 1, 0, seed=8, masks=[[0, 1, 3, 8]])


@BOTH
def test_long_contexts_are_split_and_joined(dtype):
    check([20000], [1], 2, 1, 128, dtype, 16, None, 0, seed=9)
    check([9000, 3, 5000], [2, 40, 1], 8, 2, 64, dtype, 64, None, 0, seed=10)
    check([9000, 3, 5000], [2, 40, 1], 8, 2, 64, dtype, 64, 3000, 4, seed=11)


@BOTH
def test_many_sequences(dtype):
    """More sequences than a workgroup has threads, empty ones among them."""
    r = random.Random(12)
    n = 300
    ctx = [r.choice([0, 1, 15, 16, 17, 120]) for _ in range(n)]
    drafts = [r.choice([0, 1, 1, 1, 2]) for _ in range(n)]
    check(ctx, drafts, 2, 1, 64, dtype, 16, None, 0, seed=12)


@BOTH
def test_pages_that_nothing_sees_are_not_read(dtype):
    """Pages behind the window have been given away: their numbers in the
    table are nonsense.  The first draft stands at ctx, so keys up to ctx -
    window are behind it."""
    page, ctx, window, sinks = 16, 500, 100, 4
    dead = [(0, p) for p in range(1, (ctx - window + 1) // page)]
    check([ctx], [5], 4, 2, 64, dtype, page, window, sinks, seed=13, dead=dead)
    check([ctx], [5], 4, 2, 64, dtype, page, window, 0, seed=13, dead=dead + [(0, 0)])
    check([ctx], [3], 4, 2, 64, dtype, page, window, sinks, seed=13, dead=dead, masks=[[0, 1, 2]])


@BOTH
def test_masked_places_may_hold_anything(dtype):
    """Infinities and NaN in a draft's row reach only the drafts that see it."""
    page, ctx, T = 16, 300, 5
    cache = Cache([ctx + T], page, 1, 64, dtype, 14)
    q = torch.randn(T, 4, 64, generator=torch.Generator().manual_seed(15)).to(dtype)
    masks = [[1, 3, 5, 9, 19]]                       # draft 2 is seen by itself alone
    k, v, table = cache.on_gpu()
    clean, clean_lse = sdl.tree_attention(q.cuda(), k, v, table, i32([ctx]), i32([0, T]), i64(masks[0]))
    for value in (float("inf"), float("-inf"), float("nan")):
        number, row = cache.table[0][(ctx + 2) // page], (ctx + 2) % page
        k2, v2 = k.clone(), v.clone()
        k2[number, row], v2[number, row] = value, value
        o, lse = sdl.tree_attention(q.cuda(), k2, v2, table, i32([ctx]), i32([0, T]), i64(masks[0]))
        keep = [0, 1, 3, 4]
        # the same sums in another order: twice the bound of either
        tol = 8 * torch.finfo(dtype).eps
        assert bool(((o[keep] - clean[keep]).abs() <= tol * (1 + clean[keep].abs())).all())
        assert torch.equal(lse[:, keep].isfinite(), clean_lse[:, keep].isfinite())
        assert bool(((lse[:, keep] - clean_lse[:, keep]).abs() <= 1e-4).all())
        assert not bool(torch.isfinite(o[2]).all())


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("drafts", [1, 40])
def test_an_infinite_value_beside_masked_keys(dtype, D, drafts):
    """The last first key, and the first and last key of the window, hold an
    infinite value: its element of the output is infinite for the drafts that
    see it, and no masked key of the same tile makes it no number."""
    ctx, window, sinks, page, d = 700, 41, 3, 16, 5
    for at in (sinks - 1, ctx + drafts - window, ctx + drafts - 1):
        cache = Cache([ctx + drafts], page, 1, D, dtype, 31)
        cache.rows_v[0][at, 0, d] = float("inf")
        cache.v[cache.table[0][at // page], at % page, 0, d] = float("inf")
        q = torch.randn(drafts, 4, D, generator=torch.Generator().manual_seed(32)).to(dtype)
        k, v, table = cache.on_gpu()
        o, lse = sdl.tree_attention(q.cuda(), k, v, table, i32([ctx]), i32([0, drafts]), window=window, sinks=sinks)
        seen = chain_seen(ctx, drafts, window, sinks)
        sees = seen[:, at]
        finite = cache.rows_v[0][:, 0].double()
        finite[at, d] = 0
        for h in range(4):
            f = head_forward(q[:, h].double(), cache.rows_k[0][:, 0].double(), finite, seen, D ** -0.5, dtype)
            f["o"][sees, d] = float("inf")
            assert_close(o[:, h], f["o"], 2 * f["o_tol"], f"o, key {at}")
            assert_close(lse[h], f["lse"], 2 * f["lse_tol"], "lse")


@BOTH
def test_pages_that_no_mask_names_are_not_read(dtype):
    """Pages that no draft sees hold nonsense in the table, whatever the reason."""
    # both drafts stand at ctx + 1: key ctx - window + 1, the last of page 24, is behind them
    dead = [(0, p) for p in range(1, 25)]
    check([500], [2], 4, 2, 64, dtype, 16, 102, 4, seed=35, dead=dead, masks=[[3, 3]])
    check([500], [2], 4, 2, 64, dtype, 16, 102, 0, seed=35, dead=dead + [(0, 0)], masks=[[3, 3]])
    # drafts past the 64th are seen by none
    bits = [(0x9E3779B97F4A7C15 * (i + 1)) & (1 << 64) - 1 for i in range(150)]
    check([60], [150], 2, 1, 64, dtype, 16, None, 0, seed=36, dead=[(0, p) for p in range(8, 14)], masks=[bits])
    # drafts that no mask names
    check([64, 30], [40, 3], 2, 1, 128, dtype, 16, None, 0, seed=37, dead=[(0, 5), (0, 6)],
          masks=[[b & 0xffff for b in bits[:40]], [1, 3, 7]])
    # named drafts that the window hides: the last one stands 39 behind them
    check([64], [40], 2, 1, 64, dtype, 16, 2, 0, seed=38, dead=[(0, p) for p in (0, 1, 2, 4, 5)],
          masks=[[0] * 39 + [(1 << 40) - 1]])
    # nothing is seen
    check([100, 20], [3, 1], 2, 1, 64, dtype, 16, 1, 0, seed=39, dead=[(0, p) for p in range(7)],
          masks=[[0, 0, 0], [1]])


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,drafts", [(700, 1), (700, 40), (20000, 2)])
def test_values_near_the_end_of_the_range(dtype, D, ctx, drafts):
    """Values of up to 2^126: their weighted mean is finite, their sum with
    weights that are not yet divided is not."""
    cache = Cache([ctx + drafts], 16, 1, D, dtype, 33)
    for row in [cache.rows_v[0]] + list(cache.v):
        row[..., 3] = (row[..., 3].abs() + 1).clamp(max=3) * 2.0 ** 124
    q = torch.randn(drafts, 4, D, generator=torch.Generator().manual_seed(34)).to(dtype)
    k, v, table = cache.on_gpu()
    o, lse = sdl.tree_attention(q.cuda(), k, v, table, i32([ctx]), i32([0, drafts]), window=15000, sinks=2)
    seen = chain_seen(ctx, drafts, 15000, 2)
    for h in range(4):
        f = head_forward(q[:, h].double(), cache.rows_k[0][:, 0].double(), cache.rows_v[0][:, 0].double(), seen,
                         D ** -0.5, dtype)
        assert_close(o[:, h], f["o"], 2 * f["o_tol"], "o")
        assert_close(lse[h], f["lse"], 2 * f["lse_tol"], "lse")


def test_strided_pools_and_queries():
    """Pools that are one layer of a larger tensor, queries cut from a fused
    tensor."""
    for dtype in (F32, BF16):
        cache = Cache([90, 31], 16, 2, 64, dtype, 16)
        pools = torch.stack([cache.k, cache.v], 2).cuda()      # [pages, page, 2, Hkv, D]
        q = torch.randn(4, 6, 64, generator=torch.Generator().manual_seed(17)).to(dtype)
        fused = torch.cat([torch.zeros(4, 2, 64, dtype=dtype), q], 1).cuda()
        ctx, rp = i32([87, 30]), i32([0, 3, 4])
        a = (i32(cache.table), ctx, rp)
        o, lse = sdl.tree_attention(q[:, :4].contiguous().cuda(), cache.k.cuda(), cache.v.cuda(), *a)
        o2, lse2 = sdl.tree_attention(fused[:, 2:6], pools[:, :, 0], pools[:, :, 1], *a)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_rows_of_no_sequence_are_left():
    cache = Cache([90, 31], 16, 2, 64, F32, 18)
    q = torch.full((12, 4, 64), float("nan"), device="cuda")
    q[3:7] = torch.randn(4, 4, 64, device="cuda")
    o = torch.full_like(q, 7.0)
    lse = torch.full((4, 12), 7.0, device="cuda")
    k, v, table = cache.on_gpu()
    sdl.tree_attn_paged(q, k, v, table, i32([87, 30]), i32([3, 6, 7]), None, o, lse)
    torch.cuda.synchronize()
    assert bool((o[:3] == 7).all()) and bool((o[7:] == 7).all())
    assert bool((lse[:, :3] == 7).all()) and bool((lse[:, 7:] == 7).all())
    assert bool(torch.isfinite(o[3:7]).all()) and not bool((o[3:7] == 7).all(dim=2).any())


def test_repeats_streams_and_graphs():
    sets = []
    for seed in (19, 20):
        cache = Cache([3000, 700, 20], 16, 2, 128, BF16, seed)
        q = torch.randn(9, 8, 128, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()
        sets.append((q, *cache.on_gpu(), i32([2996, 697, 18]), i32([0, 4, 7, 9])))
    eager = [sdl.tree_attention(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(i, sdl.tree_attention(*sets[i], stream=streams[i])) for _ in range(4) for i in (0, 1)]
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, eager[i]))
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sdl.tree_attention(*s))
        graphs.append(g)
    for _ in range(4):
        for out in outs:
            for x in out:
                x.zero_()
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(x, y) for x, y in zip(outs[i], eager[i]))
        assert torch.equal(sdl.tree_attention(*sets[0])[0], eager[0][0])
        torch.cuda.synchronize()


def test_lengths_that_grow_under_a_captured_call():
    """One captured call serves the sequences as they grow: lengths are read
    on the device."""
    cache = Cache([400, 60], 16, 1, 64, F32, 21)
    k, v, table = cache.on_gpu()
    q = torch.randn(2, 2, 64, device="cuda")
    ctx, rp = i32([0, 0]), i32([0, 1, 2])
    sdl.tree_attention(q, k, v, table, ctx, rp)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sdl.tree_attention(q, k, v, table, ctx, rp)
    for c in ([0, 0], [17, 3], [130, 59], [399, 40]):
        ctx.copy_(i32(c))
        g.replay()
        torch.cuda.synchronize()
        want = sdl.tree_attention(q, k, v, table, i32(c), rp)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_pool_past_32_bits():
    """Pages whose first element lies past 2^32."""
    page, D = 64, 128
    pages = (1 << 32) // (page * D) + 10
    if torch.cuda.mem_get_info()[0] < 2 * pages * page * D * 2 + (4 << 30):
        pytest.skip("needs 21 GB")
    cache = Cache([200], page, 1, D, BF16, 22)
    q = torch.randn(2, 4, D, generator=torch.Generator().manual_seed(23)).to(BF16).cuda()
    k, v, table = cache.on_gpu()
    want = sdl.tree_attention(q, k, v, table, i32([198]), i32([0, 2]))
    big_k = torch.empty((pages, page, 1, D), dtype=BF16, device="cuda")
    big_v = torch.empty_like(big_k)
    moved = [pages - 1 - 2 * i for i in range(table.shape[1])]
    for p, number in enumerate(moved):
        big_k[number], big_v[number] = k[table[0, p]], v[table[0, p]]
    got = sdl.tree_attention(q, big_k, big_v, i32([moved]), i32([198]), i32([0, 2]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # and the moves
    sdl.copy_pages(big_k[None], big_v[None], i32([moved[0]]), i32([pages - 8]))
    assert torch.equal(big_k[pages - 8], big_k[moved[0]])
    rows = big_k[moved[3]].clone()
    sdl.compact_pages(big_k[None], big_v[None], i32([moved]), i32([192]), i32([[1, 5]]))
    assert torch.equal(big_k[moved[3], 0], rows[1]) and torch.equal(big_k[moved[3], 1], rows[5])


# ------------------------------------------------------------------ pages

@pytest.mark.parametrize("dtype", [F32, BF16, torch.uint8])
@pytest.mark.parametrize("layers,pages,page,row", [(1, 3, 1, (16,)), (3, 20, 16, (2, 64)), (2, 9, 24, (3, 48)),
                                                   (2, 5, 700, (1, 80))])
def test_copy_pages(dtype, layers, pages, page, row):
    g = torch.Generator().manual_seed(pages)
    k = torch.randint(0, 200, (layers, pages, page) + row, generator=g).to(dtype)
    v = torch.randint(0, 200, (layers, pages, page) + row, generator=g).to(dtype)
    src = [0, 1, -1, 0, pages, 1, -1][:pages + 2]
    dst = [2, -1, 0, pages - 1 if pages > 3 else -1, 1, 2 ** 31 - 1, -1][:pages + 2]
    want_k, want_v = k.clone(), v.clone()
    for a, b in zip(src, dst):
        if 0 <= a < pages and 0 <= b < pages:
            want_k[:, b], want_v[:, b] = k[:, a], v[:, a]
    kc, vc = k.cuda(), v.cuda()
    sdl.copy_pages(kc, vc, i32(src), i32(dst))
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v)
    sdl.copy_pages(kc, vc, i32([]), i32([]))
    assert torch.equal(kc.cpu(), want_k)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_compact_pages(dtype, page):
    """Kept drafts within a page, across pages, from page to page; none kept,
    all kept; lists longer than a batch of rows; tables that end early."""
    r = random.Random(page)
    layers, Hkv, D = 3, 2, 24
    ctx = [0, 3, page, 7, 2 * page - 1, 5]
    drafts = [20, 33, 8, 1, 64, 12]
    keep = [[0, 3, 4, 9], [1, 2, 32], [], [0], sorted(r.sample(range(64), 20)), list(range(12))]
    keep[2] = list(range(2, 8))
    n = [-(-(c + t) // page) for c, t in zip(ctx, drafts)]
    wide, pages = max(n), sum(n) + 1
    order = list(range(pages))
    r.shuffle(order)
    table, at = [], 0
    for x in n:
        table.append(order[at:at + x] + [-1] * (wide - x))
        at += x
    g = torch.Generator().manual_seed(page)
    k = torch.randn(layers, pages, page, Hkv, D, generator=g).to(dtype)
    v = torch.randn(layers, pages, page, Hkv, D, generator=g).to(dtype)
    want_k, want_v = k.clone(), v.clone()
    for s in range(len(ctx)):
        for t, a in enumerate(keep[s]):
            f, to = ctx[s] + a, ctx[s] + t
            for x, y in ((k, want_k), (v, want_v)):
                y[:, table[s][to // page], to % page] = x[:, table[s][f // page], f % page]
    longest = max(len(x) for x in keep)
    kc, vc = k.cuda(), v.cuda()
    lists = i32([x + [-1] + [5] * (longest - len(x)) for x in keep])   # nothing counts behind a negative entry
    sdl.compact_pages(kc, vc, i32(table), i32(ctx), lists)
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v)
    # entries past the table, and pages that are not there, are passed over
    kc, vc = k.cuda(), v.cuda()
    sdl.compact_pages(kc, vc, i32(table), i32(ctx), i32([[2 ** 30] + [-1] * 2 for _ in ctx]))
    gone = [[-1] * wide for _ in ctx]
    sdl.compact_pages(kc, vc, i32(gone), i32(ctx), i32([[1, 2, 3] for _ in ctx]))
    assert torch.equal(kc.cpu(), k) and torch.equal(vc.cpu(), v)


def test_the_longest_lists():
    """Lists padded to what one launch holds, and one entry more."""
    layers, most = 64, (1 << 24) // 128 - 1
    k = torch.randn(layers, 3, 1, 1, 4, device="cuda")
    v = torch.randn_like(k)
    want_k, want_v = k.clone(), v.clone()
    want_k[:, 2], want_v[:, 2] = k[:, 0], v[:, 0]
    src = torch.full((most + 1,), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    src[most - 1], dst[most - 1] = 0, 2
    sdl.copy_pages(k, v, src[:most], dst[:most])
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    with pytest.raises(sdl.SpmmError):
        sdl.copy_pages(k, v, src, dst)
    most = (1 << 24) - 1
    table = torch.full((most + 1, 2), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(most + 1, dtype=torch.int32, device="cuda")
    keep = torch.full((most + 1, 1), -1, dtype=torch.int32, device="cuda")
    table[most - 1, 0], table[most - 1, 1], keep[most - 1] = 1, 2, 1
    want_k[:1, 1], want_v[:1, 1] = want_k[:1, 2], want_v[:1, 2]
    sdl.compact_pages(k[:1], v[:1], table[:most], ctx[:most], keep[:most])
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    with pytest.raises(sdl.SpmmError):
        sdl.compact_pages(k[:1], v[:1], table, ctx, keep)


def test_one_pool_as_both():
    """A pool given twice: copying does the same twice, compaction would move
    rows that have moved already."""
    x = torch.randn(2, 6, 16, 2, 32, device="cuda")
    want = x.clone()
    want[:, 4] = want[:, 1]
    sdl.copy_pages(x, x, i32([1]), i32([4]))
    assert torch.equal(x, want)
    for k, v in ((x, x), (x[:1], x[:1]), (x.view(-1)[:1024 * 3].view(1, 3, 16, 2, 32), x.view(-1)[1024:1024 * 4].view(
            1, 3, 16, 2, 32))):
        with pytest.raises(ValueError, match="overlap"):
            sdl.compact_pages(k, v, i32([[0, 1]]), i32([3]), i32([[1, 3]]))
    with pytest.raises(ValueError, match="overlap"):
        sdl.copy_pages(k, v, i32([1]), i32([2]))
    sdl.compact_pages(x[:1], x[1:], i32([[0, 1]]), i32([3]), i32([[1, 3]]))
    empty = x[:, :0]
    sdl.compact_pages(empty, empty, i32([[0, 1]]), i32([3]), i32([[1, 3]]))
    want[:, 0, 3:5] = want[:, 0, 4:7:2]
    assert torch.equal(x, want)


def test_pages_in_a_graph_and_on_a_stream():
    k = torch.randn(2, 8, 16, 2, 64, device="cuda")
    v = torch.randn(2, 8, 16, 2, 64, device="cuda")
    src, dst = i32([0, 1]), i32([2, 3])
    g = torch.cuda.CUDAGraph()
    k0, v0 = k.clone(), v.clone()
    with torch.cuda.graph(g):
        sdl.copy_pages(k, v, src, dst)
    stream = torch.cuda.Stream()
    for i in range(4):
        k.copy_(k0 + i)
        v.copy_(v0 - i)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(k[:, 2:4], k0[:, :2] + i) and torch.equal(v[:, 2:4], v0[:, :2] - i)
    sdl.compact_pages(k, v, i32([[4, 5]]), i32([14]), i32([[1, 3]]), stream=stream)
    stream.synchronize()
    assert torch.equal(k[:, 4, 14], k0[:, 4, 15] + 3) and torch.equal(k[:, 4, 15], k0[:, 5, 1] + 3)


# ------------------------------------------------------------ all together

@BOTH
def test_prefill_fork_draft_accept_answer(dtype):
    """Prompts are encoded by window attention, their rows go into pages, one
    sequence forks, both branches draft a tree, the accepted path moves to the
    front, and the next token is answered: every output equals attention over
    the plain sequence of kept tokens."""
    Hq, Hkv, D, page, window, sinks = 4, 2, 64, 16, 48, 3
    g = torch.Generator().manual_seed(30)

    def normal(n, h):
        return torch.randn(n, h, D, generator=g).to(dtype)

    lens = [37, 90]
    q, k, v = normal(127, Hq), normal(127, Hkv), normal(127, Hkv)
    qs = starts(lens)
    a = dict(window=window, sinks=sinks)
    o, lse = sdl.window_attention(q.cuda(), k.cuda(), v.cuda(), i32(qs), **a)
    want = window_ref(q, k, v, qs, qs, window, sinks)
    assert_close(o, want["o"], want["o_tol"], "prefill")

    pages = 32
    kp = torch.zeros(1, pages, page, Hkv, D, dtype=dtype, device="cuda")
    vp = torch.zeros_like(kp)
    table = [[0, 1, 2, 3, 4, 5, 6, 7], [8, 9, 10, 11, 12, 13, 14, 15]]

    def write(row, pos, kk, vv):
        pos = torch.arange(pos, pos + kk.shape[0])
        number = torch.tensor(row)[pos // page].cuda()
        kp[0, number, (pos % page).cuda()] = kk.cuda()
        vp[0, number, (pos % page).cuda()] = vv.cuda()

    for s in (0, 1):
        write(table[s], 0, k[qs[s]:qs[s + 1]], v[qs[s]:qs[s + 1]])
    # sequence 0 forks: full pages are shared, the partly filled one is copied
    table.append(table[0][:2] + [16, 17, 18, 19, 20, 21])
    sdl.copy_pages(kp, vp, i32([table[0][2]]), i32([16]))
    held = [[k[0:37], v[0:37]], [k[37:127], v[37:127]], [k[0:37], v[0:37]]]
    ctx = [37, 90, 37]

    masks = [[1, 3, 5, 11, 21, 43], [1, 3], [1, 2, 5, 10, 26]]
    path = [[0, 1, 3, 5], [0], [1, 3, 4]]
    drafts = [len(m) for m in masks]
    ds = starts(drafts)
    dq, dk, dv = normal(ds[-1], Hq), normal(ds[-1], Hkv), normal(ds[-1], Hkv)
    for s in range(3):
        write(table[s], ctx[s], dk[ds[s]:ds[s + 1]], dv[ds[s]:ds[s + 1]])
    o, _ = sdl.tree_attention(dq.cuda(), kp[0], vp[0], i32(table), i32(ctx), i32(ds),
                              i64([m for x in masks for m in x]), **a)
    for s in range(3):
        for t in range(drafts[s]):
            line = [b for b in range(drafts[s]) if masks[s][t] >> b & 1]
            kk = torch.cat([held[s][0], dk[ds[s]:ds[s + 1]][line]])
            vv = torch.cat([held[s][1], dv[ds[s]:ds[s + 1]][line]])
            want = window_ref(dq[ds[s] + t:ds[s] + t + 1], kk, vv, [0, 1], [0, len(kk)], window, sinks)
            assert_close(o[ds[s] + t:ds[s] + t + 1], want["o"], 2 * want["o_tol"], f"draft {s}, {t}")

    sdl.compact_pages(kp, vp, i32(table), i32(ctx), i32([x + [-1] * (4 - len(x)) for x in path]))
    for s in range(3):
        held[s] = [torch.cat([held[s][i], x[ds[s]:ds[s + 1]][path[s]]]) for i, x in ((0, dk), (1, dv))]
        ctx[s] += len(path[s])
    nq, nk, nv = normal(3, Hq), normal(3, Hkv), normal(3, Hkv)
    for s in range(3):
        write(table[s], ctx[s], nk[s:s + 1], nv[s:s + 1])
    o, _ = sdl.tree_attention(nq.cuda(), kp[0], vp[0], i32(table), i32(ctx), i32([0, 1, 2, 3]), **a)
    for s in range(3):
        kk, vv = torch.cat([held[s][0], nk[s:s + 1]]), torch.cat([held[s][1], nv[s:s + 1]])
        want = window_ref(nq[s:s + 1], kk, vv, [0, 1], [0, len(kk)], window, sinks)
        assert_close(o[s:s + 1], want["o"], 2 * want["o_tol"], f"answer {s}")
