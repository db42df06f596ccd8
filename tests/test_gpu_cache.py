"""Writing a paged cache, and a paged cache held in 8 bits (include/cache.h),
against their definitions (tests/cache_ref.py, tests/attn_ref.py)."""
import math
import random

import pytest
import torch

import sparse_dense_linear_amd as sdl
from attn_ref import SLACK, U, assert_close, chain_seen, head_forward, tree_seen
from cache_ref import (E4M3, INT8, MOST, append_ref, codes_of, compact_ref, places, rotate, rotation_tolerance,
                       scale_of_top, values)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
CODES = pytest.mark.parametrize("held", [E4M3, INT8], ids=["e4m3", "i8"])


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


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


def same_bits(got, want, what):
    """Bit for bit, but for which NaN."""
    got, want = got.cpu(), want.cpu()
    assert got.dtype == want.dtype and got.shape == want.shape, what
    nan = got.float().isnan() if got.dtype != INT8 else torch.zeros(got.shape, dtype=torch.bool)
    want_nan = want.float().isnan() if want.dtype != INT8 else nan
    assert torch.equal(nan, want_nan), f"{what}: {int((nan != want_nan).sum())} elements are NaN in one only"
    size = got.element_size()
    differ = (bits(got) != bits(want)).view(*got.shape, size).any(-1) if got.numel() else nan
    bad = (differ & ~nan).nonzero()
    if len(bad):
        at = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {len(bad)} of {got.numel()} differ; first at {at}: "
                             f"{float(got[at])!r}, not {float(want[at])!r}")


def page_table(lengths, page, seed, more=2):
    """Page numbers in random order; entries past a sequence are nonsense."""
    r = random.Random(seed)
    need = [-(-n // page) for n in lengths]
    pool = sum(need) + more
    order = list(range(pool))
    r.shuffle(order)
    wide, at, table = max(need + [1]), 0, []
    for n in need:
        table.append(order[at:at + n] + [-1000000] * (wide - n))
        at += n
    return table, pool


class CodeCache:
    """A paged cache of codes: scales of any size, no powers of two; unused rows
    hold NaN (77 where there is none) and unused blocks the scale NaN."""

    def __init__(self, lengths, page, block, Hkv, D, held, seed, dead=(), power=None):
        g = torch.Generator().manual_seed(seed)
        self.table, pool = page_table(lengths, page, seed)
        shape = (pool, page, Hkv, D)
        self.k = (torch.full(shape, math.nan).to(held) if held is E4M3 else torch.full(shape, 77, dtype=INT8))
        self.v = self.k.clone()
        self.ks = torch.full((pool, page // block, Hkv), math.nan)
        self.vs = self.ks.clone()
        self.rows_k, self.rows_v = [], []
        for s, n in enumerate(lengths):
            for pool_, scale, rows in ((self.k, self.ks, self.rows_k), (self.v, self.vs, self.rows_v)):
                blocks = -(-n // block)
                sc = (torch.rand(blocks, Hkv, generator=g) + 0.5) / (MOST[held] / 4)
                if power is not None:                     # of two; the values of all sizes
                    sc = torch.exp2(sc.log2().round())
                    if pool_ is self.v:
                        sc = sc * torch.exp2(torch.randint(-3, 4, sc.shape, generator=g).float())
                x = torch.randn(n, Hkv, D, generator=g)
                if power is not None:
                    sc, x = sc * 2.0 ** power, x * 2.0 ** power
                each = sc.repeat_interleave(block, 0)[:n]
                code = codes_of((x / each[..., None]).clamp(-MOST[held], MOST[held]), held)
                for b in range(blocks):
                    number, first = self.table[s][b * block // page], b * block % page
                    here = code[b * block:(b + 1) * block]
                    pool_[number, first:first + len(here)] = here
                    scale[number, first // block] = sc[b]
                rows.append(values(code, each))
        for s, p in dead:
            number = self.table[s][p]
            self.k[number] = self.v[number] = math.nan if held is E4M3 else 77
            self.ks[number] = self.vs[number] = math.nan
            self.table[s][p] = -1000000

    def on_gpu(self):
        return (self.k.cuda(), self.v.cuda(), i32(self.table)), {"k_scale": self.ks.cuda(), "v_scale": self.vs.cuda()}


def head_codes(q, k, v, seen, scale, dtype):
    """head_forward of values code * scale.  The kernels round a score once more
    (times the scale of its key), and a weight (times the scale of its value): U
    of each."""
    f = head_forward(q, k, v, seen, scale, dtype)
    mag = torch.where(seen, (q.abs() @ k.abs().T) * scale, 0.0)
    more = U * (mag.amax(1) if mag.shape[1] else torch.zeros(q.shape[0], dtype=q.dtype))
    f["lse_tol"] = f["lse_tol"] + more
    f["o_tol"] = f["o_tol"] + SLACK * (2 * more + U)[:, None] * (f["p"] @ v.abs())
    return f


def want_rows(q, qs, rows_k, rows_v, seen_of, Hkv, sc, dtype):
    Hq = q.shape[1]
    want = {n: torch.zeros(q.shape, dtype=torch.float64) for n in ("o", "o_tol")}
    want |= {n: torch.zeros((Hq, q.shape[0]), dtype=torch.float64) for n in ("lse", "lse_tol")}
    for s in range(len(qs) - 1):
        a = slice(qs[s], qs[s + 1])
        seen = seen_of(s)
        for h in range(Hq):
            f = head_codes(q[a, h].double(), rows_k[s][:, h * Hkv // Hq], rows_v[s][:, h * Hkv // Hq], seen, sc, dtype)
            want["o"][a, h], want["o_tol"][a, h] = f["o"], f["o_tol"]
            want["lse"][h, a], want["lse_tol"][h, a] = f["lse"], f["lse_tol"]
    return want


def check(ctx, drafts, Hq, Hkv, D, dtype, held, page, block, window, sinks, masks="tree", seed=0, dead=(),
          scale=None, power=None):
    r = random.Random(seed)
    cache = CodeCache([c + t for c, t in zip(ctx, drafts)], page, block, Hkv, D, held, seed, dead, power)
    q = torch.randn(sum(drafts), Hq, D, generator=torch.Generator().manual_seed(seed + 1)).to(dtype)
    qs = starts(drafts)
    if masks == "tree":
        masks = [random_tree(t, r) for t in drafts]
    w = sdl.NO_WINDOW if window is None else window
    pools, scales = cache.on_gpu()
    tree = None if masks is None else i64([m for x in masks for m in x])
    o, lse = sdl.tree_attention(q.cuda(), *pools, i32(ctx), i32(qs), tree, window=window, sinks=sinks, scale=scale,
                                **scales)
    torch.cuda.synchronize()
    assert o.dtype == dtype and lse.dtype == F32
    want = want_rows(q, qs, cache.rows_k, cache.rows_v,
                     lambda s: chain_seen(ctx[s], drafts[s], w, sinks) if masks is None else
                     tree_seen(ctx[s], masks[s], w, sinks), Hkv, 1 / math.sqrt(D) if scale is None else scale, dtype)
    # the joining of partial results rounds once more for each of them: a
    # factor 2 on the fp32 part covers up to as many parts as keys
    assert_close(o, want["o"], 2 * want["o_tol"], "o")
    assert_close(lse, want["lse"], 2 * want["lse_tol"], "lse")


# ------------------------------------------------------------- attention

@TYPES
@CODES
@pytest.mark.parametrize("page,block", [(1, 1), (7, 7), (16, 4), (16, 1), (24, 8), (64, 64), (128, 2), (300, 25)])
def test_pages_and_blocks(dtype, held, page, block):
    check([0, 1, 200, 515], [3, 1, 9, 2], 4, 2, 64, dtype, held, page, block, None, 0, seed=page)


@TYPES
@CODES
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
def test_head_sizes(dtype, held, D):
    check([130, 0, 33], [5, 2, 1], 4, 4, D, dtype, held, 16, 8, 60, 3, seed=D)
    check([130, 0, 33], [40, 2, 1], 2, 1, D, dtype, held, 16, 8, 60, 3, seed=D)


@TYPES
@CODES
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (40, 4), (129, 128), (500, 17), (None, 5)])
def test_windows(dtype, held, window, sinks):
    check([700, 260, 20], [12, 33, 4], 2, 1, 64, dtype, held, 16, 16, window, sinks, seed=3)
    check([700, 260, 20, 5000], [1, 1, 1, 1], 4, 1, 128, dtype, held, 16, 16, window, sinks, seed=3)


@TYPES
@CODES
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (6, 2), (8, 1), (16, 1), (40, 1)])
@pytest.mark.parametrize("drafts", [[1, 1], [3, 17], [64, 40]])
def test_shared_heads(dtype, held, Hq, Hkv, drafts):
    """From one column of a matrix to many blocks of them."""
    check([300, 77], drafts, Hq, Hkv, 64, dtype, held, 32, 16, 200, 2, seed=Hq)


@TYPES
@CODES
@pytest.mark.parametrize("power", [0, -90, 60, 112])
@pytest.mark.parametrize("drafts", [[1, 1], [40, 9], [130, 64]])
def test_scales_of_powers_of_two(dtype, held, power, drafts):
    """As append_pages writes them, whole tiles of them and tiles that a page of
    another sequence's end cuts; small and large, within what is widened with its
    scale and past it."""
    masks = None if max(drafts) > 64 else "tree"
    check([700, 77], drafts, 4, 2, 64, dtype, held, 32, 8, 300, 2, masks=masks, seed=11, power=power,
          scale=2.0 ** (-3 - power))


@TYPES
@CODES
def test_chains(dtype, held):
    """No masks: causal pieces, of any length."""
    check([300, 0, 64], [1, 130, 65], 4, 2, 64, dtype, held, 16, 16, None, 0, masks=None, seed=4)
    check([300, 0, 640], [1, 130, 65], 4, 1, 128, dtype, held, 16, 4, 70, 3, masks=None, seed=5)


@TYPES
@CODES
def test_masks_that_see_nothing_or_anything(dtype, held):
    """Rows that see no draft, and none of the cache; drafts that see later
    ones; bits past the drafts; drafts past the 64th."""
    check([0, 0, 9], [2, 3, 2], 2, 1, 64, dtype, held, 8, 4, None, 0, seed=6,
          masks=[[0, 2], [0, 0, 0], [0, (1 << 64) - 1]])
    check([5, 300], [3, 70], 2, 1, 64, dtype, held, 8, 8, 4, 0, seed=7,
          masks=[[0b111, 0b100, 0], [(0x9E3779B97F4A7C15 * (i + 1)) & (1 << 64) - 1 for i in range(70)]])
    check([50], [4], 2, 1, 64, dtype, held, 8, 2, 1, 0, seed=8, masks=[[0, 1, 3, 8]])


@TYPES
@CODES
def test_long_contexts_are_split_and_joined(dtype, held):
    check([20000], [1], 2, 1, 128, dtype, held, 16, 16, None, 0, seed=9)
    check([9000, 3, 5000], [2, 40, 1], 8, 2, 64, dtype, held, 64, 16, None, 0, seed=10)
    check([9000, 3, 5000], [2, 40, 1], 8, 2, 64, dtype, held, 64, 32, 3000, 4, seed=11)
    check([9000, 3, 5000], [2, 1, 1], 8, 2, 96, dtype, held, 100, 25, 3000, 4, seed=11)


@TYPES
@CODES
def test_many_sequences(dtype, held):
    """More sequences than a workgroup has threads, empty ones among them."""
    r = random.Random(12)
    n = 300
    ctx = [r.choice([0, 1, 15, 16, 17, 120]) for _ in range(n)]
    drafts = [r.choice([0, 1, 1, 1, 2]) for _ in range(n)]
    check(ctx, drafts, 2, 1, 64, dtype, held, 16, 8, None, 0, seed=12)


@TYPES
@CODES
@pytest.mark.parametrize("many", [1, 40])
def test_pages_that_nothing_sees_are_not_read(dtype, held, many):
    """Pages behind the window, and those of drafts that no mask names, hold
    nonsense in the table, and their scales are NaN."""
    page, ctx, window, sinks = 16, 500, 100, 4
    dead = [(0, p) for p in range(1, (ctx - window + 1) // page)]
    check([ctx], [many], 4, 2, 64, dtype, held, page, 8, window, sinks, seed=13, dead=dead)
    check([ctx], [many], 4, 2, 64, dtype, held, page, 8, window, 0, seed=13, dead=dead + [(0, 0)])
    check([64, 30], [40, 3], 2, 1, 128, dtype, held, 16, 16, None, 0, seed=37, dead=[(0, 5), (0, 6)],
          masks=[[(0x9E3779B97F4A7C15 * (i + 1)) & 0xffff for i in range(40)], [1, 3, 7]])
    check([100, 20], [3, 1], 2, 1, 64, dtype, held, 16, 16, 1, 0, seed=39, dead=[(0, p) for p in range(7)],
          masks=[[0, 0, 0], [1]])


@TYPES
@CODES
@pytest.mark.parametrize("what", ["code", "nan scale", "infinite scale"])
def test_masked_places_may_hold_anything(dtype, held, what):
    """What a draft's row or the scale of its block holds reaches only the drafts
    that see it."""
    if what == "code" and held is INT8:
        return                                          # every code is a number
    page, block, ctx, T = 16, 1, 300, 5
    cache = CodeCache([ctx + T], page, block, 1, 64, held, 14)
    q = torch.randn(T, 4, 64, generator=torch.Generator().manual_seed(15)).to(dtype)
    masks = [1, 3, 5, 9, 19]                            # draft 2 is seen by itself alone
    args = (i32([ctx]), i32([0, T]), i64(masks))
    pools, scales = cache.on_gpu()
    clean, clean_lse = sdl.tree_attention(q.cuda(), *pools, *args, **scales)
    number, row = cache.table[0][(ctx + 2) // page], (ctx + 2) % page
    if what == "code":
        cache.k[number, row] = cache.v[number, row] = math.nan
    else:
        cache.ks[number, row] = cache.vs[number, row] = math.nan if what == "nan scale" else math.inf
    pools, scales = cache.on_gpu()
    o, lse = sdl.tree_attention(q.cuda(), *pools, *args, **scales)
    keep = [0, 1, 3, 4]
    # the same sums in another order: twice the bound of either
    tol = 8 * torch.finfo(dtype).eps
    assert bool(((o[keep] - clean[keep]).abs() <= tol * (1 + clean[keep].abs())).all())
    assert torch.equal(lse[:, keep].isfinite(), clean_lse[:, keep].isfinite())
    assert bool(((lse[:, keep] - clean_lse[:, keep]).abs() <= 1e-4).all())
    assert not bool(torch.isfinite(o[2]).all())


@TYPES
@CODES
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("drafts", [1, 40])
def test_an_infinite_value_beside_masked_keys(dtype, held, D, drafts):
    """A value of infinite scale at the edges of what is seen: infinite for the
    drafts that see it, and no masked key makes it no number."""
    ctx, window, sinks, page = 700, 41, 3, 16
    for at in (sinks - 1, ctx + drafts - window, ctx + drafts - 1):
        cache = CodeCache([ctx + drafts], page, 1, 1, D, held, 31)
        number = cache.table[0][at // page]
        cache.v[number, at % page, 0] = 1
        cache.vs[number, at % page, 0] = math.inf
        q = torch.randn(drafts, 4, D, generator=torch.Generator().manual_seed(32)).to(dtype)
        pools, scales = cache.on_gpu()
        o, lse = sdl.tree_attention(q.cuda(), *pools, i32([ctx]), i32([0, drafts]), window=window, sinks=sinks,
                                    **scales)
        seen = chain_seen(ctx, drafts, window, sinks)
        v = cache.rows_v[0][:, 0].clone()
        v[at] = 0
        for h in range(4):
            f = head_codes(q[:, h].double(), cache.rows_k[0][:, 0], v, seen, D ** -0.5, dtype)
            f["o"][seen[:, at]] = math.inf
            assert_close(o[:, h], f["o"], 2 * f["o_tol"], f"o, key {at}")
            assert_close(lse[h], f["lse"], 2 * f["lse_tol"], "lse")


@TYPES
@CODES
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,drafts", [(700, 1), (700, 40), (20000, 2)])
def test_values_near_the_end_of_the_range(dtype, held, D, ctx, drafts):
    """Values of up to 2^126: their weighted mean is finite, their sum with
    weights that are not yet divided is not."""
    cache = CodeCache([ctx + drafts], 16, 4, 1, D, held, 33)
    up = 2.0 ** 125
    cache.vs *= up
    cache.rows_v[0] *= up
    if held is E4M3:
        assert float(cache.rows_v[0].abs().max()) < 2.0 ** 127.9
    q = torch.randn(drafts, 4, D, generator=torch.Generator().manual_seed(34)).to(dtype)
    pools, scales = cache.on_gpu()
    o, lse = sdl.tree_attention(q.cuda(), *pools, i32([ctx]), i32([0, drafts]), window=15000, sinks=2, **scales)
    seen = chain_seen(ctx, drafts, 15000, 2)
    for h in range(4):
        f = head_codes(q[:, h].double(), cache.rows_k[0][:, 0], cache.rows_v[0][:, 0], seen, D ** -0.5, dtype)
        assert_close(o[:, h], f["o"], 2 * f["o_tol"], "o")
        assert_close(lse[h], f["lse"], 2 * f["lse_tol"], "lse")


@CODES
def test_strided_pools_scales_and_queries(held):
    """Pools that are one layer of a larger tensor, scales whose heads come
    first, queries cut from a fused tensor."""
    for dtype in (F32, BF16):
        for drafts in ([3, 1], [33, 20]):
            cache = CodeCache([87 + drafts[0], 30 + drafts[1]], 16, 8, 2, 64, held, 16)
            n = sum(drafts)
            q = torch.randn(n, 6, 64, generator=torch.Generator().manual_seed(17)).to(dtype)
            a = (i32(cache.table), i32([87, 30]), i32(starts(drafts)))
            o, lse = sdl.tree_attention(q[:, :4].contiguous().cuda(), cache.k.cuda(), cache.v.cuda(), *a,
                                        k_scale=cache.ks.cuda(), v_scale=cache.vs.cuda())
            pools = torch.stack([bits(cache.k), bits(cache.v)], 2).cuda().view(held)    # [pages, page, 2, Hkv, D]
            ks, vs = (x.permute(2, 0, 1).contiguous().cuda().permute(1, 2, 0) for x in (cache.ks, cache.vs))
            fused = torch.cat([torch.zeros(n, 2, 64, dtype=dtype), q], 1).cuda()
            o2, lse2 = sdl.tree_attention(fused[:, 2:6], pools[:, :, 0], pools[:, :, 1], *a, k_scale=ks, v_scale=vs)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


@CODES
def test_pages_past_32_bits(held):
    """Pages more than 2^32 bytes, and scales as far, from the first one."""
    cache = CodeCache([200], 16, 16, 2, 64, held, 51, dead=())
    step = 1 << 30
    pages = len(cache.table[0])
    order = {n: i for i, n in enumerate(cache.table[0])}
    big = [torch.empty((pages + 1) // 2 * step, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pools = [b.as_strided((pages, 16, 2, 64), (step // 2, 128, 64, 1)).view(held) for b in big]
    for p, c in zip(pools, (cache.k, cache.v)):
        for n, i in order.items():
            p[i].copy_(c[n].cuda())
    ks, vs = (x[cache.table[0]].contiguous().cuda() for x in (cache.ks, cache.vs))
    ctx, rp = i32([199]), i32([0, 1])
    for dtype in (F32, BF16):
        q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(52)).to(dtype).cuda()
        a, scales = cache.on_gpu()
        o, lse = sdl.tree_attention(q, *a, ctx, rp, **scales)
        o2, lse2 = sdl.tree_attention(q, *pools, i32([list(range(pages))]), ctx, rp, k_scale=ks, v_scale=vs)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for dtype in (F32, BF16):
        k = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(53)).to(dtype).cuda()
        near, near_scales = [p.contiguous() for p in pools], (ks.clone(), vs.clone())
        a = (i32([list(range(pages))]), i32([190]), i32([0, 5]))
        sdl.append_pages(k, k, *near, *a, k_scale=near_scales[0], v_scale=near_scales[1])
        sdl.append_pages(k, k, *pools, *a, k_scale=ks, v_scale=vs)
        for x, y in zip((*pools, ks, vs), (*near, *near_scales)):
            assert torch.equal(bits(x), bits(y))


@CODES
@pytest.mark.parametrize("drafts", [(3, 1), (40, 30)])
def test_rows_of_no_sequence_are_left(held, drafts):
    n = sum(drafts)
    cache = CodeCache([87 + drafts[0], 30 + drafts[1]], 16, 4, 2, 64, held, 18)
    q = torch.full((n + 8, 4, 64), math.nan, device="cuda")
    q[3:3 + n] = torch.randn(n, 4, 64, device="cuda")
    o = torch.full_like(q, 7.0)
    lse = torch.full((4, n + 8), 7.0, device="cuda")
    pools, scales = cache.on_gpu()
    sdl.tree_attn_paged(q, *pools, i32([87, 30]), i32(starts(drafts, 3)), None, o, lse, **scales)
    torch.cuda.synchronize()
    assert bool((o[:3] == 7).all()) and bool((o[3 + n:] == 7).all())
    assert bool((lse[:, :3] == 7).all()) and bool((lse[:, 3 + n:] == 7).all())
    assert bool(torch.isfinite(o[3:3 + n]).all()) and not bool((o[3:3 + n] == 7).all(dim=2).any())


@CODES
def test_repeats_streams_and_graphs(held):
    sets = []
    for seed in (19, 20):
        cache = CodeCache([3000, 700, 20], 16, 8, 2, 128, held, seed)
        q = torch.randn(9, 8, 128, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()
        pools, scales = cache.on_gpu()
        sets.append(((q, *pools, i32([2996, 697, 18]), i32([0, 4, 7, 9])), scales))
        sets.append(((q[:3].contiguous(), *pools, i32([2999, 699, 19]), i32([0, 1, 2, 3])), scales))
    eager = [sdl.tree_attention(*s, **sc) for s, sc in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [(i, sdl.tree_attention(*sets[i][0], **sets[i][1], stream=streams[i])) for _ in range(4)
           for i in range(len(sets))]
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, eager[i]))
    graphs, outs = [], []
    for s, sc in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sdl.tree_attention(*s, **sc))
        graphs.append(g)
    for _ in range(4):
        for out in outs:
            for x in out:
                x.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for out, e in zip(outs, eager):
            assert all(torch.equal(x, y) for x, y in zip(out, e))
        assert torch.equal(sdl.tree_attention(*sets[0][0], **sets[0][1])[0], eager[0][0])
        torch.cuda.synchronize()


# ---------------------------------------------------------------- appending

def tables(positions, rotated, seed=0):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(rotated // 2, dtype=torch.float64) / max(1, rotated // 2))
    return angle.cos().float(), angle.sin().float()


def a_pool(pool, page, block, Hkv, D, kind, dtype, g):
    """Pools that are full of something, and their scales (powers of two)."""
    if kind is None:
        return (torch.randn(pool, page, Hkv, D, generator=g).to(dtype),
                torch.randn(pool, page, Hkv, D, generator=g).to(dtype), None, None)
    out = []
    for _ in range(2):
        out.append(codes_of((torch.randn(pool, page, Hkv, D, generator=g) * MOST[kind] / 4).clamp(
            -MOST[kind], MOST[kind]), kind))
    for _ in range(2):
        out.append(2.0 ** torch.randint(-9, -3, (pool, page // block, Hkv), generator=g).float())
    return out


def check_append(ctx, new, Hq, Hkv, D, dtype, kind, page, block, rotated, interleaved=False, masks=None, seed=0,
                 first=0, behind=0, k=None, v=None, angles=None, change=None, table=None):
    """One call against the definition, bit for bit, and its rotation against 64 bits."""
    g = torch.Generator().manual_seed(seed)
    rp = starts(new, first)
    T = rp[-1] + behind
    made, pool = page_table([c + n for c, n in zip(ctx, new)], page, seed)
    table = made if table is None else table
    q = torch.randn(T, Hq, D, generator=g).to(dtype) if Hq else None
    k = torch.randn(T, Hkv, D, generator=g).to(dtype) if k is None else k
    v = torch.randn(T, Hkv, D, generator=g).to(dtype) if v is None else v
    kp, vp, ks, vs = a_pool(pool, page, block, Hkv, D, kind, dtype, g)
    if change is not None:
        change(kp, vp, ks, vs, table)
    cos, sin = tables(angles or max([c + n for c, n in zip(ctx, new)] + [1]), rotated) if rotated else (None, None)
    flat = None if masks is None else [0] * first + [m for x in masks for m in x] + [0] * behind
    gpu = [x.cuda() for x in (kp, vp)]
    kw = {} if kind is None else {"k_scale": ks.cuda(), "v_scale": vs.cuda()}
    out = torch.full_like(q, 7.0).cuda() if Hq else None
    got = sdl.append_pages(k.cuda(), v.cuda(), *gpu, i32(table), i32(ctx), i32(rp), q=q.cuda() if Hq else None,
                           cos=cos.cuda() if rotated else None, sin=sin.cuda() if rotated else None,
                           tree=None if flat is None else i64(flat), interleaved=interleaved, q_out=out, **kw)
    torch.cuda.synchronize()
    assert got is out
    want = append_ref(k, v, kp, vp, table, ctx, rp, q, cos, sin, flat, interleaved, ks, vs)
    same_bits(gpu[0], kp, "keys")
    same_bits(gpu[1], vp, "values")
    if kind is not None:
        same_bits(kw["k_scale"], ks, "scales of keys")
        same_bits(kw["v_scale"], vs, "scales of values")
    if Hq:
        want[:first], want[rp[-1]:] = 7.0, 7.0
        same_bits(got, want, "q")
        if rotated and rp[-1] > first and angles is None:
            stand = places(ctx, rp, flat)[0][first:]
            c, s = cos[stand], sin[stand]
            exact = rotate(q[first:rp[-1]], c, s, interleaved, torch.float64)
            off = (got[first:rp[-1]].cpu().double() - exact).abs()
            assert bool((off <= rotation_tolerance(q[first:rp[-1]], c, s, dtype)).all())
    return kp, vp, ks, vs, table


KINDS = pytest.mark.parametrize("kind", [None, E4M3, INT8], ids=["as-is", "e4m3", "i8"])


@TYPES
@KINDS
@pytest.mark.parametrize("page,block", [(1, 1), (7, 7), (16, 4), (24, 8), (64, 64), (100, 25), (256, 128)])
def test_append_pages_and_blocks(dtype, kind, page, block):
    check_append([0, 1, 200, 515, 16], [3, 1, 90, 2, 0], 4, 2, 64, dtype, kind, page, block, 64, seed=page)
    check_append([0, 300, 17], [300, 5, 1], 2, 1, 128, dtype, kind, page, block, 128, seed=page)


@TYPES
@KINDS
@pytest.mark.parametrize("D,rotated", [(8, 8), (16, 16), (40, 40), (48, 16), (64, 64), (64, 0), (80, 32), (96, 96),
                                       (112, 56), (128, 128), (128, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_head_sizes(dtype, kind, D, rotated, interleaved):
    if kind is not None and D % 16:
        return                                             # refused, in test_cache_host.py
    check_append([0, 21, 5], [5, 2, 30], 6, 3, D, dtype, kind, 16, 8, rotated, interleaved, seed=D)


@TYPES
@KINDS
@pytest.mark.parametrize("Hq,Hkv", [(0, 1), (0, 5), (1, 1), (7, 7), (40, 8), (64, 1)])
def test_append_heads(dtype, kind, Hq, Hkv):
    check_append([9, 0], [4, 35], Hq, Hkv, 64, dtype, kind, 16, 16, 64, seed=Hq)


@TYPES
@KINDS
def test_append_drafts_stand_where_their_mask_says(dtype, kind):
    r = random.Random(5)
    drafts = [1, 17, 64, 3]
    check_append([0, 100, 31, 7], drafts, 4, 2, 64, dtype, kind, 16, 8, 64, masks=[random_tree(t, r) for t in drafts])
    # nothing seen, later ones, bits past the drafts, drafts past the 64th
    check_append([5, 8, 0], [3, 70, 1], 2, 1, 64, dtype, kind, 16, 8, 32, masks=[
        [0, 0b100, (1 << 64) - 1], [(0x9E3779B97F4A7C15 * (i + 1)) & (1 << 64) - 1 for i in range(70)], [0]])


@TYPES
@KINDS
def test_append_many_sequences_and_rows_of_none(dtype, kind):
    r = random.Random(12)
    for n in (65, 300, 5000):
        ctx = [r.choice([0, 1, 7, 8, 9]) for _ in range(n)]
        new = [r.choice([0, 1, 1, 2, 9]) for _ in range(n)]
        check_append(ctx, new, 2, 1, 16, dtype, kind, 8, 4, 16, seed=n, first=3, behind=5)
    check_append([4, 4], [0, 0], 2, 1, 16, dtype, kind, 8, 4, 16, first=2, behind=3)


@TYPES
@KINDS
def test_append_rows_whose_page_is_out_of_range_are_passed_over(dtype, kind):
    def break_table(kp, vp, ks, vs, table):
        table[0][1] = -1
        table[1][0] = len(kp)
        table[1][1] = 1 << 30
        for row in table:
            del row[4:]
    check_append([10, 0, 60], [50, 40, 20], 2, 1, 64, dtype, kind, 16, 8, 64, change=break_table)


@TYPES
@KINDS
def test_append_positions_past_the_tables_are_nan(dtype, kind):
    kp, vp, ks, vs, table = check_append([3, 60], [4, 10], 2, 1, 64, dtype, kind, 16, 16, 32, angles=63)
    if kind is None:
        assert bool(kp[table[1][63 // 16], 63 % 16, :, :32].isnan().all())


@TYPES
@CODES
def test_append_scales(dtype, held):
    """Raised for larger rows, kept for smaller ones, begun anew with a block;
    zero, tiny and huge values; scales that another program chose."""
    for power in (-149, -133, -126, -60, -7, 0, 9, 100, 119):
        for top in (1.0, 1.5, 1.75, 1.7578125, 1.984375, 1.9921875):
            x = torch.zeros(3, 1, 16)
            x[0, 0, 0], x[1, 0, 3], x[2, 0, 15] = top * 2.0 ** power, -top * 2.0 ** power / 3, 0.0
            x = x.to(dtype)
            check_append([6], [3], 0, 1, 16, dtype, held, 8, 4, 0, k=x, v=x.flip(0))

    def foreign(kp, vp, ks, vs, table):
        ks.mul_(1.3)
        vs.copy_(torch.where(torch.rand(vs.shape) < 0.5, vs * 1e-3, vs * 777.0))

    torch.manual_seed(1)
    for seed in range(4):
        check_append([5, 30, 17, 3], [1, 3, 20, 1], 0, 3, 64, dtype, held, 16, 8, 32, seed=seed, change=foreign)


@TYPES
@CODES
def test_append_values_that_are_no_finite_numbers(dtype, held):
    for value in (math.inf, -math.inf, math.nan):
        k = torch.randn(12, 2, 64, generator=torch.Generator().manual_seed(3)).to(dtype)
        k[2, 1, 5] = value
        kp, vp, ks, vs, table = check_append([5], [12], 0, 2, 64, dtype, held, 16, 8, 0, k=k, v=k.flip(2))
        number = table[0][0]
        if held is INT8:
            assert bool(ks[number, 0, 1].isnan()) and not bool(ks[number, 0, 0].isnan())
        else:
            assert int(kp[number].float().isnan().sum()) == 1
    # a scale that has become NaN stays so until the block is begun anew
    def lost(kp, vp, ks, vs, table):
        ks.fill_(math.nan)
    kp, vp, ks, vs, table = check_append([5], [12], 0, 2, 64, dtype, held, 16, 8, 0, change=lost)
    assert bool(ks[table[0][0], 0].isnan().all()) and not bool(ks[table[0][0], 1].isnan().any())


@TYPES
@CODES
def test_codes_are_as_near_as_their_type_allows(dtype, held):
    """Against 64 bits: half a step of a code (e4m3: 2^-4 of the value, or half of
    its smallest number), and the roundings to fp32 before."""
    T, D = 40, 64
    g = torch.Generator().manual_seed(8)
    x = (torch.randn(T, 1, D, generator=g) * 2.0 ** torch.randint(-4, 4, (T, 1, 1), generator=g)).to(dtype)
    kp, vp, ks, vs, table = check_append([3], [T], 0, 1, D, dtype, held, 16, 8, 64, k=x, v=x)
    cos, sin = tables(3 + T, 64)
    exact = {"k": rotate(x, cos[3:], sin[3:], False, torch.float64), "v": x.double()}
    for n, pool, scale in (("k", kp, ks), ("v", vp, vs)):
        for t in range(T):
            p = 3 + t
            s = scale[table[0][p // 16], p % 16 // 8, 0].double()
            got = pool[table[0][p // 16], p % 16, 0].double() * s
            want = exact[n][t, 0]
            half = torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10) if held is E4M3 else s / 2
            assert bool(((got - want).abs() <= half + 8 * U * exact[n][t].abs().max()).all())


@CODES
def test_rows_one_by_one_as_at_once(held):
    """A block's scale is that of its largest value either way.  e4m3: so are the
    codes, but for those below the smallest normal one; integers are rounded
    anew when a scale is raised: each time half a step more."""
    T, D = 32, 64
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T, 2, D, generator=g) * 2.0 ** torch.randint(-3, 3, (T, 1, 1), generator=g)
    pools = [codes_of(torch.zeros(2, 16, 2, D), held).cuda() for _ in range(4)]
    scales = [torch.full((2, 2, 2), 2.0 ** -40, device="cuda") for _ in range(4)]
    table, xs = i32([[0, 1]]), x.cuda()
    sdl.append_pages(xs, xs, *pools[:2], table, i32([0]), i32([0, T]), k_scale=scales[0], v_scale=scales[1])
    for t in range(T):
        sdl.append_pages(xs[t:t + 1], xs[t:t + 1], *pools[2:], table, i32([t]), i32([0, 1]), k_scale=scales[2],
                         v_scale=scales[3])
    assert torch.equal(scales[0], scales[2]) and torch.equal(scales[1], scales[3])
    a, b = (p.float().cpu() for p in (pools[0], pools[2]))
    if held is E4M3:
        normal = a.abs() >= 2.0 ** -6
        assert torch.equal(a[normal], b[normal]) and bool(((a - b).abs() <= 2.0 ** -9).all())
    else:
        # x / s, s / 2, ..: the sum of half a step, a quarter, ... is below one
        assert bool(((a - b).abs() <= 1).all())


@KINDS
def test_append_strided_operands_and_in_place(kind):
    """q, k and v cut from one fused tensor, pools that are a layer of a larger
    one, q rotated where it lies."""
    for dtype in (F32, BF16):
        g = torch.Generator().manual_seed(21)
        fused = torch.randn(30, 8, 64, generator=g).to(dtype).cuda()
        q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:8]
        kp, vp, ks, vs = (None if x is None else x.cuda() for x in a_pool(6, 16, 8, 2, 64, kind, dtype, g))
        cos, sin = (x.cuda() for x in tables(80, 64))
        a = (i32([[4, 1, 0], [2, 5, 3]]), i32([7, 20]), i32([0, 18, 30]))
        kw = dict(cos=cos, sin=sin)
        layered = torch.stack([kp.view(torch.uint8), vp.view(torch.uint8)], 2).view(kp.dtype)    # [pages, page, 2, ..]
        ls = {}
        if kind is not None:
            ls = dict(k_scale=ks.permute(2, 0, 1).contiguous().permute(1, 2, 0),
                      v_scale=vs.permute(2, 0, 1).contiguous().permute(1, 2, 0))
            kw |= dict(k_scale=ks, v_scale=vs)
        out = sdl.append_pages(k.contiguous(), v.contiguous(), kp, vp, *a, q=q.contiguous(), **kw)
        kw |= ls
        again = sdl.append_pages(k, v, layered[:, :, 0], layered[:, :, 1], *a, q=q, q_out=q, **kw)
        assert again is q
        assert torch.equal(q, out)
        assert torch.equal(bits(layered[:, :, 0]), bits(kp)) and torch.equal(bits(layered[:, :, 1]), bits(vp))
        if kind is not None:
            assert torch.equal(ls["k_scale"], ks) and torch.equal(ls["v_scale"], vs)


@KINDS
def test_append_streams_and_graphs(kind):
    """Captured once, replayed with contexts that grow: each replay against the
    same calls made one by one."""
    dtype, n = BF16, 3
    g = torch.Generator().manual_seed(22)
    pools = [None if x is None else x.cuda() for x in a_pool(9, 16, 8, 2, 64, kind, dtype, g)]
    eager = [None if x is None else x.clone() for x in pools]
    cos, sin = (x.cuda() for x in tables(100, 64))
    q, k, v = (torch.zeros(n, h, 64, dtype=dtype, device="cuda") for h in (4, 2, 2))
    table, ctx, rp = i32([[0, 3, 6], [1, 4, 7], [2, 5, 8]]), i32([5, 7, 0]), i32([0, 1, 2, 3])

    def call(p, c, stream=None):
        kw = {} if kind is None else dict(k_scale=p[2], v_scale=p[3])
        return sdl.append_pages(k, v, p[0], p[1], table, c, rp, q=q, cos=cos, sin=sin, stream=stream, **kw)

    graph = torch.cuda.CUDAGraph()
    saved = [None if x is None else x.clone() for x in pools]
    with torch.cuda.graph(graph):
        out = call(pools, ctx)
    for x, y in zip(pools, saved):
        if x is not None:
            assert torch.equal(bits(x), bits(y))           # capturing writes nothing
    other = torch.cuda.Stream()
    for step in range(12):
        for t in (q, k, v):
            t.copy_((torch.randn(t.shape, generator=g) * 2.0 ** (step % 5)).to(dtype))
        torch.cuda.synchronize()
        graph.replay()
        want = call(eager, ctx.clone(), stream=other)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for x, y in zip(pools, eager):
            if x is not None:
                assert torch.equal(bits(x), bits(y))
        ctx += 1


# -------------------------------------------------------------------- moves

def layered(layers, pool, page, block, heads, D, held, seed):
    g = torch.Generator().manual_seed(seed)
    made = [a_pool(pool, page, block, heads, D, held, None, g) for _ in range(layers)]
    return [torch.stack([m[i].view(torch.uint8) if i < 2 else m[i] for m in made]).view(held if i < 2 else F32)
            for i in range(4)]


@CODES
def test_copies_take_their_scales_with_them(held):
    k, v, ks, vs = layered(3, 7, 24, 8, 3, 48, held, 1)
    src, dst = [0, 3, -1, 0, 9, 2], [5, 1, 4, 6, 4, 70]
    gpu = [x.cuda() for x in (k, v, ks, vs)]
    sdl.copy_pages(gpu[0], gpu[1], i32(src), i32(dst), k_scale=gpu[2], v_scale=gpu[3])
    for x in (k, v, ks, vs):
        for a, b in zip(src, dst):
            if 0 <= a < 7 and 0 <= b < 7:
                x[:, b] = x[:, a].clone()
    for x, y in zip(gpu, (k, v, ks, vs)):
        assert torch.equal(bits(x), bits(y))
    # one pool as both
    sdl.copy_pages(gpu[0], gpu[0], i32([1]), i32([2]), k_scale=gpu[2], v_scale=gpu[2])
    assert torch.equal(bits(gpu[0][:, 1]), bits(gpu[0][:, 2])) and torch.equal(gpu[2][:, 1], gpu[2][:, 2])


def check_compact(held, layers, page, block, heads, D, ctx, keep, seed=0, change=None, rows=None):
    most = max([len(x) for x in keep])
    keep = [x + [-1] * (most - len(x)) for x in keep]
    lengths = [c + (max(x + [0]) + 1 if rows is None else rows) for c, x in zip(ctx, keep)]
    table, pool = page_table(lengths, page, seed)
    want = layered(layers, pool, page, block, heads, D, held, seed)
    if change is not None:
        change(*want, table)
    gpu = [x.cuda() for x in want]
    sdl.compact_pages(gpu[0], gpu[1], i32(table), i32(ctx), i32(keep), k_scale=gpu[2], v_scale=gpu[3])
    compact_ref(want[0], want[1], table, ctx, keep, want[2], want[3])
    for x, y, n in zip(gpu, want, ("keys", "values", "scales of keys", "scales of values")):
        same_bits(x, y, n)


@CODES
@pytest.mark.parametrize("page,block", [(1, 1), (8, 8), (16, 4), (24, 8), (64, 16), (128, 128)])
def test_compact(held, page, block):
    r = random.Random(page)
    ctx = [0, 5, 16, 31, 100, 7, 3]
    keep = [sorted(r.sample(range(64), n)) for n in (1, 8, 20, 64, 5)] + [[], [0, 1, 2]]
    check_compact(held, 3, page, block, 2, 64, ctx, keep, seed=page)
    # lists of up to eight, of neighbours and of drafts far apart
    for n in (1, 3, 8):
        keep = [sorted(r.sample(range(m), n)) for m in (8, 9, 20, 64, 30)] + [[], list(range(n))]
        check_compact(held, 3, page, block, 2, 64, ctx, keep, seed=page + n)


@CODES
@pytest.mark.parametrize("heads,D", [(1, 16), (3, 48), (8, 128), (24, 80), (40, 112), (2, 96)])
def test_compact_heads(held, heads, D):
    """Up to rows of more columns than a workgroup takes in a turn."""
    keep = [[1, 2, 3, 9, 30], [0, 4, 5, 6, 7, 8, 20]]
    check_compact(held, 2, 16, 8, heads, D, [3, 13], keep, seed=D)
    check_compact(held, 2, 16, 8, heads, D, [3, 13], [x + [40, 41, 50] for x in keep], seed=D)


@CODES
@pytest.mark.parametrize("kept", [3, 12])
def test_moves_past_32_bits(held, kept):
    """Pages more than 2^32 bytes from the first one of a layer, in the last of two
    layers, against the same pages in a small pool."""
    page, block, heads, D, few = 16, 8, 2, 64, 6
    small = [x.cuda() for x in layered(2, few, page, block, heads, D, held, 31)]
    pages = (1 << 32) // (page * heads * D) + few
    at = [pages - 1, 0, pages - 2, 5, (1 << 31) // (page * heads * D), pages // 2]
    big = [torch.empty((2, pages, *x.shape[2:]), dtype=torch.uint8, device="cuda").view(held) for x in small[:2]]
    big += [torch.empty((2, pages, *x.shape[2:]), device="cuda") for x in small[2:]]
    for b, x in zip(big, small):
        for i, n in enumerate(at):
            b[:, n].copy_(x[:, i])
    keep = i32([[2 * t + 1 for t in range(kept)]])
    for pools, name in ((small, list(range(few))), (big, at)):
        kw = dict(k_scale=pools[2], v_scale=pools[3])
        sdl.copy_pages(*pools[:2], i32([name[0]]), i32([name[3]]), **kw)
        sdl.compact_pages(*pools[:2], i32([[name[1], name[3], name[2], name[4], name[5]]]), i32([19]), keep, **kw)
    torch.cuda.synchronize()
    for b, x in zip(big, small):
        for i, n in enumerate(at):
            assert torch.equal(bits(b[:, n]), bits(x[:, i])), (i, n)


@CODES
def test_compact_long_lists(held):
    """More kept rows than are found at once, in one block and over many."""
    check_compact(held, 1, 256, 256, 1, 32, [40, 250], [list(range(1, 180)), list(range(0, 400, 2))])
    check_compact(held, 2, 16, 4, 1, 32, [1, 9], [list(range(3, 150)), list(range(0, 300, 2))])


@CODES
def test_compact_scales_and_places_out_of_range(held):
    def foreign(k, v, ks, vs, table):
        ks.mul_(1.37)
        vs[:, ::2].mul_(1e-3)
        vs[:, 1::3] = math.nan
        table[0][2] = -1
        table[1][1] = 1 << 30
        table[2][0] = len(ks[0])
    check_compact(held, 2, 16, 8, 2, 64, [3, 30, 5], [[2, 9, 40, 60], [1, 3, 20], [0, 1, 14, 15]], change=foreign)
    check_compact(held, 2, 16, 8, 2, 64, [3, 30], [[2, 9, 40, 90], [1, 3, 20]], rows=30)
    more = [[2, 9, 40, 60, 61, 62, 63, 70, 71, 72], [1, 3, 20], list(range(14)) + [15]]
    check_compact(held, 2, 16, 8, 2, 64, [3, 30, 5], more, change=foreign)
    check_compact(held, 2, 16, 8, 2, 64, [3, 30], more[:2], rows=30)


@CODES
def test_compact_in_a_graph(held):
    want = layered(2, 8, 16, 8, 2, 64, held, 4)
    table = [[3, 1, 0, 2], [7, 4, 6, 5]]
    keep = [[0, 12, 20, -1], [11, 13, -1, -1]]
    gpu, ctx = [x.cuda() for x in want], i32([3, 9])
    args = (i32(table), ctx, i32(keep))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdl.compact_pages(gpu[0], gpu[1], *args, k_scale=gpu[2], v_scale=gpu[3])
    at = [3, 9]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        compact_ref(want[0], want[1], table, at, keep, want[2], want[3])
        for x, y in zip(gpu, want):
            same_bits(x, y, "replayed")
        ctx += 2
        at = [a + 2 for a in at]


# ------------------------------------------------------------------ together

@TYPES
@KINDS
def test_prompt_drafts_acceptance_and_next_token(dtype, kind):
    """As they are used: a prompt into the cache, a fork, trees of drafts, their
    attention, the accepted path to the front, and the next token."""
    Hq, Hkv, D, page, block, pages = 4, 2, 64, 16, 8, 24
    g = torch.Generator().manual_seed(40)
    r = random.Random(41)
    cos, sin = tables(200, D)
    pools = [None if x is None else x[None].contiguous() for x in a_pool(pages, page, block, Hkv, D, kind, dtype, g)]
    gpu = [None if x is None else x.cuda() for x in pools]
    table = [list(range(0, 8)), list(range(8, 16)), list(range(16, 24))]
    rows = {}                                             # what a sequence's positions hold, rotated, in 64 bits

    def scales(p):
        return {} if kind is None else dict(k_scale=p[2][0], v_scale=p[3][0])

    def step(ctx, new, masks):
        T = sum(new)
        q, k, v = (torch.randn(T, h, D, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
        rp = starts(new)
        flat = None if masks is None else [m for x in masks for m in x]
        tree = None if flat is None else i64(flat)
        qr = sdl.append_pages(k.cuda(), v.cuda(), gpu[0][0], gpu[1][0], i32(table), i32(ctx), i32(rp), q=q.cuda(),
                              cos=cos.cuda(), sin=sin.cuda(), tree=tree, **scales(gpu))
        want_q = append_ref(k, v, pools[0][0], pools[1][0], table, ctx, rp, q, cos, sin, flat,
                            **scales(pools))
        same_bits(qr, want_q, "q")
        o, lse = sdl.tree_attention(qr, gpu[0][0], gpu[1][0], i32(table), i32(ctx), i32(rp), tree, **scales(gpu))
        torch.cuda.synchronize()

        def cached(pool, scale, s):
            at = range(ctx[s] + new[s])
            x = torch.stack([pool[0, table[s][p // page], p % page] for p in at]).double() if len(at) else \
                torch.zeros(0, Hkv, D, dtype=torch.float64)
            if scale is not None and len(at):
                x = x * torch.stack([scale[0, table[s][p // page], p % page // block] for p in at])[..., None].double()
            return x

        n = len(ctx)
        want = want_rows(want_q, rp, [cached(pools[0], pools[2], s) for s in range(n)],
                         [cached(pools[1], pools[3], s) for s in range(n)],
                         lambda s: chain_seen(ctx[s], new[s], sdl.NO_WINDOW, 0) if masks is None else
                         tree_seen(ctx[s], masks[s], sdl.NO_WINDOW, 0), Hkv, D ** -0.5, dtype)
        assert_close(o, want["o"], 2 * want["o_tol"], "o")
        assert_close(lse, want["lse"], 2 * want["lse_tol"], "lse")
        for x, y in zip(gpu, pools):
            if x is not None:
                same_bits(x, y, "pools")

    step([0, 0, 0], [37, 50, 0], None)                    # two prompts
    # the second one forks: its partly filled page is copied, the others are shared
    sc = {} if kind is None else dict(k_scale=gpu[2], v_scale=gpu[3])
    sdl.copy_pages(gpu[0], gpu[1], i32([table[1][3]]), i32([table[2][3]]), **sc)
    for x in pools:
        if x is not None:
            x[:, table[2][3]] = x[:, table[1][3]]
    table[2][:3] = table[1][:3]
    ctx = [37, 50, 50]
    for _ in range(3):
        drafts = [r.randint(1, 30) for _ in ctx]
        masks = [random_tree(t, r) for t in drafts]
        step(ctx, drafts, masks)
        keep = []
        for t, m in zip(drafts, masks):                   # the path to some draft
            leaf = r.randrange(t)
            keep.append([a for a in range(t) if m[leaf] >> a & 1])
        most = max(map(len, keep))
        full = [x + [-1] * (most - len(x)) for x in keep]
        sdl.compact_pages(gpu[0], gpu[1], i32(table), i32(ctx), i32(full), **sc)
        if kind is None:
            for pool in pools[:2]:
                for s, path in enumerate(keep):
                    for t, a in enumerate(path):
                        f, to = ctx[s] + a, ctx[s] + t
                        pool[:, table[s][to // page], to % page] = pool[:, table[s][f // page], f % page].clone()
        else:
            compact_ref(pools[0], pools[1], table, ctx, full, pools[2], pools[3])
        ctx = [c + len(x) for c, x in zip(ctx, keep)]
        step(ctx, [1, 1, 1], None)
        ctx = [c + 1 for c in ctx]


# ----------------------------------------------------------------- refusals

def refused(exc, match, f, *a, **kw):
    with pytest.raises(exc, match=match):
        f(*a, **kw)


@CODES
def test_attention_refuses(held):
    q = torch.zeros(4, 4, 64, device="cuda")
    pages = torch.zeros(3, 16, 2, 64).to(held).cuda()
    sc = torch.ones(3, 2, 2, device="cuda")
    a = (i32([[0, 1]]), i32([20]), i32([0, 4]))

    def call(q=q, k=pages, v=pages, ks=sc, vs=sc, **kw):
        return sdl.tree_attention(q, k, v, *a, k_scale=ks, v_scale=vs, **kw)

    call()
    refused(TypeError, "k_scale", call, ks=None)
    refused(TypeError, "v_scale", call, vs=None)
    refused(TypeError, "float32 or bfloat16", call, q=q.half())
    refused(TypeError, "float8_e4m3fn or int8", call, k=pages.float(), v=pages.float())
    other = INT8 if held is E4M3 else E4M3
    refused(TypeError, "one element type", call, v=pages.view(other))
    refused(TypeError, "without scales", call, ks=None, vs=None)
    refused(TypeError, "scales must be float32", call, ks=sc.double(), vs=sc.double())
    refused(ValueError, "same GPU", call, ks=sc.cpu())
    refused(ValueError, "pages, blocks", call, ks=sc[:2], vs=sc[:2])
    refused(ValueError, "pages, blocks", call, ks=sc[..., :1], vs=sc[..., :1])
    refused(ValueError, "pages, blocks", call, ks=sc[0], vs=sc[0])
    three = torch.ones(3, 3, 2, device="cuda")
    refused(ValueError, "must divide", call, ks=three, vs=three)
    refused(ValueError, "same strides", call, vs=sc.permute(2, 0, 1).contiguous().permute(1, 2, 0))
    refused(ValueError, "same strides", call, v=pages.transpose(1, 2).contiguous().transpose(1, 2))
    refused(sdl.SpmmError, "multiple of 16", call, q=q[..., :24], k=pages[..., :24], v=pages[..., :24])
    refused(sdl.SpmmError, "window", call, window=0)
    o, lse = torch.empty_like(q), torch.empty(4, 4, device="cuda")
    refused(TypeError, "o that of q", sdl.tree_attn_paged, q, pages, pages, *a, None, o.bfloat16(), lse, k_scale=sc,
            v_scale=sc)
    refused(ValueError, "overlap", sdl.tree_attn_paged, q, pages, pages, *a, None, q, lse, k_scale=sc, v_scale=sc)


@KINDS
def test_append_refuses(kind):
    k, q = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, 4, 64, device="cuda")
    kp, vp, ks, vs = (None if x is None else x.cuda()
                      for x in a_pool(3, 16, 8, 2, 64, kind, F32, torch.Generator().manual_seed(1)))
    cos = torch.ones(50, 32, device="cuda")
    a = (i32([[0, 1]]), i32([20]), i32([0, 4]))

    def call(k=k, v=k, kp=kp, vp=vp, a=a, ks=ks, vs=vs, **kw):
        return sdl.append_pages(k, v, kp, vp, *a, k_scale=ks, v_scale=vs, **kw)

    before = [None if x is None else x.clone() for x in (kp, vp, ks, vs)]
    refused(TypeError, "float32 or bfloat16", call, k=k.half())
    refused(TypeError, "element type", call, v=k.bfloat16())
    refused(ValueError, "three dimensions", call, k=k[0])
    refused(ValueError, "shape", call, v=k[:3])
    refused(ValueError, "pools must not overlap", call, vp=kp)
    refused(ValueError, "heads of k", call, k=k[:, :1], v=k[:, :1])
    refused(ValueError, "D of q", call, k=k[..., :32], v=k[..., :32])
    refused(ValueError, "four dimensions", call, kp=kp[0], vp=vp[0])
    refused(sdl.SpmmError, "rows of the pools overlap", call, kp=kp[:1].expand(3, 16, 2, 64),
            vp=vp[:1].expand(3, 16, 2, 64))
    refused(ValueError, "cos must have two", call, cos=cos[0], sin=cos[0])
    refused(TypeError, "sin", call, cos=cos)
    refused(TypeError, "cos", call, sin=cos)
    refused(TypeError, "float32", call, cos=cos.double(), sin=cos.double())
    refused(ValueError, "contiguous", call, cos=cos.t(), sin=cos.t())
    refused(sdl.SpmmError, "rotated", call, cos=torch.cat([cos, cos], 1), sin=torch.cat([cos, cos], 1))
    refused(sdl.SpmmError, "multiple of 8", call, cos=cos[:, :2].contiguous(), sin=cos[:, :2].contiguous())
    refused(TypeError, "64-bit masks", call, tree=i32([1, 1, 1, 1]))
    refused(ValueError, "shape", call, tree=i64([1, 1]))
    refused(TypeError, "int32", call, a=(a[0], a[1].long(), a[2]))
    refused(ValueError, "shape", call, a=(a[0], a[1], a[2][:1]))
    refused(ValueError, "two dimensions", call, a=(a[0][0], a[1], a[2]))
    refused(ValueError, "goes with q", call, q_out=q)
    refused(ValueError, "three dimensions", call, q=q[:3])
    refused(ValueError, "three dimensions", call, q=q[..., :32])
    refused(ValueError, "have heads", call, q=q[:, :0])
    refused(sdl.SpmmError, "multiple of Hkv", call, q=q[:, :3].contiguous())
    refused(ValueError, "overlap", call, q=q, q_out=q.as_strided(q.shape, (64, 256, 1)))
    refused(sdl.SpmmError, "overlap", call, q=q, q_out=torch.zeros(1, 4, 64, device="cuda").expand(4, 4, 64))
    refused(ValueError, "overlap", call, q=q[:, :2], q_out=k)
    if kind is not None:
        refused(TypeError, "v_scale", call, vs=None)
        refused(ValueError, "scales must not overlap", call, vs=ks)
        refused(sdl.SpmmError, "scales overlap", call, ks=ks[:, :1].expand(3, 2, 2), vs=vs[:, :1].expand(3, 2, 2))
        refused(TypeError, "without scales", call, ks=None, vs=None)
    else:
        refused(TypeError, "float8_e4m3fn or int8", call, ks=torch.ones(3, 2, 2, device="cuda"),
                vs=torch.ones(3, 2, 2, device="cuda"))
    torch.cuda.synchronize()
    for x, y in zip((kp, vp, ks, vs), before):
        if x is not None:
            assert torch.equal(bits(x), bits(y))


@CODES
def test_moves_refuse(held):
    kp, vp, ks, vs = (x.cuda() for x in layered(2, 4, 16, 8, 2, 64, held, 1))
    one = i32([0])
    for f, a in ((sdl.copy_pages, (one, i32([1]))), (sdl.compact_pages, (i32([[0, 1]]), one, i32([[1]])))):
        def call(kp=kp, vp=vp, ks=ks, vs=vs):
            f(kp, vp, *a, k_scale=ks, v_scale=vs)

        refused(TypeError, "k_scale", call, ks=None)
        refused(TypeError, "v_scale", call, vs=None)
        refused(TypeError, "float8_e4m3fn or int8", call, kp=kp.float(), vp=vp.float())
        refused(TypeError, "float32", call, ks=ks.double(), vs=vs.double())
        refused(ValueError, "same GPU", call, ks=ks.cpu())
        refused(ValueError, "five dimensions", call, kp=kp.flatten(3), vp=vp.flatten(3))
        refused(ValueError, "layers, pages", call, ks=ks[:1], vs=vs[:1])
        refused(ValueError, "must be contiguous", call, ks=ks.transpose(0, 1).contiguous().transpose(0, 1))
        refused(ValueError, "overlap", call, vs=ks)
        refused(ValueError, "must divide", call, ks=ks[:, :, :1].expand(2, 4, 3, 2).contiguous(),
                vs=vs[:, :, :1].expand(2, 4, 3, 2).contiguous())
        refused(sdl.SpmmError, "multiple of 16", call, kp=kp[..., :24].contiguous(), vp=vp[..., :24].contiguous())
