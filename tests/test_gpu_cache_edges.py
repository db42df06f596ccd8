"""A paged cache that is appended to and held in 8 bits (include/cache.h) at the edges of
its definition: contexts, values and scales that calls seldom have."""
import math

import pytest
import torch

import sparse_dense_linear_amd as sdl
from attn_ref import assert_close, tree_seen
from cache_ref import E4M3, INT8, MOST, codes_of, scale_of_top
from test_gpu_cache import CODES, F32, KINDS, TYPES, CodeCache, a_pool, bits, i32, i64, tables, want_rows

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@TYPES
@KINDS
@pytest.mark.parametrize("ctx", [-1, -3, -8, -17, -(1 << 30)])
def test_append_in_front_of_a_sequence(dtype, kind, ctx):
    """Rows at negative positions are passed over and their rotated elements are NaN; the
    rows behind them are as if they came alone."""
    new, page, block, D, rotated = 12, 16, 8, 64, 32
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(new, h, D, generator=g).to(dtype).cuda() for h in (4, 2, 2))
    cos, sin = (x.cuda() for x in tables(20, rotated))
    made = [None if x is None else x.cuda() for x in a_pool(3, page, block, 2, D, kind, dtype, g)]
    got, want = ([None if x is None else x.clone() for x in made] for _ in range(2))
    table, front = i32([[1, 2]]), min(-ctx, new)

    def call(pools, first, at):
        kw = {} if kind is None else dict(k_scale=pools[2], v_scale=pools[3])
        a = (x[first:].contiguous() for x in (k, v))
        return sdl.append_pages(*a, pools[0], pools[1], table, i32([at]), i32([0, new - first]),
                                q=q[first:].contiguous(), cos=cos, sin=sin, **kw)

    out = call(got, 0, ctx)
    if front < new:
        assert torch.equal(out[front:], call(want, front, 0))
    assert bool(out[:front, :, :rotated].isnan().all())
    assert torch.equal(out[:front, :, rotated:], q[:front, :, rotated:])
    for x, y in zip(got, want):
        assert x is None or torch.equal(bits(x), bits(y))


def held_as(x, scale, held):
    """The codes of finite x, in 64 bits: the nearest one whose value is finite in fp32,
    of two that are as near the even one."""
    every = torch.arange(256, dtype=torch.uint8).view(held)
    every = every[every.float().isfinite() & (every.float() >= -MOST[held])]
    every = every[(every.float() * scale).isfinite()]
    even = every.view(torch.uint8) % 2 if held is E4M3 else every % 2 != 0
    off = (every.double() * float(scale) - x.double()[..., None]).abs() / float(scale)
    return every.float()[(off * 2.0 ** 40 + even.double()).argmin(-1)]


@TYPES
@CODES
def test_finite_values_are_read_as_finite(dtype, held):
    """Next to the end of fp32's range, where the nearest code would be read as infinite."""
    top = float(torch.finfo(dtype).max)
    end = 2.0 ** 128
    for most in (0.9, 0.96, 0.96875, 0.97, 0.9921875, 0.99609375):
        x = torch.zeros(3, 1, 16)
        for i, part in enumerate((1.0, 0.999, 0.97, 0.9375, 0.8, 0.51, 0.25, 0.01)):
            x[i % 3, 0, i], x[i % 3, 0, i + 8] = most * part * end, -most * part * end
        x = x.to(dtype)
        x[1, 0, 15] = top
        assert bool(x.isfinite().all())
        pools = [codes_of(torch.zeros(1, 16, 1, 16), held).cuda() for _ in range(2)]
        ks, vs = (torch.zeros(1, 2, 1, device="cuda") for _ in range(2))
        sdl.append_pages(x.cuda(), x.cuda(), *pools, i32([[0]]), i32([0]), i32([0, 3]), k_scale=ks, v_scale=vs)
        for pool, scale in zip(pools, (ks, vs)):
            scale = scale[0, 0, 0].cpu()
            assert float(scale) == scale_of_top(top, held)
            assert torch.equal(pool[0, :3].cpu().float(), held_as(x.float(), scale, held))
            assert bool((pool[0, :3].cpu().float() * scale).isfinite().all())
        # and so is attention of the first row alone
        q = torch.zeros(1, 1, 16, dtype=dtype, device="cuda")
        o, lse = sdl.tree_attention(q, *pools, i32([[0]]), i32([0]), i32([0, 1]), k_scale=ks, v_scale=vs)
        assert torch.equal(o[0].float(), (pool[0, 0].float() * vs[0, 0, 0]).to(dtype).float()) and float(lse) == 0.0


@pytest.mark.parametrize("kept", [2, 9])
def test_integers_whose_scale_rises_are_read_as_finite(kept):
    """127 * 2^121 under a scale of 2^122: 63.5, whose nearest even code would be read as
    infinite.  Raised by appending, and by moves (both kernels) into another block."""
    top = torch.finfo(F32).max
    small, large = (torch.full((1, 1, 16), x, device="cuda") for x in (127 * 2.0 ** 121, top))
    small[0, 0, 1] = -small[0, 0, 1]
    want = torch.full((1, 16), 63.0)
    want[0, 1] = -63.0

    def pool():
        return ([codes_of(torch.zeros(1, 32, 1, 16), INT8).cuda() for _ in range(2)],
                dict(zip(("k_scale", "v_scale"), (torch.ones(1, 2, 1, device="cuda") for _ in range(2)))))

    table = i32([[0]])
    pools, scales = pool()
    for t, x in enumerate((small, large)):
        sdl.append_pages(x, x, *pools, table, i32([t]), i32([0, 1]), **scales)
    for p, s in zip(pools, scales.values()):
        assert float(s[0, 0, 0]) == 2.0 ** 122
        assert torch.equal(p[0, 0].cpu().float(), want) and torch.equal(p[0, 1].cpu().float(), want.abs())
    # the same two rows, each of a block of its own, brought together
    pools, scales = pool()
    for t, x in ((3, small), (16, large)):
        sdl.append_pages(x, x, *pools, table, i32([t]), i32([0, 1]), **scales)
    keep = [0, 13] + [-1] * (kept - 2)
    sdl.compact_pages(*(p[None] for p in pools), table, i32([3]), i32([keep]),
                      **{n: s[None] for n, s in scales.items()})
    for p, s in zip(pools, scales.values()):
        assert float(s[0, 0, 0]) == 2.0 ** 122
        assert torch.equal(p[0, 3].cpu().float(), want) and torch.equal(p[0, 4].cpu().float(), want.abs())


@TYPES
@KINDS
@pytest.mark.parametrize("ctx,drafts", [(131071, 1), (9000, 40)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_one_value_that_is_no_finite_number_costs_little(dtype, kind, ctx, drafts, bad):
    """The outputs and log-sums beside it are what they are without it; and where a row of
    values or what append_pages writes for one holds it, finding that out takes no longer
    than some turns over the cache (a look at one value after another took 100 ms at the
    longer context, the call without such a value 0.1 ms)."""
    page, Hkv, Hq, D, at = 64, 2, 8, 128, ctx - 300
    g = torch.Generator(device="cuda").manual_seed(7)
    pages = -(-(ctx + drafts) // page)
    shape = (pages, page, Hkv, D)
    q = torch.randn(drafts, Hq, D, device="cuda", generator=g).to(dtype)
    k, v = (torch.randn(shape, device="cuda", generator=g) * 16 for _ in range(2))
    scales = {}
    if kind is None:
        k, v = (x.to(dtype) / 16 for x in (k, v))
    else:
        k, v = (codes_of(x.clamp(-100, 100), kind) for x in (k, v))
        scales = {n: torch.full((pages, page, Hkv), 2.0 ** -4, device="cuda") for n in ("k_scale", "v_scale")}
    args = (i32([list(range(pages))]), i32([ctx]), i32([0, drafts]))
    clean, clean_lse = sdl.tree_attention(q, k, v, *args, **scales)
    where, columns = (at // page, at % page, 1), [37]
    if kind is None:
        v[where][37] = bad
    else:
        v.view(torch.uint8)[where][37] = 0x7f if kind is E4M3 and math.isnan(bad) else 1
        if kind is INT8 or math.isinf(bad):            # which such codes cannot be: all of the row is
            v.view(torch.uint8)[where] = 1
            scales["v_scale"][where], columns = bad, list(range(D))
    took = []
    for _ in range(3):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        o, lse = sdl.tree_attention(q, k, v, *args, **scales)
        end.record()
        torch.cuda.synchronize()
        took.append(begin.elapsed_time(end))
    # an infinite scale is taken from the definition, whose sums have another order: scores
    # of 128 products (whose sizes add up to less than 16), and ctx / 64 weights to a lane
    tol = 0.0 if columns == [37] or math.isnan(bad) else 2 * (128 * 16 + ctx / 64 + 64) * 2.0 ** -24
    assert bool(((lse - clean_lse).abs() <= tol).all())
    assert torch.equal(o[:, :Hq // 2], clean[:, :Hq // 2])
    rest = [d for d in range(D) if d not in columns]
    got = o[:, Hq // 2:]
    assert bool(got[..., columns].isnan().all() if math.isnan(bad) else (got[..., columns] == bad).all())
    assert torch.equal(got[..., rest], clean[:, Hq // 2:][..., rest])
    assert tol > 0 or min(took) < 20.0, took


@TYPES
@CODES
@pytest.mark.parametrize("ctx,drafts", [(131071, 1), (9000, 40)])
def test_a_key_that_is_no_number_costs_nothing(dtype, held, ctx, drafts):
    """What append_pages writes for a key that is not finite: all results of its head are
    no numbers, the others what they are without it."""
    page, Hkv, Hq, D, at = 64, 2, 8, 128, ctx - 300
    g = torch.Generator(device="cuda").manual_seed(8)
    pages = -(-(ctx + drafts) // page)
    q = torch.randn(drafts, Hq, D, device="cuda", generator=g).to(dtype)
    k, v = (codes_of((torch.randn(pages, page, Hkv, D, device="cuda", generator=g) * 16).clamp(-100, 100), held)
            for _ in range(2))
    scales = {n: torch.full((pages, page, Hkv), 2.0 ** -4, device="cuda") for n in ("k_scale", "v_scale")}
    args = (i32([list(range(pages))]), i32([ctx]), i32([0, drafts]))
    clean, clean_lse = sdl.tree_attention(q, k, v, *args, **scales)
    if held is INT8:
        scales["k_scale"][at // page, at % page, 1] = math.nan
    else:
        k.view(torch.uint8)[at // page, at % page, 1, 37] = 0x7f
    took = []
    for _ in range(3):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        o, lse = sdl.tree_attention(q, k, v, *args, **scales)
        end.record()
        torch.cuda.synchronize()
        took.append(begin.elapsed_time(end))
    assert torch.equal(o[:, :4], clean[:, :4]) and torch.equal(lse[:4], clean_lse[:4])
    assert bool(o[:, 4:].isnan().all()) and bool(lse[4:].isnan().all())
    assert min(took) < 5.0, took


@TYPES
@CODES
def test_a_draft_that_is_no_finite_number_and_is_not_kept(dtype, held):
    """Its block's context: as it was in e4m3, lost in integers until the block is begun
    anew; other heads and blocks as they were."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(21, 2, 64, generator=g).to(dtype).cuda()
    table = i32([[1, 0]])
    pools = [codes_of(torch.zeros(2, 16, 2, 64), held).cuda() for _ in range(2)]
    scales = dict(zip(("k_scale", "v_scale"), (torch.ones(2, 2, 2, device="cuda") for _ in range(2))))
    q = torch.randn(1, 2, 64, generator=g).to(dtype).cuda()

    def append(rows, at):
        sdl.append_pages(rows, rows, *pools, table, i32([at]), i32([0, len(rows)]), **scales)

    def answer(keys):                                      # of keys 0 .. keys - 1
        return sdl.tree_attention(q, *pools, table, i32([keys - 1]), i32([0, 1]), **scales)

    append(x[:20], 0)                                      # blocks of 8: the third has 4 rows
    before, block = answer(20), answer(16)
    bad = x[20:].clone()
    bad[0, 1, 7] = math.inf
    append(bad, 20)
    o, lse = answer(20)
    if held is E4M3:
        # a scale that a draft raises costs e4m3 nothing
        assert torch.equal(o, before[0]) and torch.equal(lse, before[1])
    else:
        assert torch.equal(o[:, 0], before[0][:, 0]) and torch.equal(lse[0], before[1][0])
        assert bool(o[:, 1].isnan().all()) and bool(lse[1].isnan().all())
    assert all(torch.equal(a, b) for a, b in zip(answer(16), block))
    append(x[16:20], 16)
    assert all(torch.equal(a, b) for a, b in zip(answer(20), before))


@TYPES
@CODES
@pytest.mark.parametrize("what", ["code", "nan scale", "infinite scale"])
@pytest.mark.parametrize("T", [5, 40])
def test_masked_places_against_the_definition(dtype, held, what, T):
    """A draft whose row or scale is no finite number: the drafts that do not see it have
    the results of the definition; its own are no numbers, or infinite where the
    definition's are."""
    page, block, ctx, at, D = 16, 1, 300, 2, 64
    if what == "code" and held is INT8:
        return                                             # every code is a number
    for pool in ("k", "v"):
        cache = CodeCache([ctx + T], page, block, 1, D, held, 14)
        number, row = cache.table[0][(ctx + at) // page], (ctx + at) % page
        code, scale, rows = (cache.k, cache.ks, cache.rows_k) if pool == "k" else (cache.v, cache.vs, cache.rows_v)
        if what == "code":
            code[number, row] = math.nan
        else:
            scale[number, row] = math.nan if what == "nan scale" else math.inf
        q = torch.randn(T, 4, D, generator=torch.Generator().manual_seed(15)).to(dtype)
        masks = [(1 << a | 1) & ~(1 << at) for a in range(T)]
        masks[at] = 1 << at | 1                            # seen by itself alone
        pools, scales = cache.on_gpu()
        o, lse = sdl.tree_attention(q.cuda(), *pools, i32([ctx]), i32([0, T]), i64(masks), **scales)
        keep = [t for t in range(T) if t != at]
        rows[0][ctx + at] = 0.0                            # of no draft that is kept
        want = want_rows(q, [0, T], cache.rows_k, cache.rows_v,
                         lambda s: tree_seen(ctx, masks, sdl.NO_WINDOW, 0), 1, D ** -0.5, dtype)
        assert_close(o[keep], want["o"][keep], 2 * want["o_tol"][keep], "o")
        assert_close(lse[:, keep], want["lse"][:, keep], 2 * want["lse_tol"][:, keep], "lse")
        if pool == "v":
            # weights do not depend on it: the log-sum is right, the outputs are what the
            # sums with it are
            assert_close(lse[:, at], want["lse"][:, at], 2 * want["lse_tol"][:, at], "lse")
            sign = code[number, row, 0].float().sign()
            if what != "infinite scale":
                assert bool(o[at].isnan().all())
            else:
                got = o[at].cpu().float()
                assert bool(torch.where(sign == 0, got.isnan(), got == sign * math.inf).all())
        elif what != "infinite scale":
            assert bool(o[at].isnan().all()) and bool(lse[:, at].isnan().all())
        else:
            # s = scale * <q, code>: plus infinity, or minus infinity and so no weight
            up = (q[at].double() @ code[number, row, 0].double()) > 0
            assert bool(up.any()) and not bool(up.all())
            assert bool(o[at, up].isnan().all()) and bool((lse[up, at] == math.inf).all())
            alone = want_rows(q, [0, T], cache.rows_k, cache.rows_v,
                              lambda s: tree_seen(ctx, [1] * T, sdl.NO_WINDOW, 0), 1, D ** -0.5, dtype)
            assert_close(o[at, ~up], alone["o"][at, ~up], 2 * alone["o_tol"][at, ~up], "o")
            assert_close(lse[~up, at], alone["lse"][~up, at], 2 * alone["lse_tol"][~up, at], "lse")
