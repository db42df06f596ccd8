"""Writing a paged cache, and a paged cache held in 8 bits: the measured cases,
their plain forms and their values in 64 bits.

append   new rows of k and v, packed by row pointers, go into the pages behind
         their sequence's context; k and q are rotated by their position on
         the way.  Pools of q's type, or of 8 bits with a scale for each block
         of positions and head: the smallest power of two that holds the
         block's largest value, raised (and the earlier rows of the block
         written anew) where new rows need more.  Returns (q rotated, the
         pools, their scales).
attend   attention of drafted tokens (one answered token; a piece of a prompt)
         over pools of 8 bits: value = code * scale.  Returns (o, lse).
compact  the kept drafts of pools of 8 bits move to the front of their
         sequence's drafts in every layer, into blocks whose scale is the
         largest of those that their rows come from.  Returns the pools and
         their scales.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HELD = {"e4m3": (torch.float8_e4m3fn, 448.0), "i8": (torch.int8, 127.0)}
NEG = -math.inf


def _ints(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(int(x)) for x in values)


def _spread(count, low, high, seed):
    """`count` lengths between low and high, spread over their logarithm."""
    r = random.Random(seed)
    return _text(math.exp(r.uniform(math.log(low), math.log(high))) for _ in range(count))


def _append(name, dtype, held, ctx, new, hq, hkv, d, rotated, interleaved, page, block, tree=False):
    return {"name": name, "op": "append", "dtype": dtype, "held": held, "ctx": ctx, "new": new, "hq": hq,
            "hkv": hkv, "d": d, "rotated": rotated, "interleaved": interleaved, "page": page, "block": block,
            "tree": tree}


def _attend(name, form, dtype, held, ctx, drafts, hq, hkv, d, page, block, window, sinks):
    return {"name": name, "op": "attend", "form": form, "dtype": dtype, "held": held, "ctx": ctx,
            "drafts": drafts, "hq": hq, "hkv": hkv, "d": d, "page": page, "block": block, "window": window,
            "sinks": sinks}


def _compact(name, held, layers, pool, page, block, hkv, d, count, drafts):
    return {"name": name, "op": "compact", "held": held, "layers": layers, "pool": pool, "page": page,
            "block": block, "hkv": hkv, "d": d, "count": count, "drafts": drafts}


def listed():
    far = 1 << 30
    return [
        # three answers that have just begun, in full precision: latency counts
        _append("append_small_f32", "f32", "none", "0,333,1000", "1,1,4", 16, 16, 96, 96, True, 24, 24),
        # prompts of very different lengths, two of them continued
        _append("append_prompts_bf16", "bf16", "none", "0,0,128,0,77", "8192,4096,2500,1333,263", 32, 8, 128,
                128, False, 64, 64),
        # one token of a batch of answers, into 8 bits: every block has earlier rows
        _append("append_answers_e4m3", "bf16", "e4m3", _spread(128, 100, 8192, 1), _text([1] * 128), 32, 8, 128,
                128, False, 16, 16),
        # prompts into 8 bits
        _append("append_prompts_e4m3", "bf16", "e4m3", "0,300,0,1000,5", "4096,2048,1500,500,48", 32, 8, 128,
                128, False, 64, 16),
        # trees of drafts, with a part of each head rotated
        _append("append_drafts_e4m3", "bf16", "e4m3", _spread(16, 500, 12000, 2), _spread(16, 16, 64, 3), 32, 4,
                128, 64, True, 32, 8, tree=True),
        # three answers that have just begun, q in full precision: latency counts
        _attend("answer_small_i8", "tree", "f32", "i8", "0,333,1000", "1,1,4", 16, 16, 96, 24, 8, far, 0),
        # a batch of answers, one token each: the cache's bytes count
        _attend("answer_batch_e4m3", "tree", "bf16", "e4m3", _spread(64, 1000, 16384, 1), _text([1] * 64), 32, 8,
                128, 64, 16, far, 0),
        # two answers behind very long contexts
        _attend("answer_long_i8", "tree", "bf16", "i8", "131072,40001", "1,1", 32, 8, 128, 128, 128, far, 0),
        # trees of drafts for a batch of answers, with a window and first tokens
        _attend("draft_trees_e4m3", "tree", "bf16", "e4m3", _spread(16, 500, 12000, 2), _spread(16, 16, 64, 3),
                32, 4, 128, 32, 32, 4096, 4),
        # the next piece of prompts that are taken in pieces, beside one that is answering
        _attend("prompt_piece_e4m3", "chain", "bf16", "e4m3", "8192,2500,20000", "1024,700,1", 32, 8, 128, 64,
                16, far, 0),
        # the accepted drafts of two answers
        _compact("accept_small_e4m3", "e4m3", 4, 64, 24, 8, 4, 96, 2, 32),
        # the accepted drafts of a batch
        _compact("accept_e4m3", "e4m3", 32, 1024, 16, 16, 8, 128, 128, 64),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["append", "append", "attend", "attend", "attend", "chain", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([32, 64, 80, 96, 112, 128, 128])
    page, block = rng.choice([(1, 1), (16, 16), (16, 4), (24, 8), (32, 32), (64, 16), (100, 25), (128, 128)])
    if op == "append":
        n, held = log(1, 48), rng.choice(["none", "e4m3", "e4m3"])
        new = [log(1, 4000 // n + 1) if rng.random() < 0.6 else 1 for _ in range(n)]
        tree = rng.random() < 0.3
        new = [min(x, 64) if tree else x for x in new]
        ctx = [log(1, 6000) if rng.random() < 0.8 else 0 for _ in range(n)]
        return _drop(_append("", dtype, held, _text(ctx), _text(new), hq, hkv, d, rng.choice([d, d, 16, d // 16 * 8]),
                             rng.random() < 0.5, page, block, tree))
    if op == "attend":
        n, most = log(1, 48), rng.choice([1, 1, 9, 33, 64])
        ctx = [log(1, 8000) if rng.random() < 0.95 else 0 for _ in range(n)]
        return _drop(_attend("", "tree", dtype, rng.choice(["e4m3", "i8"]), _text(ctx),
                             _text(rng.randint(1, most) for _ in range(n)), hq, hkv, d, page, block,
                             rng.choice([1 << 30, log(10, 6000)]), rng.choice([0, 4, 17])))
    if op == "chain":
        n = rng.choice([1, 2, 3, 5])
        return _drop(_attend("", "chain", dtype, rng.choice(["e4m3", "i8"]), _text(log(1, 6000) for _ in range(n)),
                             _text(log(1, 600) for _ in range(n)), hq, hkv, d, page, block,
                             rng.choice([1 << 30, log(10, 6000)]), rng.choice([0, 4, 17])))
    layers, count = log(1, 24), log(1, 64)
    page, block = rng.choice([(8, 8), (16, 16), (16, 4), (24, 8), (64, 16)])
    need = count * (2 + 80 // page)
    return _drop(_compact("", "e4m3", layers, log(need, 600) if need < 600 else need, page, block, hkv, d, count,
                          log(40, 64)))


def _drop(case):
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    return {"append": _prepare_append, "attend": _prepare_attend, "compact": _prepare_compact}[case["op"]](
        case, seed)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _starts(lengths):
    out = [0]
    for x in lengths:
        out.append(out[-1] + x)
    return out


def _device(values, dtype):
    return torch.tensor(values, dtype=dtype).cuda()


def _exponent(top, held):
    """The scale for a largest value: the smallest power of two, not below
    2^-126, with top <= most * scale."""
    m, e = torch.frexp(top)
    least, at = {"e4m3": (0.875, 9), "i8": (0.9921875, 7)}[held]
    e = torch.where(m <= least, e - at, e - at + 1).clamp(min=-126)
    return torch.where(top == 0, -126, e)


def _pool(shape, held, block, g):
    """Codes [.., pages, page, heads, d] and scales [.., pages, page / block, heads] of
    normal values whose size differs by head and block."""
    *lead, page, heads, d = shape
    t, most = HELD[held]
    codes = torch.empty(shape, dtype=t, device="cuda")
    scale = torch.empty((*lead, page // block, heads), device="cuda")
    flat, flat_scale = codes.view(-1, page // block, block, heads, d), scale.view(-1, page // block, heads)
    size = 2 ** torch.empty(heads, 1, device="cuda").uniform_(-2, 2, generator=g)
    step = max(1, (1 << 25) // (page * heads * d))
    for a in range(0, flat.shape[0], step):
        x = torch.randn(flat[a:a + step].shape, device="cuda", generator=g) * size
        top = x.abs().amax((2, 4))
        # integers as another program may have laid them out, with any scale
        s = torch.ldexp(torch.ones_like(top), _exponent(top, held)) if held == "e4m3" else top / most
        y = x / s[:, :, None, :, None]
        flat[a:a + step] = (y.round() if held == "i8" else y).to(t)
        flat_scale[a:a + step] = s
    return codes, scale


def _pages(lengths, page, seed, more=3):
    """Page numbers of sequences, in any order, and how many there are."""
    need = [-(-n // page) for n in lengths]
    pool = sum(need) + more
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [0] * (max(need) - n))
        at += n
    return table, pool


def _masks(drafts, r):
    """Masks of a random tree of drafts: each token sees itself and what its parent sees."""
    m = []
    for a in range(drafts):
        parent = r.randint(max(-1, a - 9), a - 1) if a else -1
        m.append((m[parent] if parent >= 0 else 0) | (1 << a))
    return [x - (1 << 64) if x >> 63 else x for x in m]


def _prepare_append(case, seed):
    g, r, t = _generator(seed), random.Random(seed), TYPES[case["dtype"]]
    ctx, new, page, block = _ints(case["ctx"]), _ints(case["new"]), case["page"], case["block"]
    starts, d, hkv = _starts(new), case["d"], case["hkv"]
    table, pool = _pages([c + n for c, n in zip(ctx, new)], page, seed)
    shape = (pool, page, hkv, d)

    def normal(heads):
        size = 2 ** torch.empty(heads, 1, device="cuda").uniform_(-2, 2, generator=g)
        return (torch.randn(starts[-1], heads, d, device="cuda", generator=g) * size).to(t)

    s = {"case": case, "q": normal(case["hq"]), "k": normal(hkv), "v": normal(hkv),
         "table": _device(table, torch.int32), "ctx": _device(ctx, torch.int32),
         "rowptr": _device(starts, torch.int32), "tree": None, "k_scale": None, "v_scale": None}
    for n in ("k", "v"):
        if case["held"] == "none":
            s[n + "_pages"] = torch.randn(shape, device="cuda", generator=g).to(t)
        else:
            s[n + "_pages"], s[n + "_scale"] = _pool(shape, case["held"], block, g)
    # tables of the rotation, of all positions
    half = case["rotated"] // 2
    rate = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(max(c + n for c, n in zip(ctx, new)), dtype=torch.float64)[:, None] * rate
    s["cos"], s["sin"] = angle.cos().float().cuda(), angle.sin().float().cuda()
    if case["tree"]:
        s["tree"] = _device([m for n in new for m in _masks(n, r)], torch.int64)
    # for the plain form: each row's sequence and place, and the blocks that new rows fall into
    s["seq"] = _device([i for i, n in enumerate(new) for _ in range(n)], torch.int64)
    s["row"] = _device([a for n in new for a in range(n)], torch.int64)
    blocks, rows, old = [], [], []
    for i, (c, n) in enumerate(zip(ctx, new)):
        for b in range(c // block, (c + n - 1) // block + 1):
            p = range(b * block, (b + 1) * block)
            blocks.append(table[i][b * block // page] * (page // block) + b * block % page // block)
            rows.append([starts[i] + x - c if c <= x < c + n else -1 for x in p])
            old.append([x < c for x in p])
    if case["held"] != "none":
        s["blocks"], s["rows"], s["old"] = (_device(blocks, torch.int64), _device(rows, torch.int64),
                                            _device(old, torch.bool))
    return s


def _prepare_attend(case, seed):
    g, r, t = _generator(seed), random.Random(seed), TYPES[case["dtype"]]
    ctx, dr, page = _ints(case["ctx"]), _ints(case["drafts"]), case["page"]
    starts = _starts(dr)
    table, pool = _pages([c + n for c, n in zip(ctx, dr)], page, seed)
    shape = (pool, page, case["hkv"], case["d"])
    s = {"case": case, "q": torch.randn(starts[-1], case["hq"], case["d"], device="cuda", generator=g).to(t),
         "table": _device(table, torch.int32), "ctx": _device(ctx, torch.int32),
         "q_rowptr": _device(starts, torch.int32), "tree": None}
    for n in ("k", "v"):
        s[n], s[n + "_scale"] = _pool(shape, case["held"], case["block"], g)
    if case["form"] == "tree":
        s["tree"] = _device([m for n in dr for m in _masks(n, r)], torch.int64)
    # which row of q is draft a of sequence n, and the way back
    most = max(dr)
    s["rows"] = _device([[starts[n] + min(a, dr[n] - 1) for a in range(most)] for n in range(len(dr))],
                        torch.int64)
    s["inverse"] = _device([n * most + a for n in range(len(dr)) for a in range(dr[n])], torch.int64)
    s["keys"] = max(c + n for c, n in zip(ctx, dr))
    return s


def _prepare_compact(case, seed):
    g, r = _generator(seed), random.Random(seed)
    page, block, n = case["page"], case["block"], case["count"]
    s = {"case": case}
    for x in ("k", "v"):
        s[x], s[x + "_scale"] = _pool((case["layers"], case["pool"], page, case["hkv"], case["d"]), case["held"],
                                      block, g)
    order = list(range(case["pool"]))
    r.shuffle(order)
    wide = case["pool"] // n
    ctx, table, keep = [], [], []
    for i in range(n):
        # a context that its first page holds in part; the kept path goes on from the
        # first draft to drafts of later levels, which lie behind the blocks that
        # rows move into, so that a second pass finds what the first one found
        ctx.append(r.randint(0, page - 1))
        table.append(order[i * wide:(i + 1) * wide])
        kept = r.randint(1, 8)
        first = kept + block - 1
        path = sorted(r.sample(range(first, max(case["drafts"], first + 8)), kept - 1))
        keep.append([0] + path + [-1] * (8 - kept))
    s["ctx"], s["table"] = _device(ctx, torch.int32), _device(table, torch.int32)
    s["keep"] = _device(keep, torch.int32)
    return s


# -------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"append": _plain_append, "attend": _plain_attend, "compact": _plain_compact}[case["op"]](state, case)


def _outputs(*x):
    return tuple(t for t in x if t is not None)


def _own(s, case):
    import sparse_dense_linear_amd as sdl
    if case["op"] == "append":
        q = sdl.append_pages(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["ctx"], s["rowptr"],
                             q=s["q"], cos=s["cos"], sin=s["sin"], tree=s["tree"],
                             interleaved=case["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return _outputs(q, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    if case["op"] == "attend":
        return sdl.tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["q_rowptr"], s["tree"],
                                  window=case["window"], sinks=case["sinks"], k_scale=s["k_scale"],
                                  v_scale=s["v_scale"])
    sdl.compact_pages(s["k"], s["v"], s["table"], s["ctx"], s["keep"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"])
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _bits(tree):
    return (tree[:, None] >> torch.arange(64, device="cuda")) & 1


def _rotated(x, cos, sin, interleaved):
    """x [rows, heads, d] in 32 bits, cos and sin [rows, 1, half]."""
    half = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _codes(y, held):
    """Codes of values that are divided by their scale already, as bytes."""
    if held == "i8":
        return y.round().to(torch.int8).view(torch.uint8)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s, case):
    t, page, block, hkv, d = s["q"].dtype, case["page"], case["block"], case["hkv"], case["d"]
    at = s["ctx"].long()[s["seq"]] + s["row"]
    place = at
    if s["tree"] is not None:
        count = (s["rowptr"][1:] - s["rowptr"][:-1]).long()[s["seq"]]
        named = _bits(s["tree"]) * (torch.arange(64, device="cuda") < count[:, None])
        place = s["ctx"].long()[s["seq"]] + (named.sum(-1) - 1).clamp(min=0)
    cos, sin = s["cos"][place][:, None], s["sin"][place][:, None]
    q = _rotated(s["q"].float(), cos, sin, case["interleaved"]).to(t)
    k, v = _rotated(s["k"].float(), cos, sin, case["interleaved"]), s["v"].float()
    if case["held"] == "none":
        row = s["table"].long()[s["seq"], at // page] * page + at % page
        for pool, x in ((s["k_pages"], k), (s["v_pages"], v)):
            pool.view(-1, hkv, d)[row] = x.to(t)
        return q, s["k_pages"], s["v_pages"]
    held, old, fresh = case["held"], s["old"][:, :, None, None], (s["rows"] >= 0)[:, :, None, None]
    for pool, scale, x in ((s["k_pages"], s["k_scale"], k), (s["v_pages"], s["v_scale"], v)):
        codes, scales = pool.view(torch.uint8).view(-1, block, hkv, d), scale.view(-1, hkv)
        new = torch.where(fresh, x[s["rows"].clamp(min=0)], 0.0)                  # [blocks, block, hkv, d]
        top = new.abs().amax((1, 3))
        need = torch.ldexp(torch.ones_like(top), _exponent(top, held))
        before = scales[s["blocks"]]
        now = torch.where(s["old"].any(1)[:, None], torch.maximum(need, before), need)
        kept = codes[s["blocks"]]
        values = kept.view(pool.dtype).float() * before[:, None, :, None]
        made = _codes(torch.where(fresh, new, values) / now[:, None, :, None], held)
        codes[s["blocks"]] = torch.where(fresh | old, made, kept)
        scales[s["blocks"]] = now
    return q, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _softmax(x, seen):
    """(weights, lse) of the scores x where `seen`; rows that see nothing: 0 and -inf."""
    x = x.masked_fill(~seen, NEG)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    return p / torch.where(total == 0, torch.ones_like(total), total), lse


def _plain_attend(s, case):
    hq, hkv, d, page, block = case["hq"], case["hkv"], case["d"], case["page"], case["block"]
    n, most = s["rows"].shape
    group, scale, t = hq // hkv, d ** -0.5, s["q"].dtype
    j = torch.arange(s["keys"], device="cuda")
    number, inside = s["table"].long()[:, j // page], j % page                 # [n, keys]
    of = number * (page // block) + inside // block

    def rows(pool, scales):  # [n, hkv, keys, d]
        x = pool.reshape(-1, hkv, d)[number * page + inside].float()
        return (x * scales.view(-1, hkv)[of][..., None]).permute(0, 2, 1, 3).contiguous()

    k, v = rows(s["k"], s["k_scale"]), rows(s["v"], s["v_scale"])
    q = s["q"].float()[s["rows"]].view(n, most, hkv, group, d).permute(0, 2, 1, 3, 4)
    q = q.reshape(n, hkv, most * group, d)
    ctx, count = s["ctx"].long(), (s["q_rowptr"][1:] - s["q_rowptr"][:-1]).long()
    if case["form"] == "tree":
        bits = _bits(s["tree"])[s["rows"]]                                     # [n, most, 64]
        bits = bits * (torch.arange(64, device="cuda") < count[:, None])[:, None]
        pos = ctx[:, None] + bits.sum(-1) - 1                                  # [n, most]
        draft = (j - ctx[:, None]).clamp(-1, 64)                               # [n, keys]
        own_pos = pos.gather(1, draft.clamp(0, most - 1))                      # position of a draft's key
        kpos = torch.where(draft < 0, j.expand(n, -1), own_pos)
        tree = torch.gather(bits, 2, draft.clamp(0, 63)[:, None].expand(-1, most, -1)) > 0
        seen = (draft < 0)[:, None] | (tree & (draft < 64)[:, None])
    else:
        pos = ctx[:, None] + torch.arange(most, device="cuda")
        kpos = j.expand(n, -1)
        seen = kpos[:, None] <= pos[:, :, None]
    near = (pos[:, :, None] - kpos[:, None] < case["window"]) | (kpos < case["sinks"])[:, None]
    seen = (seen & near)[:, None, :, None].expand(n, 1, most, group, -1).reshape(n, 1, most * group, -1)
    w, lse = _softmax((q @ k.transpose(-1, -2).contiguous()) * scale, seen)

    def packed(x):
        return (x.view(n, hkv, most, group, -1).permute(0, 2, 1, 3, 4)
                .reshape(n * most, hq, -1)[s["inverse"]])

    return packed(w @ v).to(t), packed(lse)[:, :, 0].t().contiguous()


def _plain_compact(s, case):
    layers, page, block, hkv, d = case["layers"], case["page"], case["block"], case["hkv"], case["d"]
    keep, ctx, table = s["keep"].long(), s["ctx"].long(), s["table"].long()
    n, most = keep.shape
    spans = (block - 1 + most + block - 1) // block
    # the blocks from the context's last one on, and where their rows come from
    to = (ctx // block * block)[:, None] + torch.arange(spans * block, device="cuda")      # [n, rows]
    draft = to - ctx[:, None]
    kept = keep.gather(1, draft.clamp(0, most - 1))
    held = (draft < 0) | ((draft < most) & (kept >= 0))
    of = torch.where(held & (draft >= 0), ctx[:, None] + kept, to)
    last = table.shape[1] * page - 1

    def place(p):
        p = p.clamp(max=last)
        return table.gather(1, p // page) * page + p % page

    of, to_block = place(of), place(to)[:, ::block] // block                                # [n, spans]
    moved = (held & (draft >= 0)).view(n, spans, block).any(-1)
    held = held.view(1, n, spans, block, 1) & moved[None, :, :, None, None]
    for pool, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        rows, scales = pool.view(torch.uint8).view(layers, -1, hkv, d), scale.view(layers, -1, hkv)
        before = scales[:, of // block].view(layers, n, spans, block, hkv)
        now = torch.where(held, before, 0.0).amax(3)                                        # [layers, n, spans, hkv]
        values = rows[:, of].view(pool.dtype).float().view(layers, n, spans, block, hkv, d) * before[..., None]
        made = _codes(values / torch.where(now == 0, 1.0, now)[:, :, :, None, :, None], case["held"])
        layer, seq, span = torch.nonzero(moved.expand(layers, n, spans), as_tuple=True)
        at = to_block[seq, span]
        blocks = rows.view(layers, -1, block, hkv, d)
        chosen = held[0, seq, span][:, :, :, None]
        blocks[layer, at] = torch.where(chosen, made[layer, seq, span], blocks[layer, at])
        scales[layer, at] = now[layer, seq, span]
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


# ----------------------------------------------------------------- values

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "compact": _exact_compact}[case["op"]](s, case)


def _power(top, most):
    """The smallest power of two, not below 2^-126, that `most` times holds."""
    e = torch.ceil(torch.log2(top / most))
    e = torch.where(top > most * torch.exp2(e), e + 1, e)
    e = torch.where(top <= most * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp(min=-126.0))


def _exact_append(s, case):
    """The codes are not rounded here."""
    page, block, half = case["page"], case["block"], case["rotated"] // 2
    ctx, new, table = _ints(case["ctx"]), _ints(case["new"]), s["table"].tolist()
    masks = None if s["tree"] is None else s["tree"].tolist()
    at, places, where = 0, [], []
    for i, (c, n) in enumerate(zip(ctx, new)):
        for a in range(n):
            places.append(c + a if masks is None else
                          c + max(0, bin(masks[at + a] & ((1 << min(n, 64)) - 1)).count("1") - 1))
            where.append((table[i][(c + a) // page], (c + a) % page))
        at += n
    places = torch.tensor(places).cuda()
    turn = torch.complex(s["cos"][places].double(), s["sin"][places].double())[:, None]

    def rotated(x):
        x = x.double()
        y = x.clone()
        if case["interleaved"]:
            z = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2]) * turn
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    q, k, v = rotated(s["q"]), rotated(s["k"]), s["v"].double()
    pages, rows = (torch.tensor(x).cuda() for x in zip(*where))
    pools, scales = [], []
    for pool, scale, x in ((s["k_pages"], s["k_scale"], k), (s["v_pages"], s["v_scale"], v)):
        out = pool.double()
        if scale is None:
            out[pages, rows] = x
            pools.append(out)
            continue
        most = HELD[case["held"]][1]
        sc = scale.double()
        a = 0
        for i, (c, n) in enumerate(zip(ctx, new)):
            for b in range(c // block, (c + n - 1) // block + 1):
                lo, hi = max(c, b * block), min(c + n, (b + 1) * block)
                number, first = table[i][b * block // page], b * block % page
                rows_new = x[a + lo - c:a + hi - c]
                now = _power(rows_new.abs().amax((0, 2)), most)
                if lo > b * block:
                    before = sc[number, first // block]
                    now = torch.maximum(now, before)
                    out[number, first:first + lo - b * block] *= (before / now)[:, None]
                out[number, first + lo - b * block:first + hi - b * block] = rows_new / now[:, None]
                sc[number, first // block] = now
            a += n
        pools.append(out)
        scales.append(sc)
    return (q, *pools, *scales)


def _exact_attend(s, case):
    q = s["q"].double()
    o, lse = torch.zeros_like(q), torch.full((q.shape[1], q.shape[0]), NEG, dtype=torch.float64, device="cuda")
    masks = None if s["tree"] is None else s["tree"].tolist()
    group, page, block, at = case["hq"] // case["hkv"], case["page"], case["block"], 0
    for n, (c, m) in enumerate(zip(_ints(case["ctx"]), _ints(case["drafts"]))):
        ids = s["table"][n, :-(-(c + m) // page)].long()

        def rows(pool, scale):
            x = pool[ids].double() * scale[ids].double().repeat_interleave(block, 1)[..., None]
            return x.reshape(-1, case["hkv"], case["d"])[:c + m]

        k, v = rows(s["k"], s["k_scale"]), rows(s["v"], s["v_scale"])
        if masks is None:
            i, j = torch.arange(c, c + m, device="cuda")[:, None], torch.arange(c + m, device="cuda")
            seen = j <= i
        else:
            places = [c + bin(masks[at + a] & ((1 << m) - 1)).count("1") - 1 for a in range(m)]
            j = torch.cat([torch.arange(c), torch.tensor(places)]).cuda()
            i = torch.tensor(places).cuda()[:, None]
            seen = torch.tensor([[True] * c + [bool(masks[at + a] >> b & 1) for b in range(m)]
                                 for a in range(m)]).cuda()
        seen = seen & ((i - j < case["window"]) | (j < case["sinks"]))
        for h in range(case["hq"]):
            x = torch.where(seen, q[at:at + m, h] @ k[:, h // group].T / math.sqrt(case["d"]), NEG)
            ll = torch.logsumexp(x, 1)
            w = torch.where(seen, torch.exp(x - torch.where(ll == NEG, 0.0, ll)[:, None]), 0.0)
            o[at:at + m, h], lse[h, at:at + m] = w @ v[:, h // group], ll
        at += m
    return o, lse


def _exact_compact(s, case):
    """The codes are not rounded here."""
    page, block = case["page"], case["block"]
    out = []
    scales = []
    for pool, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        x, sc = pool.double(), scale.double()
        for row, c, kept in zip(s["table"].tolist(), s["ctx"].tolist(), s["keep"].tolist()):
            kept = [a for a in kept if a >= 0]
            for b in range(c // block, (c + len(kept) - 1) // block + 1):
                first = b * block
                rows = [(p, p if p < c else c + kept[p - c])
                        for p in range(first, min(first + block, c + len(kept)))]
                come = torch.stack([sc[:, row[f // page], f % page // block] for _, f in rows], 1)
                values = torch.stack([x[:, row[f // page], f % page] for _, f in rows], 1) * come[..., None]
                now = come.amax(1)
                for e, (p, _) in enumerate(rows):
                    x[:, row[p // page], p % page] = values[:, e] / now[..., None]
                sc[:, row[first // page], first % page // block] = now
        out.append(x)
        scales.append(sc)
    return (*out, *scales)


# ------------------------------------------------------------------- work

def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "compact":
        # of up to eight kept drafts, four and a half in the mean, all but the first move: read and written
        return {"bytes": case["layers"] * 2 * hkv * (2 * 3.5 * d + 4) * case["count"], "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        new, ctx, block = _ints(case["new"]), _ints(case["ctx"]), case["block"]
        rows = sum(new)
        held = 1 if case["held"] != "none" else size
        n = rows * d * (2 * case["hq"] * size + 2 * hkv * (size + held)) + 4 * rows * case["rotated"]
        if case["held"] != "none":
            n += 8 * hkv * sum((c + x - 1) // block - c // block + 1 for c, x in zip(ctx, new))
        return {"bytes": n, "flops": 3 * rows * case["rotated"] * (case["hq"] + hkv)}
    pairs = rows = scales = 0
    for c, m in zip(_ints(case["ctx"]), _ints(case["drafts"])):
        seen = min(c, case["window"] + case["sinks"]) + m
        rows += seen
        scales += seen // case["block"] + 1
        # a tree's drafts are counted as seen by all
        pairs += seen * m if case["form"] == "tree" else sum(
            min(c + a + 1, case["window"]) + min(case["sinks"], max(0, c + a + 1 - case["window"])) for a in range(m))
    heads = sum(_ints(case["drafts"])) * case["hq"]
    return {"bytes": 2 * hkv * (rows * d + 4 * scales) + 2 * heads * d * size + 4 * heads,
            "flops": 4 * pairs * case["hq"] * d}
