"""Attention over a window with first tokens that stay visible, attention of
drafted tokens over a paged cache, and the moves of the cache's pages: the
measured cases, their plain forms and their values in 64 bits.

window  q [Tq, Hq, D], k and v [Tk, Hkv, D]: sequences packed one after
        another, cut by row pointers.  The queries of a sequence are its last
        positions: query i of Lq has position i + Lk - Lq.  A query at
        position p sees key j when j <= p and (p - j < window or j < sinks).
        "fwd" returns (o, lse); "train" one step, (o, lse, dq, dk, dv).
tree    one group of drafted tokens for each sequence, their keys and values
        already in the cache behind the context; bit a of a token's mask says
        that it sees draft a of its sequence.  A token's position is
        context + (number of drafts it sees) - 1.  Returns (o, lse).
pages   "copy": pages dst[i] <- src[i] in every layer (a fork's partly filled
        pages); "compact": the kept drafts move to the front of their
        sequence's drafts in every layer.  Both return the two pools.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NEG = -math.inf
BLOCK = 128  # queries of one block of the plain form


def _ints(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(int(x)) for x in values)


def _spread(count, low, high, seed):
    """`count` lengths between low and high, spread over their logarithm."""
    r = random.Random(seed)
    return _text(math.exp(r.uniform(math.log(low), math.log(high))) for _ in range(count))


def _window(name, form, dtype, q, k, hq, hkv, d, window, sinks):
    c = {"name": name, "op": "window", "form": form, "dtype": dtype, "q": q, "k": k, "hq": hq,
         "hkv": hkv, "d": d, "window": window, "sinks": sinks}
    return c


def _tree(name, dtype, ctx, drafts, hq, hkv, d, page, window, sinks):
    return {"name": name, "op": "tree", "dtype": dtype, "ctx": ctx, "drafts": drafts, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "window": window, "sinks": sinks}


def _pages(name, form, dtype, layers, pool, page, hkv, d, count, drafts):
    return {"name": name, "op": "pages", "form": form, "dtype": dtype, "layers": layers,
            "pool": pool, "page": page, "hkv": hkv, "d": d, "count": count, "drafts": drafts}


def listed():
    long = "4096,2048,1500,500,48"
    return [
        # a batch of prompts of very different lengths, encoded at once
        _window("prefill_bf16", "fwd", "bf16", "8192,4096,2500,1333,263", "8192,4096,2500,1333,263",
                32, 8, 128, 1024, 4),
        # the next piece of prompts that are taken in pieces, beside one that is answering
        _window("prefill_piece_bf16", "fwd", "bf16", "512,512,300,1", "16384,9000,300,4097",
                32, 8, 128, 4096, 16),
        # a small training step, bound by its launches
        _window("train_small_bf16", "train", "bf16", "200,57", "200,57", 4, 4, 64, 48, 2),
        # a training step of packed documents
        _window("train_bf16", "train", "bf16", long, long, 32, 8, 128, 1024, 4),
        # the same in full precision, with a head size that is not a power of two
        _window("train_f32", "train", "f32", "1024,700,301", "1024,700,301", 8, 4, 80, 300, 4),
        # three answers that have just begun, in full precision: latency counts
        _tree("answer_small_f32", "f32", "0,333,1000", "1,1,4", 16, 16, 96, 24, 1 << 30, 0),
        # a batch of answers, one token each: the cache's bytes count
        _tree("answer_batch_bf16", "bf16", _spread(64, 1000, 16384, 1), _text([1] * 64), 32, 8, 128,
              64, 1 << 30, 0),
        # trees of drafts for a batch of answers, with a window and first tokens
        _tree("draft_trees_bf16", "bf16", _spread(16, 500, 12000, 2), _spread(16, 16, 64, 3), 32, 4,
              128, 32, 4096, 4),
        # one answer forks into a few
        _pages("fork_small_f32", "copy", "f32", 4, 64, 16, 4, 64, 3, 0),
        # a beam step over a batch: the partly filled pages of each fork
        _pages("fork_bf16", "copy", "bf16", 32, 1024, 16, 8, 128, 250, 0),
        # the accepted drafts of two answers
        _pages("accept_small_f32", "compact", "f32", 4, 64, 24, 4, 96, 2, 32),
        # the accepted drafts of a batch
        _pages("accept_bf16", "compact", "bf16", 32, 1024, 16, 8, 128, 128, 64),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    dtype = rng.choice(["bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([40, 64, 72, 96, 128, 128])
    op = rng.choice(["fwd", "train", "tree", "tree", "copy", "compact"])
    if op in ("fwd", "train"):
        hq = hkv * rng.choice([1, 2, 4])
        total, n = log(20, 8192 if op == "fwd" else 4096), rng.choice([1, 2, 3, 5, 8])
        q = [max(1, int(total * rng.uniform(0.2, 1) / n)) for _ in range(n)]
        k = [x + (log(1, 2000) if op == "fwd" and rng.random() < 0.5 else 0) for x in q]
        return _drop(_window("", op, dtype, _text(q), _text(k), hq, hkv, d, log(1, 1500),
                             rng.choice([0, 1, 4, 16, 33])))
    if op == "tree":
        n, most = log(1, 48), rng.choice([1, 1, 9, 33, 64])
        hq = hkv * rng.choice([1, 3, 4, 8])
        ctx = [log(1, 8000) if rng.random() < 0.95 else 0 for _ in range(n)]
        return _drop(_tree("", dtype, _text(ctx), _text(rng.randint(1, most) for _ in range(n)), hq,
                           hkv, d, rng.choice([1, 16, 24, 32, 64, 100]),
                           rng.choice([1 << 30, log(10, 6000)]), rng.choice([0, 4, 17])))
    layers, page, count = log(1, 24), rng.choice([8, 16, 24, 64]), log(1, 64)
    drafts = log(9, 64)
    return _drop(_pages("", op, dtype, layers, log(count * (2 + 80 // page), 600) if count * (2 + 80 // page) < 600
                        else count * (2 + 80 // page), page, hkv, d, count, drafts if op == "compact" else 0))


def _drop(case):
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    return {"window": _prepare_window, "tree": _prepare_tree, "pages": _prepare_pages}[case["op"]](
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


def _prepare_window(case, seed):
    g, t = _generator(seed), TYPES[case["dtype"]]
    ql, kl = _ints(case["q"]), _ints(case["k"])
    qs, ks = _starts(ql), _starts(kl)
    d = case["d"]

    def normal(rows, heads):
        return torch.randn(rows, heads, d, device="cuda", generator=g).to(t)

    s = {"case": case, "q": normal(qs[-1], case["hq"]), "k": normal(ks[-1], case["hkv"]),
         "v": normal(ks[-1], case["hkv"]), "do": normal(qs[-1], case["hq"]),
         "q_rowptr": _device(qs, torch.int32), "k_rowptr": _device(ks, torch.int32)}
    # the blocks of the plain form: BLOCK queries of one sequence and the keys
    # that any of them sees
    rows, pos, keys, kpos, inverse = [], [], [], [], [0] * qs[-1]
    for n in range(len(ql)):
        for b in range(0, ql[n], BLOCK):
            r = list(range(b, min(b + BLOCK, ql[n])))
            at = len(rows) * BLOCK
            for i in r:
                inverse[qs[n] + i] = at + i - b
            p = [i + kl[n] - ql[n] for i in r]
            low = max(0, min(p) - case["window"] + 1)
            seen = list(range(min(case["sinks"], low))) + list(range(low, p[-1] + 1))
            rows.append([qs[n] + i for i in r] + [0] * (BLOCK - len(r)))
            pos.append(p + [-1] * (BLOCK - len(r)))
            keys.append([ks[n] + j for j in seen])
            kpos.append(seen)
    most = max(1, max(len(x) for x in keys))
    s["rows"] = _device(rows, torch.int64)
    s["pos"] = _device(pos, torch.int64)
    s["keys"] = _device([x + [0] * (most - len(x)) for x in keys], torch.int64)
    s["kpos"] = _device([x + [1 << 40] * (most - len(x)) for x in kpos], torch.int64)
    s["inverse"] = _device(inverse, torch.int64)
    return s


def _masks(drafts, r):
    """Masks of a random tree of drafts: each token sees itself and what its parent sees."""
    m = []
    for a in range(drafts):
        parent = r.randint(max(-1, a - 9), a - 1) if a else -1
        m.append((m[parent] if parent >= 0 else 0) | (1 << a))
    return [x - (1 << 64) if x >> 63 else x for x in m]


def _prepare_tree(case, seed):
    g, r, t = _generator(seed), random.Random(seed), TYPES[case["dtype"]]
    ctx, dr, page = _ints(case["ctx"]), _ints(case["drafts"]), case["page"]
    starts = _starts(dr)
    need = [-(-(c + n) // page) for c, n in zip(ctx, dr)]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [0] * (max(need) - n))
        at += n
    shape = (pool, page, case["hkv"], case["d"])
    s = {"case": case, "q": torch.randn(starts[-1], case["hq"], case["d"], device="cuda", generator=g).to(t),
         "k": torch.randn(shape, device="cuda", generator=g).to(t),
         "v": torch.randn(shape, device="cuda", generator=g).to(t),
         "table": _device(table, torch.int32), "ctx": _device(ctx, torch.int32),
         "q_rowptr": _device(starts, torch.int32),
         "tree": _device([m for n in dr for m in _masks(n, r)], torch.int64)}
    # which row of q is draft a of sequence n, and the way back
    most = max(dr)
    s["rows"] = _device([[starts[n] + min(a, dr[n] - 1) for a in range(most)] for n in range(len(dr))],
                        torch.int64)
    s["inverse"] = _device([n * most + a for n in range(len(dr)) for a in range(dr[n])], torch.int64)
    s["keys"] = max(c + n for c, n in zip(ctx, dr))
    return s


def _prepare_pages(case, seed):
    g, r, t = _generator(seed), random.Random(seed), TYPES[case["dtype"]]
    shape = (case["layers"], case["pool"], case["page"], case["hkv"], case["d"])
    s = {"case": case, "k": torch.randn(shape, device="cuda", generator=g).to(t),
         "v": torch.randn(shape, device="cuda", generator=g).to(t)}
    order = list(range(case["pool"]))
    r.shuffle(order)
    n, page = case["count"], case["page"]
    if case["form"] == "copy":
        s["dst"] = _device(order[:n], torch.int32)
        s["src"] = _device([r.choice(order[n:]) for _ in range(n)], torch.int32)
        return s
    ctx, table, keep, at = [], [], [], 0
    wide = case["pool"] // n
    for _ in range(n):
        # a context that its first page holds in part, and drafts in levels of
        # eight: the path that is kept has one of each level, and nothing
        # that moves is written over by what moves before it, so that a
        # second pass finds what the first one found
        ctx.append(r.randint(0, page - 1))
        table.append(order[at:at + wide])
        at += wide
        path, levels = [0], (case["drafts"] - 1) // 8
        kept = r.randint(1, min(8, 1 + levels))
        path += [r.randint(max(kept, 8 * e + 1), 8 * e + 8) for e in range(kept - 1)]
        keep.append(path + [-1] * (8 - kept))
    s["ctx"], s["table"] = _device(ctx, torch.int32), _device(table, torch.int32)
    s["keep"] = _device(keep, torch.int32)
    return s


# -------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"window": _plain_window, "tree": _plain_tree, "pages": _plain_pages}[case["op"]](state, case)


def _own(s, case):
    import sparse_dense_linear_amd as sdl
    if case["op"] == "window":
        a = dict(window=case["window"], sinks=case["sinks"])
        o, lse = sdl.window_attention(s["q"], s["k"], s["v"], s["q_rowptr"], s["k_rowptr"], **a)
        if case["form"] == "fwd":
            return o, lse
        dq, dk, dv = sdl.window_attention_backward(s["do"], s["q"], s["k"], s["v"], o, lse,
                                                   s["q_rowptr"], s["k_rowptr"], **a)
        return o, lse, dq, dk, dv
    if case["op"] == "tree":
        return sdl.tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["q_rowptr"], s["tree"],
                                  window=case["window"], sinks=case["sinks"])
    if case["form"] == "copy":
        sdl.copy_pages(s["k"], s["v"], s["src"], s["dst"])
    else:
        sdl.compact_pages(s["k"], s["v"], s["table"], s["ctx"], s["keep"])
    return s["k"], s["v"]


def _softmax(x, seen):
    """(weights, lse) of the scores x where `seen`; rows that see nothing: 0 and -inf."""
    x = x.masked_fill(~seen, NEG)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    return p / torch.where(total == 0, torch.ones_like(total), total), lse


def _plain_window(s, case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n, group, scale = s["rows"].shape[0], case["hq"] // case["hkv"], case["d"] ** -0.5
    t = s["q"].dtype

    def blocked(x):  # [rows, hq, d] -> [n, hkv, group * BLOCK, d]
        return (x.float()[s["rows"]].view(n, BLOCK, hkv, group, d).permute(0, 2, 3, 1, 4)
                .reshape(n, hkv, group * BLOCK, d))

    def packed(x):  # the way back
        return (x.view(n, hkv, group, BLOCK, -1).permute(0, 3, 1, 2, 4)
                .reshape(n * BLOCK, hq, -1)[s["inverse"]])

    q = blocked(s["q"])
    k = s["k"].float()[s["keys"]].permute(0, 2, 1, 3).contiguous()
    v = s["v"].float()[s["keys"]].permute(0, 2, 1, 3).contiguous()
    p, j = s["pos"][:, :, None], s["kpos"][:, None, :]
    seen = (j <= p) & ((p - j < case["window"]) | (j < case["sinks"]))
    seen = seen[:, None, None].expand(n, 1, group, BLOCK, -1).reshape(n, 1, group * BLOCK, -1)
    w, lse = _softmax((q @ k.transpose(-1, -2).contiguous()) * scale, seen)
    o = w @ v
    out = [packed(o).to(t), packed(lse)[:, :, 0].t().contiguous()]
    if case["form"] == "fwd":
        return tuple(out)
    do = blocked(s["do"]) * (s["pos"] >= 0)[:, None, None, :, None].expand(n, 1, group, BLOCK, 1).reshape(
        n, 1, group * BLOCK, 1)
    delta = (do * o).sum(-1, keepdim=True)
    ds = w * (do @ v.transpose(-1, -2).contiguous() - delta) * scale
    dq = packed(ds @ k).to(t)

    def summed(x):  # [n, hkv, keys, d] -> [tk, hkv, d]
        out = torch.zeros(s["k"].shape, dtype=torch.float32, device=x.device)
        return out.index_add_(0, s["keys"].reshape(-1), x.permute(0, 2, 1, 3).reshape(-1, hkv, d)).to(t)

    dk = summed(ds.transpose(-1, -2).contiguous() @ q)
    dv = summed(w.transpose(-1, -2).contiguous() @ do)
    return out[0], out[1], dq, dk, dv


def _plain_tree(s, case):
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    n, most = s["rows"].shape
    group, scale, t = hq // hkv, d ** -0.5, s["q"].dtype
    j = torch.arange(s["keys"], device="cuda")
    at = s["table"].long()[:, j // page] * page + j % page            # [n, keys]
    k = s["k"].reshape(-1, hkv, d)[at].float().permute(0, 2, 1, 3)     # [n, hkv, keys, d]
    v = s["v"].reshape(-1, hkv, d)[at].float().permute(0, 2, 1, 3).contiguous()
    q = s["q"].float()[s["rows"]].view(n, most, hkv, group, d).permute(0, 2, 1, 3, 4)
    q = q.reshape(n, hkv, most * group, d)
    bits = (s["tree"][s["rows"]][:, :, None] >> torch.arange(64, device="cuda")) & 1  # [n, most, 64]
    count = (s["q_rowptr"][1:] - s["q_rowptr"][:-1]).long()
    bits = bits * (torch.arange(64, device="cuda") < count[:, None])[:, None]
    ctx = s["ctx"].long()
    pos = ctx[:, None] + bits.sum(-1) - 1                               # [n, most]
    draft = (j - ctx[:, None]).clamp(-1, 64)                            # [n, keys]
    own_pos = pos.gather(1, draft.clamp(0, most - 1))                   # position of a draft's key
    kpos = torch.where(draft < 0, j.expand(n, -1), own_pos)
    tree = torch.gather(bits, 2, draft.clamp(0, 63)[:, None].expand(-1, most, -1)) > 0
    seen = (draft < 0)[:, None] | (tree & (draft < 64)[:, None])
    near = (pos[:, :, None] - kpos[:, None] < case["window"]) | (kpos < case["sinks"])[:, None]
    seen = (seen & near)[:, None, :, None].expand(n, 1, most, group, -1).reshape(n, 1, most * group, -1)
    w, lse = _softmax((q @ k.transpose(-1, -2).contiguous()) * scale, seen)

    def packed(x):
        return (x.view(n, hkv, most, group, -1).permute(0, 2, 1, 3, 4)
                .reshape(n * most, hq, -1)[s["inverse"]])

    return packed(w @ v).to(t), packed(lse)[:, :, 0].t().contiguous()


def _plain_pages(s, case):
    if case["form"] == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        s["k"][:, dst] = s["k"][:, src]
        s["v"][:, dst] = s["v"][:, src]
        return s["k"], s["v"]
    page = case["page"]
    keep = s["keep"].long()
    to = s["ctx"].long()[:, None] + torch.arange(keep.shape[1], device="cuda")
    of = torch.where(keep < 0, to, s["ctx"].long()[:, None] + keep)     # what is not kept stays
    table = s["table"].long()

    def place(p):
        return (table.gather(1, p // page) * page + p % page).reshape(-1)

    flat = (case["layers"], case["pool"] * page, case["hkv"], case["d"])
    a, b = place(of), place(to)
    for x in (s["k"].view(flat), s["v"].view(flat)):
        x[:, b] = x[:, a]
    return s["k"], s["v"]


# ----------------------------------------------------------------- values

def exact(case, seed):
    s = prepare(case, seed)
    return {"window": _exact_window, "tree": _exact_tree, "pages": _exact_pages}[case["op"]](s, case)


def _attend(q, k, v, seen, scale):
    """One head in 64 bits: q [a, d], k and v [b, d], seen [a, b] -> o, lse, weights."""
    x = torch.where(seen, (q @ k.T) * scale, torch.full((), NEG, dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(x, 1)
    w = torch.where(seen, torch.exp(x - torch.where(lse == NEG, 0.0, lse)[:, None]), 0.0)
    return w @ v, lse, w


def _exact_window(s, case):
    q, k, v, do = (s[x].double() for x in ("q", "k", "v", "do"))
    o, lse = torch.zeros_like(q), torch.full((q.shape[1], q.shape[0]), NEG, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    scale, group = 1 / math.sqrt(case["d"]), case["hq"] // case["hkv"]
    ql, kl = _ints(case["q"]), _ints(case["k"])
    a0 = b0 = 0
    for lq, lk in zip(ql, kl):
        for c in range(0, lq, 1024):
            i = torch.arange(c, min(c + 1024, lq), device="cuda")[:, None] + lk - lq
            lo = max(0, c + lk - lq - case["window"] + 1)
            top = int(i[-1]) + 1
            j = torch.cat([torch.arange(min(case["sinks"], lo)), torch.arange(lo, max(lo, top))]).cuda()
            seen = (j <= i) & ((i - j < case["window"]) | (j < case["sinks"]))
            at = slice(a0 + c, a0 + c + i.shape[0])
            for h in range(case["hq"]):
                kk, vv = k[b0 + j, h // group], v[b0 + j, h // group]
                oo, ll, w = _attend(q[at, h], kk, vv, seen, scale)
                o[at, h], lse[h, at] = oo, ll
                if case["form"] == "train":
                    g = do[at, h]
                    ds = w * (g @ vv.T - (g * oo).sum(1, keepdim=True)) * scale
                    dq[at, h] = ds @ kk
                    dk[b0 + j, h // group] += ds.T @ q[at, h]
                    dv[b0 + j, h // group] += w.T @ g
        a0, b0 = a0 + lq, b0 + lk
    return (o, lse) if case["form"] == "fwd" else (o, lse, dq, dk, dv)


def _exact_tree(s, case):
    q = s["q"].double()
    o, lse = torch.zeros_like(q), torch.full((q.shape[1], q.shape[0]), NEG, dtype=torch.float64, device="cuda")
    masks = s["tree"].tolist()
    group, page, at = case["hq"] // case["hkv"], case["page"], 0
    for n, (c, m) in enumerate(zip(_ints(case["ctx"]), _ints(case["drafts"]))):
        ids = s["table"][n, :-(-(c + m) // page)].long()
        k = s["k"][ids].reshape(-1, case["hkv"], case["d"])[:c + m].double()
        v = s["v"][ids].reshape(-1, case["hkv"], case["d"])[:c + m].double()
        places = [c + bin(masks[at + a] & ((1 << m) - 1)).count("1") - 1 for a in range(m)]
        j = torch.cat([torch.arange(c), torch.tensor(places)]).cuda()
        i = torch.tensor(places).cuda()[:, None]
        seen = torch.tensor([[True] * c + [bool(masks[at + a] >> b & 1) for b in range(m)] for a in range(m)]).cuda()
        seen &= (i - j < case["window"]) | (j < case["sinks"])
        for h in range(case["hq"]):
            o[at:at + m, h], lse[h, at:at + m], _ = _attend(q[at:at + m, h], k[:, h // group], v[:, h // group],
                                                            seen, 1 / math.sqrt(case["d"]))
        at += m
    return o, lse


def _exact_pages(s, case):
    k, v = s["k"].double(), s["v"].double()
    if case["form"] == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            k[:, b], v[:, b] = k[:, a], v[:, a]
        return k, v
    page = case["page"]
    for row, c, kept in zip(s["table"].tolist(), s["ctx"].tolist(), s["keep"].tolist()):
        for t, a in enumerate(x for x in kept if x >= 0):
            f, g = c + a, c + t
            k[:, row[g // page], g % page] = k[:, row[f // page], f % page]
            v[:, row[g // page], g % page] = v[:, row[f // page], f % page]
    return k, v


# ------------------------------------------------------------------- work

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] == "pages":
        row = case["layers"] * 2 * case["hkv"] * d * size
        if case["form"] == "copy":
            return {"bytes": 2 * row * case["page"] * case["count"], "flops": 0}
        # on average half of the kept path; its first token stays where it is
        kept = min(8, 1 + (case["drafts"] - 1) // 8)
        return {"bytes": row * case["count"] * max(1, kept - 1), "flops": 0}
    if case["op"] == "tree":
        pairs = rows = 0
        for c, m in zip(_ints(case["ctx"]), _ints(case["drafts"])):
            seen = min(c, case["window"] + case["sinks"]) + m
            rows += seen
            pairs += seen * m
        heads = sum(_ints(case["drafts"])) * case["hq"]
        return {"bytes": 2 * rows * case["hkv"] * d * size + 2 * heads * d * size + 4 * heads,
                "flops": 4 * pairs * case["hq"] * d}
    pairs = 0
    ql, kl = _ints(case["q"]), _ints(case["k"])
    for lq, lk in zip(ql, kl):
        # query at position p sees min(p + 1, window) keys of the window and
        # min(sinks, what lies before it) first ones
        pairs += sum(min(p + 1, case["window"]) + min(case["sinks"], max(0, p + 1 - case["window"]))
                     for p in range(max(0, lk - lq), lk))
    q, kv = sum(ql) * case["hq"] * d * size, sum(kl) * case["hkv"] * d * size
    lse = 4 * sum(ql) * case["hq"]
    if case["form"] == "fwd":
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs * case["hq"] * d}
    # one step: q, k, v and do read, o, lse, dq, dk and dv written
    return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * pairs * case["hq"] * d}
