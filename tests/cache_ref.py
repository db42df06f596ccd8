"""Writing and moving rows of a paged cache from their definition (CPU), for the
tests of include/cache.h.

The definition rounds every product, sum and quotient once to fp32, so what it
stores is defined bit by bit: the same elementary operations of torch on fp32
tensors give it.  `rotated64` and the bounds of `code_tolerance` hold it
against 64 bits."""
from __future__ import annotations

import math

import torch

E4M3, INT8 = torch.float8_e4m3fn, torch.int8
MOST = {E4M3: 448.0, INT8: 127.0}
U = 2.0 ** -24


def scale_of_top(top, held):
    """The smallest power of two, at least 2^-126, with top <= MOST * scale."""
    if not top > 0:
        return 2.0 ** -126
    e = math.frexp(top / MOST[held])[1]        # top / MOST < 2^e (64 bits hold the quotient's side of a power)
    if top <= MOST[held] * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -126)


def codes_of(x, held):
    """Codes of fp32 values that are divided by their scale already."""
    return x.round().to(torch.int8) if held is INT8 else x.to(E4M3)


def values(codes, scale):
    """code * scale in 64 bits; scale broadcasts over the last dimension."""
    return codes.double() * scale.double()[..., None]


def rotate(x, cos, sin, interleaved, real=torch.float32):
    """x [rows, heads, D]; cos and sin [rows, R / 2]."""
    x, c, s = x.to(real), cos.to(real)[:, None], sin.to(real)[:, None]
    half = cos.shape[1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def rotation_tolerance(x, cos, sin, dtype):
    """How far a rotated value may be from 64 bits: two products and a sum in
    fp32 (each off by U of what it is, at most |x| |c| + |y| |s| <= size), and one
    rounding to dtype."""
    size = x.double().abs().amax(-1, keepdim=True) * 2 * max(float(cos.abs().max()), float(sin.abs().max()), 1.0)
    return size * (3 * U) + (size * torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0)


def places(ctx, rowptr, tree):
    """Where each row stands, and its position in the pages; -1: of no sequence."""
    T = rowptr[-1]
    stand, at, seq = [0] * T, [-1] * T, [-1] * T
    for s in range(len(ctx)):
        n = rowptr[s + 1] - rowptr[s]
        for t in range(n):
            r = rowptr[s] + t
            at[r], seq[r] = ctx[s] + t, s
            if tree is None:
                stand[r] = ctx[s] + t
            else:
                seen = bin(tree[r] & ((1 << min(n, 64)) - 1)).count("1")
                stand[r] = ctx[s] + max(seen, 1) - 1
    return stand, at, seq


def append_ref(k, v, k_pages, v_pages, table, ctx, rowptr, q=None, cos=None, sin=None, tree=None, interleaved=False,
               k_scale=None, v_scale=None):
    """The call on CPU tensors (table, ctx, rowptr and tree as lists); changes
    the pools and scales it is given and returns the rotated q, whose rows of no
    sequence are zero."""
    pages, page = k_pages.shape[:2]
    stand, at, seq = places(ctx, rowptr, tree)
    T = len(at)
    if cos is not None:
        rows = torch.tensor([min(p, cos.shape[0]) for p in stand], dtype=torch.int64)
        far = torch.full((1, cos.shape[1]), math.nan)
        c, s = torch.cat([cos, far])[rows], torch.cat([sin, far])[rows]
        turned = rotate(k[:T], c, s, interleaved)
        out = None if q is None else rotate(q[:T], c, s, interleaved).to(q.dtype)
    else:
        turned, out = k[:T].float(), None if q is None else q[:T].clone()
    if out is not None:
        whole = torch.zeros_like(q)
        for r in range(T):
            if seq[r] >= 0:
                whole[r] = out[r]
        out = whole

    def number(s, pos):
        p = pos // page
        n = table[s][p] if p < len(table[s]) else -1
        return n if 0 <= n < pages else -1

    for pool, scale, x in ((k_pages, k_scale, turned), (v_pages, v_scale, v[:T].float())):
        if scale is None:
            for r in range(T):
                n = number(seq[r], at[r]) if seq[r] >= 0 else -1
                if n >= 0:
                    pool[n, at[r] % page] = x[r].to(pool.dtype)
            continue
        held, block = pool.dtype, page // scale.shape[1]
        for s in range(len(ctx)):
            first, end = ctx[s], ctx[s] + rowptr[s + 1] - rowptr[s]
            if end == first:
                continue
            for begin in range(first // block * block, end, block):
                n = number(s, begin)
                if n < 0:
                    continue
                lo, hi = max(first, begin), min(end, begin + block)
                b, i0 = begin % page // block, begin % page
                new = x[rowptr[s] + lo - first:rowptr[s] + hi - first]
                for h in range(pool.shape[2]):
                    y = new[:, h].clone()
                    top = y.abs()
                    top = float(top[top.isfinite()].max()) if bool(top.isfinite().any()) else 0.0
                    now = torch.tensor(scale_of_top(top, held))
                    if held is INT8 and not bool(y.isfinite().all()):
                        now = torch.tensor(math.nan)
                    before = scale[n, b, h].clone()
                    if lo > begin and not bool(now.isnan()):
                        now = torch.maximum(now, before)
                    if lo > begin and bool(now != before):
                        old = pool[n, i0:i0 + lo - begin, h]
                        pool[n, i0:i0 + lo - begin, h] = codes_of(old.float() * before / now, held)
                    y[~y.isfinite()] = math.nan
                    pool[n, i0 + lo - begin:i0 + hi - begin, h] = codes_of(y / now, held)
                    scale[n, b, h] = now
    return out


def compact_ref(k_pool, v_pool, table, ctx, keep, k_scale, v_scale):
    """compact_pages of pools of codes, on CPU tensors and lists."""
    pages, page = k_pool.shape[1:3]
    block = page // k_scale.shape[2]

    def place(s, pos):
        p = pos // page
        n = table[s][p] if 0 <= p < len(table[s]) else -1
        return (n, pos % page) if 0 <= n < pages else None

    for pool, scale in ((k_pool, k_scale), (v_pool, v_scale)):
        held = pool.dtype
        for s in range(len(ctx)):
            kept = []
            for a in keep[s]:
                if a < 0:
                    break
                kept.append(a)
            end = ctx[s] + len(kept)
            for begin in range(ctx[s] // block * block, end, block):
                to = place(s, begin)
                if to is None:
                    continue
                rows = []                       # (place in the block, where it comes from)
                for p in range(max(begin, ctx[s]), min(begin + block, end)):
                    of = place(s, ctx[s] + kept[p - ctx[s]])
                    if of is not None:
                        rows.append((p - begin, of))
                if not rows:
                    continue
                rows = [(p - begin, (to[0], to[1] + p - begin)) for p in range(begin, min(ctx[s], begin + block))] + rows
                come = torch.stack([scale[:, n, i // block] for _, (n, i) in rows], 1)       # [layers, rows, heads]
                code = torch.stack([pool[:, n, i].float() for _, (n, i) in rows], 1)
                now = come[:, 0]
                for i in range(1, come.shape[1]):
                    now = torch.maximum(now, come[:, i])
                made = torch.where((come == now[:, None])[..., None], code,
                                   codes_of(code * come[..., None] / now[:, None, :, None], held).float())
                for i, (p, _) in enumerate(rows):
                    pool[:, to[0], to[1] + p] = made[:, i].to(held)
                scale[:, to[0], to[1] // block] = now
