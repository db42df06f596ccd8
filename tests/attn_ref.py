"""Attention from its definition in 64 bits (CPU), with the bound of each
element's error, for the tests of the attention operators.

The bounds are first order in the roundings of the kernels, which the
interface states: sums and softmax statistics in fp32, weights and score
gradients rounded to the element type once as operands, results rounded once.
u = 2^-24 is half a step of fp32; uw and uo are half a step of the element
type for those two roundings (uw = 0 for fp32, where nothing is rounded
below).  A fp32 sum of n products is taken to be off by at most 2 n u times
the sum of their magnitudes (any order, matrix instructions included), a
base-2 exponential or logarithm by 8 u.  SLACK covers products of two
roundings."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
SLACK = 1.05


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def seen_window(lq, lk, window, sinks):
    i = torch.arange(lq)[:, None] + lk - lq
    j = torch.arange(lk)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def head_forward(q, k, v, seen, scale, dtype):
    """q [a, d], k, v [b, d] (float64), seen [a, b] -> dict of o, lse, the
    weights p, and bounds of |error|: o_tol, lse_tol, p_rel."""
    uw = half_step(dtype) if dtype != torch.float32 else 0.0
    uo = half_step(dtype)
    D, n = q.shape[1], max(1, int(seen.sum(1).max()) if seen.numel() else 1)
    x = (q @ k.T) * scale
    mag = (q.abs() @ k.abs().T) * scale
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, 1) if x.shape[1] else torch.full((x.shape[0],), -math.inf, dtype=x.dtype)
    p = torch.where(seen, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
    # a score: its sum, then the factor and the subtraction of the maximum
    ds = torch.where(seen, 2 * D * U * mag + 4 * U * mag + 2 * U, 0.0)
    ds = ds.amax(1) if ds.shape[1] else torch.zeros(ds.shape[0], dtype=x.dtype)
    lse_tol = ds + (2 * n + 16) * U + 4 * U * torch.where(lse == -math.inf, 0.0, lse).abs()
    p_rel = 2 * ds + (2 * n + 32) * U          # against the sum of the same errors
    o = p @ v
    o_tol = SLACK * ((p_rel + uw + 2 * n * U)[:, None] * (p @ v.abs()) + uo * o.abs()) + 1e-30
    return {"o": o, "lse": lse, "p": p, "o_tol": o_tol, "lse_tol": lse_tol + 1e-30, "p_rel": p_rel,
            "uw": uw, "uo": uo, "n": n}


def head_backward(f, q, k, v, do, scale):
    """Gradients of sum(o * do) of one head from head_forward's answer; the
    sums over heads are the caller's.  Returns values and bounds without the
    last rounding (mag_*: what fp32 sums of them scale with)."""
    p, o = f["p"], f["o"]
    D = q.shape[1]
    lse = torch.where(f["lse"] == -math.inf, 0.0, f["lse"])
    # weights again from q, k and the stored lse
    p_rel = f["p_rel"] + f["lse_tol"] + 4 * U * lse.abs() + 16 * U
    dp, mag = do @ v.T, do.abs() @ v.abs().T
    delta = (do * o).sum(1)
    delta_tol = (do.abs() * f["o_tol"]).sum(1) + 2 * D * U * (do * o).abs().sum(1)
    ds = p * (dp - delta[:, None])
    ds_tol = p * (p_rel[:, None] * (dp - delta[:, None]).abs() + 2 * D * U * mag + delta_tol[:, None] +
                  2 * U * (dp.abs() + delta.abs()[:, None])) + f["uw"] * ds.abs()
    dv_tol = p.T @ ((p_rel + f["uw"])[:, None] * do.abs())
    return {"dq": ds @ k * scale, "dk": ds.T @ q * scale, "dv": p.T @ do,
            "dq_tol": ds_tol @ k.abs() * scale, "dk_tol": ds_tol.T @ q.abs() * scale, "dv_tol": dv_tol,
            "dq_mag": ds.abs() @ k.abs() * scale, "dk_mag": ds.abs().T @ q.abs() * scale,
            "dv_mag": p.T @ do.abs()}


def window_ref(q, k, v, q_rowptr, k_rowptr, window, sinks, scale=None, do=None):
    """Values and bounds for packed sequences (tensors of the kernels' inputs,
    on the CPU; row pointers as lists).  Rows of no sequence: NaN."""
    dtype = q.dtype
    Hq, Hkv, D = q.shape[1], k.shape[1], q.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    G = Hq // Hkv
    nan = float("nan")
    out = {"o": torch.full(q.shape, nan, dtype=torch.float64),
           "lse": torch.full((Hq, q.shape[0]), nan, dtype=torch.float64)}
    out["o_tol"], out["lse_tol"] = torch.zeros_like(out["o"]), torch.zeros_like(out["lse"])
    if do is not None:
        for n, t in (("dq", q), ("dk", k), ("dv", k)):
            out[n] = torch.full(t.shape, nan, dtype=torch.float64)
            out[n + "_tol"] = torch.zeros(t.shape, dtype=torch.float64)
    uo = half_step(dtype)
    for s in range(len(q_rowptr) - 1):
        a, b = slice(q_rowptr[s], q_rowptr[s + 1]), slice(k_rowptr[s], k_rowptr[s + 1])
        lq, lk = a.stop - a.start, b.stop - b.start
        seen = seen_window(lq, lk, window, sinks)
        if do is not None:
            acc = {n: torch.zeros((lk, Hkv, D), dtype=torch.float64)
                   for n in ("dk", "dv", "dk_tol", "dv_tol", "dk_mag", "dv_mag")}
        for h in range(Hq):
            qq, kk, vv = q[a, h].double(), k[b, h // G].double(), v[b, h // G].double()
            f = head_forward(qq, kk, vv, seen, scale, dtype)
            out["o"][a, h], out["o_tol"][a, h] = f["o"], f["o_tol"]
            out["lse"][h, a], out["lse_tol"][h, a] = f["lse"], f["lse_tol"]
            if do is not None:
                g = head_backward(f, qq, kk, vv, do[a, h].double(), scale)
                out["dq"][a, h] = g["dq"]
                out["dq_tol"][a, h] = SLACK * (g["dq_tol"] + 2 * f["n"] * U * g["dq_mag"] +
                                               uo * g["dq"].abs()) + 1e-30
                for n in acc:
                    acc[n][:, h // G] += g[n]
        if do is not None:
            n = max(1, lq * G)
            for x in ("dk", "dv"):
                out[x][b] = acc[x]
                out[x + "_tol"][b] = SLACK * (acc[x + "_tol"] + 2 * n * U * acc[x + "_mag"] +
                                              uo * acc[x].abs()) + 1e-30
    return out


def tree_seen(ctx, masks, window, sinks):
    """[T, ctx + T] of one sequence."""
    T = len(masks)
    kept = [m & ((1 << T) - 1) & ((1 << 64) - 1) for m in masks]
    place = [ctx + max(bin(m).count("1"), 1) - 1 for m in kept]
    kpos = torch.tensor(list(range(ctx)) + place, dtype=torch.int64)
    pos = torch.tensor(place, dtype=torch.int64)[:, None]
    named = torch.tensor([[True] * ctx + [a < 64 and bool(m >> a & 1) for a in range(T)] for m in kept],
                         dtype=torch.bool)
    return named.reshape(T, ctx + T) & ((pos - kpos < window) | (kpos < sinks))


def chain_seen(ctx, T, window, sinks):
    return seen_window(T, ctx + T, window, sinks)


def assert_close(got, want, tol, what):
    """|got - want| <= tol element by element; infinities and NaN must agree."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, not {tuple(want.shape)}"
    odd = ~torch.isfinite(want)
    same = (got == want) | (got.isnan() & want.isnan())
    bad = torch.where(odd, ~same, ~((got - want).abs() <= tol))
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        err = ((got - want).abs() / tol)[bad & ~odd]
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} elements outside their bound (worst "
            f"{float(err.max()) if err.numel() else math.inf:.3g} times); first at {at}: "
            f"{float(got[at])!r}, not {float(want[at])!r} within {float(tol[at]):.3g}")
