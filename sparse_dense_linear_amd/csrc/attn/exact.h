// exact.h -- single rows of attention from their definition, by one
// wavefront.
//
// The tiled kernels give a masked pair the weight 0 and multiply it with the
// row of V (K, q, do) all the same; where that row holds an infinity or a
// NaN the product is NaN, though the pair is not part of the result.  A row
// that comes out of a tiled kernel non-finite is therefore computed once
// more here, from the pairs that are seen alone, if a row that a masked pair
// of its tiles brought in is not finite (any_odd): a few dozen rows at the
// edges of the window.  An output whose sum left the range of fp32 before it was
// divided (weights reach 2^8 there, TooLarge) is computed again too.  So
// infinities and NaN that are seen cost no more than those two looks, and the
// tiles pay one test per output.  Finite data come here only so, and for a
// draft that sees no key.  A row all of whose elements have become NaN is not
// followed to its end.
#pragma once

#include "tile.h"

namespace sdl {

__device__ inline float wave_max(float x)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        x = fmaxf(x, __shfl_xor(x, d));
    return x;
}

__device__ inline float wave_sum(float x)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        x += __shfl_xor(x, d);
    return x;
}

// Whether one of rows from .. to - 1 (row(j): where it starts) that counts(j)
// lets through has an element that is not finite.
template <class T, class Row, class Counts>
__device__ inline bool any_odd(Row row, Counts counts, int from, int to, int D, int lane)
{
    bool odd = false;
    for (int j = from + lane; j < to; j += 64) {
        if (!counts(j))
            continue;
        const T *p = row(j);
        for (int d = 0; d < D; d += 8) {
            const Frag<T> x = load8(p + d);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                odd = odd || !finite((float)x[e]);
        }
    }
    return __any(odd);
}

template <class T, class Row>
__device__ inline bool any_odd(Row row, int from, int to, int D, int lane)
{
    return any_odd<T>(row, [](int) { return true; }, from, to, D, lane);
}

// Whether an output is infinite or no number though no value that it sums up is:
// first the columns in which some value is not finite (of rows that may be
// more than a query sees), then, for each output, what it holds in the others.
template <class T>
struct TooLarge {
    bool odd0 = false, odd1 = false;           // of the lane's columns, lane and lane + 64
    template <class Row, class Counts>
    __device__ void look(Row val, Counts counts, int from, int to, int D, int lane)
    {
#pragma unroll 4
        for (int j = from; j < to; ++j) {
            if (!counts(j))
                continue;
            const T *v = val(j);
            odd0 = odd0 || (lane < D && !finite((float)v[lane]));
            odd1 = odd1 || (lane + 64 < D && !finite((float)v[lane + 64]));
        }
    }
    __device__ bool operator()(const T *o, int D, int lane) const
    {
        return __any((lane < D && !odd0 && !finite((float)o[lane])) ||
                     (lane + 64 < D && !odd1 && !finite((float)o[lane + 64])));
    }
};

// Whether every lane's share of a row has become NaN.
__device__ inline bool all_nan(float a0, float a1, int D, int lane)
{
    return __all((lane >= D || a0 != a0) && (lane + 64 >= D || a1 != a1));
}

template <class T>
__device__ inline float dot_row(const T *a, const T *b, int D)
{
    float s = 0.0f;
    for (int d = 0; d < D; d += 8) {
        const Frag<T> x = load8(a + d), y = load8(b + d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s = fmaf((float)x[e], (float)y[e], s);
    }
    return s;
}

// Adds w * row[d] to (a0: d = lane, a1: d = lane + 64).
template <class T>
__device__ inline void add_row(const T *row, float w, int D, int lane, float &a0, float &a1)
{
    if (lane < D)
        a0 = fmaf(w, (float)row[lane], a0);
    if (lane + 64 < D)
        a1 = fmaf(w, (float)row[lane + 64], a1);
}

template <class T>
__device__ inline void put_row(T *row, float a0, float a1, int D, int lane)
{
    if (lane < D)
        row[lane] = (T)a0;
    if (lane + 64 < D)
        row[lane + 64] = (T)a1;
}

// o and lse of one query over keys 0 .. a - 1 and b .. c - 1 (a <= b) that
// seen(j) lets through; key(j) and val(j) are their rows.  c2 = scale *
// log2(e).  No key at all: 0 and -infinity.  have_lse: *lse is right already.
// Three passes: the maximum, the sum, and the values by weights that are divided
// already, whose sum leaves the range of fp32 only where the result does.
template <class T, class Key, class Val, class SeenAt>
__device__ inline void exact_row(const T *q, Key key, Val val, SeenAt seen, int a, int b, int c,
                                 int D, float c2, T *o, float *lse, bool have_lse, int lane)
{
    const float nan = __builtin_nanf("");
    float top = SDL_NEG_INF, total = 0.0f, inv = 0.0f, a0 = 0.0f, a1 = 0.0f;
    bool any = false;
    for (int pass = 0; pass < 3; ++pass) {
        for (int j0 = 0; j0 < c; j0 += 64) {
            if (j0 >= a && j0 + 64 <= b)
                continue;
            const int j = j0 + lane;
            const bool in = j < c && (j < a || j >= b) && seen(j);
            const float x = in ? dot_row(q, key(j), D) * c2 : SDL_NEG_INF;
            if (pass == 0) {
                if (__any(x != x)) {           // a score that is no number: nor is the softmax
                    put_row(o, nan, nan, D, lane);
                    if (lane == 0)
                        *lse = nan;
                    return;
                }
                top = fmaxf(top, x);
                any = any || __any(in);
                continue;
            }
            const float p = in ? __builtin_amdgcn_exp2f(x - (top == SDL_NEG_INF ? 0.0f : top)) : 0.0f;
            if (pass == 1) {
                total += p;
                continue;
            }
            for (uint64_t left = __ballot(in); left != 0; left &= left - 1) {
                const int n = __ffsll((unsigned long long)left) - 1;
                add_row(val(j0 + n), __shfl(p, n) * inv, D, lane, a0, a1);
            }
            if (have_lse && all_nan(a0, a1, D, lane)) {
                put_row(o, nan, nan, D, lane);
                return;
            }
        }
        if (pass == 0) {
            top = wave_max(top);
            if (top == __builtin_inff()) {     // an infinite score: infinity over infinity
                put_row(o, nan, nan, D, lane);
                if (lane == 0)
                    *lse = top;
                return;
            }
        } else if (pass == 1) {
            total = wave_sum(total);
            inv = 1.0f / total;
        }
    }
    put_row(o, a0, a1, D, lane);               // no key at all: the sums are empty
    if (lane == 0)
        *lse = any ? kLn2 * (top + __builtin_amdgcn_logf(total)) : SDL_NEG_INF;
}

// What a row of the gradients needs of the other operands.
template <class T>
struct GradRows {
    const T *q, *k, *v, *dout;      // first query / key of the sequence, at the head
    int64_t q_stride, k_stride, v_stride, dout_stride;
    const float *lse, *delta;       // of the first query, at the head
};

// dq of query i from keys 0 .. a - 1 and b .. c - 1 that seen(j) lets through.
template <class T, class SeenAt>
__device__ inline void exact_dq_row(const GradRows<T> &r, int i, float delta, SeenAt seen, int a,
                                    int b, int c, int D, float c2, float scale, T *dq, int lane)
{
    const T *q = r.q + (int64_t)i * r.q_stride, *g = r.dout + (int64_t)i * r.dout_stride;
    const float lse2 = r.lse[i] * kLog2e;
    float a0 = 0.0f, a1 = 0.0f;
    for (int j0 = 0; j0 < c; j0 += 64) {
        if (j0 >= a && j0 + 64 <= b)
            continue;
        const int j = j0 + lane;
        const bool in = j < c && (j < a || j >= b) && seen(j);
        float ds = 0.0f;
        if (in) {
            const float p =
                __builtin_amdgcn_exp2f(dot_row(q, r.k + (int64_t)j * r.k_stride, D) * c2 - lse2);
            ds = p * (dot_row(g, r.v + (int64_t)j * r.v_stride, D) - delta);
        }
        for (uint64_t left = __ballot(in); left != 0; left &= left - 1) {
            const int n = __ffsll((unsigned long long)left) - 1;
            add_row(r.k + (int64_t)(j0 + n) * r.k_stride, __shfl(ds, n), D, lane, a0, a1);
        }
        if (all_nan(a0, a1, D, lane))
            break;
    }
    put_row(dq, a0 * scale, a1 * scale, D, lane);
}

// Adds what queries i0 .. i1 - 1 of one head that seen(i) lets through give
// to dk and dv of key j.
template <class T, class SeenAt>
__device__ inline void exact_dkv_add(const GradRows<T> &r, int j, SeenAt seen, int i0, int i1, int D,
                                     float c2, int lane, float (&dk)[2], float (&dv)[2])
{
    const T *k = r.k + (int64_t)j * r.k_stride, *v = r.v + (int64_t)j * r.v_stride;
    for (int b = i0; b < i1; b += 64) {
        const int i = b + lane;
        const bool in = i < i1 && seen(i);
        float p = 0.0f, ds = 0.0f;
        if (in) {
            p = __builtin_amdgcn_exp2f(dot_row(r.q + (int64_t)i * r.q_stride, k, D) * c2 -
                                       r.lse[i] * kLog2e);
            ds = p * (dot_row(r.dout + (int64_t)i * r.dout_stride, v, D) - r.delta[i]);
        }
        for (uint64_t left = __ballot(in); left != 0; left &= left - 1) {
            const int n = __ffsll((unsigned long long)left) - 1;
            add_row(r.q + (int64_t)(b + n) * r.q_stride, __shfl(ds, n), D, lane, dk[0], dk[1]);
            add_row(r.dout + (int64_t)(b + n) * r.dout_stride, __shfl(p, n), D, lane, dv[0], dv[1]);
        }
        if (all_nan(dk[0], dk[1], D, lane) && all_nan(dv[0], dv[1], D, lane))
            break;
    }
}

// Whether a key or value that the tiles of queries p0 .. p1 brought in behind
// a mask is not finite.  Tiles of KT keys: those of the first `sinks` keys
// (first_tiles of them) and from tile `band` on.
template <class T, class Key, class Val>
__device__ inline bool odd_masked_keys(const Seen &seen, Key key, Val val, int p0, int p1, int first_tiles,
                                       int band, int KT, int lk, int D, int lane)
{
    auto odd = [&](int from, int to) {
        to = to < lk ? to : lk;
        return any_odd<T>(key, from, to, D, lane) || any_odd<T>(val, from, to, D, lane);
    };
    const int from = band * KT > seen.sinks ? band * KT : seen.sinks;
    // past the queries, behind the window, behind the first keys (and the
    // sequence's last key, which stands for those past its end)
    return odd(p0 > 0 ? p0 : 0, (p1 / KT + 1) * KT) || odd(from, p1 - seen.window + 1) ||
           odd(seen.sinks, first_tiles * KT) || odd(lk - 1, lk);
}

}  // namespace sdl
