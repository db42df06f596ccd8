// tree_codes.h -- attention of drafted tokens over a paged cache of codes of 8
// bits.
//
// tree_stream: blocks of up to 16 query rows (T * Hq / Hkv), as one answered token
// of each sequence has.  It is bound by the read of the cache, and the codes go
// from memory into registers with no barrier between tiles: each wavefront walks
// keys of its own, 32 to a step.
//   Scores: lane (c, part) takes codes 16 part .. + 15 (and 64 further) of key c;
//   eight of them are an operand of 32 terms whose order along D is the lanes'
//   own, and q is held in the same order.  Loads of half rows (four lanes to a key
//   of 128 bytes) reach 5.5 TB/s and no more, so keys are loaded by whole rows and
//   change lanes in LDS, which is the wavefront's own.
//   Values: it loads DP / 16 codes from (DP / 16) c on of the eight keys whose
//   weights it holds; bytes of key pairs are put side by side (one permutation
//   for two pairs) and widened.
// The 16 columns of a matrix are COLS query rows (16, or up to 8 of them) times 16 /
// COLS steps: the scores of two steps are moved into one register, column by column,
// before the softmax, which so works on full wavefronts; each step's weights are an
// operand whose other columns are zero.  A column keeps a maximum and a sum of its
// own, and the columns of a row are joined at the end.
// Wavefronts of a workgroup take neighbouring heads (up to four) of the same keys:
// rows of 128 bytes that are read together lie beside each other in memory.
// 64 answers of 1000 to 16384 positions, 8 heads of 128, 697 MB in 131 us = 5.3 TB/s
// (reading alone 7.1).  Each further byte costs what 6.6 TB/s cost; 25 us are the start
// (six loads that wait for each other) and the last turns, which end at different
// times, and 6 more the join.
// Codes are exact in bf16.  q in fp32 is the sum of three bf16 parts (8 bits
// each, exact), whose products with a code are exact too, so that three
// instructions of bf16 do what eight of fp32 would; weights are taken as two
// parts (16 bits), for q in fp32 as three.  The matrix cores have the time.
#pragma once

#include "tree_impl.h"

namespace sdl {

namespace {

// x as a sum of bf16 numbers: truncated ones, which leave an exact rest of 8 bits
// less each, and the last rounded to nearest.  Infinities and NaN go into the first.
template <int PARTS>
__device__ inline void split(const f32x8 &x, bf16x8 (&p)[PARTS])
{
    f32x8 rest = x;
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (i == PARTS - 1) {
                p[i][e] = (__bf16)rest[e];
                continue;
            }
            const bool f = finite(rest[e]);
            const float top = f ? __uint_as_float(__float_as_uint(rest[e]) & 0xffff0000) : rest[e];
            p[i][e] = (__bf16)top;
            rest[e] = f ? rest[e] - top : 0.0f;
        }
}

// The same of finite numbers: the truncated parts of two numbers are one
// permutation.
template <int PARTS>
__device__ inline void split_finite(const f32x8 &x, bf16x8 (&p)[PARTS])
{
    f32x8 rest = x;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        if (i == PARTS - 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                p[i][e] = (__bf16)rest[e];
            continue;
        }
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = __float_as_uint(rest[2 * e]), hi = __float_as_uint(rest[2 * e + 1]);
            w[e] = __builtin_amdgcn_perm(hi, lo, 0x07060302);
            rest[2 * e] -= __uint_as_float(lo & 0xffff0000);
            rest[2 * e + 1] -= __uint_as_float(hi & 0xffff0000);
        }
        p[i] = __builtin_bit_cast(bf16x8, w);
    }
}

// A key's or value's rows of a step on their way: 64 or 128 codes each.
template <int DP>
struct StepRows {
    static constexpr int kVal = DP / 16, kLoads = DP / 32, kLanes = DP / 16;   // of keys: loads, lanes of a row
    u32x4 k[kLoads];
    typedef std::conditional_t<kVal == 8, uint2, uint32_t> Val;
    Val v[8];
};

__device__ inline uint32_t word_of(uint2 x, int i) { return i == 0 ? x.x : x.y; }
__device__ inline uint32_t word_of(uint32_t x, int) { return x; }

__device__ inline uint2 load_val(const char *p, uint2)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 x = __builtin_nontemporal_load((const u32x2 *)p);
    return make_uint2(x[0], x[1]);
}
__device__ inline uint32_t load_val(const char *p, uint32_t) { return __builtin_nontemporal_load((const uint32_t *)p); }


// Division by a number that the host has prepared (Divisor), for x < 2^31.
__device__ inline int divided(int x, const Divisor &d) { return (int)(__umulhi((uint32_t)x << 1, d.factor) >> d.shift); }

__device__ inline int64_t uniform(int64_t x)
{
    return (int64_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)x);
}

// TOGETHER: 16 keys that begin at a multiple of 16 lie in one page, and four in one
// block of scales.  Else each key is found by itself.
template <class T, class H, int DP, int COLS, bool TOGETHER>
__global__ __launch_bounds__(kAttnThreads, stream_per_cu(sizeof(T), DP)) void tree_stream(TreeArgs a)
{
    constexpr int QP = sizeof(T) == 4 ? 3 : 1, PP = sizeof(T) == 4 ? 3 : 2;
    constexpr int HALVES = DP / 64, VAL = DP / 16, LANES = StepRows<DP>::kLanes, LOADS = StepRows<DP>::kLoads,
                   STEPS = 16 / COLS, kTurn = 32 * STEPS;
    typedef Tile<float, DP, 16> Out;
    __shared__ __align__(16) char lds[4 * Out::kBytes];
    __shared__ Drafts drafts;
    __shared__ float tops[4][16], totals[4][16];
    __shared__ int redo[4][16];
    // !TOGETHER: of three turns, where keys lie, and their scales
    constexpr int SLOTS = TOGETHER ? 1 : 3;
    __shared__ __align__(16) int64_t place_of[4][SLOTS][32];
    __shared__ __align__(16) float scale_of[4][SLOTS][2][32];

    const int t = threadIdx.x, lane = t & 63, c = lane & 15, part = lane >> 4, cls = c / COLS;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int heads = a.wave_heads, wh = wave % heads, wk = wave / heads;
    const int group = a.Hq / a.Hkv;
    const float c2 = a.scale * kLog2e;
    const Slots slots(a);

    Span span;
    if (!span.begin<H>(a, slots))
        return;
    int64_t at = uniform(span.at), base = uniform(span.base);
    const int64_t stop = uniform(span.stop);
    int seq = __builtin_amdgcn_readfirstlane(span.seq);
    bool later = false;
    while (at < stop) {
        Unit u = unit_of<H>(a, seq);
        int64_t mine = (int64_t)key_groups<H>(a) * u.blocks * u.tiles;
        while (at >= base + mine) {            // the next sequence that has tiles
            base += mine;
            ++seq;
            u = unit_of<H>(a, seq);
            mine = (int64_t)key_groups<H>(a) * u.blocks * u.tiles;
        }
        const int unit = (int)Spans::divide(at - base, u.tiles);
        const int hg = unit / u.blocks, block = unit % u.blocks, hk = hg * heads + wh;
        const int n0 = (int)(at - base - (int64_t)unit * u.tiles);
        const int n1 = stop - at < u.tiles - n0 ? n0 + (int)(stop - at) : u.tiles;
        const int rows = u.drafts * group;

        __syncthreads();
        if (t < 64)
            redo[t >> 4][t & 15] = 0;
        if (wave == 3 && a.tree != nullptr)
            find_drafts(a, u, lane, drafts);

        // this lane's query
        const int r = block * COLS + c % COLS;
        const int token = (r < rows ? r : rows - 1) / group, head = hk * group + (r < rows ? r : rows - 1) % group;
        DraftSeen seen;
        seen.ctx = u.ctx;
        seen.drafts = u.drafts;
        seen.window = a.window;
        seen.sinks = a.sinks;
        seen.mask = a.tree != nullptr ? draft_mask(a.tree[u.q_begin + token], u.drafts) : 0;
        seen.pos = a.tree != nullptr ? draft_place(u.ctx, seen.mask) : u.ctx + token;
        seen.place = a.tree != nullptr ? drafts.place : nullptr;
        const T *q = (const T *)a.q + (int64_t)(u.q_begin + token) * a.q_row + head * a.q_head;
        bf16x8 qf[2 * HALVES][QP];
#pragma unroll
        for (int s = 0; s < 2 * HALVES; ++s) {
            const int d = 64 * (s >> 1) + 16 * part + 8 * (s & 1);
            const Frag<T> x = d < a.D ? load8(q + d) : zero_frag<T>();
            if constexpr (QP == 1)
                qf[s][0] = x;
            else
                split<QP>(x, qf[s]);
        }

        f32x4 O[VAL];
#pragma unroll
        for (int e = 0; e < VAL; ++e)
            O[e] = f32x4(0.0f);
        float top = SDL_NEG_INF, total = 0.0f;
        // A weight times an infinite scale has no second part.  Such units come out
        // as if a score were infinite, and are computed again.
        bool strange = false;

        const int32_t *table = a.table + (int64_t)seq * a.table_stride;
        const char *kp = (const char *)a.k_pages + hk * a.head_stride, *vp = (const char *)a.v_pages + hk * a.head_stride;
        const float *kscale = a.k_scale + hk * a.scale_head, *vscale = a.v_scale + hk * a.scale_head;
        // the lane's codes of a key and of a value, and its row of a load of keys
        const int kd = 16 * (lane % LANES) < a.D ? 16 * (lane % LANES) : a.D - 16, k_row = lane / LANES;
        const int vd = VAL * c < a.D ? VAL * c : a.D - VAL;
        auto first = [&](int n) { return first_key(u, n) + kTurn * wk; };

        StepRows<DP> x;
        // Keys of a step into LDS: whole rows come from memory, 8 or 4 lanes to a row,
        // and go out by 16 rows, 4 lanes to a row.  Pieces of a row are exchanged by its
        // number, so that neither counts bank conflicts.
        char *const keys = lds + wave * Out::kBytes;
        auto piece_at = [&](int r, int piece) {
            return r * DP + ((piece ^ (r >> (DP == 64 ? 1 : 0) & (LANES - 1))) << 4);
        };
        auto stage = [&](const u32x4 (&k)[LOADS]) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                *(u32x4 *)(keys + piece_at(i * (64 / LANES) + k_row, lane % LANES)) = k[i];
        };
        // scores of a step's keys
        auto scores = [&](f32x4 (&s)[2]) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b] = f32x4(0.0f);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    const u32x4 w = *(const u32x4 *)(keys + piece_at(16 * b + c, 4 * h + part));
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const auto lo = wide_bf16<H>(w[2 * e]), hi = wide_bf16<H>(w[2 * e + 1]);
                        const bf16x8 f = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                        for (int i = 0; i < QP; ++i)
                            s[b] = mma16(f, qf[2 * h + e][i], s[b]);
                    }
                }
            }
        };
        // weights of scores that are scaled already
        auto weights = [&](f32x4 (&s)[2]) {
            float most = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                               fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
            most = max_quarters(most) * c2;
            if (__any(most > top + kLazy)) {
                const float now = fmaxf(top, most);
                const float less = now == SDL_NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(top - now);
                top = now;
                total *= less;
#pragma unroll
                for (int e = 0; e < VAL; ++e)
                    O[e] *= less;
            }
            const float ref = top == SDL_NEG_INF ? 0.0f : top;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[b][i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], c2, -ref));
            total += ((s[0][0] + s[0][1]) + (s[0][2] + s[0][3])) + ((s[1][0] + s[1][1]) + (s[1][2] + s[1][3]));
        };
        // two columns of the values at a time: the bytes of two keys side by side
        auto values = [&](const typename StepRows<DP>::Val (&v)[8], const bf16x8 (&pf)[PP]) {
#pragma unroll
            for (int e = 0; e < VAL; e += 2) {
                bf16x4 w[4];
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    w[m] = wide_bf16<H>(__builtin_amdgcn_perm(word_of(v[2 * m + 1], e >> 2), word_of(v[2 * m], e >> 2),
                                                              (e & 3) == 0 ? 0x05010400 : 0x07030602));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    bf16x8 f;
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        f[2 * m] = w[m][2 * i];
                        f[2 * m + 1] = w[m][2 * i + 1];
                    }
#pragma unroll
                    for (int k = 0; k < PP; ++k)
                        O[e + i] = mma16(f, pf[k], O[e + i]);
                }
            }
        };

        __syncthreads();                       // what the drafts see is there
        // What some draft sees: of the context, as SeenRows; of the drafts, these bits
        // (a chain: all of them).
        const int low = a.tree != nullptr ? __builtin_amdgcn_readfirstlane(drafts.low) : u.low;
        const int sinks = a.sinks < u.ctx ? a.sinks : u.ctx;
        const uint64_t named = a.tree != nullptr ? __ballot(drafts.named[lane] != 0) : 0;
        auto any_seen = [&](int j, int count) {         // of keys j .. j + count - 1
            const int e = j + count < u.end ? j + count - 1 : u.end - 1;
            const bool cached = j < sinks || (e < u.ctx - 1 ? e : u.ctx - 1) >= (j > low ? j : low);
            const int d0 = j > u.ctx ? j - u.ctx : 0, d1 = e - u.ctx;
            if (a.tree == nullptr)
                return cached || d1 >= d0;
            const uint64_t which = ((uint64_t)2 << (((d1 < 63 ? d1 : 63) - d0) & 63)) - 1;
            return cached || (d1 >= d0 && d0 < 64 && (named >> (d0 & 63) & which) != 0);
        };
        // a tile of which this wavefront sees all: nothing to mask
        auto whole = [&](int n) {
            const int j0 = first(n), j1 = j0 + kTurn - 1;
            return all_seen(a, u, j0, j1) && j1 < u.ctx && (u.end - 1 - j0 < a.window || j1 < a.sinks);
        };
        // the next tile that holds a key that is seen, n1 if there is none
        auto after = [&](int n) {
            do
                ++n;
            while (n < n1 && !any_seen(first(n), kTurn));
            return n < n1 ? n : n1;
        };

        // Turns of STEPS steps.  The values lag a turn behind the keys: each step takes
        // scores of one turn and values of the turn before, whose softmax lies between,
        // while the loads of the next step are under way.  No load in the loop stands
        // behind a branch: the compiler then counts them, and waits for no more than it
        // needs.  So keys that no draft sees are taken from the start of the pool (there
        // is one, since some key of the tile is seen), and in tiles that are not whole
        // scores are masked and such keys' values become zero.
        struct Turn {
            int n, slot;
            int64_t at[2];                     // TOGETHER: of the lane's two groups of 16 keys (those of its column's step)
            float ks[2], vs[2];                // and the scales of its four keys of each
        };
        const int last_page = divided(u.end > 0 ? u.end - 1 : 0, a.by_page);
        int id[2], in[2];                      // in < 0: not seen
        float scale_k = 0.0f, scale_v = 0.0f;
        auto find = [&](int n) {
            constexpr int GROUPS = TOGETHER ? 2 : 1, KEYS = TOGETHER ? 16 : 1;
#pragma unroll
            for (int b = 0; b < GROUPS; ++b) {
                const int j = first(n) + (TOGETHER ? 32 * cls + 16 * b : (lane & 31)), p = divided(j, a.by_page);
                const int number = table[p < last_page ? p : last_page];
                const bool read = any_seen(j, KEYS);
                in[b] = read ? j - p * a.page : -1;
                id[b] = read ? number : 0;
            }
        };
        auto keep = [&](Turn &to, int n, int slot) {
            to.n = n;
            to.slot = slot;
            if constexpr (TOGETHER) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const bool read = any_seen(first(n) + 32 * cls + 16 * b + 4 * part, 4);
                    const int in_block = divided(read ? in[b] + 4 * part : 0, a.by_block);
                    const int64_t s = (int64_t)id[b] * a.scale_page + in_block * a.scale_block;
                    to.ks[b] = kscale[read ? s : 0];
                    to.vs[b] = vscale[read ? s : 0];
                    to.ks[b] = read ? to.ks[b] : 0.0f;
                    to.vs[b] = read ? to.vs[b] : 0.0f;
                    to.at[b] = in[b] >= 0 ? (int64_t)id[b] * a.page_stride + (int64_t)in[b] * a.row_stride : 0;
                }
            } else {
                const bool read = in[0] >= 0;
                const int64_t s = (int64_t)id[0] * a.scale_page + divided(read ? in[0] : 0, a.by_block) * a.scale_block;
                scale_k = kscale[read ? s : 0];
                scale_v = vscale[read ? s : 0];
                scale_k = read ? scale_k : 0.0f;
                scale_v = read ? scale_v : 0.0f;
                place_of[wave][slot][lane & 31] = read ? (int64_t)id[0] * a.page_stride + (int64_t)in[0] * a.row_stride : 0;
            }
        };
        auto keep_scales = [&](int slot) {
            if constexpr (!TOGETHER) {
                scale_of[wave][slot][0][lane & 31] = scale_k;
                scale_of[wave][slot][1][lane & 31] = scale_v;
                strange = strange || fabsf(scale_v) == __builtin_inff();
            }
        };
        const uint32_t row = (uint32_t)a.row_stride, k_off = k_row * row + kd, v_off = 4 * part * row + vd;
        auto begin = [&](const char *pool, const Turn &of, int b, int step) {
            const int l = COLS * step;
            return pool + ((int64_t)__builtin_amdgcn_readlane((int)(of.at[b] >> 32), l) << 32 |
                           (uint32_t)__builtin_amdgcn_readlane((int)of.at[b], l));
        };
        auto fetch_k = [&](const Turn &of, int step, u32x4 (&k)[LOADS]) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const char *p;
                if constexpr (TOGETHER)
                    p = begin(kp, of, 2 * i / LOADS, step) + i % (LOADS / 2) * (64 / LANES) * (uint64_t)row + k_off;
                else
                    p = kp + place_of[wave][of.slot][i * (64 / LANES) + k_row] + kd;
                k[i] = __builtin_nontemporal_load((const u32x4 *)p);
            }
        };
        typedef typename StepRows<DP>::Val Val;
        auto fetch_v = [&](const Turn &of, int step, Val (&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const char *p;
                if constexpr (TOGETHER)
                    p = begin(vp, of, i >> 2, step) + (i & 3) * (uint64_t)row + v_off;
                else
                    p = vp + place_of[wave][of.slot][16 * (i >> 2) + 4 * part + (i & 3)] + vd;
                v[i] = load_val(p, Val());
            }
        };
        // the scores of a step into the columns that are its
        auto merge = [&](f32x4 (&y)[2], const f32x4 (&s)[2], auto step) {
            constexpr int st = decltype(step)::value;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if constexpr (st == 0)
                        y[b][i] = s[b][i];
                    else
                        y[b][i] = __int_as_float(__builtin_amdgcn_update_dpp(
                            __float_as_int(y[b][i]), __float_as_int(s[b][i]), 0x118, 0xf, 0xc, false));
        };
        bf16x8 pf[PP];
        bool masked = false;
        auto softmax = [&](f32x4 (&y)[2], const Turn &of) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if constexpr (TOGETHER)
                    y[b] *= of.ks[b];
                else
                    times_scales<4>(y[b], scale_of[wave][of.slot][0] + 16 * b + 4 * part);
            masked = !whole(of.n);
            if (masked) {
                const int j = first(of.n) + 32 * cls + 4 * part;
                int hidden = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    hidden |= seen(j + 16 * (i >> 2) + (i & 3)) ? 0 : 1 << i;
                hidden = renewed(hidden);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i >> 2][i & 3] = hidden >> i & 1 ? SDL_NEG_INF : y[i >> 2][i & 3];
            }
            weights(y);
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if constexpr (TOGETHER) {
                    y[b] *= of.vs[b];
                    strange = strange || fabsf(of.vs[b]) == __builtin_inff();
                } else {
                    times_scales<4>(y[b], scale_of[wave][of.slot][1] + 16 * b + 4 * part);
                }
            split_finite<PP>(__builtin_shufflevector(y[0], y[1], 0, 1, 2, 3, 4, 5, 6, 7), pf);
        };
        auto apply = [&](const Turn &of, int step, Val (&v)[8]) {
            if (masked) {
                const int j = first(of.n) + 32 * step + 4 * part;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = any_seen(j + 16 * (i >> 2) + (i & 3), 1) ? v[i] : Val();
            }
            if constexpr (STEPS == 1) {
                values(v, pf);
            } else {
                bf16x8 only[PP];
#pragma unroll
                for (int k = 0; k < PP; ++k)
                    only[k] = cls == step ? pf[k] : zero_frag<__bf16>();
                values(v, only);
            }
        };
        auto steps = [&](auto f) {             // f(step, as a constant)
            f(std::integral_constant<int, 0>());
            if constexpr (STEPS > 1)
                f(std::integral_constant<int, 1>());
        };
        int n = after(n0 - 1);
        if (n < n1) {
            Turn last, now, next;
            f32x4 y[2], s[2];
            find(n);
            keep(now, n, 0);
            keep_scales(0);
            int m = after(n), then = m < n1 ? after(m) : n1;      // the tiles after this one
            find(m < n1 ? m : n);
            // of the first turn all keys at once, and of the last one all values: there
            // is nothing else to do while they are under way
            u32x4 first_k[STEPS][LOADS];
            steps([&](auto step) { fetch_k(now, step, first_k[step]); });
            keep(next, m < n1 ? m : n, 1);
            keep_scales(1);
            find(then < n1 ? then : next.n);
            fetch_v(now, 0, x.v);
            fetch_k(next, 0, x.k);
            keep_order();
            steps([&](auto step) {
                stage(first_k[step]);
                scores(s);
                merge(y, s, step);
            });
#pragma unroll 1
            while (m < n1) {
                last = now;
                now = next;
                m = then;
                then = m < n1 ? after(m) : n1;
                keep(next, m < n1 ? m : now.n, now.slot == 2 ? 0 : now.slot + 1);
                find(then < n1 ? then : next.n);
                keep_order();
                softmax(y, last);
                steps([&](auto step) {
                    stage(x.k);
                    keep_order();
                    if (step + 1 < STEPS)
                        fetch_k(now, step + 1, x.k);
                    else
                        fetch_k(next, 0, x.k);
                    keep_order();
                    scores(s);
                    merge(y, s, step);
                    apply(last, step, x.v);
                    keep_order();
                    if (step + 1 < STEPS)
                        fetch_v(last, step + 1, x.v);
                    else
                        fetch_v(now, 0, x.v);
                    keep_order();
                });
                keep_scales(next.slot);
            }
            Val last_v[STEPS][8];
            steps([&](auto step) {
                if (step > 0)
                    fetch_v(now, step, last_v[step]);
            });
            keep_order();
            softmax(y, now);
            steps([&](auto step) { apply(now, step, step > 0 ? last_v[step] : x.v); });
        }
        if (__any(strange)) {
            top = __builtin_inff();
            total = __builtin_nanf("");
        }

        // ---- join the columns of a row, then the wavefronts of a head, and write
        total = sum_quarters(total);
        if constexpr (STEPS > 1) {
            // row_ror:8
            float best = top;
            best = fmaxf(best, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(best), 0x128, 15, 15, true)));
            const float f = best == SDL_NEG_INF ? 0.0f : __builtin_amdgcn_exp2f(top - best);
            top = best;
            auto joined = [&](float v) {
                v *= f;
                return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x128, 15, 15, true));
            };
            total = joined(total);
#pragma unroll
            for (int e = 0; e < VAL; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    O[e][i] = joined(O[e][i]);
        }
        if (part == 0) {
            tops[wave][c] = top;
            totals[wave][c] = total;
        }
        // row 4 part + i of result e is column VAL (4 part + i) + e of the output
        if (c < COLS)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < VAL; e += 4)
                    store4((float *)(lds + wave * Out::kBytes + Out::at(c, (VAL * (4 * part + i) + e) / 4)), O[e][i],
                           O[e + 1][i], O[e + 2][i], O[e + 3][i]);
        __syncthreads();
        const bool done = n0 == 0 && n1 == u.tiles;
        const int64_t slot = 2 * (int64_t)span.w + (later ? 1 : 0);
        constexpr int kOutPieces = DP / 4;
        for (int m = t; m < heads * COLS * kOutPieces; m += kAttnThreads) {
            const int lr = m / kOutPieces % COLS, h = m / kOutPieces / COLS, p = m % kOutPieces;
            const int rr = block * COLS + lr;
            if (rr >= rows)
                continue;
            float best = SDL_NEG_INF;
            for (int w = h; w < 4; w += heads)
                best = fmaxf(best, tops[w][lr]);
            const float ref = best == SDL_NEG_INF ? 0.0f : best;
            float sum = 0.0f;
            f32x4 o = f32x4(0.0f);
            for (int w = h; w < 4; w += heads) {
                const float f = __builtin_amdgcn_exp2f(tops[w][lr] - ref);
                sum = fmaf(f, totals[w][lr], sum);
                const f32x4 v = *(const f32x4 *)(lds + w * Out::kBytes + Out::at(lr, p));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = fmaf(f, v[e], o[e]);
            }
            if (!done) {
                const int64_t to = (slot * heads + h) * COLS + lr;
                *(f32x4 *)(slots.out + to * DP + 4 * p) = o;
                if (p == 0) {
                    slots.stat[to * 2] = best;
                    slots.stat[to * 2 + 1] = sum;
                }
                continue;
            }
            finish<T, H>(a, u.q_begin + rr / group, (hg * heads + h) * group + rr % group, p, best, sum, o, &redo[h][lr]);
        }
        __syncthreads();
        if (done)
            for (int h = 0; h < heads; ++h)
                finish_again<T, H>(a, u, seq, hg * heads + h, block * COLS, COLS, redo[h], drafts, wave, lane);
        at += n1 - n0;
        later = true;
    }
}

// Blocks of 32 to 128 query rows, RG groups of C of them; the 4 / RG wavefronts of a
// group share the keys of a tile.  Tiles of 128 keys are widened to bf16 on their way
// into LDS, once for all query groups; the next tile is under way while one is worked
// on.  Where all scales of a tile are powers of two that cannot leave bf16's range, as
// append writes them, they go into the widening, which is exact still; else they are
// applied to scores and weights.
// q in fp32 is taken in three bf16 parts, weights too (tree_stream); for q in bf16 the
// weights are rounded to bf16, once, as they are over rows of bf16.  (Two parts, as
// tree_stream has them: pieces of prompts 354 us against 295, trees of drafts 94 against
// 84; errors against 64 bits 0.0017, which is the rounding of the result, instead of
// 0.0022.)
// A piece of 1024 queries behind 8192 keys and two more sequences, 32 heads of 128 on
// 8: 179 GFLOP in 272 us = 660 TFLOP/s; integers, with scales that are no powers of two,
// 322 us.  It is
// bound by LDS, 82 % of what row reads alone reach: each wavefront of 32 queries reads
// the whole tile.
// (Two buffers of 64 keys with one barrier to a tile instead of two: prompt pieces 418
// us against 355, most of it the finding and widening of rows, which every tile
// waits for.)
constexpr int kTileKeys8 = 128;

template <class T, class H, int DP, int DU, int C, int RG>
__global__ __launch_bounds__(kAttnThreads, 2) void tree_tiles(TreeArgs a)
{
    constexpr int KS = 4 / RG, RB = C * RG, KEYS = kTileKeys8;
    constexpr int QP = sizeof(T) == 4 ? 3 : 1;
    typedef Cols<__bf16, DP, DU, KEYS, C> Co;
    typedef typename Co::Acc Acc;
    constexpr int STEPS = Co::kSteps, DB = Co::kBlocks;
    typedef Tile<__bf16, DP, KEYS> Tl;
    typedef Tile<float, DP, C> Out;
    constexpr int kPieces = DP / 16, kPiecesPer = KEYS * kPieces / kAttnThreads;
    constexpr int kBytes = 2 * Tl::kBytes > 4 * Out::kBytes ? 2 * Tl::kBytes : 4 * Out::kBytes;
    static_assert(kPiecesPer * kAttnThreads == KEYS * kPieces, "whole pieces per thread");
    static_assert(KEYS / C % KS == 0, "keys for every wavefront of a group");
    __shared__ __align__(16) char lds[kBytes];
    __shared__ Drafts drafts;
    __shared__ float tops[4][C], totals[4][C];
    __shared__ int redo[RB];
    __shared__ int64_t place_of[2][KEYS];          // of a tile's rows, in the pools
    __shared__ __align__(16) float scale_of[2][2][KEYS];
    __shared__ int folds[2][2];                    // whether the scales of half a tile go into its rows
    __shared__ int strange;                        // an infinite scale, which has no second part (tree_stream)

    const int t = threadIdx.x, lane = t & 63, part = lane / C;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int group = a.Hq / a.Hkv;
    const int rg = wave % RG, ks = wave / RG;
    const float c2 = a.scale * kLog2e;
    const Slots slots(a);

    Span span;
    if (!span.begin<H>(a, slots))
        return;
    int64_t at = uniform(span.at), base = uniform(span.base);
    const int64_t stop = uniform(span.stop);
    int seq = __builtin_amdgcn_readfirstlane(span.seq);
    bool later = false;
    while (at < stop) {
        Unit u = unit_of<H>(a, seq);
        int64_t mine = (int64_t)a.Hkv * u.blocks * u.tiles;
        while (at >= base + mine) {            // the next sequence that has tiles
            base += mine;
            ++seq;
            u = unit_of<H>(a, seq);
            mine = (int64_t)a.Hkv * u.blocks * u.tiles;
        }
        const int unit = (int)Spans::divide(at - base, u.tiles);
        const int hk = unit / u.blocks, block = unit % u.blocks;
        const int n0 = (int)(at - base - (int64_t)unit * u.tiles);
        const int n1 = stop - at < u.tiles - n0 ? n0 + (int)(stop - at) : u.tiles;
        const int rows = u.drafts * group;

        __syncthreads();
        if (t < RB)
            redo[t] = 0;
        if (t == 0)
            strange = 0;
        if (wave == 3 && a.tree != nullptr)    // (the first one finds the rows)
            find_drafts(a, u, lane, drafts);

        // this lane's query
        const int r = block * RB + C * rg + lane % C;
        const int token = (r < rows ? r : rows - 1) / group, head = hk * group + (r < rows ? r : rows - 1) % group;
        BlockSeen seen;
        seen.mask = a.tree != nullptr ? draft_mask(a.tree[u.q_begin + token], u.drafts) : 0;
        seen.pos = a.tree != nullptr ? draft_place(u.ctx, seen.mask) : u.ctx + token;
        seen.cached = a.tree != nullptr ? u.ctx : seen.pos + 1;
        const T *q = (const T *)a.q + (int64_t)(u.q_begin + token) * a.q_row + head * a.q_head;
        bf16x8 qf[STEPS][QP];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int d = Co::kTerms * s + 8 * part;
            const Frag<T> x = d < a.D ? load8(q + d) : zero_frag<T>();
            if constexpr (QP == 1)
                qf[s][0] = x;
            else
                split<QP>(x, qf[s]);
        }

        Acc O[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
            O[d] = Acc(0.0f);
        float top = SDL_NEG_INF, total = 0.0f;

        // A chain's block ends where its last row stands: later tiles hold nothing for it,
        // later keys nothing for a wavefront.  Its rows see all keys up to the first one's
        // place (of a tree, the context) that are in the window of the last.
        int e1 = n1, first_pos = u.ctx - 1, last_pos = u.end - 1, low = u.low;
        if (a.tree == nullptr) {
            auto stands = [&](int last) { return u.ctx + (last < rows ? last : rows - 1) / group; };
            first_pos = stands(block * RB + C * rg);
            last_pos = stands(block * RB + C * rg + C - 1);
            low = window_low(first_pos, a.window);
            const int e = u.first_tiles + stands(block * RB + RB - 1) / KEYS - u.band + 1;
            e1 = e < n1 ? (e > n0 ? e : n0) : n1;
        }
        const int32_t *table = a.table + (int64_t)seq * a.table_stride;
        const H *kp = (const H *)a.k_pages + hk * a.head_stride, *vp = (const H *)a.v_pages + hk * a.head_stride;
        struct Rows {                          // a thread's share of a tile on its way
            u32x4 k[kPiecesPer], v[kPiecesPer];
        };
        int id = 0, in_page = 0;               // in_page < 0: a row that is not read
        float scale_k = 0.0f, scale_v = 0.0f;
        auto whole = [&](int n) { return all_seen(a, u, first_key(u, n), first_key(u, n) + KEYS - 1); };
        auto find_row = [&](int n) {
            const int j = first_key(u, n) + t;
            in_page = -1;
            if (whole(n) || seen_rows(a, u, drafts)(j)) {
                const int p = divided(j, a.by_page);
                in_page = j - p * a.page;
                id = table[p];
            }
        };
        auto keep_row = [&](int n) {
            place_of[n & 1][t] = in_page < 0 ? -1 : (int64_t)id * a.page_stride + (int64_t)in_page * a.row_stride;
            scale_k = scale_v = 0.0f;
            if (in_page >= 0) {
                const int64_t s =
                    (int64_t)id * a.scale_page + divided(in_page, a.by_block) * a.scale_block + hk * a.scale_head;
                scale_k = a.k_scale[s];
                scale_v = a.v_scale[s];
            }
        };
        auto folding = [](float s) {           // 2^-100 .. 2^100, or a row that is not read
            const uint32_t b = __float_as_uint(s);
            return b == 0 || ((b & 0x807fffff) == 0 && b >> 23 >= 27 && b >> 23 <= 227);
        };
        auto keep_scales = [&](int n) {
            scale_of[n & 1][0][t] = scale_k;
            scale_of[n & 1][1][t] = scale_v;
            const bool all = __all(folding(scale_k) && folding(scale_v));
            const bool odd = __any(fabsf(scale_v) == __builtin_inff());
            if (lane == 0) {
                folds[n & 1][wave] = all;
                if (odd)
                    strange = 1;
            }
        };
        auto fetch = [&](int n, Rows &to) {
            const int tt = renewed(t);
            int64_t from[kPiecesPer];          // all of them before the loads, which then go out together
#pragma unroll
            for (int i = 0; i < kPiecesPer; ++i)
                from[i] = place_of[n & 1][(tt + i * kAttnThreads) / kPieces];
            auto load = [&](bool all) {
#pragma unroll
                for (int i = 0; i < kPiecesPer; ++i) {
                    const int p = (tt + i * kAttnThreads) % kPieces;
                    const int d = p * 16 < a.D ? p * 16 : a.D - 16;
                    if (!all) {
                        to.k[i] = u32x4(0);
                        to.v[i] = u32x4(0);
                    }
                    if (all || from[i] >= 0) {
                        to.k[i] = *(const u32x4 *)(kp + from[i] + d);
                        to.v[i] = *(const u32x4 *)(vp + from[i] + d);
                    }
                }
            };
            if (whole(n))
                load(true);
            else
                load(false);
        };
        auto put = [&](int n, const Rows &of) {
            char *kt = lds, *vt = kt + Tl::kBytes;
            const bool fold = (folds[n & 1][0] & folds[n & 1][1]) != 0;
#pragma unroll
            for (int i = 0; i < kPiecesPer; ++i) {
                const int m = t + i * kAttnThreads, row = m / kPieces, p = m % kPieces;
                const float sk = fold ? scale_of[n & 1][0][row] : 1.0f, sv = fold ? scale_of[n & 1][1][row] : 1.0f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // (new to the compiler here, which else widens all pieces first and
                    // has no registers for them)
                    uint32_t k[2] = {of.k[i][2 * h], of.k[i][2 * h + 1]}, v[2] = {of.v[i][2 * h], of.v[i][2 * h + 1]};
                    asm volatile("" : "+v"(k[0]), "+v"(k[1]), "+v"(v[0]), "+v"(v[1]) : : "memory");
                    const auto k0 = wide_scaled<H>(k[0], sk), k1 = wide_scaled<H>(k[1], sk);
                    const auto v0 = wide_scaled<H>(v[0], sv), v1 = wide_scaled<H>(v[1], sv);
                    *(bf16x8 *)(kt + Tl::at(row, 2 * p + h)) = __builtin_shufflevector(k0, k1, 0, 1, 2, 3, 4, 5, 6, 7);
                    *(bf16x8 *)(vt + Tl::at(row, 2 * p + h)) = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
                }
            }
        };
        __syncthreads();                       // what the drafts see is there
        if (a.tree != nullptr)
            seen.keep_near(drafts.place, a.window, a.sinks);
        const bool finds = t < KEYS;           // the first two wavefronts
        if (finds && n0 < e1) {
            find_row(n0);
            keep_row(n0);
            keep_scales(n0);
            if (n0 + 1 < e1) {
                find_row(n0 + 1);
                keep_row(n0 + 1);
            }
        }
        Rows next;
        __syncthreads();
        if (n0 < e1)
            fetch(n0, next);
        for (int n = n0; n < e1; ++n) {
            const char *kt = lds, *vt = kt + Tl::kBytes;
            const bool fold = (folds[n & 1][0] & folds[n & 1][1]) != 0;
            put(n, next);
            const bool find = finds && n + 2 < e1;
            if (finds && n + 1 < e1)
                keep_scales(n + 1);            // loaded a tile ago
            if (find)
                find_row(n + 2);
            if (n + 1 < e1)
                fetch(n + 1, next);
            __syncthreads();
#pragma unroll 1
            for (int b = ks; b < KEYS / C; b += KS) {
                const int j0 = first_key(u, n) + C * b, j1 = j0 + C - 1;
                if (j0 > last_pos || (j1 < low && j0 >= a.sinks) || block * RB + C * rg >= rows)
                    continue;
                const int rows_at = renewed(Co::row_base(lane) + C * b * Tl::kRowBytes);
                const int cols_at = renewed(Co::col_base(lane) + C * b * Tl::kRowBytes);
                Acc x = Acc(0.0f);
                chain<STEPS, 4>([&](int i) { return Co::key_frag(kt, rows_at, i); },
                                [&](int i, bf16x8 f) {
#pragma unroll
                                    for (int k = 0; k < QP; ++k)
                                        x = Co::mul(f, qf[i][k], x);
                                });
                if (!fold)
                    times_scales<Co::kAcc>(x, scale_of[n & 1][0] + C * b + 4 * part);
                if (!(j1 <= first_pos && (last_pos - j0 < a.window || j1 < a.sinks))) {
                    const uint32_t bits = renewed((int)(seen(j0, u.ctx, a.window, a.sinks) >> (4 * part)));
#pragma unroll
                    for (int i = 0; i < Co::kAcc; ++i)
                        x[i] = bits >> Co::key_of(i) & 1 ? x[i] : SDL_NEG_INF;
                }
                const float most = Co::most(x) * c2;
                if (__any(most > top + kLazy)) {
                    const float now = fmaxf(top, most);
                    const float less = now == SDL_NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(top - now);
                    top = now;
                    total *= less;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < Co::kAcc; ++i)
                            O[d][i] *= less;
                }
                const float ref = top == SDL_NEG_INF ? 0.0f : top;
                float sums[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < Co::kAcc; ++i) {
                    x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], c2, -ref));
                    sums[i & 1] += x[i];
                }
                total += sums[0] + sums[1];
                if (!fold)
                    times_scales<Co::kAcc>(x, scale_of[n & 1][1] + C * b + 4 * part);
                // bf16 parts of the weights: one for q in bf16, rounded here
                typename Co::Weights pf[QP][Co::kGroups];
#pragma unroll
                for (int k = 0; k < QP; ++k) {
                    Acc z = x;
                    if (k < QP - 1)
#pragma unroll
                        for (int i = 0; i < Co::kAcc; ++i) {
                            z[i] = __uint_as_float(__float_as_uint(x[i]) & 0xffff0000);
                            x[i] -= z[i];
                        }
#pragma unroll
                    for (int i = 0; i < Co::kGroups; ++i)
                        pf[k][i] = Co::weights(z, i);
                }
                chain<Co::kGroups * DB, 4>(
                    [&](int i) { return Co::val_frag(vt, cols_at, i / DB, i % DB); },
                    [&](int i, typename Co::Weights f) {
#pragma unroll
                        for (int k = 0; k < QP; ++k)
                            O[i % DB] = Co::apply(f, pf[k][i / DB], O[i % DB]);
                    });
            }
            if (find)
                keep_row(n + 2);
            __syncthreads();
        }
        if (QP > 1 && strange != 0) {
            top = __builtin_inff();
            total = __builtin_nanf("");
        }

        // ---- join the wavefronts of a query group, and write
        total = Co::sum(total);
        if (part == 0) {
            tops[wave][lane] = top;
            totals[wave][lane] = total;
        }
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < Co::kAcc / 4; ++g)
                store4((float *)(lds + wave * Out::kBytes +
                                 Out::at(lane % C, (C * d + Co::key_of(4 * g)) / 4 + part)),
                       O[d][4 * g], O[d][4 * g + 1], O[d][4 * g + 2], O[d][4 * g + 3]);
        __syncthreads();
        join_waves<T, H, DP, DU, C, RG>(a, u, {span.w, seq, hk, block, n0, n1, later}, slots, lds, tops, totals, redo,
                                        drafts, wave, lane);
        at += n1 - n0;
        later = true;
    }
}

// Joins the slots of units that were cut, a row's pieces by the lanes of part of a
// wavefront and its spans by the wavefronts in turn: 250 spans to a unit take 9 us,
// with every span added by the same lanes 27.
template <class T, class H, int DP>
__global__ __launch_bounds__(1024) void join_codes(TreeArgs a, int numbers)
{
    constexpr int PIECES = DP / 4, ROWS = 64 / PIECES;
    __shared__ __align__(16) f32x4 outs[16][64];
    __shared__ float tops[16][ROWS], sums[16][ROWS];
    __shared__ int redo[ROWS];
    __shared__ Drafts drafts;
    const int t = threadIdx.x, lane = t & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int RB = a.block_rows, group = a.Hq / a.Hkv;
    const int row0 = blockIdx.y * ROWS, lr = lane / PIECES, p = lane % PIECES;
    const Slots slots(a);
    Cut cut;
    if (!cut.find<H>(a, slots, numbers, row0, lane))
        return;
    const int heads = wave_heads<H>(a), r = cut.block * RB + row0 + lr;
    float best = SDL_NEG_INF, sum = 0.0f;
    f32x4 o = f32x4(0.0f);
#pragma unroll 4
    for (int w = cut.w0 + wave; w <= cut.w1; w += waves) {
        const int64_t slot = w == cut.w0 ? cut.slot0 : 2 * (int64_t)w;
        const int64_t at = (slot * heads + cut.hk % heads) * RB + row0 + lr;
        const float top = slots.stat[2 * at], total = slots.stat[2 * at + 1];
        const f32x4 x = *(const f32x4 *)(slots.out + at * DP + 4 * p);
        const float now = fmaxf(best, top), ref = now == SDL_NEG_INF ? 0.0f : now;
        const float mine = __builtin_amdgcn_exp2f(best - ref), theirs = __builtin_amdgcn_exp2f(top - ref);
        best = now;
        sum = fmaf(theirs, total, mine * sum);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = fmaf(theirs, x[e], mine * o[e]);
    }
    outs[wave][lane] = o;
    if (p == 0) {
        tops[wave][lr] = best;
        sums[wave][lr] = sum;
    }
    if (t < ROWS)
        redo[t] = 0;
    __syncthreads();
    if (wave == 0 && r < cut.u.drafts * group) {
        best = SDL_NEG_INF;
        for (int w = 0; w < waves; ++w)
            best = fmaxf(best, tops[w][lr]);
        const float ref = best == SDL_NEG_INF ? 0.0f : best;
        sum = 0.0f;
        o = f32x4(0.0f);
        for (int w = 0; w < waves; ++w) {
            const float f = __builtin_amdgcn_exp2f(tops[w][lr] - ref);
            const f32x4 x = outs[w][lane];
            sum = fmaf(f, sums[w][lr], sum);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fmaf(f, x[e], o[e]);
        }
        finish<T, H>(a, cut.u.q_begin + r / group, cut.hk * group + r % group, p, best, sum, o, redo + lr);
    }
    __syncthreads();
    if (!__any(lane < ROWS && redo[lane] != 0))        // the same in all wavefronts
        return;
    if (wave == 0 && a.tree != nullptr)
        find_drafts(a, cut.u, lane, drafts);
    __syncthreads();
    finish_again<T, H>(a, cut.u, cut.seq, cut.hk, cut.block * RB + row0, ROWS, redo, drafts, wave, lane, waves);
}

template <class T, class H, int DP>
hipError_t launch_stream(const TreeArgs &a, hipStream_t stream)
{
    if (!a.together)
        tree_stream<T, H, DP, 16, false><<<a.workers, kAttnThreads, 0, stream>>>(a);
    else if (a.block_rows == 8)
        tree_stream<T, H, DP, 8, true><<<a.workers, kAttnThreads, 0, stream>>>(a);
    else
        tree_stream<T, H, DP, 16, true><<<a.workers, kAttnThreads, 0, stream>>>(a);
    // spans to a unit, in the mean: 16 wavefronts to a row of many (a batch of 64 answers
    // has 4, whose rows are joined side by side: 6 us)
    const int64_t units = (int64_t)a.S * (a.Hkv / a.wave_heads);
    if (a.workers / units < 16)
        return launch_join<T, H, DP, DP>(a, stream);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    constexpr int ROWS = 256 / DP;
    const int64_t numbers = join_numbers(a);
    join_codes<T, H, DP><<<dim3((uint32_t)(numbers * a.Hkv), (a.block_rows + ROWS - 1) / ROWS), 1024, 0, stream>>>(
        a, (int)numbers);
    return hipGetLastError();
}

template <class T, class H, int DP, int DU>
hipError_t launch_codes(const TreeArgs &a, hipStream_t stream)
{
    if (a.block_rows <= 16)
        return launch_stream<T, H, DP>(a, stream);
    // 16 queries to a wavefront where q in three parts leaves no registers for 32
    if (a.block_rows == 32) {
        tree_tiles<T, H, DP, DU, 16, 2><<<a.workers, kAttnThreads, 0, stream>>>(a);
    } else if constexpr (sizeof(T) == 4) {
        tree_tiles<T, H, DP, DU, 16, 4><<<a.workers, kAttnThreads, 0, stream>>>(a);
    } else {
        if (a.block_rows == 64)
            tree_tiles<T, H, DP, DU, 32, 2><<<a.workers, kAttnThreads, 0, stream>>>(a);
        else
            tree_tiles<T, H, DP, DU, 32, 4><<<a.workers, kAttnThreads, 0, stream>>>(a);
    }
    return launch_join<T, H, DP, DU>(a, stream);
}

// By the head's size, for q of type T.
template <class T, class H>
hipError_t launch_codes_sized(const TreeArgs &a, hipStream_t stream)
{
    return a.D <= 64 ? launch_codes<T, H, 64, 64>(a, stream)
                     : (a.D <= 96 ? launch_codes<T, H, 128, 96>(a, stream) : launch_codes<T, H, 128, 128>(a, stream));
}

}  // namespace

}  // namespace sdl
