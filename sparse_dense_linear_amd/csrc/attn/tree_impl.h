// tree_impl.h -- attention of drafted tokens over a paged cache: how the work is
// cut, joined and finished, for caches whose rows are of the type of q (H = T,
// tree.hip) or codes of 8 bits with a scale for each block of positions and head
// (H = E4M3, Int8; tree_codes.h).
//
// A sequence has ctx cached keys and T drafts whose keys follow them in the
// cache; draft t sees the context (through the window and the first keys)
// and the drafts that its mask names.  One answered token is T = 1.
//
// The T * (Hq / Hkv) queries that share a key head are the columns of one
// matrix product with its keys, so each cached row is read once for all of
// them (for as many as a block holds; more take another turn over L2).
//
// Work is counted in tiles of keys over (sequence, key head, block of
// queries) and cut into equal spans, one per workgroup, so that ragged
// batches and single long sequences fill the GPU alike.  A unit that lies
// within one span is finished there; one that is cut leaves its running
// maximum, sum and unnormalised output (fp32) in a slot of each span it
// touches, and a second launch joins them in span order: no atomics, the
// same result every time.
#pragma once

#include "ops.h"
#include "draft.h"
#include "exact.h"
#include "held.h"
#include "tile.h"
#include "spmm.h"

namespace sdl {

namespace {

// Keys of a tile of rows of the type of q: with 16 queries to a block, three
// workgroups share a CU and each has half a tile.
__host__ __device__ constexpr int tile_keys(int block_rows) { return block_rows == 16 ? 64 : 128; }

// Key heads that are worked on together by one workgroup: more than one where
// codes are streamed (tree_codes.h).
template <class H>
__device__ inline int wave_heads(const TreeArgs &a)
{
    if constexpr (kCodes<H>)
        return a.wave_heads;
    else
        return 1;
}
template <class H>
__device__ inline int key_groups(const TreeArgs &a) { return kCodes<H> ? a.Hkv / wave_heads<H>(a) : a.Hkv; }

// What sequence s asks for.
struct Unit {
    int q_begin, drafts, ctx, end;   // end: ctx + drafts
    int low;                         // first key of the window (any draft's)
    int first_tiles, band, tiles;    // key tiles [0, first_tiles) and [band, ..)
    int blocks;                      // blocks of queries
    int tile_keys;
};

template <class H>
__device__ inline Unit unit_of(const TreeArgs &a, int s)
{
    Unit u;
    u.q_begin = a.q_rowptr[s];
    u.drafts = a.q_rowptr[s + 1] - u.q_begin;
    u.ctx = a.ctx[s];
    u.end = u.ctx + u.drafts;
    u.low = u.ctx - a.window + 1 > 0 ? u.ctx - a.window + 1 : 0;
    if constexpr (kCodes<H>)
        u.tile_keys = a.tile_keys;
    else
        u.tile_keys = tile_keys(a.block_rows);
    u.band = u.low / u.tile_keys;
    u.first_tiles = (a.sinks + u.tile_keys - 1) / u.tile_keys;
    u.first_tiles = u.first_tiles < u.band ? u.first_tiles : u.band;
    u.tiles = u.first_tiles + (u.end + u.tile_keys - 1) / u.tile_keys - u.band;
    u.blocks = (u.drafts * (a.Hq / a.Hkv) + a.block_rows - 1) / a.block_rows;
    return u;
}

__device__ inline int first_key(const Unit &u, int n)
{
    return (n < u.first_tiles ? n : u.band + n - u.first_tiles) * u.tile_keys;
}

// f of all lanes' x, in each lane; f takes them in any order, f(x, x) is x.
template <class F>
__device__ inline int wave_of(int x, F f)
{
    // within a row of 16 lanes, turned by 8, 4, 2 and 1
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0x128, 15, 15, true));
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0x124, 15, 15, true));
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0x122, 15, 15, true));
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0x121, 15, 15, true));
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = f((int)r[0], (int)r[1]);
    r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return f((int)r[0], (int)r[1]);
}

// What all drafts of a sequence see together, and where each of them stands
// (in LDS).
struct Drafts {
    int place[64], named[64], low;
};

// By one wavefront; a.tree is not null.
__device__ inline void find_drafts(const TreeArgs &a, const Unit &u, int lane, Drafts &to)
{
    const uint64_t *masks = a.tree + u.q_begin;
    int low = u.ctx;
    uint64_t named = 0;
    int place = 0;
    for (int t = lane; t < u.drafts; t += 64) {
        const int at = count_draft(masks, u.ctx, u.drafts, a.window, a.sinks, t, low, named);
        place = t < 64 ? at : place;
    }
    low = wave_of(low, [](int x, int y) { return x < y ? x : y; });
    auto either = [](int x, int y) { return x | y; };
    const uint32_t named0 = wave_of((int)named, either), named1 = wave_of((int)(named >> 32), either);
    if (lane < u.drafts)
        to.place[lane] = place;
    to.named[lane] = (lane < 32 ? named0 : named1) >> (lane & 31) & 1;
    if (lane == 0)
        to.low = low;
}

// Tiles reach over keys that no draft sees.  Those are zero in LDS: what a
// masked pair multiplies by its weight of 0 is then no row that is seen
// elsewhere and may be infinite.
__device__ inline SeenRows seen_rows(const TreeArgs &a, const Unit &u, const Drafts &drafts)
{
    if (a.tree == nullptr)
        return {u.ctx, u.end, u.low, a.sinks, nullptr};
    return {u.ctx, u.end, drafts.low, a.sinks, drafts.named};
}

// Whether that need not be asked, as every key of j0 .. j1 is seen whatever the
// masks are: no draft stands further than 63 behind the context.
__device__ inline bool all_seen(const TreeArgs &a, const Unit &u, int j0, int j1)
{
    return a.tree == nullptr ? j1 < u.end && (j0 >= u.low || j1 < a.sinks)
                             : j1 < u.ctx && (j0 >= u.low + 63 || j1 < a.sinks);
}

// Row j of a pool.
template <class H>
struct PoolRows {
    const TreeArgs &a;
    const int32_t *table;
    const H *base;                    // at the key head
    const float *scale;               // (codes only)
    __device__ auto operator()(int j) const
    {
        const int p = j / a.page, in = j - p * a.page;
        const H *row = base + (int64_t)table[p] * a.page_stride + (int64_t)in * a.row_stride;
        if constexpr (kCodes<H>)
            return CodeRow<H>{row, scale[(int64_t)table[p] * a.scale_page + in / a.block * a.scale_block]};
        else
            return row;
    }
};

// Whether a row that some draft does not see, but that its tiles brought in as
// another one does, is not finite: keys that the window of the last draft has left,
// and the drafts.
template <class H>
__device__ bool odd_unseen(const TreeArgs &a, const Unit &u, const SeenRows &rows, const PoolRows<H> &k,
                           const PoolRows<H> &v, int D, int lane)
{
    if (u.drafts == 1)
        return false;                          // it sees all that is brought in
    const int left = u.end - a.window < u.ctx ? u.end - a.window : u.ctx;
    auto odd = [&](const PoolRows<H> &x) {
        return any_odd(x, rows.low, left, D, lane) || any_odd(x, rows, u.ctx, u.end, D, lane);
    };
    return odd(k) || odd(v);
}

// The spans: `workers` of them (at most one for each tile), span w from
// tile span_start(w) on.
struct Spans {
    int64_t tiles;
    int workers;
    __device__ int64_t start(int w) const { return divide(w * tiles, workers); }
    // the span that holds a tile
    __device__ int of(int64_t tile) const
    {
        return (int)divide((tile + 1) * workers + tiles - 1, tiles) - 1;
    }
    // of non-negative numbers; 64 bits cost some hundred instructions
    __device__ static int64_t divide(int64_t x, int64_t y)
    {
        return (x | y) >> 32 == 0 ? (uint32_t)x / (uint32_t)y : x / y;
    }
};

// Workspace: first tile of every sequence (S + 1), then for each span two
// slots (its first and its last unit) of maximum and sum, then their outputs.
struct Slots {
    int64_t *base;
    float *stat, *out;
    __device__ explicit Slots(const TreeArgs &a)
    {
        base = (int64_t *)a.partial;
        stat = a.partial + 2 * (((int64_t)a.S + 1 + 31) / 32 * 32);
        out = stat + (int64_t)2 * a.workers * a.slot_rows * 2;
    }
};

// A workgroup's span, and the sequence that holds its first tile.
struct Span {
    int w, seq;
    int64_t at, stop;      // tiles
    int64_t base;          // first tile of the sequence

    // By all threads of the workgroup; false: it has none.
    template <class H>
    __device__ bool begin(const TreeArgs &a, const Slots &slots)
    {
        __shared__ int64_t scan[4];
        __shared__ int found;
        __shared__ int64_t found_base;
        const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
        // the total of all tiles, then the sequence
        Spans spans;
        spans.tiles = 0;
        int64_t n = 0;
        for (int s0 = 0; s0 < a.S; s0 += kAttnThreads) {
            n = 0;
            if (s0 + t < a.S) {
                const Unit u = unit_of<H>(a, s0 + t);
                n = (int64_t)key_groups<H>(a) * u.blocks * u.tiles;
            }
            int64_t all = n;
            for (int d = 32; d > 0; d >>= 1)
                all += __shfl_xor(all, d);
            if (lane == 0)
                scan[wave] = all;
            __syncthreads();
            spans.tiles += scan[0] + scan[1] + scan[2] + scan[3];
            __syncthreads();
        }
        spans.workers = spans.tiles < a.workers ? (int)spans.tiles : a.workers;
        if ((int)blockIdx.x >= spans.workers)
            return false;
        w = xcd_order(blockIdx.x, spans.workers);
        at = spans.start(w);
        stop = spans.start(w + 1);
        int64_t sum = 0;
        for (int s0 = 0; s0 < a.S; s0 += kAttnThreads) {
            if (a.S > kAttnThreads) {          // else as it was
                n = 0;
                if (s0 + t < a.S) {
                    const Unit u = unit_of<H>(a, s0 + t);
                    n = (int64_t)key_groups<H>(a) * u.blocks * u.tiles;
                }
            }
            int64_t upto = n;                  // inclusive sum over the wavefront
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t y = __shfl_up(upto, d);
                if (lane >= d)
                    upto += y;
            }
            if (lane == 63)
                scan[wave] = upto;
            __syncthreads();
            for (int i = 0; i < wave; ++i)
                upto += scan[i];
            upto += sum;
            if (s0 + t < a.S) {
                if (upto - n <= at && at < upto) {
                    found = s0 + t;
                    found_base = upto - n;
                }
                if (w == 0) {
                    slots.base[s0 + t] = upto - n;
                    if (s0 + t == a.S - 1)
                        slots.base[a.S] = upto;
                }
            }
            sum += scan[0] + scan[1] + scan[2] + scan[3];
            __syncthreads();
        }
        seq = found;
        base = found_base;
        return true;
    }
};

// A finished row lr of a block: four elements of its output from the sum of
// weights and the unnormalised values.  redo[lr]: 1, the output is to be
// computed again if a row that is masked is not finite, or its sum became too
// large; 2, the sum of weights too (no key was seen, or a score is infinite
// or no number).  Over codes a score is no number where a key holds a NaN, or its scale
// is one, and then nor are the results: they are right as they are.
template <class T, class H>
__device__ inline void finish(const TreeArgs &a, int64_t token, int head, int p, float best, float sum,
                              const f32x4 &o, int *redo)
{
    const float lse = kLn2 * (best + __builtin_amdgcn_logf(sum));
    const float inv = 1.0f / sum;
    bool clean = finite(lse);
    if (4 * p < a.D) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = o[e] * inv;
            clean = clean && finite(y[e]);
        }
        store4((T *)a.o + (token * a.Hq + head) * a.D + 4 * p, y[0], y[1], y[2], y[3]);
    }
    if (p == 0)
        a.lse[head * a.Tq + token] = lse;
    if (!clean && !(kCodes<H> && sum != sum && best < __builtin_inff()))
        atomicMax(redo, finite(lse) ? 1 : 2);
}

// What finish() left to do in rows first .. first + count - 1 of a sequence's
// query rows, by the `waves` wavefronts of a workgroup, all of them; place: the
// drafts' positions.
template <class T, class H>
__device__ inline void finish_again(const TreeArgs &a, const Unit &u, int seq, int hk, int first, int count,
                                    const int *redo, const Drafts &drafts, int wave, int lane, int waves = 4)
{
    bool some = false, outputs = false;
    for (int lr = lane; lr < count; lr += 64)
        some = some || redo[lr] != 0, outputs = outputs || redo[lr] == 1;
    // (so seldom that no loop behind this is worth a register of one before it)
    if (__builtin_expect_with_probability(__any(some) == 0, 1, 0.999999))
        return;
    lane = renewed(lane);      // what goes by the lane is found here, not kept all along
    const int group = a.Hq / a.Hkv;
    const int32_t *table = a.table + (int64_t)seq * a.table_stride;
    const PoolRows<H> key{a, table, (const H *)a.k_pages + hk * a.head_stride, a.k_scale + hk * a.scale_head};
    const PoolRows<H> val{a, table, (const H *)a.v_pages + hk * a.head_stride, a.v_scale + hk * a.scale_head};
    const SeenRows rows = seen_rows(a, u, drafts);
    const bool odd = odd_unseen<H>(a, u, rows, key, val, a.D, lane);
    OddColumns values;
    if (!odd && __any(outputs)) {              // (the same for the whole workgroup)
        const int gap = a.sinks < u.low ? a.sinks : u.low;
        auto key_of = [&](int i) { return i < gap ? i : i - gap + u.low; };
        values.look([&](int i) { return val(key_of(i)); }, [&](int i) { return rows(key_of(i)); }, 0,
                    gap + u.end - u.low, a.D, lane, wave, waves);
        values.join(lane, wave);
    }
    for (int lr = wave; lr < count; lr += waves) {
        const int why = redo[lr];              // uniform over the wavefront
        if (why == 0)
            continue;
        const int r = first + lr, t = r / group, head = hk * group + r % group;
        const int64_t token = u.q_begin + t;
        T *o = (T *)a.o + (token * a.Hq + head) * a.D;
        if (why == 1 && !odd && !too_large(values, o, a.D, lane))
            continue;
        DraftSeen seen;
        seen.ctx = u.ctx;
        seen.drafts = u.drafts;
        seen.window = a.window;
        seen.sinks = a.sinks;
        seen.mask = a.tree != nullptr ? draft_mask(a.tree[u.q_begin + t], u.drafts) : 0;
        seen.pos = a.tree != nullptr ? draft_place(u.ctx, seen.mask) : u.ctx + t;
        seen.place = a.tree != nullptr ? drafts.place : nullptr;
        exact_row<T>((const T *)a.q + token * a.q_row + head * a.q_head, key, val, seen,
                     a.sinks < u.low ? a.sinks : u.low, u.low, u.end, a.D, a.scale * kLog2e,
                     o, a.lse + head * a.Tq + token, why == 1, lane);
    }
}

// Which part of which unit a workgroup has worked on: key tiles n0 .. n1 - 1, the
// first or a later piece of its span.
struct Piece {
    int w, seq, hk, block, n0, n1;
    bool later;
};

// Joins the wavefronts of each query group, whose outputs lie in lds (Tile<float,
// DP, C> for each wavefront) with their maxima and sums, and writes: the unit's
// results if the piece is all of it, else a slot.
template <class T, class H, int DP, int DU, int C, int RG>
__device__ inline void join_waves(const TreeArgs &a, const Unit &u, const Piece &c, const Slots &slots, const char *lds,
                                  const float (&tops)[4][C], const float (&totals)[4][C], int *redo,
                                  const Drafts &drafts, int wave, int lane)
{
    constexpr int KS = 4 / RG, RB = C * RG;
    typedef Tile<float, DP, C> Out;
    const int group = a.Hq / a.Hkv, rows = u.drafts * group;
    const bool done = c.n0 == 0 && c.n1 == u.tiles;
    const int64_t slot = 2 * (int64_t)c.w + (c.later ? 1 : 0);
    constexpr int kOutPieces = DU / 4;
    for (int m = threadIdx.x; m < RB * kOutPieces; m += kAttnThreads) {
        const int lr = m / kOutPieces, p = m % kOutPieces;
        const int rr = c.block * RB + lr;
        if (rr >= rows)
            break;
        float best = SDL_NEG_INF;
#pragma unroll
        for (int k = 0; k < KS; ++k)
            best = fmaxf(best, tops[k * RG + lr / C][lr % C]);
        const float ref = best == SDL_NEG_INF ? 0.0f : best;
        float sum = 0.0f;
        f32x4 o = f32x4(0.0f);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int wv = k * RG + lr / C;
            const float f = __builtin_amdgcn_exp2f(tops[wv][lr % C] - ref);
            sum = fmaf(f, totals[wv][lr % C], sum);
            const f32x4 x = *(const f32x4 *)(lds + wv * Out::kBytes + Out::at(lr % C, p));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fmaf(f, x[e], o[e]);
        }
        if (!done) {
            float *to = slots.out + (slot * RB + lr) * DP + 4 * p;
            *(f32x4 *)to = o;
            if (p == 0) {
                slots.stat[(slot * RB + lr) * 2] = best;
                slots.stat[(slot * RB + lr) * 2 + 1] = sum;
            }
            continue;
        }
        finish<T, H>(a, u.q_begin + rr / group, c.hk * group + rr % group, p, best, sum, o, redo + lr);
    }
    __syncthreads();
    if (done)
        finish_again<T, H>(a, u, c.seq, c.hk, c.block * RB, RB, redo, drafts, wave, lane);
}

// A unit that spans have cut, for its joining workgroup.
struct Cut {
    Unit u;
    int seq, hk, block, w0, w1;      // spans w0 .. w1
    int64_t slot0;                   // of the first; a unit that goes on is a span's first piece

    // By each wavefront; false: nothing to join from row0 of the block on.
    template <class H>
    __device__ bool find(const TreeArgs &a, const Slots &slots, int numbers, int row0, int lane)
    {
        const int RB = a.block_rows, group = a.Hq / a.Hkv;
        const int number = blockIdx.x % numbers;
        hk = blockIdx.x / numbers;
        const int64_t tiles = slots.base[a.S];
        // (all queries are fewer than 2^31)
        auto first = [&](int s) { return (int)((uint32_t)a.q_rowptr[s] * (uint32_t)group / (uint32_t)RB) + s; };
        int left = a.S;              // the last sequence whose first number is <= number
        seq = 0;
        while (left > 1) {
            const int step = (left + 63) / 64, s = seq + lane * step;
            const bool at = lane * step < left && first(s) <= number;
            const int n = __popcll(__ballot(at)) - 1;
            if (n < 0)
                return false;
            seq += n * step;
            left = left - n * step < step ? left - n * step : step;
        }
        u = unit_of<H>(a, seq);
        block = number - first(seq);
        if (block < 0 || block >= u.blocks || block * RB + row0 >= u.drafts * group)
            return false;
        Spans spans;
        spans.tiles = tiles;
        spans.workers = tiles < a.workers ? (int)tiles : a.workers;
        const int64_t from = slots.base[seq] + (int64_t)(hk / wave_heads<H>(a) * u.blocks + block) * u.tiles;
        w0 = spans.of(from);
        w1 = spans.of(from + u.tiles - 1);
        slot0 = 2 * (int64_t)w0 + (spans.start(w0) >= from ? 0 : 1);
        return w0 != w1;
    }
};

constexpr int kJoinRows = 16;      // query rows of a joining workgroup

// Joins the slots of the spans that a unit was cut over (units within one
// span are written already), kJoinRows of its rows to a workgroup.  Units are numbered
// without a list, as find_seq_tile does: the rows of sequence s, in blocks,
// have the numbers from rowptr[s] * group / rows + s on.
template <class T, class H, int DP, int DU>
__global__ __launch_bounds__(kAttnThreads) void tree_join(TreeArgs a, int numbers)
{
    __shared__ int redo[kJoinRows];
    __shared__ Drafts drafts;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int RB = a.block_rows, group = a.Hq / a.Hkv;
    const int row0 = blockIdx.y * kJoinRows;
    const Slots slots(a);
    Cut cut;
    if (!cut.find<H>(a, slots, numbers, row0, lane))
        return;
    const Unit &u = cut.u;
    const int hk = cut.hk, block = cut.block, rows = u.drafts * group, heads = wave_heads<H>(a);

    if (t < kJoinRows)
        redo[t] = 0;
    __syncthreads();
    constexpr int kOutPieces = DU / 4;
    for (int m = t; m < kJoinRows * kOutPieces; m += kAttnThreads) {
        const int lr = m / kOutPieces, p = m % kOutPieces;
        const int r = block * RB + row0 + lr;
        if (r >= rows || row0 + lr >= RB)
            break;
        float best = SDL_NEG_INF, sum = 0.0f;
        f32x4 o = f32x4(0.0f);
        auto add = [&](int64_t slot) {
            const int64_t row = (slot * heads + hk % heads) * RB + row0 + lr;
            const float top = slots.stat[2 * row], total = slots.stat[2 * row + 1];
            const f32x4 x = *(const f32x4 *)(slots.out + row * DP + 4 * p);
            const float now = fmaxf(best, top), ref = now == SDL_NEG_INF ? 0.0f : now;
            const float mine = __builtin_amdgcn_exp2f(best - ref), theirs = __builtin_amdgcn_exp2f(top - ref);
            best = now;
            sum = fmaf(theirs, total, mine * sum);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fmaf(theirs, x[e], mine * o[e]);
        };
        add(cut.slot0);
#pragma unroll 4
        for (int w = cut.w0 + 1; w <= cut.w1; ++w)     // a unit that goes on is a span's first
            add(2 * (int64_t)w);
        finish<T, H>(a, u.q_begin + r / group, hk * group + r % group, p, best, sum, o, redo + lr);
    }
    __syncthreads();
    if (!__any(lane < kJoinRows && redo[lane] != 0))    // the same in all wavefronts
        return;
    if (wave == 0 && a.tree != nullptr)
        find_drafts(a, u, lane, drafts);
    __syncthreads();
    finish_again<T, H>(a, u, cut.seq, hk, block * RB + row0, kJoinRows, redo, drafts, wave, lane);
}

// Blocks of queries that the join numbers, of one key head.
int64_t join_numbers(const TreeArgs &a) { return a.Tq * (a.Hq / a.Hkv) / a.block_rows + a.S; }

template <class T, class H, int DP, int DU>
hipError_t launch_join(const TreeArgs &a, hipStream_t stream)
{
    hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    const int64_t numbers = join_numbers(a);
    tree_join<T, H, DP, DU><<<dim3((uint32_t)(numbers * a.Hkv), (a.block_rows + kJoinRows - 1) / kJoinRows), kAttnThreads, 0, stream>>>(
        a, (int)numbers);
    return hipGetLastError();
}

}  // namespace

}  // namespace sdl
