// tree.hip -- attention of drafted tokens over a paged cache.
//
// A sequence has ctx cached keys and T drafts whose keys follow them in the
// cache; draft t sees the context (through the window and the first keys)
// and the drafts that its mask names.  One answered token is T = 1.
//
// The T * (Hq / Hkv) queries that share a key head are the columns of one
// matrix product with its keys, so each cached row is read once for all of
// them (for up to 32 * RG of them; more take another turn over L2).
//
// Work is counted in tiles of keys over (sequence, key head, block of
// queries) and cut into equal spans, one per workgroup, so that ragged
// batches and single long sequences fill the GPU alike.  A unit that lies
// within one span is finished there; one that is cut leaves its running
// maximum, sum and unnormalised output (fp32) in a slot of each span it
// touches, and a second launch joins them in span order: no atomics, the
// same result every time.
//
// One answered token of each sequence is bound by the read of the cache: 64
// sequences, 1.39 GB in 225 us = 6.2 TB/s (a plain read reaches 7.1), 6 us
// for the join.  Drafts of up to 64 tokens with 8 heads on one are bound by
// latency, two workgroups to a CU: 23 GFLOP in 73 us and 12 for the join.
#include "ops.h"
#include "draft.h"
#include "exact.h"
#include "tile.h"
#include "spmm.h"

namespace sdl {

namespace {

// Keys of a tile: with 16 queries to a block, three workgroups share a CU and
// each has half a tile.
__host__ __device__ constexpr int tile_keys(int block_rows) { return block_rows == 16 ? 64 : 128; }

// What sequence s asks for.
struct Unit {
    int q_begin, drafts, ctx, end;   // end: ctx + drafts
    int low;                         // first key of the window (any draft's)
    int first_tiles, band, tiles;    // key tiles [0, first_tiles) and [band, ..)
    int blocks;                      // blocks of queries
    int tile_keys;
};

__device__ inline Unit unit_of(const TreeArgs &a, int s)
{
    Unit u;
    u.q_begin = a.q_rowptr[s];
    u.drafts = a.q_rowptr[s + 1] - u.q_begin;
    u.ctx = a.ctx[s];
    u.end = u.ctx + u.drafts;
    u.low = u.ctx - a.window + 1 > 0 ? u.ctx - a.window + 1 : 0;
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

// Row j of a pool, and whether a row that some draft does not see, but that
// its tiles brought in, is not finite: keys at the lower end of the window,
// and the drafts.
template <class T>
struct PoolRows {
    const TreeArgs &a;
    const int32_t *table;
    const T *base;                    // at the key head
    __device__ const T *operator()(int j) const
    {
        const int p = j / a.page;
        return base + (int64_t)table[p] * a.page_stride + (int64_t)(j - p * a.page) * a.row_stride;
    }
};

template <class T>
__device__ bool odd_unseen(const Unit &u, const SeenRows &rows, const PoolRows<T> &k, const PoolRows<T> &v, int D,
                           int lane)
{
    const int edge = u.low + u.drafts < u.ctx ? u.low + u.drafts : u.ctx;
    auto odd = [&](const PoolRows<T> &x) {
        return any_odd<T>(x, rows.low, edge, D, lane) || any_odd<T>(x, rows, u.ctx, u.end, D, lane);
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
        out = stat + (int64_t)2 * a.workers * a.block_rows * 2;
    }
};

// A workgroup's span, and the sequence that holds its first tile.
struct Span {
    int w, seq;
    int64_t at, stop;      // tiles
    int64_t base;          // first tile of the sequence

    // By all threads of the workgroup; false: it has none.
    __device__ bool begin(const TreeArgs &a, const Slots &slots)
    {
        __shared__ int64_t scan[4];
        __shared__ int found;
        __shared__ int64_t found_base;
        const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
        // the total of all tiles, then the sequence
        Spans spans;
        spans.tiles = 0;
        for (int s0 = 0; s0 < a.S; s0 += kAttnThreads) {
            int64_t n = 0;
            if (s0 + t < a.S) {
                const Unit u = unit_of(a, s0 + t);
                n = (int64_t)a.Hkv * u.blocks * u.tiles;
            }
            for (int d = 32; d > 0; d >>= 1)
                n += __shfl_xor(n, d);
            if (lane == 0)
                scan[wave] = n;
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
            int64_t n = 0;
            if (s0 + t < a.S) {
                const Unit u = unit_of(a, s0 + t);
                n = (int64_t)a.Hkv * u.blocks * u.tiles;
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
// or no number).
template <class T>
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
    if (!clean)
        atomicMax(redo, finite(lse) ? 1 : 2);
}

// What finish() left to do in rows first .. first + count - 1 of a sequence's
// query rows, by the four wavefronts of a workgroup; place: the drafts'
// positions.
template <class T>
__device__ inline void finish_again(const TreeArgs &a, const Unit &u, int seq, int hk, int first, int count,
                                    const int *redo, const Drafts &drafts, int wave, int lane)
{
    const int group = a.Hq / a.Hkv;
    bool some = false, outputs = false;
    for (int lr = lane; lr < count; lr += 64)
        some = some || redo[lr] != 0, outputs = outputs || redo[lr] == 1;
    if (!__any(some))
        return;
    const int32_t *table = a.table + (int64_t)seq * a.table_stride;
    const PoolRows<T> key{a, table, (const T *)a.k_pages + hk * a.head_stride};
    const PoolRows<T> val{a, table, (const T *)a.v_pages + hk * a.head_stride};
    const SeenRows rows = seen_rows(a, u, drafts);
    const bool odd = odd_unseen<T>(u, rows, key, val, a.D, lane);
    TooLarge<T> too_large;
    if (!odd && __any(outputs)) {
        too_large.look(val, rows, 0, a.sinks < u.low ? a.sinks : u.low, a.D, lane);
        too_large.look(val, rows, u.low, u.end, a.D, lane);
    }
    for (int lr = wave; lr < count; lr += 4) {
        const int why = redo[lr];              // uniform over the wavefront
        if (why == 0)
            continue;
        const int r = first + lr, t = r / group, head = hk * group + r % group;
        const int64_t token = u.q_begin + t;
        T *o = (T *)a.o + (token * a.Hq + head) * a.D;
        if (why == 1 && !odd && !too_large(o, a.D, lane))
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

// Where sequences fill one block of 16 queries in the mean, most keys are read
// once, and keeping them in the caches would only push out what is read again.
// (64 answers: 231 us against 255; trees of drafts, several blocks each, 83
// against 76 the other way round.)
template <bool ONCE>
__device__ inline u32x4 load_once(const u32x4 *p)
{
    return ONCE ? __builtin_nontemporal_load(p) : *p;
}

// Workgroups to a CU that registers and LDS allow.
template <class T, int DP>
constexpr int per_cu(int block_rows)
{
    const int tile = 2 * tile_keys(block_rows) * DP * (int)sizeof(T);
    return tile <= 16384 ? 4 : (tile <= 32768 && block_rows == 16 ? 3 : (tile <= 65536 ? 2 : 1));
}

// RG groups of C queries; the 4 / RG wavefronts of a group share the keys of
// a tile.
template <class T, int DP, int DU, int C, int RG>
__global__ __launch_bounds__(kAttnThreads, (per_cu<T, DP>(C * RG))) void tree_attn(TreeArgs a)
{
    constexpr int KS = 4 / RG;                 // wavefronts that share a query group's keys
    constexpr int RB = C * RG;                 // queries of a block
    constexpr int kTileKeys = tile_keys(RB);
    typedef Cols<T, DP, DU, kTileKeys, C> Co;
    typedef typename Co::Acc Acc;
    constexpr int STEPS = Co::kSteps, DB = Co::kBlocks;
    typedef Tile<T, DP, kTileKeys> Tl;
    typedef Tile<float, DP, C> Out;
    constexpr int kPiecesPer = kTileKeys * Tl::kPieces / kAttnThreads;
    constexpr int kBytes = 2 * Tl::kBytes > 4 * Out::kBytes ? 2 * Tl::kBytes : 4 * Out::kBytes;
    __shared__ __align__(16) char lds[kBytes];
    __shared__ Drafts drafts;
    __shared__ float tops[4][C], totals[4][C];
    __shared__ int redo[RB];
    __shared__ int64_t place_of[2][kTileKeys];     // of a tile's rows, in the pools

    const int t = threadIdx.x, lane = t & 63, part = lane / C;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int group = a.Hq / a.Hkv;
    const int rg = wave % RG, ks = wave / RG;
    const float c2 = a.scale * kLog2e;
    const Slots slots(a);

    Span span;
    if (!span.begin(a, slots))
        return;
    const int w = span.w;
    int64_t at = span.at, base = span.base;
    const int64_t stop = span.stop;
    int seq = span.seq;

    // ---- the units of the span, one piece after another
    int64_t piece_no = 0;
    while (at < stop) {
        Unit u = unit_of(a, seq);
        int64_t mine = (int64_t)a.Hkv * u.blocks * u.tiles;
        while (at >= base + mine) {            // the next sequence that has tiles
            base += mine;
            ++seq;
            u = unit_of(a, seq);
            mine = (int64_t)a.Hkv * u.blocks * u.tiles;
        }
        const int unit = (int)Spans::divide(at - base, u.tiles);
        const int hk = unit / u.blocks, block = unit % u.blocks;
        const int n0 = (int)(at - base - (int64_t)unit * u.tiles);
        const int n1 = stop - at < u.tiles - n0 ? n0 + (int)(stop - at) : u.tiles;
        const int rows = u.drafts * group;

        // the drafts' positions, and what they see together
        __syncthreads();
        if (t < RB)
            redo[t] = 0;
        if (wave == 3 && a.tree != nullptr)    // (the first ones find the rows)
            find_drafts(a, u, lane, drafts);

        // this lane's query
        const int r = block * RB + C * rg + lane % C;
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
        Frag<T> qf[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            qf[s] = Co::kTerms * s + 8 * part < a.D ? load8(q + Co::kTerms * s + 8 * part) : zero_frag<T>();

        Acc O[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
            O[d] = Acc(0.0f);
        float top = SDL_NEG_INF, total = 0.0f;

        // Rows pass through registers: a tile's rows are under way while the
        // tile before it is worked on, in both workgroups of a CU, which is
        // what keeps HBM busy (LDS alone could not hold as much).  Where the
        // rows lie is found two tiles ahead, once for each row.
        const int32_t *table = a.table + (int64_t)seq * a.table_stride;
        const T *kp = (const T *)a.k_pages + hk * a.head_stride, *vp = (const T *)a.v_pages + hk * a.head_stride;
        u32x4 pk[kPiecesPer], pv[kPiecesPer];
        int id = 0, in_page = 0;               // in_page < 0: a row that is not read
        auto whole = [&](int n) { return all_seen(a, u, first_key(u, n), first_key(u, n) + kTileKeys - 1); };
        auto find_row = [&](int n) {
            const int j = first_key(u, n) + t;
            in_page = -1;
            if (whole(n) || seen_rows(a, u, drafts)(j)) {
                const int p = j / a.page;
                in_page = j - p * a.page;
                id = table[p];
            }
        };
        auto keep_row = [&](int n) {
            place_of[n & 1][t] = in_page < 0 ? -1 : (int64_t)id * a.page_stride + (int64_t)in_page * a.row_stride;
        };
        auto fetch = [&](int n) {
            const int tt = renewed(t);
            int64_t at[kPiecesPer];            // all of them before the loads, which then go out together
#pragma unroll
            for (int i = 0; i < kPiecesPer; ++i)
                at[i] = place_of[n & 1][(tt + i * kAttnThreads) / Tl::kPieces];
            auto load = [&](bool all) {
#pragma unroll
                for (int i = 0; i < kPiecesPer; ++i) {
                    const int p = (tt + i * kAttnThreads) % Tl::kPieces;
                    const int d = p * Tl::kElems < a.D ? p * Tl::kElems : a.D - Tl::kElems;
                    if (!all) {
                        pk[i] = u32x4(0);
                        pv[i] = u32x4(0);
                    }
                    if (all || at[i] >= 0) {
                        pk[i] = load_once<C == 16>((const u32x4 *)(kp + at[i] + d));
                        pv[i] = load_once<C == 16>((const u32x4 *)(vp + at[i] + d));
                    }
                }
            };
            if (whole(n))
                load(true);
            else
                load(false);
        };
        if (a.tree != nullptr && !(whole(n0) && (n0 + 1 >= n1 || whole(n0 + 1))))
            __syncthreads();                   // what the drafts see is there
        if (t < kTileKeys) {
            find_row(n0);
            keep_row(n0);
            if (n0 + 1 < n1) {
                find_row(n0 + 1);
                keep_row(n0 + 1);
            }
        }
        __syncthreads();
        fetch(n0);
        for (int n = n0; n < n1; ++n) {
            char *kt = lds, *vt = lds + Tl::kBytes;
#pragma unroll
            for (int i = 0; i < kPiecesPer; ++i) {
                const int m = t + i * kAttnThreads;
                *(u32x4 *)(kt + Tl::at(m / Tl::kPieces, m % Tl::kPieces)) = pk[i];
                *(u32x4 *)(vt + Tl::at(m / Tl::kPieces, m % Tl::kPieces)) = pv[i];
            }
            const bool find = t < kTileKeys && n + 2 < n1;
            if (find)
                find_row(n + 2);
            if (n + 1 < n1)
                fetch(n + 1);
            __syncthreads();
#pragma unroll 1
            for (int b = ks; b < kTileKeys / C; b += KS) {
                const int j0 = first_key(u, n) + C * b, j1 = j0 + C - 1;
                if (j0 >= u.end || (j1 < u.low && j0 >= a.sinks) || block * RB + C * rg >= rows)
                    continue;
                const int rows_at = renewed(Co::row_base(lane) + C * b * Tl::kRowBytes);
                const int cols_at = renewed(Co::col_base(lane) + C * b * Tl::kRowBytes);
                Acc x = Acc(0.0f);
                chain<STEPS, 4>([&](int i) { return Co::key_frag(kt, rows_at, i); },
                                [&](int i, Frag<T> f) { x = Co::mul(f, qf[i], x); });
                if (!(j1 < u.ctx && (u.end - 1 - j0 < a.window || j1 < a.sinks))) {
                    const int j = renewed(j0 + 4 * part);
#pragma unroll
                    for (int i = 0; i < Co::kAcc; ++i)
                        if (!seen(j + Co::key_of(i)))
                            x[i] = SDL_NEG_INF;
                }
                const float most = Co::most(x) * c2;
                if (__any(most > top + kLazy)) {
                    const float now = fmaxf(top, most);
                    const float keep = now == SDL_NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(top - now);
                    top = now;
                    total *= keep;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < Co::kAcc; ++i)
                            O[d][i] *= keep;
                }
                const float ref = top == SDL_NEG_INF ? 0.0f : top;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < Co::kAcc; ++i) {
                    x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], c2, -ref));
                    sum += x[i];
                }
                total += sum;
                typename Co::Weights pf[Co::kGroups];
#pragma unroll
                for (int i = 0; i < Co::kGroups; ++i)
                    pf[i] = Co::weights(x, i);
                chain<Co::kGroups * DB, 4>(
                    [&](int i) { return Co::val_frag(vt, cols_at, i / DB, i % DB); },
                    [&](int i, typename Co::Weights f) { O[i % DB] = Co::apply(f, pf[i / DB], O[i % DB]); });
            }
            if (find)
                keep_row(n + 2);
            __syncthreads();
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
        const bool done = n0 == 0 && n1 == u.tiles;
        const int64_t slot = 2 * (int64_t)w + (piece_no == 0 ? 0 : 1);
        constexpr int kOutPieces = DU / 4;
        for (int m = t; m < RB * kOutPieces; m += kAttnThreads) {
            const int lr = m / kOutPieces, p = m % kOutPieces;
            const int rr = block * RB + lr;
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
            finish<T>(a, u.q_begin + rr / group, hk * group + rr % group, p, best, sum, o, redo + lr);
        }
        __syncthreads();
        if (done)
            finish_again<T>(a, u, seq, hk, block * RB, RB, redo, drafts, wave, lane);
        at += n1 - n0;
        ++piece_no;
    }
}

constexpr int kJoinRows = 16;      // query rows of a joining workgroup

// Joins the slots of the spans that a unit was cut over (units within one
// span are written already), kJoinRows of its rows to a workgroup.  Units are numbered
// without a list, as find_seq_tile does: the rows of sequence s, in blocks,
// have the numbers from rowptr[s] * group / rows + s on.
template <class T, int DP, int DU>
__global__ __launch_bounds__(kAttnThreads) void tree_join(TreeArgs a, int numbers)
{
    __shared__ int redo[kJoinRows];
    __shared__ Drafts drafts;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int RB = a.block_rows, group = a.Hq / a.Hkv;
    const int hk = blockIdx.x / numbers, number = blockIdx.x % numbers;
    const Slots slots(a);
    const int64_t tiles = slots.base[a.S];
    int seq = 0, left = a.S;                   // the last sequence whose first number is <= number
    while (left > 1) {
        const int step = (left + 63) / 64, s = seq + lane * step;
        const bool at = lane * step < left && (int64_t)a.q_rowptr[s] * group / RB + s <= number;
        const int n = __popcll(__ballot(at)) - 1;
        if (n < 0)
            return;
        seq += n * step;
        left = left - n * step < step ? left - n * step : step;
    }
    const Unit u = unit_of(a, seq);
    const int block = number - (int)((int64_t)u.q_begin * group / RB + seq);
    const int rows = u.drafts * group;
    const int row0 = blockIdx.y * kJoinRows;
    if (block < 0 || block >= u.blocks || block * RB + row0 >= rows)
        return;
    Spans spans;
    spans.tiles = tiles;
    spans.workers = tiles < a.workers ? (int)tiles : a.workers;
    const int64_t from = slots.base[seq] + (int64_t)(hk * u.blocks + block) * u.tiles;
    const int w0 = spans.of(from), w1 = spans.of(from + u.tiles - 1);
    if (w0 == w1)
        return;
    const int64_t slot0 = 2 * (int64_t)w0 + (spans.start(w0) >= from ? 0 : 1);

    if (t < kJoinRows)
        redo[t] = 0;
    __syncthreads();
    constexpr int kOutPieces = DU / 4;
    for (int m = t; m < kJoinRows * kOutPieces; m += kAttnThreads) {
        const int lr = m / kOutPieces, p = m % kOutPieces;
        const int r = block * RB + row0 + lr;
        if (r >= rows)
            break;
        float best = SDL_NEG_INF, sum = 0.0f;
        f32x4 o = f32x4(0.0f);
        auto add = [&](int64_t slot) {
            const int64_t row = slot * RB + row0 + lr;
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
        add(slot0);
#pragma unroll 4
        for (int w = w0 + 1; w <= w1; ++w)     // a unit that goes on is a span's first
            add(2 * (int64_t)w);
        finish<T>(a, u.q_begin + r / group, hk * group + r % group, p, best, sum, o, redo + lr);
    }
    __syncthreads();
    if (!__any(lane < kJoinRows && redo[lane] != 0))    // the same in all wavefronts
        return;
    if (wave == 0 && a.tree != nullptr)
        find_drafts(a, u, lane, drafts);
    __syncthreads();
    finish_again<T>(a, u, seq, hk, block * RB + row0, kJoinRows, redo, drafts, wave, lane);
}

// Blocks of queries that the join numbers, of one key head.
int64_t join_numbers(const TreeArgs &a) { return a.Tq * (a.Hq / a.Hkv) / a.block_rows + a.S; }

template <class T, int DP, int DU>
hipError_t launch(const TreeArgs &a, hipStream_t stream)
{
    if (a.block_rows == 16)
        tree_attn<T, DP, DU, 16, 1><<<a.workers, kAttnThreads, 0, stream>>>(a);
    else if (a.block_rows == 32)
        tree_attn<T, DP, DU, 32, 1><<<a.workers, kAttnThreads, 0, stream>>>(a);
    else if (a.block_rows == 64)
        tree_attn<T, DP, DU, 32, 2><<<a.workers, kAttnThreads, 0, stream>>>(a);
    else
        tree_attn<T, DP, DU, 32, 4><<<a.workers, kAttnThreads, 0, stream>>>(a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    const int64_t numbers = join_numbers(a);
    tree_join<T, DP, DU><<<dim3((uint32_t)(numbers * a.Hkv), a.block_rows / kJoinRows), kAttnThreads, 0, stream>>>(
        a, (int)numbers);
    return hipGetLastError();
}

}  // namespace

TreeShape tree_shape(int dtype, int64_t S, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D)
{
    TreeShape sh;
    const int DP = D <= 64 ? 64 : 128;
    // as many queries to a block as the mean sequence fills
    const int64_t rows = S > 0 ? (Tq + S - 1) / S * (Hq / Hkv) : 0;
    sh.block_rows = rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128));
    // as many workgroups as the 256 CUs hold at once
    if (dtype == SPMM_DTYPE_BF16)
        sh.workers = 256 * (DP == 64 ? per_cu<__bf16, 64>(sh.block_rows) : per_cu<__bf16, 128>(sh.block_rows));
    else
        sh.workers = 256 * (DP == 64 ? per_cu<float, 64>(sh.block_rows) : per_cu<float, 128>(sh.block_rows));
    sh.bytes = 4 * (2 * ((S + 1 + 31) / 32 * 32) + 2 * (int64_t)sh.workers * sh.block_rows * (2 + DP));
    return sh;
}

int64_t tree_threads(const TreeArgs &a)
{
    const int64_t join = join_numbers(a) * a.Hkv, most = join > a.workers ? join : a.workers;
    return most * kAttnThreads;
}

hipError_t launch_tree(int dtype, const TreeArgs &a, hipStream_t stream)
{
    if (dtype == SPMM_DTYPE_BF16)
        return a.D <= 64 ? launch<__bf16, 64, 64>(a, stream)
                         : (a.D <= 96 ? launch<__bf16, 128, 96>(a, stream) : launch<__bf16, 128, 128>(a, stream));
    return a.D <= 64 ? launch<float, 64, 64>(a, stream)
                     : (a.D <= 96 ? launch<float, 128, 96>(a, stream) : launch<float, 128, 128>(a, stream));
}

}  // namespace sdl
