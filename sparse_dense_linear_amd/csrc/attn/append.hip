// append.hip -- new rows of a paged cache, rotated by their position on the way.
//
// A row of D elements is taken in groups of eight by D / 8 lanes.  A rotated
// group holds four pairs (x, y), in halves elements 4 g .. and rotated / 2 +
// 4 g .., else 8 g .. 8 g + 7, so that a lane needs four cosines and four
// sines, 4 g .., either way; they serve all heads of a row.
//
// Pools of codes need the largest value of each block of positions and head
// before the first code is written: a wavefront takes one block of one head
// and one pool, and keeps its rows in registers, or reads them again from L2
// where there are more than it holds.
//
// Bound by memory: 16384 rows of bf16, 48 heads of 128, 411 MB in 81 us = 5.1 TB/s,
// the rate of a large copy; 8192 rows into codes, 189 MB in 37 us (46 with caches that
// other work has filled).  A batch of single rows takes 6 to 8 us, a launch and four
// loads that wait for each other: the sequence, its context, the page, the scale.
#include "ops.h"

#include "cache.h"
#include "draft.h"
#include "exact.h"
#include "held.h"
#include "tile.h"

namespace sdl {

namespace {

constexpr int kWaves = kAttnThreads / 64;

// Lanes of a row, for heads of up to 8 * LPR elements.
template <int LPR> constexpr int kRowsPer = 64 / LPR;       // rows of a wavefront

__device__ inline f32x4 load4(const __bf16 *p)
{
    const bf16x4 x = *(const bf16x4 *)p;
    return f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
}
__device__ inline f32x4 load4(const float *p) { return *(const f32x4 *)p; }

struct Angles {
    f32x4 c, s;
};

// A lane's group of a row: where its two quads lie, and their rotation.
struct Group {
    int g, d0, d1;
    bool in, turned;
    __device__ Group(const AppendArgs &a, int g_) : g(g_)
    {
        in = 8 * g < a.D;
        turned = 8 * g < a.rotated;
        const bool halves = turned && a.interleaved == 0;
        d0 = halves ? 4 * g : 8 * g;
        d1 = halves ? a.rotated / 2 + 4 * g : 8 * g + 4;
    }
    // of the position where a row stands
    __device__ Angles angles(const AppendArgs &a, int place) const
    {
        const float nan = __builtin_nanf("");
        Angles t = {f32x4(nan), f32x4(nan)};
        if (turned && has_angles(place, a.angles)) {
            const int64_t at = (int64_t)place * (a.rotated / 2) + 4 * g;
            t.c = *(const f32x4 *)(a.cosines + at);
            t.s = *(const f32x4 *)(a.sines + at);
        }
        return t;
    }
    // every product and sum rounded by itself
    __device__ void turn(const AppendArgs &a, const Angles &t, f32x4 &x, f32x4 &y) const
    {
#pragma clang fp contract(off)
        if (!turned)
            return;
        if (a.interleaved == 0) {
            const f32x4 u = x * t.c - y * t.s;
            y = y * t.c + x * t.s;
            x = u;
        } else {
            const f32x4 p = {x[0], x[2], y[0], y[2]}, q = {x[1], x[3], y[1], y[3]};
            const f32x4 u = p * t.c - q * t.s, v = q * t.c + p * t.s;
            x = f32x4{u[0], v[0], u[1], v[1]};
            y = f32x4{u[2], v[2], u[3], v[3]};
        }
    }
};

// The last i of 0 .. S - 1 with first(i) <= x, -1 if there is none, first being
// non-decreasing: 64 places looked at at once, by a wavefront.
template <class First>
__device__ inline int last_not_above(First first, int S, int64_t x, int lane)
{
    int at = 0, left = S;
    do {
        const int step = (left + 63) / 64, i = at + lane * step;
        const bool is = lane * step < left && first(i) <= x;
        const int n = __popcll(__ballot(is)) - 1;
        if (n < 0)
            return -1;
        at += n * step;
        left = left - n * step < step ? left - n * step : step;
    } while (left > 1);
    return at;
}

// A sequence's rows, and where they stand.
struct Rowed {
    int first, count, ctx;
    __device__ Rowed(const AppendArgs &a, int seq)
    {
        first = a.rowptr[seq];
        count = a.rowptr[seq + 1] - first;
        ctx = a.ctx[seq];
    }
    __device__ int place(const AppendArgs &a, int t) const
    {
        return a.tree != nullptr ? draft_place(ctx, draft_mask(a.tree[first + t], count)) : ctx + t;
    }
};

// Number of the page that holds a position, -1 if there is none.
__device__ inline int64_t page_of(const AppendArgs &a, int seq, int pos)
{
    const int p = pos / a.page;
    if (pos < 0 || p >= a.table_stride)
        return -1;
    const int number = a.table[(int64_t)seq * a.table_stride + p];
    return number >= 0 && number < a.pages ? number : -1;
}

// Heads of a wavefront, all of which are loaded before one is stored (17000 rows of 48
// heads: 80 us, with four such turns to a wavefront, which find their rows once, 85).
constexpr int kHeads = 4;

// Rows of q and, where the pools hold them as they are, of k and v: kRowsPer
// rows to a wavefront and kHeads heads of them, counted through q, k and v.
template <class T, bool CODES, int LPR>
__device__ inline void move_rows(const AppendArgs &a, uint32_t wave, int lane)
{
    constexpr int ROWS = kRowsPer<LPR>;
    const int all = a.Hq + (CODES ? 0 : 2 * a.Hkv), parts = (all + kHeads - 1) / kHeads;
    if (all == 0)
        return;
    const int h = (int)(wave % (uint32_t)parts) * kHeads;
    const int64_t first = (int64_t)(wave / (uint32_t)parts) * ROWS;
    if (first >= a.T)
        return;
    int seq = -1;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int s = last_not_above([&](int n) { return a.rowptr[n]; }, a.S, first + i, lane);
        if (lane / LPR == i)
            seq = s;
    }
    const int64_t row = first + lane / LPR;
    const Group group(a, lane % LPR);
    if (seq < 0 || row >= a.rowptr[seq + 1] || !group.in)
        return;
    const Rowed rows(a, seq);
    const int t = (int)row - rows.first, pos = rows.ctx + t;
    const Angles angles = group.angles(a, rows.place(a, t));
    int64_t at = -1;                                       // of the row in the pools
    if (!CODES) {
        const int64_t number = page_of(a, seq, pos);
        if (number >= 0)
            at = number * a.page_stride + (int64_t)(pos % a.page) * a.row_stride;
    }
    f32x4 x[kHeads], y[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (h + i >= all)
            break;
        const bool is_q = h + i < a.Hq, is_k = h + i < a.Hq + a.Hkv;
        const Rows &from = is_q ? a.q : (is_k ? a.k : a.v);
        const int head = h + i - (is_q ? 0 : (is_k ? a.Hq : a.Hq + a.Hkv));
        const T *p = (const T *)from.base + row * from.row_stride + head * from.head_stride;
        x[i] = load4(p + group.d0);
        y[i] = load4(p + group.d1);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (h + i >= all)
            break;
        const bool is_q = h + i < a.Hq, is_k = h + i < a.Hq + a.Hkv;
        const int head = h + i - (is_q ? 0 : (is_k ? a.Hq : a.Hq + a.Hkv));
        if (is_k)
            group.turn(a, angles, x[i], y[i]);
        if (!is_q && at < 0)
            continue;
        T *to = is_q ? (T *)a.q_out.base + row * a.q_out.row_stride + head * a.q_out.head_stride
                     : (T *)(is_k ? a.k_pages : a.v_pages) + at + head * a.head_stride;
        store4(to + group.d0, x[i][0], x[i][1], x[i][2], x[i][3]);
        store4(to + group.d1, y[i][0], y[i][1], y[i][2], y[i][3]);
    }
}

// Blocks of positions that a call may write to are numbered without a list:
// sequence s, whose n rows touch at most n / block + 2 of them, owns the
// numbers from rowptr[s] / block + 2 s on.
__host__ __device__ inline int64_t block_numbers(const AppendArgs &a) { return a.T / a.block + 2 * (int64_t)a.S; }

// One block of one head and one pool, by a wavefront.  (Wavefronts, positions and rows
// fit 32 bits; a division of 64 costs some hundred instructions.)
template <class T, class H, int LPR>
__device__ inline void code_block(const AppendArgs &a, uint32_t wave, int lane)
{
    constexpr int ROWS = kRowsPer<LPR>, kHold = 4;
    const uint32_t columns = 2 * (uint32_t)a.Hkv, block = (uint32_t)a.block;
    const int which = (int)(wave % columns);
    const int64_t number = wave / columns;
    const bool is_k = which < a.Hkv;
    const int head = is_k ? which : which - a.Hkv;
    const int seq = last_not_above([&](int n) { return (int64_t)((uint32_t)a.rowptr[n] / block) + 2 * (int64_t)n; },
                                   a.S, number, lane);
    if (seq < 0)
        return;
    const Rowed rows(a, seq);
    const int64_t begin =
        (block_of(rows.ctx, a.block) + number - ((uint32_t)rows.first / block + 2 * (int64_t)seq)) * block;
    const int64_t end = (int64_t)rows.ctx + rows.count;
    if (rows.count <= 0 || begin >= end)
        return;
    const int p0 = (int)begin;
    const int64_t page = page_of(a, seq, p0);
    if (page < 0)
        return;
    const int in_page = p0 % a.page;
    H *pool = (H *)(is_k ? a.k_pages : a.v_pages) + page * a.page_stride + (int64_t)in_page * a.row_stride +
              head * a.head_stride;
    float *scale_at = (is_k ? a.k_scale : a.v_scale) + page * a.scale_page +
                      in_page / a.block * a.scale_block + head * a.scale_head;
    const int lo = p0 < rows.ctx ? rows.ctx - p0 : 0;             // new rows of the block
    const int hi = end - p0 < a.block ? (int)(end - p0) : a.block;
    const float before = lo > 0 ? *scale_at : 0.0f;
    const Rows &from = is_k ? a.k : a.v;
    const T *base = (const T *)from.base + (int64_t)rows.first * from.row_stride + head * from.head_stride;
    const Group group(a, lane % LPR);
    const int mine = lo + lane / LPR;

    auto load = [&](int r, f32x4 &x, f32x4 &y) {
        const int t = p0 + r - rows.ctx;
        const T *p = base + (int64_t)t * from.row_stride;
        x = load4(p + group.d0);
        y = load4(p + group.d1);
        if (is_k)
            group.turn(a, group.angles(a, rows.place(a, t)), x, y);
    };
    float top = 0.0f;
    bool odd = false;
    auto look = [&](const f32x4 &x) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool f = finite(x[e]);
            top = fmaxf(top, f ? fabsf(x[e]) : 0.0f);
            odd = odd || !f;
        }
    };
    f32x4 x[kHold], y[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        x[i] = y[i] = f32x4(0.0f);
        if (mine + i * ROWS < hi && group.in)
            load(mine + i * ROWS, x[i], y[i]);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        look(x[i]);
        look(y[i]);
    }
    for (int r = mine + kHold * ROWS; r < hi; r += ROWS)
        if (group.in) {
            f32x4 u, w;
            load(r, u, w);
            look(u);
            look(w);
        }
    float scale = scale_of_top<H>(wave_max(top));
    if (std::is_same_v<H, Int8> && __any(odd))
        scale = __builtin_nanf("");
    if (lo > 0 && !(scale != scale))
        scale = larger_scale(before, scale);
    const Divide divide(scale);
    if (lo > 0 && scale != before && group.in) {
        // earlier rows, whose codes mean something else from now on
        for (int r = lane / LPR; r < lo; r += ROWS) {
            uint32_t *w = (uint32_t *)(pool + (int64_t)r * a.row_stride + 8 * group.g);
            const f32x4 u = wide<H>(w[0]), v = wide<H>(w[1]);
            w[0] = divide.codes<H>(f32x4{u[0] * before, u[1] * before, u[2] * before, u[3] * before});
            w[1] = divide.codes<H>(f32x4{v[0] * before, v[1] * before, v[2] * before, v[3] * before});
        }
    }
    auto put = [&](int r, f32x4 u, f32x4 w) {
        if constexpr (std::is_same_v<H, E4M3>) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[e] = finite(u[e]) ? u[e] : __builtin_nanf("");
                w[e] = finite(w[e]) ? w[e] : __builtin_nanf("");
            }
        }
        H *to = pool + (int64_t)r * a.row_stride;
        *(uint32_t *)(to + group.d0) = divide.codes<H>(u);
        *(uint32_t *)(to + group.d1) = divide.codes<H>(w);
    };
    if (group.in) {
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            if (mine + i * ROWS < hi)
                put(mine + i * ROWS, x[i], y[i]);
        for (int r = mine + kHold * ROWS; r < hi; r += ROWS) {
            f32x4 u, w;
            load(r, u, w);
            put(r, u, w);
        }
    }
    if (lane == 0)
        *scale_at = scale;
}

// The first `blocks` wavefronts take blocks of codes, the others rows.
template <class T, class H, int LPR>
__global__ __launch_bounds__(kAttnThreads) void append_kernel(AppendArgs a, int64_t blocks)
{
    const int lane = threadIdx.x & 63;
    const uint32_t wave = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (kCodes<H>) {
        if (wave < (uint32_t)blocks) {
            code_block<T, H, LPR>(a, wave, lane);
            return;
        }
    }
    move_rows<T, kCodes<H>, LPR>(a, wave - (uint32_t)blocks, lane);
}

struct AppendShape {
    int64_t blocks, waves;
};

AppendShape append_shape(int held, const AppendArgs &a)
{
    AppendShape sh;
    const bool codes = held != CACHE_AS_IS;
    const int64_t all = a.Hq + (codes ? 0 : 2 * a.Hkv), per = a.D > 64 ? kRowsPer<16> : kRowsPer<8>;
    sh.blocks = codes ? block_numbers(a) * 2 * a.Hkv : 0;
    sh.waves = sh.blocks + (a.T + per - 1) / per * ((all + kHeads - 1) / kHeads);
    return sh;
}

template <class T, class H>
hipError_t launch_as(int held, const AppendArgs &a, hipStream_t stream)
{
    const AppendShape sh = append_shape(held, a);
    const uint32_t grid = (uint32_t)((sh.waves + kWaves - 1) / kWaves);
    if (grid == 0)
        return hipSuccess;
    if (a.D > 64)
        append_kernel<T, H, 16><<<grid, kAttnThreads, 0, stream>>>(a, sh.blocks);
    else
        append_kernel<T, H, 8><<<grid, kAttnThreads, 0, stream>>>(a, sh.blocks);
    return hipGetLastError();
}

template <class T>
hipError_t launch_held(int held, const AppendArgs &a, hipStream_t stream)
{
    if (held == CACHE_E4M3)
        return launch_as<T, E4M3>(held, a, stream);
    return held == CACHE_INT8 ? launch_as<T, Int8>(held, a, stream) : launch_as<T, T>(held, a, stream);
}

}  // namespace

int64_t append_threads(int held, const AppendArgs &a)
{
    return (append_shape(held, a).waves + kWaves - 1) / kWaves * kAttnThreads;
}

hipError_t launch_append(int dtype, int held, const AppendArgs &a, hipStream_t stream)
{
    return dtype == SPMM_DTYPE_BF16 ? launch_held<__bf16>(held, a, stream) : launch_held<float>(held, a, stream);
}

}  // namespace sdl
