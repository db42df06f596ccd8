// pages.hip -- moves of a paged cache: copying pages and compacting kept
// drafts, all layers of both pools in one launch.  Bound by memory: each
// moved byte is read and written once, 16 bytes a lane.
#include "ops.h"

#include "cache.h"
#include "held.h"
#include "tile.h"

namespace sdl {

namespace {

constexpr int kCopyPieces = 4;                                  // 16-byte pieces per thread
constexpr int kCopyBytes = kAttnThreads * kCopyPieces * 16;     // per workgroup
constexpr int kKeepBatch = 8;                                   // rows a thread holds at once
constexpr int kItems = 8;                                       // layers and pools of a workgroup

// Workgroup: `parts` of them to a page of one pair, layer and pool.  Stores
// past the caches: 250 pages of 32 KB in 32 layers, 182 us (5.8 TB/s read and
// written; a large copy reaches 5.1) against 194.
__global__ __launch_bounds__(kAttnThreads) void copy_kernel(PagesArgs a, int parts)
{
    const int64_t page_bytes = a.page * a.row_bytes;
    const int64_t item = blockIdx.x / parts;
    const int64_t begin = (int64_t)(blockIdx.x % parts) * kCopyBytes;
    const int64_t pair = item % a.count, layer = item / a.count % a.layers;
    char *pool = item / a.count / a.layers == 0 ? a.k : a.v;
    const int64_t src = a.src[pair], dst = a.dst[pair];
    if (src < 0 || src >= a.pages || dst < 0 || dst >= a.pages)
        return;
    const char *from = pool + (layer * a.pages + src) * page_bytes + begin;
    char *to = pool + (layer * a.pages + dst) * page_bytes + begin;
    const int64_t left = page_bytes - begin;
    u32x4 piece[kCopyPieces];
#pragma unroll
    for (int i = 0; i < kCopyPieces; ++i) {
        const int64_t at = 16 * (int64_t)(threadIdx.x + i * kAttnThreads);
        if (at < left)
            piece[i] = *(const u32x4 *)(from + at);
    }
#pragma unroll
    for (int i = 0; i < kCopyPieces; ++i) {
        const int64_t at = 16 * (int64_t)(threadIdx.x + i * kAttnThreads);
        if (at < left)
            __builtin_nontemporal_store(piece[i], (u32x4 *)(to + at));
    }
    if (a.k_scale != nullptr && begin == 0) {              // of pools of codes
        float *scale = item / a.count / a.layers == 0 ? a.k_scale : a.v_scale;
        const int64_t n = a.page / a.block * a.heads;
        for (int64_t i = threadIdx.x; i < n; i += kAttnThreads)
            scale[(layer * a.pages + dst) * n + i] = scale[(layer * a.pages + src) * n + i];
    }
}

// Workgroup: one sequence, kItems of its (layer, pool) pairs.  Where the kept
// rows lie is found once, kKeepBatch of them at a time; a thread then takes
// a 16-byte column through them, all reads before its writes, so rows never
// wait for other threads.  (Finding them anew in every thread, with a column
// each, took 35 us for 128 sequences, 32 layers and up to 8 rows of 2 KB; this
// takes 21.)
__global__ __launch_bounds__(kAttnThreads) void compact_kernel(PagesArgs a)
{
    __shared__ int64_t from[kKeepBatch], to[kKeepBatch];      // byte offsets in a layer; -1: nothing
    __shared__ int stop;
    const int t = threadIdx.x;
    const int64_t seq = blockIdx.x, first = (int64_t)blockIdx.y * kItems;
    const int items = (int)(2 * a.layers - first < kItems ? 2 * a.layers - first : kItems);
    const uint32_t cols = (uint32_t)(a.row_bytes / 16);
    const int64_t layer_bytes = a.pages * a.page * a.row_bytes;
    const int32_t *table = a.table + seq * a.table_stride, *keep = a.keep + seq * a.kept;
    const int64_t ctx = a.ctx[seq];
    // byte offset of a position's row, -1 if it has none
    auto row_at = [&](int64_t pos) -> int64_t {
        if (pos < 0 || pos / a.page >= a.table_stride)
            return -1;
        const int64_t number = table[pos / a.page];
        if (number < 0 || number >= a.pages)
            return -1;
        return (number * a.page + pos % a.page) * a.row_bytes;
    };
    for (int64_t t0 = 0; t0 < a.kept; t0 += kKeepBatch) {
        if (t < 64) {
            const int64_t i = t0 + t;
            const bool mine = t < kKeepBatch && i < a.kept;
            const int64_t of = mine ? keep[i] : 0;
            const uint64_t ends = __ballot(mine && of < 0);    // nothing counts from the first on
            if (t < kKeepBatch) {
                const bool moves = mine && (ends & (((uint64_t)2 << t) - 1)) == 0 && of != i;
                const int64_t f = moves ? row_at(ctx + of) : -1;
                from[t] = f;
                to[t] = f < 0 ? -1 : row_at(ctx + i);
            }
            if (t == 0)
                stop = ends != 0;
        }
        __syncthreads();
        for (uint32_t m = t; m < cols * items; m += kAttnThreads) {
            const uint32_t item = m / cols, col = m - item * cols;
            const int64_t n = first + item;
            char *base = (n < a.layers ? a.k + n * layer_bytes : a.v + (n - a.layers) * layer_bytes) + 16 * (int64_t)col;
            u32x4 piece[kKeepBatch];
#pragma unroll
            for (int i = 0; i < kKeepBatch; ++i)
                if (to[i] >= 0)
                    piece[i] = *(const u32x4 *)(base + from[i]);
#pragma unroll
            for (int i = 0; i < kKeepBatch; ++i)
                if (to[i] >= 0)
                    *(u32x4 *)(base + to[i]) = piece[i];
        }
        if (stop)
            return;                            // the same for the whole workgroup
        __syncthreads();
    }
}

constexpr int kCodeItems = 4;                                   // layers and pools of a workgroup
constexpr int kCodeBatch = 64;                                  // rows found at once

// Pools of codes.  Workgroup: one sequence, kCodeItems of its (layer, pool)
// pairs; block after block of the positions that kept rows move to, in ascending
// order, which is also the order of where they come from.  A thread takes a
// 16-byte column, which belongs to one head, through the block's rows: first the
// scales of where they come from, then the rows.  Rows are read no later than
// anything is written over them, since a row never comes from before its place;
// a block's scale is written when its rows have been read.
template <class H>
__global__ __launch_bounds__(kAttnThreads) void compact_codes(PagesArgs a)
{
    __shared__ int64_t from[kCodeBatch], to[kCodeBatch];      // rows of a layer; -1: nothing
    __shared__ int first_end;
    const int t = threadIdx.x;
    const int64_t seq = blockIdx.x, first = (int64_t)blockIdx.y * kCodeItems;
    const int items = (int)(2 * a.layers - first < kCodeItems ? 2 * a.layers - first : kCodeItems);
    const uint32_t cols = (uint32_t)(a.row_bytes / 16), D = (uint32_t)(a.row_bytes / a.heads);
    const int64_t layer_rows = a.pages * a.page, layer_scales = layer_rows / a.block * a.heads;
    const int32_t *table = a.table + seq * a.table_stride, *keep = a.keep + seq * a.kept;
    const int64_t ctx = a.ctx[seq];
    // a position's row, -1 if it has none
    auto row_at = [&](int64_t pos) -> int64_t {
        if (pos < 0 || pos / a.page >= a.table_stride)
            return -1;
        const int64_t number = table[pos / a.page];
        return number < 0 || number >= a.pages ? -1 : number * a.page + pos % a.page;
    };
    // kept rows: up to the first negative entry
    if (t == 0)
        first_end = (int)a.kept;
    __syncthreads();
    for (int64_t i = t; i < a.kept; i += kAttnThreads)
        if (keep[i] < 0) {
            atomicMin(&first_end, (int)i);
            break;
        }
    __syncthreads();
    const int64_t end = ctx + first_end;
    for (int64_t begin = ctx / a.block * a.block; begin < end; begin += a.block) {
        const int64_t lo = begin > ctx ? begin : ctx, hi = begin + a.block < end ? begin + a.block : end;
        const int64_t block_row = row_at(begin);
        if (block_row < 0)
            continue;                          // the same for the whole workgroup
        auto find = [&](int64_t p0) {          // rows p0 .. p0 + kCodeBatch - 1 of the block
            __syncthreads();
            if (t < kCodeBatch) {
                const int64_t p = p0 + t;
                const int64_t f = p < hi ? row_at(ctx + keep[p - ctx]) : -1;
                from[t] = f;
                to[t] = f < 0 ? -1 : block_row + (p - begin);
            }
            __syncthreads();
        };
        if (hi - lo <= kCodeBatch)
            find(lo);
        bool any = false;
        // kMine columns to a thread, whole heads to a turn: no turn reads a scale
        // that an earlier one has written
        constexpr int kMine = 4;
        const uint32_t wide_turn = kMine * kAttnThreads / (D / 16) * (D / 16);
        for (uint32_t m0 = 0; m0 < cols * items; m0 += wide_turn) {
            const uint32_t m1 = m0 + wide_turn < cols * items ? m0 + wide_turn : cols * items;
            float scale[kMine], before[kMine];
            char *pool[kMine];
            float *scales[kMine];
#pragma unroll
            for (int c = 0; c < kMine; ++c) {
                const uint32_t m = m0 + c * kAttnThreads + t, item = m / cols, col = m - item * cols;
                const int64_t n = first + item;
                const bool is_k = n < a.layers;
                const int64_t layer = is_k ? n : n - a.layers;
                pool[c] = nullptr;
                if (m >= m1)
                    continue;
                pool[c] = (is_k ? a.k : a.v) + layer * layer_rows * a.row_bytes + 16 * (int64_t)col;
                scales[c] = (is_k ? a.k_scale : a.v_scale) + layer * layer_scales + 16 * col / D;
                before[c] = scales[c][block_row / a.block * a.heads];
                scale[c] = lo > begin ? before[c] : 0.0f;
            }
            for (int64_t p0 = lo; p0 < hi; p0 += kCodeBatch) {
                if (hi - lo > kCodeBatch)
                    find(p0);
                for (int i = 0; i < kCodeBatch && p0 + i < hi; ++i) {
                    if (from[i] < 0)
                        continue;
                    any = true;
#pragma unroll
                    for (int c = 0; c < kMine; ++c)
                        if (pool[c] != nullptr)
                            scale[c] = larger_scale(scale[c], scales[c][from[i] / a.block * a.heads]);
                }
            }
            if (!any)
                break;                         // the same for the whole workgroup
            auto convert = [&](int c, int64_t source, int64_t dest, float old) {
                const u32x4 x = *(const u32x4 *)(pool[c] + source * a.row_bytes);
                const Divide divide(scale[c]);
                u32x4 y = x;
                if (old != scale[c])
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4 u = wide<H>(x[e]);
                        y[e] = divide.codes<H>(f32x4{u[0] * old, u[1] * old, u[2] * old, u[3] * old});
                    }
                *(u32x4 *)(pool[c] + dest * a.row_bytes) = y;
            };
#pragma unroll
            for (int c = 0; c < kMine; ++c)
                if (pool[c] != nullptr && scale[c] != before[c])
                    for (int64_t p = begin; p < lo; ++p)
                        convert(c, block_row + (p - begin), block_row + (p - begin), before[c]);
            for (int64_t p0 = lo; p0 < hi; p0 += kCodeBatch) {
                if (hi - lo > kCodeBatch)
                    find(p0);
                for (int i = 0; i < kCodeBatch && p0 + i < hi; ++i) {
                    if (from[i] < 0)
                        continue;
#pragma unroll
                    for (int c = 0; c < kMine; ++c) {
                        if (pool[c] == nullptr)
                            continue;
                        const float old = scales[c][from[i] / a.block * a.heads];
                        if (from[i] != to[i] || old != scale[c])
                            convert(c, from[i], to[i], old);
                    }
                }
            }
            __syncthreads();                   // all have read the scales
#pragma unroll
            for (int c = 0; c < kMine; ++c) {
                const uint32_t m = m0 + c * kAttnThreads + t, col = m % cols;
                if (pool[c] != nullptr && 16 * col % D == 0)
                    scales[c][block_row / a.block * a.heads] = scale[c];
            }
        }
        __syncthreads();                       // and written them
    }
}

// The same for lists of up to kFew kept drafts.  All rows and the scales of where they
// come from are read at once, then all are written: no row waits for another, and
// blocks neither (128 sequences, 32 layers, up to 8 rows of 1 KB: 21 us, taking row
// after row 34; 75 MB, of which few lie together).  Longer lists go row after row
// (compact_codes): 8 kept of 64 drafts 27 us (integers 31), 9 42 (46), 16 82 (86).
// Workgroup: one sequence, `items` of its (layer, pool) pairs, as many as have a thread
// for each 16-byte column.
constexpr int kFew = 8;

template <class H>
__global__ __launch_bounds__(kAttnThreads) void compact_few(PagesArgs a, int items)
{
    __shared__ int64_t from[kFew], to[kFew];       // rows of a layer; -1: nothing
    __shared__ int64_t from_block[kFew], to_block[kFew];
    const int t = threadIdx.x;
    const int64_t seq = blockIdx.x, first = (int64_t)blockIdx.y * items, ctx = a.ctx[seq];
    const uint32_t cols = (uint32_t)(a.row_bytes / 16), D = (uint32_t)(a.row_bytes / a.heads);
    const int64_t left = 2 * a.layers - first;
    const uint32_t all = cols * (uint32_t)(left < items ? left : items);
    const int64_t layer_rows = a.pages * a.page, layer_scales = layer_rows / a.block * a.heads;
    if (t < 64) {
        const int32_t *table = a.table + seq * a.table_stride, *keep = a.keep + seq * a.kept;
        const bool mine = t < kFew && t < a.kept;
        const int64_t of = mine ? keep[t] : 0;
        const uint64_t ends = __ballot(mine && of < 0);        // nothing counts from the first on
        // a position's row and block, -1 if it has none (positions and sizes fit 32 bits;
        // a division of 64 costs some hundred instructions)
        const uint32_t page = (uint32_t)a.page, block = (uint32_t)a.block, blocks = page / block;
        auto find = [&](int64_t pos, int64_t &row, int64_t &block_row) {
            row = -1;
            const uint32_t p = (uint32_t)pos / page, in = (uint32_t)pos - p * page;
            if (pos < 0 || p >= a.table_stride)
                return;
            const int64_t number = table[p];
            if (number < 0 || number >= a.pages)
                return;
            row = number * page + in;
            block_row = number * blocks + in / block;
        };
        if (t < kFew) {
            const bool counts = mine && (ends & (((uint64_t)2 << t) - 1)) == 0;
            int64_t f = -1, g = -1, f_block = 0, g_block = 0;
            if (counts) {
                find(ctx + of, f, f_block);
                find(ctx + t, g, g_block);
            }
            const bool moves = f >= 0 && g >= 0;
            from[t] = moves ? f : -1;
            to[t] = moves ? g : -1;
            from_block[t] = moves ? f_block : 0;
            to_block[t] = moves ? g_block : 0;
        }
    }
    __syncthreads();
    const int off = (int)(ctx % a.block);                      // rows of the context in the first block
    int which[kFew];                                           // block of the i-th place
    which[0] = 0;
#pragma unroll
    for (int i = 1, in = off; i < kFew; ++i) {
        in = in + 1 == (int)a.block ? 0 : in + 1;
        which[i] = which[i - 1] + (in == 0 ? 1 : 0);
    }
    const uint32_t turn = kAttnThreads / (D / 16) * (D / 16);  // whole heads
    for (uint32_t m0 = 0; m0 < all; m0 += turn) {
        const uint32_t m = m0 + t, item = m / cols, col = m - item * cols;
        const bool in = (uint32_t)t < turn && m < all;
        char *pool = nullptr;
        float *scales = nullptr;
        u32x4 piece[kFew];
        float come[kFew], before = 0.0f, now[kFew];
        if (in) {
            const int64_t n = first + item, layer = n < a.layers ? n : n - a.layers;
            pool = (n < a.layers ? a.k : a.v) + layer * layer_rows * a.row_bytes + 16 * (int64_t)col;
            scales = (n < a.layers ? a.k_scale : a.v_scale) + layer * layer_scales + 16 * col / D;
#pragma unroll
            for (int i = 0; i < kFew; ++i) {
                come[i] = 0.0f;
                if (from[i] >= 0) {
                    come[i] = scales[from_block[i] * a.heads];
                    piece[i] = *(const u32x4 *)(pool + from[i] * a.row_bytes);
                }
            }
            // the block of the context's last row, if a kept row moves into it
            int into = -1;
#pragma unroll
            for (int i = kFew - 1; i >= 0; --i)
                into = which[i] == 0 && from[i] >= 0 ? i : into;
            if (off > 0 && into >= 0)
                before = scales[to_block[into] * a.heads];
            // the largest so far of each block (where nothing comes from: 0), then of all
            now[0] = larger_scale(before, come[0]);
#pragma unroll
            for (int i = 1; i < kFew; ++i)
                now[i] = which[i] == which[i - 1] ? larger_scale(now[i - 1], come[i]) : come[i];
#pragma unroll
            for (int i = kFew - 2; i >= 0; --i)
                now[i] = which[i] == which[i + 1] ? now[i + 1] : now[i];
            auto convert = [&](u32x4 x, float old, const Divide &divide) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x4 u = wide<H>(x[e]);
                    x[e] = divide.codes<H>(f32x4{u[0] * old, u[1] * old, u[2] * old, u[3] * old});
                }
                return x;
            };
            if (off > 0 && into >= 0 && now[into] != before) {
                const Divide divide(now[into]);
                const int64_t row = to[into] - into - off;     // the block's first
                for (int r = 0; r < off; ++r) {
                    u32x4 *p = (u32x4 *)(pool + (row + r) * a.row_bytes);
                    *p = convert(*p, before, divide);
                }
            }
#pragma unroll
            for (int i = 0; i < kFew; ++i)
                if (from[i] >= 0 && (from[i] != to[i] || come[i] != now[i]))
                    *(u32x4 *)(pool + to[i] * a.row_bytes) =
                        come[i] != now[i] ? convert(piece[i], come[i], Divide(now[i])) : piece[i];
        }
        __syncthreads();                       // all have read the scales
        if (in && 16 * col % D == 0) {
#pragma unroll
            for (int i = 0; i < kFew; ++i)
                if (from[i] >= 0)
                    scales[to_block[i] * a.heads] = now[i];
        }
        __syncthreads();
    }
}

}  // namespace

int64_t pages_copy_parts(int64_t page_bytes) { return (page_bytes + kCopyBytes - 1) / kCopyBytes; }

hipError_t launch_pages_copy(const PagesArgs &a, hipStream_t stream)
{
    const int64_t parts = pages_copy_parts(a.page * a.row_bytes);
    copy_kernel<<<dim3((uint32_t)(2 * a.layers * a.count * parts)), kAttnThreads, 0, stream>>>(a, (int)parts);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const PagesArgs &a, hipStream_t stream)
{
    const dim3 grid((uint32_t)a.count, (uint32_t)((2 * a.layers + kItems - 1) / kItems));
    compact_kernel<<<grid, kAttnThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_cache_compact(int held, const PagesArgs &a, hipStream_t stream)
{
    if (a.kept <= kFew) {
        const int64_t cols = a.row_bytes / 16, fit = kAttnThreads / cols;
        const int items = (int)(fit < 1 ? 1 : (fit > 8 ? 8 : fit));
        const dim3 grid((uint32_t)a.count, (uint32_t)((2 * a.layers + items - 1) / items));
        if (held == CACHE_E4M3)
            compact_few<E4M3><<<grid, kAttnThreads, 0, stream>>>(a, items);
        else
            compact_few<Int8><<<grid, kAttnThreads, 0, stream>>>(a, items);
        return hipGetLastError();
    }
    const dim3 grid((uint32_t)a.count, (uint32_t)((2 * a.layers + kCodeItems - 1) / kCodeItems));
    if (held == CACHE_E4M3)
        compact_codes<E4M3><<<grid, kAttnThreads, 0, stream>>>(a);
    else
        compact_codes<Int8><<<grid, kAttnThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace sdl
