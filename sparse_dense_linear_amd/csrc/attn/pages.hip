// pages.hip -- moves of a paged cache: copying pages and compacting kept
// drafts, all layers of both pools in one launch.  Bound by memory: each
// moved byte is read and written once, 16 bytes a lane.
#include "ops.h"

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

}  // namespace sdl
