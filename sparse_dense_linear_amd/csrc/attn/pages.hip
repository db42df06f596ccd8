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

// Workgroup: `parts` of them to a page of one pair, layer and pool.
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
            *(u32x4 *)(to + at) = piece[i];
    }
}

// Thread: one 16-byte column of one sequence, layer and pool.  It takes the
// column through all kept rows, so rows never wait for other threads.
__global__ __launch_bounds__(kAttnThreads) void compact_kernel(PagesArgs a)
{
    // (32-bit division where the numbers allow it: the 64-bit one costs more
    // than the rest of the kernel)
    auto divide = [](int64_t x, int64_t y) {
        return ((uint64_t)x | (uint64_t)y) >> 32 == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
    };
    const int64_t cols = a.row_bytes / 16;
    const int64_t n = (int64_t)blockIdx.x * kAttnThreads + threadIdx.x;
    const int64_t item = divide(n, cols), col = n - item * cols;
    const int64_t outer = divide(item, a.count), seq = item - outer * a.count;
    if (outer >= 2 * a.layers)
        return;
    const int64_t layer = outer < a.layers ? outer : outer - a.layers;
    char *base = (outer < a.layers ? a.k : a.v) + layer * a.pages * a.page * a.row_bytes + 16 * col;
    const int32_t *table = a.table + seq * a.table_stride, *keep = a.keep + seq * a.kept;
    const int64_t ctx = a.ctx[seq];
    // byte offset of a position's row, -1 if it has none
    auto row_at = [&](int64_t pos) -> int64_t {
        if (pos < 0)
            return -1;
        const int64_t p = divide(pos, a.page);
        if (p >= a.table_stride)
            return -1;
        const int64_t number = table[p];
        if (number < 0 || number >= a.pages)
            return -1;
        return (number * a.page + pos - p * a.page) * a.row_bytes;
    };
    bool more = true;
    for (int64_t t0 = 0; t0 < a.kept && more; t0 += kKeepBatch) {
        u32x4 piece[kKeepBatch];
        int64_t to[kKeepBatch];
#pragma unroll
        for (int i = 0; i < kKeepBatch; ++i) {
            to[i] = -1;
            const int64_t of = more && t0 + i < a.kept ? keep[t0 + i] : -1;
            more = more && of >= 0;
            if (more && of != t0 + i) {
                const int64_t from = row_at(ctx + of);
                to[i] = from < 0 ? -1 : row_at(ctx + t0 + i);
                if (to[i] >= 0)
                    piece[i] = *(const u32x4 *)(base + from);
            }
        }
#pragma unroll
        for (int i = 0; i < kKeepBatch; ++i)
            if (to[i] >= 0)
                *(u32x4 *)(base + to[i]) = piece[i];
    }
}

}  // namespace

hipError_t launch_pages_copy(const PagesArgs &a, hipStream_t stream)
{
    const int64_t parts = (a.page * a.row_bytes + kCopyBytes - 1) / kCopyBytes;
    copy_kernel<<<dim3((uint32_t)(2 * a.layers * a.count * parts)), kAttnThreads, 0, stream>>>(a, (int)parts);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const PagesArgs &a, hipStream_t stream)
{
    const int64_t threads = 2 * a.layers * a.count * (a.row_bytes / 16);
    compact_kernel<<<dim3((uint32_t)((threads + kAttnThreads - 1) / kAttnThreads)), kAttnThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace sdl
