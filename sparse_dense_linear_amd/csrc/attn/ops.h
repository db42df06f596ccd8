// ops.h -- shared between the host side and the kernels of the attention
// operators and the cache's page moves.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdl {

constexpr int kAttnThreads = 256;   // 4 wavefronts
constexpr int kMaxHeadDim = 128;

// A launch holds fewer than 2^32 threads in a dimension.  The *_threads
// functions below tell the most that a call needs along x.
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;

// Packed rows of heads: element (row, head, d) at base + row * row_stride +
// head * head_stride + d.
struct Rows {
    const void *base;
    int64_t row_stride, head_stride;
};
struct OutRows {
    void *base;
    int64_t row_stride, head_stride;
};

struct WindowArgs {
    Rows q, k, v;
    const int32_t *q_rowptr, *k_rowptr;
    OutRows o;
    float *lse;               // [Hq, Tq]
    int32_t S, Hq, Hkv, D;
    int64_t Tq, Tk;
    int32_t window, sinks;
    float scale;
    // backward only
    Rows dout, out;           // do and o
    OutRows dq, dk, dv;
    float *delta;             // [Hq, Tq]
    float *partial;           // scratch: parts of split walks (forward), see
                              // window_bwd.hip (backward)
};

// Queries of a forward workgroup; the parts of `tiles` key tiles that its walk
// is split into, at most `parts`; and where they leave maximum and sum, and
// unnormalised output.
struct SplitShape {
    int32_t rows, tiles, parts;
    float *stat, *out;
};

// Whether workgroups of 128 queries make less than two rounds of the 512
// places that the GPU has for them (two to a CU): then 64 queries each, or
// split walks.
inline bool few_tiles(const WindowArgs &a) { return (a.Tq / 128 + a.S) * a.Hq < 1024; }

hipError_t launch_window_fwd(int dtype, const WindowArgs &a, hipStream_t stream);
hipError_t launch_window_bwd(int dtype, const WindowArgs &a, hipStream_t stream);
int64_t window_fwd_scratch_bytes(int dtype, const WindowArgs &a);
int64_t window_fwd_threads(int dtype, const WindowArgs &a);
int64_t window_bwd_threads(int dtype, const WindowArgs &a);
// Bytes of delta and of the partial sums (0: none) of a backward call.
int64_t window_bwd_delta_bytes(int64_t Tq, int64_t Hq);
int64_t window_bwd_partial_bytes(int64_t S, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                                 int64_t window, int64_t sinks);

// x / d for 0 <= x < 2^31 is (x * factor) >> (31 + shift).
struct Divisor {
    uint32_t factor;
    int32_t shift;
};
inline Divisor divisor(uint32_t d)
{
    int s = 0;
    while (((uint64_t)1 << s) < d)
        ++s;
    return {(uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), s};
}

// Workgroups of tree_codes.h to a CU, by the bytes of an element of q and the head's
// size, that registers have room for.
constexpr int stream_per_cu(int bytes, int DP) { return bytes == 2 && DP == 64 ? 3 : 2; }

struct TreeArgs {
    const void *q;
    int64_t q_row, q_head;    // strides
    const void *k_pages, *v_pages;
    int64_t page_stride, row_stride, head_stride;   // of both pools
    const int32_t *table;     // [S, table_stride]
    int64_t table_stride;
    const int32_t *ctx;       // [S]
    const int32_t *q_rowptr;  // [S + 1]
    const uint64_t *tree;     // [Tq] or null (a chain)
    void *o;                  // [Tq, Hq, D]
    float *lse;               // [Hq, Tq]
    int32_t S, Hq, Hkv, D, page;
    int64_t Tq;
    int32_t window, sinks;
    float scale;
    float *partial;
    int32_t workers, block_rows, slot_rows;   // launch shape (tree_shape)
    // pools of codes only: key heads of a workgroup and keys of a tile, whether 16
    // keys lie together (tree_codes.h); scales of blocks of positions, and their strides
    int32_t wave_heads, tile_keys, together, mean_rows;
    const float *k_scale, *v_scale;
    int64_t scale_page, scale_block, scale_head;
    int32_t block;
    Divisor by_page, by_block;
};

// Workgroups of the split, queries of a workgroup, and the workspace.
struct TreeShape {
    int32_t workers, block_rows, wave_heads;
    int64_t rows;                  // queries that share a key head, of the mean sequence
    int64_t bytes;
};
TreeShape tree_shape(int dtype, int held, int64_t S, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D);
int64_t tree_threads(const TreeArgs &a);
hipError_t launch_tree(int dtype, const TreeArgs &a, hipStream_t stream);
hipError_t launch_tree_e4m3(int dtype, const TreeArgs &a, hipStream_t stream);
hipError_t launch_tree_int8(int dtype, const TreeArgs &a, hipStream_t stream);

struct PagesArgs {
    char *k, *v;               // [layers, pages, page, row_bytes]
    int64_t layers, pages, page, row_bytes;
    const int32_t *src, *dst;  // copy: [count]
    const int32_t *table;      // compact: [count, table_stride]
    int64_t table_stride;
    const int32_t *ctx;        // [count]
    const int32_t *keep;       // [count, kept]
    int64_t count, kept;
    // pools of codes only (cache.h): scales [layers, pages, page / block, heads]
    float *k_scale, *v_scale;
    int64_t block, heads;
};
// Workgroups that copy a page in one layer of one pool.
int64_t pages_copy_parts(int64_t page_bytes);
hipError_t launch_pages_copy(const PagesArgs &a, hipStream_t stream);
hipError_t launch_pages_compact(const PagesArgs &a, hipStream_t stream);
hipError_t launch_cache_compact(int held, const PagesArgs &a, hipStream_t stream);

struct AppendArgs {
    Rows q, k, v;
    OutRows q_out;
    const float *cosines, *sines;   // [angles, rotated / 2]
    const int32_t *table;           // [S, table_stride]
    int64_t table_stride;
    const int32_t *ctx;             // [S]
    const int32_t *rowptr;          // [S + 1]
    const uint64_t *tree;           // [T] or null (a chain)
    void *k_pages, *v_pages;
    int64_t pages, page_stride, row_stride, head_stride;
    float *k_scale, *v_scale;       // pools of codes only
    int64_t scale_page, scale_block, scale_head;
    int32_t block;
    int32_t S, T, Hq, Hkv, D, page;
    int32_t rotated, angles, interleaved;
};
int64_t append_threads(int held, const AppendArgs &a);
hipError_t launch_append(int dtype, int held, const AppendArgs &a, hipStream_t stream);

}  // namespace sdl
