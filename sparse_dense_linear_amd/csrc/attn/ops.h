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
    int32_t workers, block_rows;   // launch shape (tree_shape)
};

// Workgroups of the split, queries of a workgroup, and the workspace.
struct TreeShape {
    int32_t workers, block_rows;
    int64_t bytes;
};
TreeShape tree_shape(int dtype, int64_t S, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D);
int64_t tree_threads(const TreeArgs &a);
hipError_t launch_tree(int dtype, const TreeArgs &a, hipStream_t stream);

struct PagesArgs {
    char *k, *v;               // [layers, pages, page, row_bytes]
    int64_t layers, pages, page, row_bytes;
    const int32_t *src, *dst;  // copy: [count]
    const int32_t *table;      // compact: [count, table_stride]
    int64_t table_stride;
    const int32_t *ctx;        // [count]
    const int32_t *keep;       // [count, kept]
    int64_t count, kept;
};
// Workgroups that copy a page in one layer of one pool.
int64_t pages_copy_parts(int64_t page_bytes);
hipError_t launch_pages_copy(const PagesArgs &a, hipStream_t stream);
hipError_t launch_pages_compact(const PagesArgs &a, hipStream_t stream);

}  // namespace sdl
