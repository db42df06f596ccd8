// api.hip -- host side of the C ABI declared in include/attn.h: checks
// arguments before any HIP call, then enqueues.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "attn.h"

#include "ops.h"
#include "internal.h"

using namespace sdl;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;      // positions and windows fit 31 bits
constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxGridY = 65535;
constexpr int64_t kMaxSinks = 128;                  // a few first tokens
constexpr int64_t kMaxStride = (int64_t)1 << 32;

spmm_status_t bad(const char *msg) { return record_error(SPMM_ERROR_INVALID_VALUE, msg); }
spmm_status_t unsupported(const char *msg) { return record_error(SPMM_ERROR_UNSUPPORTED, msg); }

spmm_status_t launched(hipError_t err, const char *what)
{
    return err == hipSuccess ? SPMM_SUCCESS : record_hip_error(err, what);
}

bool aligned(const void *p, uintptr_t a) { return (uintptr_t)p % a == 0; }

spmm_status_t check_heads(int32_t dtype, int64_t Hq, int64_t Hkv, int64_t D, int64_t window,
                          int64_t sinks, float scale, int32_t reserved)
{
    if (dtype != SPMM_DTYPE_F32 && dtype != SPMM_DTYPE_BF16)
        return bad("unknown dtype");
    if (reserved != 0)
        return bad("reserved must be 0");
    if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0)
        return bad("Hq must be a positive multiple of Hkv");
    if (Hq > 65536)
        return unsupported("at most 65536 heads");
    if (D < 1)
        return bad("D must be positive");
    if (D % 8 != 0 || D > kMaxHeadDim)
        return unsupported("D must be a multiple of 8 up to 128");
    if (window < 1)
        return bad("window must be at least 1");
    if (sinks < 0)
        return bad("sinks must not be negative");
    if (sinks > kMaxSinks)
        return unsupported("at most 128 sinks");
    if (!(scale > 0.0f) || !isfinite(scale))
        return bad("scale must be positive and finite");
    return SPMM_SUCCESS;
}

// An operand of `rows` packed rows of heads.
spmm_status_t check_rows(const attn_rows_t *r, int64_t rows, int32_t dtype, const char *null_msg)
{
    if (r == nullptr)
        return bad("an operand's description is null");
    const int64_t unit = dtype == SPMM_DTYPE_BF16 ? 8 : 4;
    if (r->row_stride < 0 || r->head_stride < 0 || r->row_stride > kMaxStride ||
        r->head_stride > kMaxStride)
        return bad("strides must be in 0 .. 2^32");
    if (r->row_stride % unit != 0 || r->head_stride % unit != 0)
        return bad("strides must be multiples of 16 bytes");
    if (rows > 0 && r->data == nullptr)
        return bad(null_msg);
    if (!aligned(r->data, 16))
        return bad("operands must be 16-byte aligned");
    return SPMM_SUCCESS;
}

// An output: as an operand, and its rows and heads must not overlap.
spmm_status_t check_out(const attn_rows_t *r, int64_t rows, int64_t heads, int64_t D, int32_t dtype,
                        const char *null_msg)
{
    const spmm_status_t st = check_rows(r, rows, dtype, null_msg);
    if (st != SPMM_SUCCESS)
        return st;
    const int64_t a = r->row_stride, b = r->head_stride;
    const bool rows_outside = (heads <= 1 || b >= D) && (rows <= 1 || a >= (heads - 1) * b + D);
    const bool heads_outside = (rows <= 1 || a >= D) && (heads <= 1 || b >= (rows - 1) * a + D);
    if (!rows_outside && !heads_outside)
        return bad("rows of an output overlap");
    return SPMM_SUCCESS;
}

Rows in_rows(const attn_rows_t *r) { return {r->data, r->row_stride, r->head_stride}; }
OutRows out_rows(const attn_rows_t *r)
{
    return {const_cast<void *>(r->data), r->row_stride, r->head_stride};
}

int32_t clamp_window(int64_t window)
{
    return (int32_t)(window < kMaxRows - 1 ? window : kMaxRows - 1);
}

spmm_status_t check_window(int32_t dtype, const attn_window_t *w)
{
    if (w == nullptr)
        return bad("shape is null");
    const spmm_status_t st =
        check_heads(dtype, w->Hq, w->Hkv, w->D, w->window, w->sinks, w->scale, w->reserved);
    if (st != SPMM_SUCCESS)
        return st;
    if (w->S < 0 || w->Tq < 0 || w->Tk < 0)
        return bad("negative size");
    if (w->S >= kMaxRows || w->Tq >= kMaxRows || w->Tk >= kMaxRows)
        return bad("S, Tq and Tk must be below 2^30");
    // so that workgroups and their numbers fit 31 bits; what a launch holds is
    // checked by the calls
    if (2 * (w->Tq / 32 + w->Tk / 32 + 2 * w->S) * w->Hq > kMaxGrid ||
        w->S * w->Hkv * (w->sinks > 0 ? w->sinks : 1) > kMaxGrid)
        return unsupported("too many workgroups: fewer sequences, rows or heads");
    return SPMM_SUCCESS;
}

void fill_window(WindowArgs &a, const attn_window_t *w)
{
    a.S = (int32_t)w->S;
    a.Hq = (int32_t)w->Hq;
    a.Hkv = (int32_t)w->Hkv;
    a.D = (int32_t)w->D;
    a.Tq = w->Tq;
    a.Tk = w->Tk;
    a.window = clamp_window(w->window);
    a.sinks = (int32_t)w->sinks;
    a.scale = w->scale;
}

spmm_status_t check_rowptrs(const int32_t *q_rowptr, const int32_t *k_rowptr)
{
    if (q_rowptr == nullptr || k_rowptr == nullptr)
        return bad("a row pointer array is null");
    if (!aligned(q_rowptr, 4) || !aligned(k_rowptr, 4))
        return bad("row pointers must be 4-byte aligned");
    return SPMM_SUCCESS;
}

struct BwdScratch {
    int64_t delta, partial;
};

BwdScratch bwd_scratch(const attn_window_t *w)
{
    return {window_bwd_delta_bytes(w->Tq, w->Hq),
            window_bwd_partial_bytes(w->S, w->Tq, w->Tk, w->Hq, w->Hkv, w->D, clamp_window(w->window),
                                     w->sinks)};
}

spmm_status_t check_tree(int32_t dtype, const attn_tree_t *w)
{
    if (w == nullptr)
        return bad("shape is null");
    const spmm_status_t st =
        check_heads(dtype, w->Hq, w->Hkv, w->D, w->window, w->sinks, w->scale, w->reserved);
    if (st != SPMM_SUCCESS)
        return st;
    if (w->S < 0 || w->Tq < 0 || w->table_stride < 0)
        return bad("negative size");
    if (w->S >= kMaxRows || w->Tq >= kMaxRows || w->table_stride >= kMaxRows)
        return bad("S, Tq and table_stride must be below 2^30");
    if (w->page < 1 || w->page >= kMaxRows)
        return bad("page must be in 1 .. 2^30 - 1");
    const int64_t unit = dtype == SPMM_DTYPE_BF16 ? 8 : 4;
    if (w->page_stride < 0 || w->row_stride < 0 || w->head_stride < 0 ||
        w->page_stride > kMaxStride || w->row_stride > kMaxStride || w->head_stride > kMaxStride)
        return bad("strides must be in 0 .. 2^32");
    if (w->page_stride % unit != 0 || w->row_stride % unit != 0 || w->head_stride % unit != 0)
        return bad("strides must be multiples of 16 bytes");
    if (w->Tq * w->Hq + w->S * w->Hkv > kMaxGrid)
        return unsupported("too many queries: Tq * Hq + S * Hkv must be below 2^31");
    return SPMM_SUCCESS;
}

spmm_status_t check_pool(const attn_pool_t *p)
{
    if (p == nullptr)
        return bad("pool is null");
    if (p->layers < 0 || p->pages < 0 || p->page < 0 || p->row_bytes < 0)
        return bad("negative size");
    if (p->layers >= kMaxRows || p->pages >= kMaxRows || p->page >= kMaxRows ||
        p->row_bytes >= kMaxRows)
        return bad("sizes of a pool must be below 2^30");
    if (p->row_bytes % 16 != 0)
        return unsupported("a row must be a multiple of 16 bytes");
    return SPMM_SUCCESS;
}

spmm_status_t check_pool_data(const attn_pool_t *p)
{
    if (p->k == nullptr || p->v == nullptr)
        return bad("a pool is null");
    if (!aligned(p->k, 16) || !aligned(p->v, 16))
        return bad("pools must be 16-byte aligned");
    return SPMM_SUCCESS;
}

PagesArgs pages_args(const attn_pool_t *p)
{
    PagesArgs a = {};
    a.k = (char *)p->k;
    a.v = (char *)p->v;
    a.layers = p->layers;
    a.pages = p->pages;
    a.page = p->page;
    a.row_bytes = p->row_bytes;
    return a;
}

// Whether 2 * layers * count * parts workgroups are more than a launch holds,
// without overflow (all below 2^60)
bool too_many(int64_t layers, int64_t count, int64_t parts)
{
    return (unsigned __int128)2 * kAttnThreads * (uint64_t)layers * (uint64_t)count >
           (unsigned __int128)kMaxThreads / (uint64_t)parts;
}

spmm_status_t check_threads(int64_t threads)
{
    return threads <= kMaxThreads ? SPMM_SUCCESS
                                  : unsupported("too many workgroups: fewer sequences, rows or heads");
}

}  // namespace

extern "C" {

spmm_status_t window_attn_fwd(int32_t dtype, const attn_window_t *shape, const attn_rows_t *q,
                              const attn_rows_t *k, const attn_rows_t *v, const int32_t *q_rowptr,
                              const int32_t *k_rowptr, const attn_rows_t *o, float *lse, void *scratch,
                              int64_t scratch_bytes, void *stream)
{
    spmm_status_t st = check_window(dtype, shape);
    if (st != SPMM_SUCCESS)
        return st;
    if ((st = check_rows(q, shape->Tq, dtype, "q is null")) != SPMM_SUCCESS ||
        (st = check_rows(k, shape->Tk, dtype, "k is null")) != SPMM_SUCCESS ||
        (st = check_rows(v, shape->Tk, dtype, "v is null")) != SPMM_SUCCESS ||
        (st = check_out(o, shape->Tq, shape->Hq, shape->D, dtype, "o is null")) != SPMM_SUCCESS)
        return st;
    if (shape->S == 0 || shape->Tq == 0)
        return SPMM_SUCCESS;
    if ((st = check_rowptrs(q_rowptr, k_rowptr)) != SPMM_SUCCESS)
        return st;
    if (lse == nullptr || !aligned(lse, 4))
        return bad("lse is null or not 4-byte aligned");
    WindowArgs a = {};
    fill_window(a, shape);
    a.q = in_rows(q);
    a.k = in_rows(k);
    a.v = in_rows(v);
    a.q_rowptr = q_rowptr;
    a.k_rowptr = k_rowptr;
    a.o = out_rows(o);
    a.lse = lse;
    a.partial = (float *)scratch;
    const int64_t need = window_fwd_scratch_bytes(dtype, a);
    if (scratch_bytes < need)
        return bad("scratch is smaller than window_attn_fwd_scratch says");
    if (need > 0 && (scratch == nullptr || !aligned(scratch, 16)))
        return bad("scratch is null or not 16-byte aligned");
    if ((st = check_threads(window_fwd_threads(dtype, a))) != SPMM_SUCCESS)
        return st;
    return launched(launch_window_fwd(dtype, a, (hipStream_t)stream), "window attention");
}

spmm_status_t window_attn_fwd_scratch(int32_t dtype, const attn_window_t *shape, int64_t *bytes)
{
    const spmm_status_t st = check_window(dtype, shape);
    if (st != SPMM_SUCCESS)
        return st;
    if (bytes == nullptr)
        return bad("bytes is null");
    WindowArgs a = {};
    fill_window(a, shape);
    *bytes = shape->S == 0 || shape->Tq == 0 ? 0 : window_fwd_scratch_bytes(dtype, a);
    return SPMM_SUCCESS;
}

spmm_status_t window_attn_bwd_scratch(const attn_window_t *shape, int64_t *bytes)
{
    const spmm_status_t st = check_window(SPMM_DTYPE_F32, shape);
    if (st != SPMM_SUCCESS)
        return st;
    if (bytes == nullptr)
        return bad("bytes is null");
    const BwdScratch s = bwd_scratch(shape);
    *bytes = s.delta + s.partial;
    return SPMM_SUCCESS;
}

spmm_status_t window_attn_bwd(int32_t dtype, const attn_window_t *shape, const attn_rows_t *dout,
                              const attn_rows_t *q, const attn_rows_t *k, const attn_rows_t *v,
                              const attn_rows_t *o, const float *lse, const int32_t *q_rowptr,
                              const int32_t *k_rowptr, const attn_rows_t *dq, const attn_rows_t *dk,
                              const attn_rows_t *dv, void *scratch, int64_t scratch_bytes, void *stream)
{
    spmm_status_t st = check_window(dtype, shape);
    if (st != SPMM_SUCCESS)
        return st;
    const int64_t Tq = shape->Tq, Tk = shape->Tk;
    if ((st = check_rows(dout, Tq, dtype, "dout is null")) != SPMM_SUCCESS ||
        (st = check_rows(q, Tq, dtype, "q is null")) != SPMM_SUCCESS ||
        (st = check_rows(k, Tk, dtype, "k is null")) != SPMM_SUCCESS ||
        (st = check_rows(v, Tk, dtype, "v is null")) != SPMM_SUCCESS ||
        (st = check_rows(o, Tq, dtype, "o is null")) != SPMM_SUCCESS ||
        (st = check_out(dq, Tq, shape->Hq, shape->D, dtype, "dq is null")) != SPMM_SUCCESS ||
        (st = check_out(dk, Tk, shape->Hkv, shape->D, dtype, "dk is null")) != SPMM_SUCCESS ||
        (st = check_out(dv, Tk, shape->Hkv, shape->D, dtype, "dv is null")) != SPMM_SUCCESS)
        return st;
    if (shape->S == 0 || (Tq == 0 && Tk == 0))
        return SPMM_SUCCESS;
    if ((st = check_rowptrs(q_rowptr, k_rowptr)) != SPMM_SUCCESS)
        return st;
    if (Tq > 0 && (lse == nullptr || !aligned(lse, 4)))
        return bad("lse is null or not 4-byte aligned");
    const BwdScratch s = bwd_scratch(shape);
    if (scratch_bytes < s.delta + s.partial)
        return bad("scratch is smaller than window_attn_bwd_scratch says");
    if (s.delta + s.partial > 0 && (scratch == nullptr || !aligned(scratch, 16)))
        return bad("scratch is null or not 16-byte aligned");
    WindowArgs a = {};
    fill_window(a, shape);
    a.q = in_rows(q);
    a.k = in_rows(k);
    a.v = in_rows(v);
    a.dout = in_rows(dout);
    a.out = in_rows(o);
    a.q_rowptr = q_rowptr;
    a.k_rowptr = k_rowptr;
    a.lse = const_cast<float *>(lse);
    a.dq = out_rows(dq);
    a.dk = out_rows(dk);
    a.dv = out_rows(dv);
    a.delta = (float *)scratch;
    a.partial = (float *)((char *)scratch + s.delta);
    if ((st = check_threads(window_bwd_threads(dtype, a))) != SPMM_SUCCESS)
        return st;
    return launched(launch_window_bwd(dtype, a, (hipStream_t)stream), "window attention backward");
}

spmm_status_t tree_attn_scratch(int32_t dtype, const attn_tree_t *shape, int64_t *bytes)
{
    const spmm_status_t st = check_tree(dtype, shape);
    if (st != SPMM_SUCCESS)
        return st;
    if (bytes == nullptr)
        return bad("bytes is null");
    *bytes = shape->S == 0 || shape->Tq == 0
                 ? 0
                 : tree_shape(dtype, shape->S, shape->Tq, shape->Hq, shape->Hkv, shape->D).bytes;
    return SPMM_SUCCESS;
}

spmm_status_t tree_attn_paged(int32_t dtype, const attn_tree_t *shape, const attn_rows_t *q,
                              const void *k_pages, const void *v_pages, const int32_t *table,
                              const int32_t *ctx, const int32_t *q_rowptr, const uint64_t *tree,
                              void *o, float *lse, void *scratch, int64_t scratch_bytes, void *stream)
{
    spmm_status_t st = check_tree(dtype, shape);
    if (st != SPMM_SUCCESS)
        return st;
    if ((st = check_rows(q, shape->Tq, dtype, "q is null")) != SPMM_SUCCESS)
        return st;
    if (shape->S == 0 || shape->Tq == 0)
        return SPMM_SUCCESS;
    if (k_pages == nullptr || v_pages == nullptr || table == nullptr || ctx == nullptr ||
        q_rowptr == nullptr || o == nullptr || lse == nullptr)
        return bad("a null pointer");
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16))
        return bad("the pools and o must be 16-byte aligned");
    if (!aligned(table, 4) || !aligned(ctx, 4) || !aligned(q_rowptr, 4) || !aligned(lse, 4) ||
        !aligned(tree, 8))
        return bad("an array is not aligned to its element size");
    const TreeShape sh = tree_shape(dtype, shape->S, shape->Tq, shape->Hq, shape->Hkv, shape->D);
    if (scratch_bytes < sh.bytes)
        return bad("scratch is smaller than tree_attn_scratch says");
    if (scratch == nullptr || !aligned(scratch, 16))
        return bad("scratch is null or not 16-byte aligned");
    TreeArgs a = {};
    a.q = q->data;
    a.q_row = q->row_stride;
    a.q_head = q->head_stride;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.page_stride = shape->page_stride;
    a.row_stride = shape->row_stride;
    a.head_stride = shape->head_stride;
    a.table = table;
    a.table_stride = shape->table_stride;
    a.ctx = ctx;
    a.q_rowptr = q_rowptr;
    a.tree = tree;
    a.o = o;
    a.lse = lse;
    a.S = (int32_t)shape->S;
    a.Hq = (int32_t)shape->Hq;
    a.Hkv = (int32_t)shape->Hkv;
    a.D = (int32_t)shape->D;
    a.page = (int32_t)shape->page;
    a.Tq = shape->Tq;
    a.window = clamp_window(shape->window);
    a.sinks = (int32_t)shape->sinks;
    a.scale = shape->scale;
    a.partial = (float *)scratch;
    a.workers = sh.workers;
    a.block_rows = sh.block_rows;
    if ((st = check_threads(tree_threads(a))) != SPMM_SUCCESS)
        return st;
    return launched(launch_tree(dtype, a, (hipStream_t)stream), "tree attention");
}

spmm_status_t pages_copy(const attn_pool_t *pool, const int32_t *src, const int32_t *dst,
                         int64_t count, void *stream)
{
    spmm_status_t st = check_pool(pool);
    if (st != SPMM_SUCCESS)
        return st;
    if (count < 0)
        return bad("negative size");
    if (count == 0 || pool->layers == 0 || pool->pages == 0 || pool->page == 0 || pool->row_bytes == 0)
        return SPMM_SUCCESS;
    if ((st = check_pool_data(pool)) != SPMM_SUCCESS)
        return st;
    if (src == nullptr || dst == nullptr || !aligned(src, 4) || !aligned(dst, 4))
        return bad("src or dst is null or not 4-byte aligned");
    if (count >= kMaxRows || too_many(pool->layers, count, pages_copy_parts(pool->page * pool->row_bytes)))
        return unsupported("too many pages for one call");
    PagesArgs a = pages_args(pool);
    a.src = src;
    a.dst = dst;
    a.count = count;
    return launched(launch_pages_copy(a, (hipStream_t)stream), "pages_copy");
}

spmm_status_t pages_compact(const attn_pool_t *pool, const int32_t *table, int64_t table_stride,
                            const int32_t *ctx, const int32_t *keep, int64_t S, int64_t kept,
                            void *stream)
{
    spmm_status_t st = check_pool(pool);
    if (st != SPMM_SUCCESS)
        return st;
    if (S < 0 || kept < 0 || table_stride < 0)
        return bad("negative size");
    if (S == 0 || kept == 0 || table_stride == 0 || pool->layers == 0 || pool->pages == 0 ||
        pool->page == 0 || pool->row_bytes == 0)
        return SPMM_SUCCESS;
    if ((st = check_pool_data(pool)) != SPMM_SUCCESS)
        return st;
    if (table == nullptr || ctx == nullptr || keep == nullptr || !aligned(table, 4) ||
        !aligned(ctx, 4) || !aligned(keep, 4))
        return bad("table, ctx or keep is null or not 4-byte aligned");
    if (S >= kMaxRows || kept >= kMaxRows || table_stride >= kMaxRows)
        return bad("S, kept and table_stride must be below 2^30");
    if (pool->layers > 4 * kMaxGridY || pool->row_bytes > kMaxRows / 16)
        return unsupported("at most 262140 layers, and 64 MiB to a row");
    if (S * kAttnThreads > kMaxThreads)
        return unsupported("too many sequences for one call");
    PagesArgs a = pages_args(pool);
    a.table = table;
    a.table_stride = table_stride;
    a.ctx = ctx;
    a.keep = keep;
    a.count = S;
    a.kept = kept;
    return launched(launch_pages_compact(a, (hipStream_t)stream), "pages_compact");
}

}  // extern "C"
