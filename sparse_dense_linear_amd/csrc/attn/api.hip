// api.hip -- host side of the C ABI declared in include/attn.h: checks
// arguments before any HIP call, then enqueues.
#include "checks.h"

using namespace sdl;

namespace {

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
    const spmm_status_t st = check_tree(dtype, CACHE_AS_IS, shape);
    if (st != SPMM_SUCCESS)
        return st;
    if (bytes == nullptr)
        return bad("bytes is null");
    *bytes = shape->S == 0 || shape->Tq == 0
                 ? 0
                 : tree_shape(dtype, CACHE_AS_IS, shape->S, shape->Tq, shape->Hq, shape->Hkv, shape->D).bytes;
    return SPMM_SUCCESS;
}

spmm_status_t tree_attn_paged(int32_t dtype, const attn_tree_t *shape, const attn_rows_t *q,
                              const void *k_pages, const void *v_pages, const int32_t *table,
                              const int32_t *ctx, const int32_t *q_rowptr, const uint64_t *tree,
                              void *o, float *lse, void *scratch, int64_t scratch_bytes, void *stream)
{
    spmm_status_t st = check_tree(dtype, CACHE_AS_IS, shape);
    if (st != SPMM_SUCCESS)
        return st;
    TreeArgs a = {};
    if ((st = check_tree_call(dtype, CACHE_AS_IS, shape, q, k_pages, v_pages, table, ctx, q_rowptr, tree, o, lse,
                              scratch, scratch_bytes, a)) != SPMM_SUCCESS ||
        a.workers == 0)
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
