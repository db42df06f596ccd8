// cache.hip -- host side of the C ABI declared in include/cache.h: checks
// arguments before any HIP call, then enqueues.
#include <utility>

#include "checks.h"

using namespace sdl;

namespace {

spmm_status_t check_codes(int32_t held)
{
    return held == CACHE_E4M3 || held == CACHE_INT8 ? SPMM_SUCCESS
                                                    : bad("held must be CACHE_E4M3 or CACHE_INT8");
}

spmm_status_t check_scales(const cache_scales_t *s, int64_t page)
{
    if (s == nullptr)
        return bad("scales is null");
    if (s->block < 1 || page % s->block != 0)
        return bad("a block must divide the page");
    if (s->page_stride < 0 || s->block_stride < 0 || s->head_stride < 0 || s->page_stride > kMaxStride ||
        s->block_stride > kMaxStride || s->head_stride > kMaxStride)
        return bad("strides of the scales must be in 0 .. 2^32");
    if (s->k == nullptr || s->v == nullptr || !aligned(s->k, 4) || !aligned(s->v, 4))
        return bad("scales are null or not 4-byte aligned");
    return SPMM_SUCCESS;
}

struct Dim {
    int64_t count, stride;
};

// Whether runs of `length` elements lie apart, in dimensions that each step over all
// of those of smaller strides (counts below 2^30, strides up to 2^32).
bool apart(Dim a, Dim b, Dim c, int64_t length)
{
    Dim d[] = {a, b, c};
    for (Dim &x : d)
        if (x.count <= 1)
            x.stride = 0;
    if (d[0].stride > d[1].stride)
        std::swap(d[0], d[1]);
    if (d[1].stride > d[2].stride)
        std::swap(d[1], d[2]);
    if (d[0].stride > d[1].stride)
        std::swap(d[0], d[1]);
    uint64_t extent = (uint64_t)length;
    for (const Dim &x : d) {
        if (x.count <= 1)
            continue;
        if ((uint64_t)x.stride < extent)
            return false;
        extent += (uint64_t)(x.count - 1) * (uint64_t)x.stride;
    }
    return true;
}

spmm_status_t check_code_heads(int64_t D)
{
    return D % 16 == 0 ? SPMM_SUCCESS : unsupported("D must be a multiple of 16 in pools of 8 bits");
}

spmm_status_t check_code_tree(int32_t dtype, int32_t held, const attn_tree_t *shape)
{
    spmm_status_t st = check_codes(held);
    if (st != SPMM_SUCCESS || (st = check_tree(dtype, held, shape)) != SPMM_SUCCESS)
        return st;
    return check_code_heads(shape->D);
}

spmm_status_t check_append(int32_t dtype, int32_t held, const cache_append_t *w)
{
    if (held != CACHE_AS_IS && held != CACHE_E4M3 && held != CACHE_INT8)
        return bad("unknown kind of pool");
    if (w == nullptr)
        return bad("shape is null");
    // no queries: as many as one key head has
    spmm_status_t st = check_heads(dtype, w->Hq == 0 ? w->Hkv : w->Hq, w->Hkv, w->D, 1, 0, 1.0f, w->reserved);
    if (st != SPMM_SUCCESS)
        return st;
    if (held != CACHE_AS_IS && (st = check_code_heads(w->D)) != SPMM_SUCCESS)
        return st;
    if (w->S < 0 || w->T < 0 || w->table_stride < 0 || w->pages < 0 || w->angles < 0)
        return bad("negative size");
    if (w->S >= kMaxRows || w->T >= kMaxRows || w->table_stride >= kMaxRows || w->pages >= kMaxRows)
        return bad("S, T, table_stride and pages must be below 2^30");
    if ((st = check_paging(w, pool_unit(dtype, held))) != SPMM_SUCCESS)
        return st;
    if (!apart({w->pages, w->page_stride}, {w->page, w->row_stride}, {w->Hkv, w->head_stride}, w->D))
        return bad("rows of the pools overlap");
    if (w->rotated < 0 || w->rotated > w->D)
        return bad("rotated must be in 0 .. D");
    if (w->rotated % 8 != 0)
        return unsupported("rotated must be a multiple of 8");
    if (w->interleaved != 0 && w->interleaved != 1)
        return bad("interleaved must be 0 or 1");
    return SPMM_SUCCESS;
}

spmm_status_t check_code_pool(const cache_pool_t *p)
{
    if (p == nullptr)
        return bad("pool is null");
    const spmm_status_t st = check_pool(&p->pool);
    if (st != SPMM_SUCCESS)
        return st;
    if (p->heads < 1 || p->heads > 65536 || p->pool.row_bytes % p->heads != 0)
        return bad("heads must divide row_bytes");
    if (p->block < 1 || p->pool.page % p->block != 0)
        return bad("a block must divide the page");
    // (a turn of the threads that move rows holds whole heads)
    if (p->pool.row_bytes / p->heads > kMaxHeadDim)
        return unsupported("D must be a multiple of 16 up to 128");
    return check_code_heads(p->pool.row_bytes / p->heads);
}

spmm_status_t check_code_pool_data(const cache_pool_t *p)
{
    const spmm_status_t st = check_pool_data(&p->pool);
    if (st != SPMM_SUCCESS)
        return st;
    if (p->k_scale == nullptr || p->v_scale == nullptr || !aligned(p->k_scale, 4) || !aligned(p->v_scale, 4))
        return bad("scales are null or not 4-byte aligned");
    return SPMM_SUCCESS;
}

bool empty(const attn_pool_t &p) { return p.layers == 0 || p.pages == 0 || p.page == 0 || p.row_bytes == 0; }

PagesArgs code_pages_args(const cache_pool_t *p)
{
    PagesArgs a = pages_args(&p->pool);
    a.k_scale = p->k_scale;
    a.v_scale = p->v_scale;
    a.block = p->block;
    a.heads = p->heads;
    return a;
}

}  // namespace

extern "C" {

spmm_status_t cache_append(int32_t dtype, int32_t held, const cache_append_t *shape, const attn_rows_t *q,
                           const attn_rows_t *k, const attn_rows_t *v, const float *cosines, const float *sines,
                           const int32_t *table, const int32_t *ctx, const int32_t *rowptr,
                           const uint64_t *tree, void *k_pages, void *v_pages, const cache_scales_t *scales,
                           const attn_rows_t *q_out, void *stream)
{
    spmm_status_t st = check_append(dtype, held, shape);
    if (st != SPMM_SUCCESS)
        return st;
    if ((st = check_rows(k, shape->T, dtype, "k is null")) != SPMM_SUCCESS ||
        (st = check_rows(v, shape->T, dtype, "v is null")) != SPMM_SUCCESS)
        return st;
    if (shape->Hq > 0 &&
        ((st = check_rows(q, shape->T, dtype, "q is null")) != SPMM_SUCCESS ||
         (st = check_out(q_out, shape->T, shape->Hq, shape->D, dtype, "q_out is null")) != SPMM_SUCCESS))
        return st;
    if (shape->S == 0 || shape->T == 0)
        return SPMM_SUCCESS;
    if (table == nullptr || ctx == nullptr || rowptr == nullptr || k_pages == nullptr || v_pages == nullptr)
        return bad("a null pointer");
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16))
        return bad("the pools must be 16-byte aligned");
    if (!aligned(table, 4) || !aligned(ctx, 4) || !aligned(rowptr, 4) || !aligned(tree, 8))
        return bad("an array is not aligned to its element size");
    if (shape->rotated > 0 && shape->angles > 0 &&
        (cosines == nullptr || sines == nullptr || !aligned(cosines, 16) || !aligned(sines, 16)))
        return bad("cosines or sines are null or not 16-byte aligned");
    if (held != CACHE_AS_IS && (st = check_scales(scales, shape->page)) != SPMM_SUCCESS)
        return st;
    if (held != CACHE_AS_IS &&
        !apart({shape->pages, scales->page_stride}, {shape->page / scales->block, scales->block_stride},
               {shape->Hkv, scales->head_stride}, 1))
        return bad("scales overlap");
    if (held == CACHE_AS_IS && scales != nullptr)
        return bad("pools of the operands' type have no scales");
    AppendArgs a = {};
    if (shape->Hq > 0) {
        a.q = in_rows(q);
        a.q_out = out_rows(q_out);
    }
    a.k = in_rows(k);
    a.v = in_rows(v);
    a.cosines = cosines;
    a.sines = sines;
    a.table = table;
    a.table_stride = shape->table_stride;
    a.ctx = ctx;
    a.rowptr = rowptr;
    a.tree = tree;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.pages = shape->pages;
    a.page_stride = shape->page_stride;
    a.row_stride = shape->row_stride;
    a.head_stride = shape->head_stride;
    if (scales != nullptr) {
        a.k_scale = scales->k;
        a.v_scale = scales->v;
        a.block = (int32_t)scales->block;
        a.scale_page = scales->page_stride;
        a.scale_block = scales->block_stride;
        a.scale_head = scales->head_stride;
    }
    a.S = (int32_t)shape->S;
    a.T = (int32_t)shape->T;
    a.Hq = (int32_t)shape->Hq;
    a.Hkv = (int32_t)shape->Hkv;
    a.D = (int32_t)shape->D;
    a.page = (int32_t)shape->page;
    a.rotated = (int32_t)shape->rotated;
    a.angles = (int32_t)(shape->angles < kMaxRows ? shape->angles : kMaxRows);
    a.interleaved = shape->interleaved;
    if ((st = check_threads(append_threads(held, a))) != SPMM_SUCCESS)
        return st;
    return launched(launch_append(dtype, held, a, (hipStream_t)stream), "cache_append");
}

spmm_status_t cache_tree_attn_scratch(int32_t dtype, int32_t held, const attn_tree_t *shape, int64_t *bytes)
{
    const spmm_status_t st = check_code_tree(dtype, held, shape);
    if (st != SPMM_SUCCESS)
        return st;
    if (bytes == nullptr)
        return bad("bytes is null");
    *bytes = shape->S == 0 || shape->Tq == 0
                 ? 0
                 : tree_shape(dtype, held, shape->S, shape->Tq, shape->Hq, shape->Hkv, shape->D).bytes;
    return SPMM_SUCCESS;
}

spmm_status_t cache_tree_attn(int32_t dtype, int32_t held, const attn_tree_t *shape, const attn_rows_t *q,
                              const void *k_pages, const void *v_pages, const cache_scales_t *scales,
                              const int32_t *table, const int32_t *ctx, const int32_t *q_rowptr,
                              const uint64_t *tree, void *o, float *lse, void *scratch,
                              int64_t scratch_bytes, void *stream)
{
    spmm_status_t st = check_code_tree(dtype, held, shape);
    if (st != SPMM_SUCCESS)
        return st;
    TreeArgs a = {};
    if ((st = check_tree_call(dtype, held, shape, q, k_pages, v_pages, table, ctx, q_rowptr, tree, o, lse, scratch,
                              scratch_bytes, a)) != SPMM_SUCCESS ||
        a.workers == 0)
        return st;
    if ((st = check_scales(scales, shape->page)) != SPMM_SUCCESS)
        return st;
    a.k_scale = scales->k;
    a.v_scale = scales->v;
    a.block = (int32_t)scales->block;
    a.scale_page = scales->page_stride;
    a.scale_block = scales->block_stride;
    a.scale_head = scales->head_stride;
    a.by_page = divisor((uint32_t)shape->page);
    a.by_block = divisor((uint32_t)scales->block);
    // 16 keys in one page, whose bytes are 32 bits apart at most, and four with one scale
    a.together = shape->page % 16 == 0 && scales->block % 4 == 0 && shape->row_stride < ((int64_t)1 << 27);
    if (a.block_rows == 16) {
        // Blocks of 8 rows where there are no more, of two steps of keys: 64 answers of 4
        // rows 136 us against 151, with integers 140 against 164.  (Blocks of 4, of four
        // steps: 137 and 142.)
        if (a.together && a.mean_rows <= 8)
            a.block_rows = 8;
        a.tile_keys = 32 * (16 / a.block_rows) * (4 / a.wave_heads);
        a.slot_rows = a.block_rows * a.wave_heads;
        if ((st = check_threads(tree_threads(a))) != SPMM_SUCCESS)
            return st;
    } else {
        a.tile_keys = 128;
    }
    return launched(held == CACHE_E4M3 ? launch_tree_e4m3(dtype, a, (hipStream_t)stream)
                                       : launch_tree_int8(dtype, a, (hipStream_t)stream),
                    "tree attention over 8 bits");
}

spmm_status_t cache_copy(const cache_pool_t *pool, const int32_t *src, const int32_t *dst, int64_t count,
                         void *stream)
{
    spmm_status_t st = check_code_pool(pool);
    if (st != SPMM_SUCCESS)
        return st;
    if (count < 0)
        return bad("negative size");
    if (count == 0 || empty(pool->pool))
        return SPMM_SUCCESS;
    if ((st = check_code_pool_data(pool)) != SPMM_SUCCESS)
        return st;
    if (src == nullptr || dst == nullptr || !aligned(src, 4) || !aligned(dst, 4))
        return bad("src or dst is null or not 4-byte aligned");
    if (count >= kMaxRows ||
        too_many(pool->pool.layers, count, pages_copy_parts(pool->pool.page * pool->pool.row_bytes)))
        return unsupported("too many pages for one call");
    PagesArgs a = code_pages_args(pool);
    a.src = src;
    a.dst = dst;
    a.count = count;
    return launched(launch_pages_copy(a, (hipStream_t)stream), "cache_copy");
}

spmm_status_t cache_compact(int32_t held, const cache_pool_t *pool, const int32_t *table, int64_t table_stride,
                            const int32_t *ctx, const int32_t *keep, int64_t S, int64_t kept, void *stream)
{
    spmm_status_t st = check_codes(held);
    if (st != SPMM_SUCCESS || (st = check_code_pool(pool)) != SPMM_SUCCESS)
        return st;
    if (S < 0 || kept < 0 || table_stride < 0)
        return bad("negative size");
    if (S == 0 || kept == 0 || table_stride == 0 || empty(pool->pool))
        return SPMM_SUCCESS;
    if ((st = check_code_pool_data(pool)) != SPMM_SUCCESS)
        return st;
    if (table == nullptr || ctx == nullptr || keep == nullptr || !aligned(table, 4) || !aligned(ctx, 4) ||
        !aligned(keep, 4))
        return bad("table, ctx or keep is null or not 4-byte aligned");
    if (S >= kMaxRows || kept >= kMaxRows || table_stride >= kMaxRows)
        return bad("S, kept and table_stride must be below 2^30");
    if (pool->pool.layers > kMaxGridY / 2 || pool->pool.row_bytes > kMaxRows / 16)
        return unsupported("at most 32767 layers, and 64 MiB to a row");
    if (S * kAttnThreads > kMaxThreads)
        return unsupported("too many sequences for one call");
    PagesArgs a = code_pages_args(pool);
    a.table = table;
    a.table_stride = table_stride;
    a.ctx = ctx;
    a.keep = keep;
    a.count = S;
    a.kept = kept;
    return launched(launch_cache_compact(held, a, (hipStream_t)stream), "cache_compact");
}

}  // extern "C"
