// checks.h -- what the host sides of attn.h and cache.h share: checks of
// arguments, made before any HIP call, and the kernels' descriptions of them.
#pragma once

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "cache.h"

#include "ops.h"
#include "internal.h"

namespace sdl {

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

// Elements of 16 bytes of a pool.
int64_t pool_unit(int32_t dtype, int32_t held)
{
    return held != CACHE_AS_IS ? 16 : (dtype == SPMM_DTYPE_BF16 ? 8 : 4);
}

// Strides and the page of pools, as attn_tree_t and cache_append_t have them.
template <class Shape>
spmm_status_t check_paging(const Shape *w, int64_t unit)
{
    if (w->page < 1 || w->page >= kMaxRows)
        return bad("page must be in 1 .. 2^30 - 1");
    if (w->page_stride < 0 || w->row_stride < 0 || w->head_stride < 0 ||
        w->page_stride > kMaxStride || w->row_stride > kMaxStride || w->head_stride > kMaxStride)
        return bad("strides must be in 0 .. 2^32");
    if (w->page_stride % unit != 0 || w->row_stride % unit != 0 || w->head_stride % unit != 0)
        return bad("strides must be multiples of 16 bytes");
    return SPMM_SUCCESS;
}

spmm_status_t check_tree(int32_t dtype, int32_t held, const attn_tree_t *w)
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
    const spmm_status_t paging = check_paging(w, pool_unit(dtype, held));
    if (paging != SPMM_SUCCESS)
        return paging;
    if (w->Tq * w->Hq + w->S * w->Hkv > kMaxGrid)
        return unsupported("too many queries: Tq * Hq + S * Hkv must be below 2^31");
    return SPMM_SUCCESS;
}

spmm_status_t check_threads(int64_t threads)
{
    return threads <= kMaxThreads ? SPMM_SUCCESS
                                  : unsupported("too many workgroups: fewer sequences, rows or heads");
}

// The rest of a call's checks once its shape is right, and its description;
// nothing to do: a.workers stays 0.
spmm_status_t check_tree_call(int32_t dtype, int32_t held, const attn_tree_t *shape, const attn_rows_t *q,
                              const void *k_pages, const void *v_pages, const int32_t *table,
                              const int32_t *ctx, const int32_t *q_rowptr, const uint64_t *tree, void *o,
                              float *lse, void *scratch, int64_t scratch_bytes, TreeArgs &a)
{
    const spmm_status_t st = check_rows(q, shape->Tq, dtype, "q is null");
    if (st != SPMM_SUCCESS)
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
    const TreeShape sh = tree_shape(dtype, held, shape->S, shape->Tq, shape->Hq, shape->Hkv, shape->D);
    if (scratch_bytes < sh.bytes)
        return bad("scratch is smaller than the call's host-only function says");
    if (scratch == nullptr || !aligned(scratch, 16))
        return bad("scratch is null or not 16-byte aligned");
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
    a.slot_rows = sh.block_rows * sh.wave_heads;
    a.wave_heads = sh.wave_heads;
    a.mean_rows = (int32_t)(sh.rows < 128 ? sh.rows : 128);
    return check_threads(tree_threads(a));
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

}  // namespace

}  // namespace sdl
