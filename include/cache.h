/*
 * cache.h -- C ABI of a paged key/value cache that is written as it is read:
 * appending rows with their rotation, and caches held in 8 bits (MI355X,
 * gfx950).  Part of the library declared in spmm.h and attn.h: the same status
 * codes, error text, rules for streams, scratch memory and capture, layout of
 * heads, packed sequences and pages.
 *
 * What a pool holds (`held`):
 *   CACHE_AS_IS  rows of the operands' type (SPMM_DTYPE_F32 or _BF16)
 *   CACHE_E4M3   floating-point codes of 8 bits: sign, 4 bits of exponent, 3 of
 *                fraction, no infinities, largest 448
 *   CACHE_INT8   integer codes, -127 .. 127 as written here (-128 may be read)
 * A pool of codes has a scale, float32, for each block of `block` positions
 * (which divides the page) and head: value = code * scale.  Scales as written
 * here are powers of two; reading takes any.  In pools of codes D is a
 * multiple of 16 (up to 128, as everywhere), and strides of the pools are in
 * codes (multiples of 16).
 *
 * How a scale is chosen.  The values that a call brings into a block are held
 * by the smallest power of two s, at least 2^-126, with
 *     max |x| <= 448 s  (e4m3)   or   127 s  (integers),
 * the maximum over the values that are finite numbers.  Where the block keeps
 * earlier rows, its scale is the larger of s and the one it had; if that
 * raises it, the codes of the earlier rows become round(code * old / new).
 * A code is round(x / scale), to nearest even, and products and quotients are
 * rounded once each to fp32.  Where x is finite and that code times its scale is
 * not, it is the next smaller code (values from 248 * 2^120 on are held as 240 *
 * 2^120, in integers from 63.5 * 2^122 on as 63 * 2^122).  With powers of two that
 * is exact but for the last rounding, so raising a scale costs codes of e4m3
 * nothing (but for those below the smallest normal one), and integers their last
 * bit.
 * A value that is not finite becomes the code NaN in e4m3.  Integers have no
 * such code: the scale of its block and head becomes NaN, and all rows of the
 * block and head read as NaN until the block is begun anew.  The earlier rows of
 * the block are lost with it (codes and scale are written over), also where the
 * value was that of a draft which is not kept.  Rows of a block behind the last one
 * that was written hold codes of no meaning.
 *
 * Preconditions, beyond those of attn.h: scales of blocks that keep rows are
 * positive (or NaN); no two sequences of a call write the same block; pools,
 * scales and outputs overlap nothing else that the call takes.
 */
#ifndef SDL_CACHE_H
#define SDL_CACHE_H

#include <stdint.h>

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CACHE_AS_IS 0
#define CACHE_E4M3  1
#define CACHE_INT8  2

/* Scales of both pools: of page number n, block b and head h at
 * n * page_stride + b * block_stride + h * head_stride (elements). */
typedef struct cache_scales {
    float *k, *v;
    int64_t block;        /* positions of a block, divides the page */
    int64_t page_stride, block_stride, head_stride;
} cache_scales_t;

/*
 * New rows go into the pages behind the context of their sequence, and are
 * rotated on the way.  Row t of sequence s (row rowptr[s] + t of q, k and v)
 * is position ctx[s] + t of the sequence: it lies where attn.h says that
 * tree_attn_paged reads it.  It stands at position ctx[s] + t too, or, with
 * masks of a tree (attn.h), where the draft stands: at ctx + n - 1 when it sees
 * n drafts, at ctx when it sees none.
 *
 * Rotation by the position a where a row stands, of the first `rotated`
 * elements of each head of q and k, c = cosines[a * rotated / 2 + i] and
 * s = sines[same], i < rotated / 2:
 *     (x, y) -> (x c - y s, y c + x s)
 * where x and y are elements i and i + rotated / 2, or, interleaved, 2 i and
 * 2 i + 1.  Each product and each sum is rounded once to fp32, the result once
 * to what it is stored as.  At positions past the tables (a >= angles) the
 * rotated elements are NaN.  cosines and sines are contiguous, 16-byte aligned;
 * rotated = 0: none, and they may be null.
 *
 * q_out takes the rotated q; it may be q itself.  Hq = 0: no queries, q and
 * q_out are not looked at.  v is stored as it is.  Rows of k and v whose table
 * index or page number (0 .. pages - 1) is out of range, or whose position is
 * negative, are passed over, in pools of codes whole blocks.  Nothing else of the pools is written but, in
 * pools of codes, the scales and the earlier rows of the blocks written to.
 * Strides by which rows of a pool, or scales, would overlap are refused.
 */
typedef struct cache_append {
    int64_t S, T;                                   /* sequences, rows */
    int64_t Hq, Hkv, D;
    int64_t page, pages;
    int64_t page_stride, row_stride, head_stride;   /* of both pools */
    int64_t table_stride;
    int64_t rotated;      /* 0 .. D, a multiple of 8 */
    int64_t angles;       /* rows of the tables */
    int32_t interleaved;  /* 0 or 1 */
    int32_t reserved;     /* must be 0 */
} cache_append_t;

/* scales: null for CACHE_AS_IS. */
spmm_status_t cache_append(int32_t dtype, int32_t held,
                           const cache_append_t *shape, const attn_rows_t *q,
                           const attn_rows_t *k, const attn_rows_t *v,
                           const float *cosines, const float *sines,
                           const int32_t *table, const int32_t *ctx,
                           const int32_t *rowptr, const uint64_t *tree,
                           void *k_pages, void *v_pages,
                           const cache_scales_t *scales,
                           const attn_rows_t *q_out, void *stream);

/*
 * tree_attn_paged over pools of codes (held: CACHE_E4M3 or CACHE_INT8): keys
 * and values are code * scale.  Codes are exact in the products; scales are
 * applied in fp32, or exactly, those of keys to the sum over the codes (which an
 * infinite one makes infinite).  Softmax weights, times the scale of their value
 * or not, are rounded to the element type, or to more bits.  Codes, scales and
 * table entries of rows that no draft sees have no effect; other rows of pages
 * that hold a row which is seen, and page 0, may be read.  k_pages and v_pages
 * are 16-byte aligned.
 */
spmm_status_t cache_tree_attn(int32_t dtype, int32_t held,
                              const attn_tree_t *shape, const attn_rows_t *q,
                              const void *k_pages, const void *v_pages,
                              const cache_scales_t *scales,
                              const int32_t *table, const int32_t *ctx,
                              const int32_t *q_rowptr, const uint64_t *tree,
                              void *o, float *lse, void *scratch,
                              int64_t scratch_bytes, void *stream);

/* Host only: scratch bytes of cache_tree_attn for this shape. */
spmm_status_t cache_tree_attn_scratch(int32_t dtype, int32_t held,
                                      const attn_tree_t *shape,
                                      int64_t *bytes);

/*
 * pages_copy and pages_compact (attn.h) for pools of codes
 * [layers, pages, page, heads, D], row_bytes = heads * D, and their scales
 * [layers, pages, page / block, heads], all contiguous.
 *
 * cache_copy copies a page's scales with it.
 *
 * cache_compact: a block that kept rows move into, or stay in, takes the
 * largest of the scales of the blocks where the rows come from that it then
 * holds (its own, if it holds rows of the context), and codes of another scale
 * become round(code * their scale / its scale).
 */
typedef struct cache_pool {
    attn_pool_t pool;
    float *k_scale, *v_scale;
    int64_t block, heads;
} cache_pool_t;

spmm_status_t cache_copy(const cache_pool_t *pool, const int32_t *src,
                         const int32_t *dst, int64_t count, void *stream);

spmm_status_t cache_compact(int32_t held, const cache_pool_t *pool,
                            const int32_t *table, int64_t table_stride,
                            const int32_t *ctx, const int32_t *keep, int64_t S,
                            int64_t kept, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SDL_CACHE_H */
