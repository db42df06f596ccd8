/*
 * attn.h -- C ABI of the attention operators and of the moves of a paged
 * key/value cache (MI355X, gfx950).  Part of the library declared in spmm.h:
 * the same status codes, element types, error text (spmm_last_error) and
 * rules for streams.
 *
 * Attention is FusedMM with a softmax between its two products, on patterns
 * that need no column list: a window with a few first keys, and a cached
 * context followed by a tree of drafts.
 *
 * Element types: SPMM_DTYPE_F32 and SPMM_DTYPE_BF16, one for all of q, k, v,
 * the output and the gradients of a call.  Products of bf16 values are exact
 * and summed in fp32; softmax statistics and all sums are fp32; the softmax
 * weights and the gradients of the scores are rounded to bf16 once, as
 * operands of the second products, and results once, when they are stored.
 * The backward call takes o as it was stored: in bf16 the products delta =
 * <dout, o> carry its rounding.  fp32 calls round nothing below fp32.
 *
 * Masks are exact: a pair that is not seen contributes nothing, whatever its
 * key, value, query or incoming gradient holds (infinities and NaN too).  A
 * query that sees no key has output 0, log-sum -infinity and no gradient.
 * Infinities and NaN in pairs that are seen go where IEEE arithmetic on the
 * definition sends them.
 *
 * Layout of heads: element (row, head, d) of an operand at
 * data + row * row_stride + head * head_stride + d, strides in elements.
 * data is 16-byte aligned and strides are multiples of 16 bytes; D is a
 * multiple of 8 from 8 to 128.  Hq is a multiple of Hkv: query head h reads
 * key head h / (Hq / Hkv).
 *
 * Packed sequences: rowptr int32[S+1], non-decreasing; sequence s owns rows
 * rowptr[s] .. rowptr[s+1]-1 (rowptr[0] may be positive).  Rows of no
 * sequence are neither read nor written, in the outputs either.
 *
 * Preconditions, as for the CSR arrays of spmm.h not checked by the fast
 * path: row pointers non-decreasing and within the row counts, page numbers
 * (of what a draft may see) within the pool, tables long enough, contexts from 0
 * on and, with their drafts, below 2^30.  Outputs, gradients and scratch memory overlap
 * neither each other nor any input: rows are written while others are still
 * read, and a row that comes out non-finite is computed again from its inputs.
 * (Inputs may overlap each other.)
 *
 * A launch holds fewer than 2^24 workgroups.  Calls that would need more (2^24
 * sequences times heads, roughly) are refused (SPMM_ERROR_UNSUPPORTED) before
 * anything is enqueued.
 *
 * Memory: calls allocate nothing.  Some take scratch memory from the
 * caller (device, 16-byte aligned, the size told by a host-only call); its
 * contents need no preparation and mean nothing afterwards.  Calls that may
 * run at the same time, or graphs that may be replayed at the same time,
 * need scratch of their own.  Every call may be captured into a graph.
 *
 * Results repeat bit for bit: no sum depends on the order of atomics.
 */
#ifndef SDL_ATTN_H
#define SDL_ATTN_H

#include <stdint.h>

#include "spmm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct attn_rows {
    const void *data;     /* written where the call says so */
    int64_t row_stride;   /* elements */
    int64_t head_stride;
} attn_rows_t;

/*
 * Window attention.  Sequence s has Lq queries (rows q_rowptr[s] ..) and Lk
 * keys (rows k_rowptr[s] ..); the queries are its last positions: query i
 * has position p = i + Lk - Lq, key j position j.  The query sees key j when
 *     j <= p  and  (p - j < window  or  j < sinks),
 * so it sees itself, window - 1 keys before it, and the first `sinks` keys
 * of its sequence.  A query at a negative position (Lq > Lk) sees nothing.
 */
typedef struct attn_window {
    int64_t S;            /* sequences */
    int64_t Tq, Tk;       /* rows of the packed queries / keys, < 2^30 */
    int64_t Hq, Hkv, D;
    int64_t window;       /* >= 1; any large value: no window */
    int64_t sinks;        /* 0 .. 128 */
    float scale;          /* > 0, finite */
    int32_t reserved;     /* must be 0 */
} attn_window_t;

/*
 * o_i = sum_j p_ij v_j with p = softmax of scale <q_i, k_j> over the keys
 * that i sees; lse[h * Tq + i] = log sum_j exp(scale <q_i, k_j>), natural
 * logarithm, float32.  lse is what the backward call needs.
 */
spmm_status_t window_attn_fwd(int32_t dtype, const attn_window_t *shape,
                              const attn_rows_t *q, const attn_rows_t *k,
                              const attn_rows_t *v, const int32_t *q_rowptr,
                              const int32_t *k_rowptr, const attn_rows_t *o,
                              float *lse, void *scratch, int64_t scratch_bytes,
                              void *stream);

/* Host only: scratch bytes of window_attn_fwd for this shape (0: none). */
spmm_status_t window_attn_fwd_scratch(int32_t dtype,
                                      const attn_window_t *shape,
                                      int64_t *bytes);

/*
 * Gradients of window_attn_fwd: with p as there,
 *     delta_i = <dout_i, o_i>          ds_ij = p_ij (<dout_i, v_j> - delta_i)
 *     dq_i = scale sum_j ds_ij k_j     dk_j = scale sum_i ds_ij q_i
 *     dv_j = sum_i p_ij dout_i
 * dk and dv sum over all query heads that share a key head.  They are
 * overwritten, for every row of every sequence (keys that no query sees:
 * zero).  o and lse are those of the forward call.
 */
spmm_status_t window_attn_bwd(int32_t dtype, const attn_window_t *shape,
                              const attn_rows_t *dout, const attn_rows_t *q,
                              const attn_rows_t *k, const attn_rows_t *v,
                              const attn_rows_t *o, const float *lse,
                              const int32_t *q_rowptr, const int32_t *k_rowptr,
                              const attn_rows_t *dq, const attn_rows_t *dk,
                              const attn_rows_t *dv, void *scratch,
                              int64_t scratch_bytes, void *stream);

/* Host only: scratch bytes of window_attn_bwd for this shape. */
spmm_status_t window_attn_bwd_scratch(const attn_window_t *shape,
                                      int64_t *bytes);

/*
 * Attention of drafted tokens over a paged cache.  Sequence s has ctx[s]
 * cached keys and the drafts q_rowptr[s] .. q_rowptr[s+1]-1; the keys and
 * values of the drafts lie in the cache behind the context.  Position j of
 * the sequence is row j % page of page table[s * table_stride + j / page]:
 * element (position, head, d) of both pools at
 * number * page_stride + (j % page) * row_stride + head * head_stride + d.
 *
 * tree: bit a of tree[row] says that the draft sees draft a of its sequence
 * (itself too, if it is to; bits past the sequence's drafts mean nothing,
 * and drafts past the 64th are seen by none).  A draft stands at position
 * ctx + n - 1 when it sees n drafts, at ctx when it sees none.  NULL: a
 * chain, draft t sees drafts 0 .. t and stands at ctx + t; any number of
 * them.  A draft at position p sees a cached key (or a draft that its mask
 * names) at position j when p - j < window or j < sinks.
 *
 * Pages that no draft sees are not read: their numbers in the table may be
 * anything.  Outputs: o [Tq, Hq, D] and lse [Hq, Tq], contiguous.
 */
typedef struct attn_tree {
    int64_t S, Tq, Hq, Hkv, D;
    int64_t page;                                   /* rows of a page, >= 1 */
    int64_t page_stride, row_stride, head_stride;   /* of both pools */
    int64_t table_stride;
    int64_t window, sinks;                          /* as attn_window_t */
    float scale;
    int32_t reserved;                               /* must be 0 */
} attn_tree_t;

spmm_status_t tree_attn_paged(int32_t dtype, const attn_tree_t *shape,
                              const attn_rows_t *q, const void *k_pages,
                              const void *v_pages, const int32_t *table,
                              const int32_t *ctx, const int32_t *q_rowptr,
                              const uint64_t *tree, void *o, float *lse,
                              void *scratch, int64_t scratch_bytes,
                              void *stream);

/* Host only: scratch bytes of tree_attn_paged for this shape. */
spmm_status_t tree_attn_scratch(int32_t dtype, const attn_tree_t *shape,
                                int64_t *bytes);

/*
 * Moves within the two pools of a cache, all layers in one launch.  A pool
 * is [layers, pages, page, row_bytes], contiguous; row_bytes (all heads of a
 * position) is a multiple of 16, the pools are 16-byte aligned and do not
 * overlap (a precondition; pages_copy may be given one pool as both).
 *
 * pages_copy: page dst[i] becomes a copy of page src[i] in every layer of
 * both pools, i < count (a fork's partly filled page).  Pairs with a number
 * outside 0 .. pages-1 are passed over, so a list may be padded with -1.  A
 * page may be the source of many pairs; the dst of the others must differ
 * from each other and from every src (a precondition).
 *
 * pages_compact: the kept drafts of sequence s move to the front of its
 * drafts: position ctx[s] + keep[s * kept + t] to ctx[s] + t, t = 0, 1, ...
 * up to the first negative entry.  The entries before it are strictly
 * ascending (a precondition: no kept row is then written over before it has
 * moved), and no two sequences share a page that is written.  An entry whose
 * table index or page number is out of range is passed over.
 */
typedef struct attn_pool {
    void *k, *v;
    int64_t layers, pages, page, row_bytes;
} attn_pool_t;

spmm_status_t pages_copy(const attn_pool_t *pool, const int32_t *src,
                         const int32_t *dst, int64_t count, void *stream);

spmm_status_t pages_compact(const attn_pool_t *pool, const int32_t *table,
                            int64_t table_stride, const int32_t *ctx,
                            const int32_t *keep, int64_t S, int64_t kept,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SDL_ATTN_H */
