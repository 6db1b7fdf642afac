/*
 * gdn_attn.h -- C ABI of the softmax-attention side of a decode step on MI355X
 * (gfx950): rotary positions of a draft tree's rows, attention of the tree over
 * a paged key/value cache, the append of the accepted path to that cache, and
 * the bookkeeping of its pages.
 *
 * Models with Gated DeltaNet layers keep some layers of ordinary softmax
 * attention.  gdn_tree.h verifies a draft tree through the former; these calls
 * verify the same tree through the latter, from the same cache record: the
 * ancestor bit rows, depths and tree status that gdn_tree_verify writes, and the
 * path that gdn_tree_commit writes.  As there, nothing is rolled back: the
 * tree's keys and values stay outside the paged cache until the accepted path is
 * known, and only its rows are then appended.
 *
 * What the calls compute, for sequence b with a cached prefix of ctx[b] rows:
 *
 *   rope    position of node i = ctx[b] + depth[i]; for each rotated pair t with
 *           angle a = position * freq[t]:  (x, y) -> amp (x cos a - y sin a,
 *                                                         y cos a + x sin a)
 *   verify  o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = e^(scale q_i.k_j - m_i),
 *           j over the ctx[b] rows of the prefix, the strict ancestors of i, and i
 *   commit  cache row ctx[b] + t = row path[t] of the tree's k and v, t < path_len
 *
 * Conventions are those of gdn_tree.h (device pointers, a negative gdn_status for
 * what the host can see, nothing allocated, nothing synchronised, kernels on
 * `stream`), except that tensors of rows and the cache need not be contiguous:
 *
 *  - gdn_attn_rows describes [rows][heads][d] with the last axis contiguous and
 *    any row and head stride, in elements, so that q, k and v can be slices of
 *    one projection's output.
 *  - gdn_paged_cache describes key and value pools [layers][pages][page_rows][h_kv][d]
 *    with the last axis contiguous and any other strides: rows first or heads
 *    first within a page.
 *  - Pointers and all these strides are multiples of 16 bytes (GDN_ERR_ALIGN).
 *    Strides are not negative (GDN_ERR_DIMS).
 *
 * Sizes: 1 <= n_nodes <= 1024; 1 <= h_kv <= 8192; h_q a multiple of h_kv, <= 2^20; n_nodes
 * h_q / h_kv <= 65536; d a multiple of 8, 8 <= d <= 256; io_dtype GDN_F32 or GDN_BF16;
 * a page's keys of one layer at most 16 GiB.
 * batch = 0 launches nothing.
 *
 * Ragged batches are those of gdn_tree.h: `offsets` (device int32 [B + 1]) gives
 * sequence b the rows offsets[b] .. offsets[b+1] - 1 of the row tensors; NULL is
 * the dense layout, rows b N .. b N + N - 1.
 */
#ifndef GDN_ATTN_H
#define GDN_ATTN_H

#include "gdn_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

/* scale: the factor of q.k, finite and > 0 (read by gdn_attn_verify alone). */
typedef struct {
    int32_t batch, n_nodes, h_q, h_kv, d, io_dtype;
    float scale;
} gdn_attn_dims;

typedef struct {
    void* data;
    int64_t row, head; /* strides in elements */
} gdn_attn_rows;

typedef struct {
    void* k;
    void* v;
    int32_t n_layers, n_pages, page_rows, h_kv, d, io_dtype;
    int64_t k_layer, k_page, k_row, k_head; /* strides in elements */
    int64_t v_layer, v_page, v_row, v_head;
} gdn_paged_cache;

/* ------------------------------------------------------------------ rope */

/* Which coordinates form pair t of the first `rot` of a head's d. */
typedef enum {
    GDN_ROPE_HALF = 0,       /* (t, t + rot / 2) */
    GDN_ROPE_INTERLEAVED = 1 /* (2 t, 2 t + 1)   */
} gdn_rope_layout;

/* rot: rotated coordinates, even, 2 <= rot <= d; the others are copied.
 * amp: factor of the rotated coordinates (1 where a long-context scaling has none). */
typedef struct {
    int32_t rot, layout;
    double amp;
} gdn_rope_dims;

/*
 * Rotate the tree's queries and keys to their nodes' positions.
 *
 *   q, k          [T][h_q][d], [T][h_kv][d]  io
 *   freq          [rot / 2] fp64  radians per position of each pair; a scaling
 *                                 for long contexts is a matter of these
 *   ctx           [B]    int32    rows of each prefix
 *   depth         [B][N] int32    depth in the tree (gdn_tree_cache.depth)
 *   q_out, k_out  as q, k; each may be its input (same data and strides)
 *
 * Angles are formed and reduced in fp64.  A node of depth < 0 (an invalid tree)
 * gets NaN rows.  Rows that belong to no sequence are not written.
 */
int gdn_attn_rope(const gdn_attn_dims* dims, const gdn_rope_dims* rope, const int32_t* offsets,
                  int64_t n_rows, const gdn_attn_rows* q, const gdn_attn_rows* k, const double* freq,
                  const int32_t* ctx, const int32_t* depth, const gdn_attn_rows* q_out,
                  const gdn_attn_rows* k_out, hipStream_t stream);

/* ------------------------------------------------------------------ verify */

/* Bytes of the workspace of gdn_attn_verify.  It is zeroed once, when it is
 * allocated; every call leaves it ready for the next.  One workspace serves
 * calls that follow each other on a stream, not concurrent ones.  They may be of
 * any dims that need no more bytes; fewer sequences or nodes never need more. */
int gdn_attn_workspace_bytes(const gdn_attn_dims* dims, size_t* bytes);

/*
 * Attention of every node of every tree over prefix and ancestors.
 *
 *   cache     layer `layer` of the pools; they hold the prefixes alone
 *   table     [B][width] int32  page of rows page_rows c .. of sequence b, at [b][c]
 *             (NULL where width is 0: no sequence has a prefix)
 *   ctx       [B] int32         rows of each prefix, 0 allowed
 *   q, k, v   [T] rows          of the tree's nodes (rotated already)
 *   anc_mask  [B][N][ceil(N/32)] int32, tree_status [B] int32: gdn_tree_cache's.
 *             Node i sees node j where bit j is set, and itself; bits from n_b
 *             on are not read as nodes.  For the next token alone N = 1, one zero
 *             word and status 0.
 *   o         [T][h_q][d] io    out
 *
 * Scores, running maximum, sum and output are fp32; with bf16 io the weights p
 * are rounded for the product with v, and the sum is that of the rounded weights: to 2^-16
 * of each at most where up to 16 rows share a key head (n_nodes h_q / h_kv), to 2^-8 where more do.  Infinities and NaN in rows that a node does not see do not reach it.
 * The o rows of a sequence are NaN where tree_status is not 0, where ctx is outside
 * [0, min(page_rows width, 2^31 - 2^16)], or where an entry of the table that the prefix needs is not
 * a page of the pool; no page is read through such an entry.
 */
int gdn_attn_verify(const gdn_attn_dims* dims, const int32_t* offsets, const gdn_paged_cache* cache,
                    int32_t layer, const int32_t* table, int32_t width, const int32_t* ctx,
                    const gdn_attn_rows* q, const gdn_attn_rows* k, const gdn_attn_rows* v,
                    const uint32_t* anc_mask, const int32_t* tree_status, const gdn_attn_rows* o,
                    void* workspace, hipStream_t stream);

/* ------------------------------------------------------------------ commit */

/*
 * Append the accepted path's keys and values to the cache.
 *
 *   path, path_len  as gdn_tree_commit (ragged: gdn_tree_commit_ragged) writes them
 *   new_len [B] int32  out: ctx + path_len; ctx where path_len <= 0; -1 where rows
 *                      have no place (ctx < 0, the table is too narrow or names no
 *                      page of the pool there, ctx + path_len > 2^31 - 1) or path has an entry that is no node:
 *                      then nothing of the sequence is appended.  Not ctx itself
 *                      (GDN_ERR_ALIAS): several workgroups read that.
 *
 * The pages that receive rows must belong to one sequence (gdn_pages_reserve).
 */
int gdn_attn_commit(const gdn_attn_dims* dims, const int32_t* offsets, const gdn_paged_cache* cache,
                    int32_t layer, const int32_t* table, int32_t width, const int32_t* ctx,
                    const gdn_attn_rows* k, const gdn_attn_rows* v, const int32_t* path,
                    const int32_t* path_len, int32_t* new_len, hipStream_t stream);

/* ------------------------------------------------------------------ pages */

/*
 * Bookkeeping of a pool of n_pages pages of page_rows rows that n_slots sequences share:
 *
 *   ref    [n_pages]        int32  sequences that hold the page; 0 is free
 *   table  [n_slots][width] int32  pages of each sequence, -1 past the held ones
 *   held   [n_slots]        int32  pages held
 *   length [n_slots]        int32  rows
 *
 * All of it stays on the device; nothing waits for the host.  The results do not
 * depend on the order in which threads run.
 * Sizes: 1 <= n_pages <= 2^30, 1 <= page_rows <= 65536, 1 <= n_slots <= 4096,
 * 1 <= width <= 2^20.
 */
typedef struct {
    int32_t n_pages, page_rows, n_slots, width;
} gdn_page_dims;

/*
 * dst_seq[i] becomes a second holder of all pages of src_seq[i], i < n.
 *   status [n] int32 out: 0; -1, and nothing done, where a slot is outside the table,
 *          dst holds pages already, dst is named by an earlier i, src is a dst of this
 *          call, or src's length and pages do not fit each other.
 */
int gdn_pages_fork(const gdn_page_dims* dims, int32_t n, const int32_t* src_seq, const int32_t* dst_seq,
                   int32_t* ref, int32_t* table, int32_t* held, int32_t* length, int32_t* status,
                   hipStream_t stream);

/*
 * Make room for need[s] more rows of each sequence s: a page of its own for a partly
 * filled last page that others hold too, then the missing pages, each the lowest
 * free one, sequences in ascending order.  Of the sequences that ask here and share a
 * last page with nobody else, the last one keeps the page itself.
 *   src, dst [n_slots] int32, count [1] int32 out: the page copies this takes
 *          (gdn_pages_copy), entries from *count on unspecified
 *   status [n_slots] int32 out: 0; -1 does not fit the table (or its length and held
 *          pages contradict each other); -2 the pool has too few pages.  A sequence
 *          whose status is not 0 is left as it was.
 * need[s] <= 0 asks for nothing.  A sequence after one that the pool was too small for
 * gets nothing either, unless it needs no page.
 */
int gdn_pages_reserve(const gdn_page_dims* dims, const int32_t* need, int32_t* ref, int32_t* table,
                      int32_t* held, const int32_t* length, int32_t* src, int32_t* dst, int32_t* count,
                      int32_t* status, hipStream_t stream);

/* Copy pages src[i] over pages dst[i], i < min(*count, n), in every layer, keys and
 * values.  No dst may be a src or another dst.  Entries that name no page are skipped. */
int gdn_pages_copy(const gdn_paged_cache* cache, int32_t n, const int32_t* src, const int32_t* dst,
                   const int32_t* count, hipStream_t stream);

/* Sequences with drop[s] != 0 give their pages back and become empty. */
int gdn_pages_free(const gdn_page_dims* dims, const int32_t* drop, int32_t* ref, int32_t* table,
                   int32_t* held, int32_t* length, hipStream_t stream);

/*
 * Move the held pages, those with ref > 0, to the front of the pool: with m pages held, the
 * i-th held page at or past m goes to the i-th free page below m.  At most n pages are
 * moved.  `held` is not read.
 *   src, dst [n] int32, count [1] int32 out: the copies (gdn_pages_copy)
 *   remap [n_pages] int32 out: where each page's rows are afterwards
 * ref and table are brought in line; table entries that name no page stay.
 */
int gdn_pages_compact(const gdn_page_dims* dims, int32_t n, int32_t* ref, int32_t* table,
                      const int32_t* held, int32_t* src, int32_t* dst, int32_t* count, int32_t* remap,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTN_H */
