/*
 * sv_cache.h -- the paged key-value cache of a verification step (libspecverify.so)
 *
 * A step on paged caches, in the order it runs:
 *   sv_cache_append     turns the rows' queries and keys to their positions and
 *                       stores keys and values in the sequences' pages;
 *   sv_paged_attention  sv_attention of sv_step.h over those pages;
 *   (LM head, logits adjustment and verification of sv_step.h and sv.h)
 *   sv_cache_commit     after sv_verify_tree: moves the accepted path's keys and
 *                       values behind the context, and advances the lengths.
 * sv_rotary turns rows alone (caches without pages; gradients).  The
 * conventions of sv.h on pointers, streams, workspaces, determinism and errors
 * hold here too.
 */
#ifndef SPECVERIFY_SV_CACHE_H
#define SPECVERIFY_SV_CACHE_H

#include "sv_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Storage type of 8-bit pages: 1 sign, 4 exponent and 3 fraction bits, largest
 * value 448, no infinities. */
#define SV_DT_F8E4M3 3
#define SV_ROTARY_MAX_DIM 512
#define SV_CACHE_MAX_PAGE 256
#define SV_CACHE_MAX_BLOCK 64

/* Pages of keys and values.  Token t of head h of page p begins `p *
 * page_stride + t * token_stride + h * head_stride` elements after k (and v);
 * its D values are contiguous.  Zero strides: dense [num_pages][Hkv][page][D].
 *   dtype   SV_DT_BF16, SV_DT_F16 or SV_DT_F8E4M3.
 *   page    tokens of a page: 16, 32, 64, 128 or 256.
 *   block   8-bit pages: tokens that share a scale: 16, 32 or 64, at most page.
 *           A stored value is byte * scale[(p * (page / block) + t / block) *
 *           Hkv + h].  Scales are finite and positive, or zero where a block is
 *           zeros.  (sv_cache_append leaves powers of two from 2^-100 on.  Of scales
 *           below 2^-126 a value may count for anything up to 2^-117.)
 *           Others (16-bit pages): ignored.
 *   k_scale, v_scale  [num_pages][page / block][Hkv] float; NULL for 16-bit pages.
 *   D       64 or 128.
 * Addresses are 16-byte aligned and so are strides in bytes (scales 4); no two
 * values of k share memory, and none of v (SV_EINVAL otherwise, also for strides
 * that interleave), nor may any of k and of v (not checked). */
typedef struct {
  void *k, *v;
  float *k_scale, *v_scale;
  int32_t dtype, num_pages, page, block, Hkv, D;
  int64_t page_stride, token_stride, head_stride;
} sv_paged_cache;

/* Frequencies for the rotations: turns[i] = inv_freq[i] / (2 pi) of a turn in
 * units of 2^-64 (whole turns left out), i < n.  HOST arrays; the caller copies
 * turns to the device.  inv_freq in radians per position, finite.  The product
 * of a position and such a number, modulo 2^64, is the angle without any loss,
 * however far the position. */
int sv_rotary_turns(const double *inv_freq, int32_t n, uint64_t *turns);

/* Rotary positions: pairs of a head's first rot values turned by position *
 * frequency.  Row r of sequence b stands at base_pos[b] + r (a window, a
 * prompt), or at base_pos[b] + the depth of node r (a tree).
 *   (a, b) -> magnitude * (a cos - b sin, b cos + a sin)
 *   x, out   [B][R] rows of x_row_stride / out_row_stride elements (0 = H * D),
 *            each H heads of D; `dtype` float32, bf16 or fp16.  out may be x
 *            (same stride); else no value of the two shares memory (other heads
 *            of the same wider rows: the same stride).  Values from rot on are
 *            copied.
 *   turns    DEVICE [rot / 2], see sv_rotary_turns.
 *   rot      even number of turned values, at most D.  (Multiples of 16 are
 *            handled 16 values at a time, others by pairs.)
 *   interleaved  0: pairs (i, i + rot / 2); 1: pairs (2 i, 2 i + 1).
 *   inverse  1: by the negative angles (with the same magnitude: the gradient of
 *            the operator).
 *   base_pos [B] int64, or NULL (= 0).
 *   row_count [B] or NULL (= R): rows to turn (clamped to [0, R]); the others of
 *            out are left as they were.
 *   parent_host  NULL, or HOST [R], a tree as in sv_verify_tree.
 * D a multiple of 16, at most SV_ROTARY_MAX_DIM.  Sines and cosines are right
 * to float32, products and sums float32, rounded once to dtype.  Rows are
 * 16-byte aligned. */
int sv_rotary(const void *x, int64_t x_row_stride, void *out, int64_t out_row_stride, int dtype,
              const uint64_t *turns, int32_t rot, int interleaved, int inverse, float magnitude,
              const int64_t *base_pos, const int32_t *row_count, const int32_t *parent_host,
              int32_t B, int32_t R, int32_t H, int32_t D, hipStream_t stream);

/* Appends rows to the pages, keys turned on the way.
 *   page_table [B] rows of table_stride int32 (0 = table_pages): token t of
 *              sequence b lies in page page_table[b][t / page].
 *   ctx_len    [B] int32: tokens that a sequence has; row r becomes token
 *              ctx_len[b] + r (nodes of a tree too, in their order).  A sequence
 *              with ctx_len[b] < 0, or with rows past table_pages * page, is left
 *              alone whole: nothing is written for it.
 *   row_count  [B] or NULL (= R): rows to append (clamped to [0, R]).
 *   parent_host  NULL: row r stands at position base_pos[b] + r; else HOST [R],
 *              a tree as in sv_verify_tree: at base_pos[b] + the node's depth.
 *   base_pos   [B] int64, or NULL (= ctx_len: the pages hold a sequence from its
 *              first token on).  Behind P tokens that the batch shares (the
 *              prefix_table of sv_paged_attention, whose own keys were appended
 *              at 0 .. P - 1) rows stand at P + ctx_len: the caller gives that.
 *   k, v       [B][R] rows of k_row_stride / v_row_stride elements (0 = Hkv * D),
 *              each Hkv heads of D, `dtype` SV_DT_BF16 or SV_DT_F16; 16-bit pages
 *              hold the same type.
 *   q, q_out   NULL (Hq = 0), or [B][R] rows of q_row_stride / q_out_row_stride
 *              elements (0 = Hq * D), Hq heads of D: the queries, turned as the
 *              keys are.  q_out may be q (same stride); else no value of the
 *              two shares memory, as for sv_rotary; none of q_out is k's or v's.
 *   turns, rot, interleaved, magnitude  as for sv_rotary, rot a multiple of 16;
 *              turns NULL (rot 0): not turned (queries are copied).
 * Values are stored unturned, keys turned and rounded once: to dtype, or in 8-bit
 * pages to the nearest 8-bit number (ties to even) of the quotient by the scale.
 * (By a scale that is no power of two, as only other programs leave them: turned
 * keys enter the quotient as float32 numbers, inexact ones with their last bit
 * set.)
 * The scale of a block of tokens and kv head, for keys and values each, with a
 * the largest finite magnitude among the call's rows in the block:
 *   a block that begins with the call's rows: the least power of two s >= 2^-100
 *     with a <= 448 s;
 *   a block with earlier tokens and a scale s0: s0 2^j, the least j >= 0 with
 *     a <= 448 s0 2^j; the earlier bytes are then divided by 2^j (exact but for
 *     what falls below the format's smallest numbers).  An s0 that is not a
 *     positive finite number counts as the first case, earlier bytes unchanged.
 * NaN and infinities are stored as NaN and do not enter the scale.  Tokens behind
 * a sequence's rows, and rows whose page number is outside [0, num_pages), are
 * not touched.  No two rows of a call may go to the same place (what it then
 * holds is one of them, or a mixture), nor blocks that another call writes. */
int sv_cache_append(const sv_paged_cache *cache, const int32_t *page_table, int64_t table_stride, int32_t table_pages,
                    const int32_t *ctx_len, const int32_t *row_count, const int32_t *parent_host, const int64_t *base_pos,
                    const void *k, int64_t k_row_stride, const void *v, int64_t v_row_stride,
                    const void *q, int64_t q_row_stride, void *q_out, int64_t q_out_row_stride, int dtype,
                    const uint64_t *turns, int32_t rot, int interleaved, float magnitude,
                    int32_t B, int32_t R, int32_t Hq, hipStream_t stream);

/* Attention of a step's rows over pages: sv_attention with the prefix and the
 * sequences' caches given by page numbers.  What differs:
 *   page_table  as for sv_cache_append; max_ctx + R <= table_pages * page.
 *   prefix_table  DEVICE [ceil(P / page)] page numbers of the P tokens that all
 *            sequences share (in front of them), NULL with P = 0.
 *   8-bit pages: keys and values are byte * scale.  The bytes enter the products
 *            exactly; scales are applied in float32 (or, powers of two, with the
 *            bytes in bf16, exactly): to a key's scores, and of the values to the
 *            exponentials before those are rounded to dtype.  (fp16: exponentials
 *            are held 2^15 times larger, relative to the largest value scale of
 *            the range; products below 2^-29 of it lose up to 2^-40 of it.)
 * Rows are a step's, as for sv_attention: windows of SV_MAX_GAMMA + 1 at most,
 * trees of SV_TREE_MAX_NODES.  (sv_cache_append takes prompts of any length; their
 * own attention is not among these operators.)
 * A page number outside [0, num_pages) among a sequence's tokens makes its rows
 * NaN, one in the prefix all rows; no memory outside the pages is read.  Table
 * entries past a sequence's tokens do not matter. */
size_t sv_paged_attention_workspace(int32_t B, int32_t R, int32_t Hq, int32_t Hkv, int32_t D, int32_t P, int32_t max_ctx);
int sv_paged_attention(const void *q, int64_t q_row_stride, int dtype, const sv_paged_cache *cache,
                       const int32_t *page_table, int64_t table_stride, int32_t table_pages,
                       const int32_t *prefix_table, int32_t P,
                       const int32_t *ctx_len, const int32_t *row_count, const int32_t *parent_host,
                       int32_t B, int32_t R, int32_t Hq, int32_t max_ctx, float scale,
                       void *out, float *lse, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Keeps a tree's accepted path: the keys and values of its nodes, stored by
 * sv_cache_append at tokens ctx_len[b] + node, move to tokens ctx_len[b] + 1 ..
 * behind the root's, in every layer.  (Their positions were the depths already.)
 *   layers   caches of one shape behind each other, layer_stride elements apart
 *            in k and v (0 = dense), their scales num_pages * (page / block) *
 *            Hkv apart; all follow the one page_table.
 *   nodes    [B] rows of nodes_stride int32 (0 = max_nodes): out_nodes of
 *            sv_verify_tree.  NULL (a window, max_nodes = 0): nothing moves, the
 *            lengths advance.  max_nodes <= 64.
 *   n_accepted [B] int32, the first that many nodes (clamped to [0, R - 1], with
 *            nodes to max_nodes too).  A node outside [1, R) ends the path.
 *   new_len  [B] or NULL: ctx_len[b] + 1 + the path's length; may be ctx_len,
 *            apart from it and from n_accepted otherwise.
 * All rows of a path are read before one is stored.  8-bit rows (byte * scale)
 * are stored as sv_cache_append stores them, at token ctx_len[b] + 1 and on
 * (products by a scale that is no power of two: rounded to float32 first).
 * A sequence with ctx_len[b] < 0 or ctx_len[b] + R > table_pages * page is left
 * alone, its length too; rows from or to pages outside [0, num_pages) are left
 * out. */
int sv_cache_commit(const sv_paged_cache *cache, int32_t layers, int64_t layer_stride,
                    const int32_t *page_table, int64_t table_stride, int32_t table_pages,
                    const int32_t *ctx_len, const int32_t *nodes, int64_t nodes_stride, int32_t max_nodes,
                    const int32_t *n_accepted, int32_t B, int32_t R, int32_t *new_len, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_SV_CACHE_H */
