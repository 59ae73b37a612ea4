/*
 * sv_step.h -- operators around a verification step (libspecverify.so)
 *
 * The target's (or draft's) side of a step, in the order a step runs them:
 *   sv_attention      the rows of a window or tree over the batch's shared
 *                     prefix, the cached context and their ancestors;
 *   sv_lmhead_quant   their logits on a 4-bit unembedding;
 *   sv_adjust_logits  penalties, biases and grammar masks on those logits;
 * and then sv_verify_window, sv_verify_greedy or sv_verify_tree of sv.h, whose
 * conventions on pointers, streams, workspaces, determinism and errors hold
 * here too.  A step's rows are those of the verify calls: gamma + 1 rows of a
 * window, or the nodes of a tree given by the same parent array.
 */
#ifndef SPECVERIFY_SV_STEP_H
#define SPECVERIFY_SV_STEP_H

#include "sv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_ADJUST_MAX_BIAS 65535
#define SV_ATTENTION_MAX_HEADS 1024
#define SV_ATTENTION_MAX_KEYS (1 << 24)

/* Logits adjustment: penalties for repeated tokens, biases and grammar masks
 * on the rows of a window or tree, before they are verified (or before a draft
 * is drawn from them).
 *   logits, out [B][R][V], `dtype`; rows of one sequence contiguous, sequences
 *               seq_stride / out_seq_stride ELEMENTS apart (0 = dense).  out is
 *               logits itself (same stride: in place), or the two lie apart
 *               (from first row to last, also where only their gaps overlap).
 *   tokens      [B] rows of tokens_stride (0 = dense) int32, the drafts.
 *   parent_host NULL: a window; row i follows tokens[b][0 .. i-1] (R - 1 are
 *               read), so target rows (R = gamma + 1) and draft rows
 *               (R = gamma) take the same array.  R <= SV_MAX_GAMMA + 1.
 *               Else HOST [R], a tree as in sv_verify_tree: row v follows the
 *               tokens tokens[b][v] of the nodes from the root's child to v
 *               (entry 0 is ignored).
 *   row_count   [B] or NULL (= R): rows of each sequence to adjust (clamped to
 *               [0, R]); the others of `out` are left as they were.
 *   history     [B] rows of history_stride (0 = history_cap) int32: the tokens
 *               so far, history_len[b] of them (NULL = history_cap; clamped to
 *               [0, history_cap]), the first prompt_len[b] the prompt (NULL =
 *               0).  NULL with history_cap 0: no history.
 *   repetition, presence, frequency [B] float or NULL (= 1, 0, 0).
 *   bias_tokens, bias_values [B][n_bias]: added to those tokens' logits.  Of
 *               several entries that name one token the last counts.
 *               n_bias <= SV_ADJUST_MAX_BIAS.
 *   allowed     NULL, or bit masks: token t of row r is allowed when bit
 *               t % 32 of word allowed[b * allowed_seq_stride +
 *               r * allowed_row_stride + t / 32] is set (strides in 32-bit
 *               words; 0 shares a mask between sequences or rows).
 * With n the occurrences of t in the history after the prompt and on the
 * row's path, and t seen when it is anywhere in the history or on the path:
 *   seen:  x = x > 0 ? x / repetition : x * repetition   (repetition > 0)
 *   n > 0: x = x - frequency * n - presence
 *   bias;  then x = -inf when t is not allowed
 * in float32, rounded once to dtype.  Tokens outside [0, V) anywhere are
 * skipped.  A disallowed logit is -inf whatever it was (NaN included); a row
 * that allows nothing becomes all -inf (a greedy argmax of 0).  Logits that
 * nothing applies to keep their bits.  In place, rows are read and written back
 * in groups of 8 tokens (4 in float32, counted from token 0), and only the
 * groups that something applies to: nothing else may write to those while the
 * call runs.  tokens may be NULL when R = 1 or no penalty is given. */
int sv_adjust_logits(const void *logits, int64_t seq_stride, void *out, int64_t out_seq_stride, int dtype,
                     const int32_t *tokens, int64_t tokens_stride, const int32_t *parent_host,
                     const int32_t *row_count, int32_t B, int32_t R, int32_t V,
                     const int32_t *history, int64_t history_stride, int32_t history_cap,
                     const int32_t *history_len, const int32_t *prompt_len,
                     const float *repetition, const float *presence, const float *frequency,
                     const int32_t *bias_tokens, const float *bias_values, int32_t n_bias,
                     const uint32_t *allowed, int64_t allowed_seq_stride, int64_t allowed_row_stride,
                     hipStream_t stream);

/* LM head on 4-bit weights with group scales: rows of logits for the verify
 * calls (or for drafting) from hidden states and a quantised unembedding.
 *   logits[m][v] = sum_k hidden[m][k] * scales[v][k / group]
 *                                     * (q[v][k] - zeros[v][k / group])
 *   hidden  [M] rows of hidden_row_stride elements (0 = K), `dtype` SV_DT_BF16
 *           or SV_DT_F16; 16-byte aligned, the stride a multiple of 8.
 *   weights [V][K / 2] bytes: q[v][k] in 0..15, even k in the low half of byte
 *           k / 2; 16-byte aligned.
 *   scales  [V][K / group], of hidden's type.
 *   zeros   [V][K / group] bytes, at most 15, or NULL (= 8).
 *   group   32, 64 or 128; K a multiple of group and of SV_LMHEAD_K_STEP, at
 *           most SV_LMHEAD_MAX_HIDDEN.
 *   out     [M] rows of out_row_stride elements (0 = V), SV_DT_F32 or hidden's
 *           type, not overlapping the inputs.  Dense rows of M = B * (gamma + 1)
 *           are the target_logits of sv_verify_window.
 *   workspace of sv_lmhead_quant_workspace bytes; that is 0 (and NULL will do)
 *           for up to 32 rows (and for sizes outside the rules).
 * Weights enter the products exactly; sums are held in float32 and rounded
 * once.  Hidden values must be finite (an infinite one makes its row NaN).
 * M <= 65535; what a dispatch cannot hold (ceil(V / 128) * ceil(M / 64) >=
 * 2^24, only the largest M and V together) is SV_EINVAL. */
size_t sv_lmhead_quant_workspace(int32_t M, int32_t K, int32_t V, int32_t group);
int sv_lmhead_quant(const void *hidden, int64_t hidden_row_stride, int dtype,
                    const uint8_t *weights, const void *scales, const uint8_t *zeros,
                    int32_t M, int32_t K, int32_t V, int32_t group,
                    void *out, int64_t out_row_stride, int out_dtype,
                    void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Attention of a step's rows: every row of a window or tree over the prefix
 * the whole batch shares, its sequence's cached context and its own ancestors
 * (what produces the hidden states the rows' logits come from).
 *   q        [B][R] rows of q_row_stride elements (0 = Hq * D), each Hq heads
 *            of D; `dtype` SV_DT_BF16 or SV_DT_F16.  D is 64 or 128.  Query
 *            head h reads kv head h / (Hq / Hkv).
 *   k_cache, v_cache  [B] caches cache_seq_stride elements apart (0 = dense),
 *            of cap tokens cache_tok_stride elements apart (0 = Hkv * D), each
 *            Hkv heads of D.  The first ctx_len[b] tokens are committed; the R
 *            rows' own keys and values follow them.
 *   prefix_k, prefix_v  P tokens prefix_tok_stride elements apart (0 = Hkv *
 *            D), seen by every row of every sequence; P = 0: none.
 *   ctx_len  [B] int32 in [0, max_ctx]; max_ctx + R <= cap.  max_ctx only
 *            bounds the lengths: work and results follow the lengths
 *            themselves, and the workspace stops growing with it after some
 *            tens of thousands.  A sequence whose length is outside gets rows
 *            of NaN, and nothing of its cache is read.
 *   row_count  [B] or NULL (= R): rows of each sequence to compute (clamped
 *            to [0, R]); the others of out and lse are left as they were, and
 *            their keys and values are not used.
 *   parent_host  NULL: a window, row i sees rows 0..i (R <= SV_MAX_GAMMA + 1);
 *            else HOST [R], a tree as in sv_verify_tree: a node sees its
 *            ancestors and itself.
 *   out      [B][R][Hq][D], dense; lse [B][R][Hq] float or NULL: the logarithm
 *            of the row's sum of exp(scale * q.k).
 * Scores, softmax statistics and sums are float32; the exponentials enter the
 * second product in dtype.  Keys and values past a sequence's rows do not
 * matter, whatever they hold, nor do those of nodes a row does not see.
 * Strides are multiples of 8 elements, tensors 16-byte aligned; workspace of
 * sv_attention_workspace bytes (0: sizes outside the rules). */
size_t sv_attention_workspace(int32_t B, int32_t R, int32_t Hq, int32_t Hkv, int32_t D, int32_t P, int32_t max_ctx);
int sv_attention(const void *q, int64_t q_row_stride, int dtype,
                 const void *k_cache, const void *v_cache, int64_t cache_seq_stride, int64_t cache_tok_stride, int32_t cap,
                 const void *prefix_k, const void *prefix_v, int64_t prefix_tok_stride, int32_t P,
                 const int32_t *ctx_len, const int32_t *row_count, const int32_t *parent_host,
                 int32_t B, int32_t R, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_ctx, float scale,
                 void *out, float *lse, void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_SV_STEP_H */
