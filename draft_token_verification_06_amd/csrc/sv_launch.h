// Kernel argument blocks and launchers (host-callable, defined in sv_kernels.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "sv_plan.h"

namespace sv {

struct WindowArgs {
  const char *t;
  int64_t t_stride_bytes;
  const char *d;
  int64_t d_stride_bytes;
  const int32_t *tokens;
  const int32_t *window_len;
  int32_t gamma, V, S;
  uint64_t seed, tag;
  const uint64_t *seq_ids;
  const int64_t *base_pos;
  const float2 *part;
  int32_t *n_accepted;
  int32_t *out_tokens;
  float *p_draft, *q_draft;
  SampleJob *jobs;
  int32_t stage_lo;   // early exit: first position of the last block (decided in the draw)
  int32_t *status;    // early exit: per-sequence status
};

struct GreedyArgs {
  const int32_t *tokens;
  const int32_t *window_len;
  int32_t gamma, V, S;
  const float2 *part;
  int32_t *n_accepted;
  int32_t *out_tokens;
};

struct TreeArgs {
  const char *t;
  const char *d;
  int64_t seq_bytes;
  const int32_t *tokens;
  int32_t V, S, R, mode;
  uint64_t seed, tag;
  const uint64_t *seq_ids;
  const int64_t *base_pos;
  const float2 *part;
  int32_t *n_accepted, *best_node, *out_tokens, *out_nodes;
  SampleJob *jobs;
  TreeMeta meta;
};

struct RollbackArgs {
  int32_t *buf_tokens;
  int32_t *buf_len;
  int32_t K, cap;
  const int32_t *verified;
  int64_t verified_stride;
  const int32_t *verified_len;
  int32_t len_offset;
};

// LM-head fused window.  GEMM rows g < M: hidden row g of A (row stride lda
// elements) against every row of W ([V][K], bf16).
struct LmGemmArgs {
  const uint16_t *A;
  int64_t lda;
  const uint16_t *W;
  int32_t M, V, K;
  int32_t RB, NT;             // row blocks, column tiles (set by the launcher)
  float2 *part;               // [M][NT] (max, sum-exp) per row and column tile
  float *gath;                // [M] logit at the row's draft token
  const int32_t *tokens;      // [B][gamma]
  int32_t gamma, rows_per_seq;
  float *out;                 // [M][V] float32 logits
};

struct LmDecideArgs {
  const float2 *stats_t, *stats_d;
  const float *gath_t, *gath_d;
  const int32_t *tokens;
  const int32_t *window_len;
  int32_t gamma, V;
  uint64_t seed, tag;
  const uint64_t *seq_ids;
  const int64_t *base_pos;
  int32_t *n_accepted, *out_tokens;
  float *p_draft, *q_draft;
  SampleJob *jobs;
  const float *rows_t, *rows_d;  // the GEMM's float32 logits, [B][gamma+1][V] / [B][gamma][V]
  int32_t *arrive;               // arrival counters of the draw, zeroed here
};

// Parents of a tree's nodes (entry 0, the root's, unused), as the last part of
// a kernel's arguments.  Window calls leave them out: a launch writes its
// arguments across the bus, at about 2 us a kilobyte.
struct TreeParents {
  uint8_t parent[kTreeMaxNodes];
};
static_assert(kTreeMaxNodes <= 256, "a parent fits a byte");

// Logits adjustment.  Row r of a sequence follows tokens[0 .. r - 1] (window)
// or carries node r of the tree given by parent.
struct AdjustArgs {
  const char *in;
  int64_t in_stride_bytes;
  char *out;
  int64_t out_stride_bytes;
  const int32_t *tokens;  // [B] rows of tokens_stride
  int64_t tokens_stride;
  const int32_t *row_count;
  int32_t R, V;
  const int32_t *history;
  int64_t history_stride;
  const int32_t *history_len, *prompt_len;
  int32_t history_cap, n_bias;
  const float *repetition, *presence, *frequency;
  const int32_t *bias_tokens;
  const float *bias_values;
  const uint32_t *allowed;
  int64_t allowed_seq_stride, allowed_row_stride;  // words
  int32_t chunks;   // token chunks per row; rows split into groups of group_rows (set by the launcher)
  int32_t row_groups, group_rows;
  int32_t in_place; // out is in: only what changes is touched
};
constexpr int kAdjustThreads = 256;
int adjust_chunks(int dtype, int V);
// parents: null for a window.
void launch_adjust_logits(int dtype, AdjustArgs A, const TreeParents *parents, int B, hipStream_t st);

// LM head on 4-bit weights: rows of h (stride lda elements) against w [V][K / 2]
// with scales [V][K / group] of h's type and zeros [V][K / group] or null (8).
struct LmQuantArgs {
  const uint16_t *h;
  int64_t lda;
  const uint8_t *w;
  const uint16_t *scales;
  const uint8_t *zeros;
  int32_t M, V, K, group;
  void *out;  // [M] rows of out_stride, float32 or h's type
  int64_t out_stride;
  int32_t out_f32;
  int32_t row_blocks;  // set by the launcher
  // calls of more than kLmQuantDirectRows rows: the rows laid out, [M][padded], and their groups' sums, [padded / group][M]
  int32_t padded;
  uint16_t *prepared;
  float *sums;
  int32_t splits, split_chunks;  // K shared out among workgroups: shares, chunks of 256 in each
  float *partial;                // [splits][M][V] where there are several
};
constexpr int kLmQuantThreads = 256;
void launch_lm_quant(int dtype, const LmQuantArgs &A, hipStream_t st);

// Attention of a step's rows.  Strides in elements; heads are D apart.  What
// the join of a row's items needs, and the rest.
struct AttendJoin {
  const int32_t *ctx_len, *row_count;
  int32_t B, R, Hq;
  int32_t max_ctx;
  int32_t prefix_parts;
  AttendSplit split;
  float scale_log2;  // magnitude of the score scale, times log2(e)
  float *part_o;     // [parts][B R Hq][D] unnormalised outputs
  float2 *part_ml;   // [parts][B R Hq] (largest product, sum)
  uint16_t *out;     // [B][R][Hq][D]
  float *lse;        // [B][R][Hq] or null
};
struct AttendArgs : AttendJoin {
  const uint16_t *q;
  int64_t q_row_stride;
  const uint16_t *k, *v;  // [B] caches of cap tokens
  int64_t seq_stride, tok_stride;
  const uint16_t *prefix_k, *prefix_v;
  int64_t prefix_tok_stride;
  int32_t Hkv, n;  // n = Hq / Hkv
  int32_t P;
  int32_t prefix_chunk, prefix_items;
  int32_t own_parts, own_tiles;
  int32_t negate;    // the scale is negative
};
void launch_attend(int dtype, int D, const AttendArgs &A, const TreeParents *parents, const AttendPlan &P, hipStream_t st);

// Launches the GEMMs of two problems (target rows, draft rows) as one grid.
void launch_lm_gemm(LmGemmArgs A0, LmGemmArgs A1, hipStream_t st);
int64_t lm_gemm_blocks(int64_t M, int V);
void launch_lm_combine(const float2 *part, int NT, int M, float2 *stats, hipStream_t st);
void launch_lm_decide(const LmDecideArgs &A, int B, hipStream_t st);

// Workspace of the split draw (several workgroups per sequence): chunk sums
// spart [B][cmax] and one arrival counter per sequence, which the launch
// before the draw zeroes.
struct DrawScratch {
  float *spart;
  int cmax;
  int32_t *arrive;
};

void launch_window_finish(int dtype, const WindowArgs &A, int B, const DrawScratch &ds, hipStream_t st);
void launch_stage_decide(int dtype, const WindowArgs &A, int B, int lo, int hi, int32_t *status, hipStream_t st);
void launch_stage_finish(int dtype, const WindowArgs &A, int B, const DrawScratch &ds, hipStream_t st);
void launch_greedy_decide(const GreedyArgs &A, int B, hipStream_t st);
void launch_tree_decide(int dtype, const TreeArgs &A, int B, hipStream_t st);
void launch_tree_finish(int dtype, SampleJob *jobs, int B, int V, const DrawScratch &ds, hipStream_t st);
// Stochastic tree: the draw kernels decide each sequence themselves (no separate decision launch).
void launch_tree_decide_draw(int dtype, const TreeArgs &A, int B, const DrawScratch &ds, hipStream_t st);
void launch_tree_walk(int dtype, const TreeArgs &A, int B, hipStream_t st);
void launch_rollback(const RollbackArgs &A, int S, int stage, hipStream_t st);

}  // namespace sv
