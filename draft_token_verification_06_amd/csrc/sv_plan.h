// Launch plan and workspace layout shared by the C-ABI layer and the kernels.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "sv_rowset.h"

namespace sv {

#ifndef SV_FIN_THREADS
#define SV_FIN_THREADS 1024
#endif
#ifndef SV_FIN_BATCH
#define SV_FIN_BATCH 2
#endif
constexpr int kFinThreads = SV_FIN_THREADS;  // sampling workgroup (one per sequence)
constexpr int kFinWaves = kFinThreads / 64;
constexpr int kFinBatch = SV_FIN_BATCH;      // chunks per pipelined batch
constexpr int kMaxVocab = 1 << 21;    // 2,097,152 tokens
// Chunks of a sampling pass: at most ceil((V + 3) / (4 kFinThreads)) (four
// slots per thread and up to 3 slots of head offset); 513 at 1024 threads.
constexpr int fin_chunks_max(int V) { return (V + 3 + kFinThreads * 4 - 1) / (kFinThreads * 4); }
constexpr int kFinMaxChunks = fin_chunks_max(kMaxVocab);
constexpr int kFinFillWorkgroups = 256;  // draw workgroups wanted per launch
constexpr int kMaxSegments = 64;      // row segments (split-row mode)
constexpr int64_t kFillWorkgroups = 16384;  // row workgroups per launch (256 CUs)
// A row splits into at most ceil(V / kMinSegment) segments: shorter segments
// leave each workgroup too few loads to cover its start-up and reduction.
constexpr int kMinSegment = 32768;

// Work item of the sampling pass of one sequence: draw from
//   w_k = p_k                       (BONUS)
//   w_k = max(0, p_k - cq * q_k)    (RESIDUAL; cq = 1 for a window or a node's
//                                    first residual, larger after several
//                                    rejected siblings)
// with p_k = 2^(t_k log2e - ct), q_k = 2^(d_k log2e - cd); the offsets carry
// the row maximum and the log of the row's normaliser.
enum : int { JOB_NONE = 0, JOB_BONUS = 1, JOB_RESIDUAL = 2 };

struct SampleJob {
  const void *t_row;
  const void *d_row;
  int32_t *out_slot;  // where the drawn token is stored
  float ct, cd;
  float v;            // sampling uniform
  int32_t mode;
  float cq;           // coefficient of q in the residual (>= 1)
  int32_t pad[5];
};
static_assert(sizeof(SampleJob) == 64, "SampleJob is one 64-byte record");

// Tree shape handed to the tree kernels by value.
constexpr int kTreeMaxDepth = 64;
struct TreeMeta {
  int32_t N;
  int32_t max_depth;
  uint64_t internal[kTreeMaxNodes / 64];  // bit v: node v has children
  int16_t parent[kTreeMaxNodes];
  int16_t rank[kTreeMaxNodes];
  int16_t first_child[kTreeMaxNodes];     // smallest child index, or -1
  int16_t next_sibling[kTreeMaxNodes];    // next larger index with the same parent, or -1
  uint8_t depth[kTreeMaxNodes];
};
static_assert(sizeof(TreeMeta) <= 2560, "tree metadata travels in the kernel arguments");

// LM-head fused path: vocabulary columns per GEMM block tile, threads per
// GEMM workgroup.
constexpr int kLmBN = 256;
constexpr int kLmGemmThreads = 512;

// A dispatch packet gives each grid dimension's size in work-items as a 32-bit
// count, so a launch of `blocks` workgroups of `threads` along one dimension
// must stay within it; the entry points reject calls whose grids would not.
constexpr int64_t kMaxGridItems = 0xFFFFFFFFll;
constexpr int64_t kMaxGridY = 65535;  // workgroups along a second dimension
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks >= 1 && blocks <= kMaxGridItems / threads; }

struct RowPlan {
  int S;        // segments per row
  int seg_len;  // elements per segment (multiple of 8)
};

inline RowPlan plan_rows(int64_t rows_total, int32_t V) {
  int64_t S = 1;
  if (rows_total < kFillWorkgroups) S = (kFillWorkgroups + rows_total - 1) / rows_total;
  int64_t cap = (V + kMinSegment - 1) / kMinSegment;
  if (cap < 1) cap = 1;
  if (S > cap) S = cap;
  if (S > kMaxSegments) S = kMaxSegments;
  int64_t seg = (V + S - 1) / S;
  seg = (seg + 7) / 8 * 8;
  S = (V + seg - 1) / seg;
  return {static_cast<int>(S), static_cast<int>(seg)};
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace sections (byte offsets); rows_per_seq counts target + draft rows.
struct Layout {
  RowPlan plan;
  int rows_per_seq;
  int cmax;  // chunk sums per sequence in the split draw
  size_t part_off, jobs_off, spart_off, status_off, arrive_off, total;
};

// op: 0 window, 1 greedy, 2 tree (n = gamma or N).
inline Layout make_layout(int op, int64_t B, int32_t n, int32_t V) {
  Layout L{};
  if (op == 0) L.rows_per_seq = 2 * n + 1;
  else if (op == 1) L.rows_per_seq = n + 1;
  else L.rows_per_seq = 2 * n;
  L.plan = plan_rows(B * L.rows_per_seq, V);
  size_t off = 0;
  L.part_off = off;
  off = align256(off + sizeof(float) * 2 * static_cast<size_t>(B) * L.rows_per_seq * L.plan.S);
  L.jobs_off = off;
  off = align256(off + (op == 1 ? 0 : sizeof(SampleJob) * static_cast<size_t>(B)));
  L.cmax = (op == 1) ? 0 : fin_chunks_max(V);
  L.spart_off = off;
  off = align256(off + sizeof(float) * static_cast<size_t>(B) * L.cmax);
  L.status_off = off;  // early-exit window: per-sequence status
  off = align256(off + (op == 0 ? sizeof(int32_t) * static_cast<size_t>(B) : 0));
  L.arrive_off = off;  // split draw: per-sequence arrival counter
  off = align256(off + (op == 1 ? 0 : sizeof(int32_t) * static_cast<size_t>(B)));
  L.total = off;
  return L;
}

// Workspace of the LM-head fused window (byte offsets).  Rows: B(gamma+1)
// target rows then B gamma draft rows.
struct LmLayout {
  int NT;  // column tiles
  int cmax;
  size_t part_off, stats_off, gath_off, jobs_off, spart_off, arrive_off, rows_t_off, rows_d_off, total;
};

inline LmLayout make_lm_layout(int64_t B, int32_t gamma, int32_t V) {
  LmLayout L{};
  const int64_t Mt = B * (gamma + 1), Md = B * gamma, M = Mt + Md;
  L.NT = (V + kLmBN - 1) / kLmBN;
  L.cmax = fin_chunks_max(V);
  size_t off = 0;
  L.part_off = off;
  off = align256(off + sizeof(float) * 2 * static_cast<size_t>(M) * L.NT);
  L.stats_off = off;
  off = align256(off + sizeof(float) * 2 * static_cast<size_t>(M));
  L.gath_off = off;
  off = align256(off + sizeof(float) * static_cast<size_t>(M));
  L.jobs_off = off;
  off = align256(off + sizeof(SampleJob) * static_cast<size_t>(B));
  L.spart_off = off;
  off = align256(off + sizeof(float) * static_cast<size_t>(B) * L.cmax);
  L.arrive_off = off;
  off = align256(off + sizeof(int32_t) * static_cast<size_t>(B));
  L.rows_t_off = off;
  off = align256(off + sizeof(float) * static_cast<size_t>(Mt) * V);
  L.rows_d_off = off;
  off = align256(off + sizeof(float) * static_cast<size_t>(Md) * V);
  L.total = off;
  return L;
}

// 4-bit LM head: the narrowest tile of a workgroup, and the workspace of a call
// with more rows than its workgroups lay out themselves (K padded to a chunk).
constexpr int kLmQuantMinCols = 16;
constexpr int kLmQuantDirectRows = 32;
constexpr int kLmQuantCols = 128;       // columns of a workgroup with more rows than that
constexpr int64_t kLmQuantSlots = 512;  // of those run at once: 2 on each of 256 CUs
// Rows of a workgroup: blocks of 64 or 80, whichever pads less.
inline int lm_quant_rows(int64_t M) { return (M + 63) / 64 * 64 <= (M + 79) / 80 * 80 ? 64 : 80; }
// Workgroups of a launch along its first dimension, at most: all rows in one
// row block up to kLmQuantDirectRows, and column tiles in eights.
inline int64_t lm_quant_blocks(int64_t M, int64_t V) {
  const int64_t cols = M <= kLmQuantDirectRows ? kLmQuantMinCols : kLmQuantCols;
  const int64_t rows = M <= kLmQuantDirectRows ? kLmQuantDirectRows : lm_quant_rows(M);
  return ((V + cols - 1) / cols + 7) / 8 * 8 * ((M + rows - 1) / rows);
}
struct LmQuantLayout {
  int32_t padded, splits, split_chunks;
  size_t sums_off, partial_off, total;
};
inline LmQuantLayout lm_quant_layout(int64_t M, int32_t K, int32_t V, int32_t group) {
  LmQuantLayout L{};
  L.splits = 1;
  if (M <= kLmQuantDirectRows) return L;
  const int chunks = (K + 255) / 256;
  L.padded = chunks * 256;
  // Few tiles leave most of the chip idle for as long as K is: K is then shared
  // out too, two chunks at least to a workgroup.
  const int64_t rows = lm_quant_rows(M);
  const int64_t tiles = (static_cast<int64_t>(V) + kLmQuantCols - 1) / kLmQuantCols * ((M + rows - 1) / rows);
  int64_t splits = (kLmQuantSlots + tiles - 1) / tiles;
  if (splits > (chunks + 1) / 2) splits = (chunks + 1) / 2;
  if (splits > 8) splits = 8;
  if (4 * tiles > 3 * kLmQuantSlots) splits = 1;
  L.split_chunks = static_cast<int32_t>((chunks + splits - 1) / splits);
  L.splits = (chunks + L.split_chunks - 1) / L.split_chunks;
  L.sums_off = align256(static_cast<size_t>(M) * L.padded * 2);
  L.partial_off = align256(L.sums_off + static_cast<size_t>(M) * (L.padded / group) * sizeof(float));
  L.total = L.partial_off + (L.splits > 1 ? align256(static_cast<size_t>(L.splits) * M * V * sizeof(float)) : 0);
  return L;
}

// Work items of an attention call.  Stacked rows (query rows times the heads of
// a group) come in tiles of 32, 64 or 128, on 1, 2 or 4 of a workgroup's waves
// (the others share a tile's keys); keys are split into ranges until the items
// fill the chip.
constexpr int kAttendThreads = 256;
constexpr int kAttendWideRows = 64;        // more stacked rows than this: tiles of 128
constexpr int64_t kAttendSlots = 512;      // workgroups that run at once: 2 on each of 256 CUs
constexpr int kAttendMinKeys = 128;        // keys per range at least (a tile)
// A sequence's own keys (context and live rows) are split by their number
// alone, so that neither the ranges nor the results follow the capacity of the
// cache: lengths up to 128, 256, 512 .. each have their range, in tiles of 128
// keys (16 bits: no division in the kernel).
constexpr int kAttendBuckets = 19;  // 128 << 18 holds the longest
struct AttendSplit {
  uint64_t tiles[5];
};
constexpr int attend_bucket(int keys) { return keys <= 128 ? 0 : 32 - __builtin_clz(static_cast<unsigned>(keys - 1) >> 7); }
// Keys per range of a sequence with `keys` of its own.
constexpr int attend_own_range(const AttendSplit &S, int keys) {
  const int j = attend_bucket(keys);
  const uint64_t word = j < 8 ? (j < 4 ? S.tiles[0] : S.tiles[1]) : j < 12 ? S.tiles[2] : j < 16 ? S.tiles[3] : S.tiles[4];
  return static_cast<int>(word >> (16 * (j & 3)) & 0xFFFF) * 128;
}
struct AttendPlan {
  int prefix_waves, own_waves;  // waves along the rows
  int prefix_parts, prefix_chunk, own_parts, own_tiles;  // own_parts: most ranges of a sequence
  AttendSplit split;
  int64_t prefix_items, own_blocks;
  size_t ml_off, total;
};

// Keys of a range when `keys` are split into `parts`: whole tiles.
inline int64_t attend_range(int64_t keys, int64_t parts) { return ((keys + parts - 1) / parts + 127) / 128 * 128; }

// Ranges of `keys` keys for `items` items of `rows` rows each: the number that
// ends first when rounds of kAttendSlots items take turns.  An item costs its
// keys, a tile's start and end, and its partial output, written and read
// again: two keys' bytes per row; a round that fills half of the slots at most,
// one item per CU, takes 13 twentieths of a full one (8 windows of 9 rows over
// 4000 keys: 4 ranges 32 us, 8 ranges 35).  Every range costs the join of a row
// two trips to memory after each other, 0.75 us or some 64 keys (one token of 32
// heads over 4000 keys: 32 ranges 27 us, 7 ranges 19, 2 ranges 32; with 42 keys 64
// windows behind 16384 tokens get 7 ranges for 3, 239 us for 223).  Where
// there is work for many rounds already (crowded), ranges of about 1024 keys
// keep the items even; longer sequences then have longer ranges, 16 of them or
// what fills the chip once, so that partial outputs do not follow the length.
inline int attend_parts(int64_t keys, int64_t items, int64_t rows, bool crowded, int64_t slots = kAttendSlots, int64_t join = 64) {
  if (crowded) {
    const int64_t fill = (slots + items - 1) / items, cap = fill > 16 ? fill : 16;
    const int64_t p = (keys + 1023) / 1024;
    return static_cast<int>(p < cap ? p : cap);
  }
  int64_t most = (keys + kAttendMinKeys - 1) / kAttendMinKeys, best = -1;
  if (most > 256) most = 256;
  int parts = 1;
  for (int64_t p = 1, step = 1; p <= most; p += step) {
    if (p == 8 * step) step *= 2;  // eight candidates, then four per doubling
    const int64_t last = items * p % slots;
    const int64_t rounds = items * p / slots * 20 + (last == 0 ? 0 : last <= slots / 2 ? 13 : 20);
    const int64_t cost = rounds * (attend_range(keys, p) + kAttendMinKeys + 2 * rows) + 20 * join * p;
    if (best < 0 || cost < best) {
      best = cost;
      parts = static_cast<int>(p);
    }
  }
  return parts;
}

inline AttendPlan plan_attention(int64_t B, int64_t R, int64_t Hq, int64_t Hkv, int D, int64_t P, int64_t max_ctx) {
  AttendPlan L{};
  const int64_t n = Hq / Hkv;
  const int64_t all = B * R * n, own = R * n;
  L.prefix_waves = all > kAttendWideRows ? 4 : 1;
  L.own_waves = own > kAttendWideRows ? 4 : own > 32 ? 2 : 1;
  const int64_t prefix_rows = 32 * L.prefix_waves, own_rows = 32 * L.own_waves;
  const int64_t tiles = (all + prefix_rows - 1) / prefix_rows;
  L.own_tiles = static_cast<int>((own + own_rows - 1) / own_rows);
  const int64_t own_items = B * Hkv * L.own_tiles;
  const int longest = attend_bucket(static_cast<int>(max_ctx + R));
  for (int j = 0; j <= longest; ++j) {
    const int64_t keys = int64_t{128} << j;
    const bool crowded = own_items * ((keys + 1023) / 1024) >= 4 * kAttendSlots;
    const int64_t range = attend_range(keys, attend_parts(keys, own_items, own < own_rows ? own : own_rows, crowded));
    L.split.tiles[j / 4] |= static_cast<uint64_t>(range / 128) << (16 * (j % 4));  // (crowded: 1024 keys or a 16th at most; else below 2^21 keys)
    const int parts = static_cast<int>((keys + range - 1) / range);
    if (parts > L.own_parts) L.own_parts = parts;
  }
  L.prefix_chunk = 1;
  if (P > 0) {
    // The prefix's items run beside the sequences' own; whatever their lengths,
    // those alone are two rounds where there are as many.
    const bool crowded = own_items >= 2 * kAttendSlots;
    L.prefix_chunk = static_cast<int>(attend_range(P, attend_parts(P, tiles * Hkv, all < prefix_rows ? all : prefix_rows, crowded)));
    L.prefix_parts = static_cast<int>((P + L.prefix_chunk - 1) / L.prefix_chunk);
    L.prefix_items = tiles * Hkv * L.prefix_parts;
  }
  L.own_blocks = (B * L.own_parts + 7) / 8 * 8 * Hkv * L.own_tiles;
  const size_t slots = static_cast<size_t>(L.prefix_parts + L.own_parts) * static_cast<size_t>(B * R * Hq);
  L.ml_off = align256(slots * static_cast<size_t>(D) * sizeof(float));
  L.total = align256(L.ml_off + slots * 2 * sizeof(float));
  return L;
}

// Attention over pages.  The rows of a sequence (times the heads of a group)
// choose the kernel: up to 16, 32 or 48 of them stay one tile (few), more go by
// tiles of 64 or 128 as above.  Tiles of 16 rows hold half of the registers: four
// workgroups on a CU, but for 16-bit heads of 128 (71 KB of LDS) and behind a
// batch's prefix (the registers of its tiles of 128 rows; with heads of 64 three
// are counted as two), two.  With two counted as such 64 windows of 4 rows over
// 300 keys, 16-bit, take 19 us for 31, 64 of them behind 4096 keys, 8-bit, 46 for
// 58; over 215 batches, lengths and prefixes the mean is 1.8% less (the worst 15%
// more: 64 single tokens over 1500 keys behind 8192).  Ranges of 1024 keys
// (crowded) begin at 4096 items for these tiles, however many run at once, as
// sequences of one range write their outputs themselves: 128 single tokens over
// 2000 keys, 16-bit, 161 us, from 2048 items on 170.  The join of pages reads 8
// ranges at a time, so that a range of a sequence costs it less (16 keys; a
// prefix's as above, where every row of the batch writes and reads one: 132 us
// with 2 of them, 138 with 8).
constexpr int64_t kPagedFewSlots = 1024;
constexpr int64_t kPagedJoin = 16;
// Most rows of a few.  (16-bit pages, 36 to 48 rows as 48 and as tiles of 64: heads
// of 128, which spill at 48, 64 windows of 9 rows over 300 keys 38 us for 32, one
// over 1000 17.7 for 13.3; heads of 64 one 12.6 for 11.1, 64 behind 2048 keys 44 for
// 40, but 64 without a prefix 16 for 24.)
constexpr int paged_few_rows(bool f8) { return f8 ? 48 : 32; }
struct PagedPlan : AttendPlan {
  int few;
  bool direct;  // a sequence of one range needs no partial outputs
};

inline PagedPlan plan_paged(int64_t B, int64_t R, int64_t Hq, int64_t Hkv, int D, int64_t P, int64_t max_ctx, bool f8) {
  PagedPlan L{};
  const int64_t n = Hq / Hkv, all = B * R * n, own = R * n;
  L.few = own <= 16 ? 16 : own <= 32 ? 32 : own <= paged_few_rows(f8) ? 48 : 0;
  L.direct = L.few > 0 && P == 0;
  L.own_waves = own > kAttendWideRows ? 4 : own > 32 ? 2 : 1;
  L.prefix_waves = all > kAttendWideRows ? 4 : 1;
  const int64_t own_rows = L.few > 0 ? L.few : 32 * L.own_waves;
  const int64_t prefix_rows = L.prefix_waves == 4 ? 128 : L.few > 0 ? L.few : 32;
  const int64_t tiles = (all + prefix_rows - 1) / prefix_rows;
  const bool batch_prefix = P > 0 && L.prefix_waves == 4;
  const int64_t slots = L.few == 16 && !batch_prefix && (f8 || D == 64) ? kPagedFewSlots : kAttendSlots;
  L.own_tiles = static_cast<int>((own + own_rows - 1) / own_rows);
  const int64_t own_items = B * Hkv * L.own_tiles;
  const int longest = attend_bucket(static_cast<int>(max_ctx + R));
  for (int j = 0; j <= longest; ++j) {
    const int64_t keys = int64_t{128} << j;
    const bool crowded = own_items * ((keys + 1023) / 1024) >= 4 * (L.few == 16 ? kPagedFewSlots : kAttendSlots);
    int64_t parts = attend_parts(keys, own_items, own < own_rows ? own : own_rows, crowded, slots, kPagedJoin);
    const int64_t range = attend_range(keys, parts);
    L.split.tiles[j / 4] |= static_cast<uint64_t>(range / 128) << (16 * (j % 4));
    parts = (keys + range - 1) / range;
    if (parts > L.own_parts) L.own_parts = static_cast<int>(parts);
  }
  L.prefix_chunk = 1;
  if (P > 0) {
    const bool crowded = own_items >= 2 * slots;
    L.prefix_chunk = static_cast<int>(attend_range(P, attend_parts(P, tiles * Hkv, all < prefix_rows ? all : prefix_rows, crowded, slots)));
    L.prefix_parts = static_cast<int>((P + L.prefix_chunk - 1) / L.prefix_chunk);
    L.prefix_items = tiles * Hkv * L.prefix_parts;
  }
  L.own_blocks = (B * L.own_parts + 7) / 8 * 8 * Hkv * L.own_tiles;
  const size_t parts = static_cast<size_t>(L.prefix_parts + L.own_parts) * static_cast<size_t>(B * R * Hq);
  L.ml_off = align256(parts * static_cast<size_t>(D) * sizeof(float));
  L.total = align256(L.ml_off + parts * 2 * sizeof(float));
  return L;
}

}  // namespace sv
