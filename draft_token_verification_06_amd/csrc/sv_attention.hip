// Attention of a step's rows (gfx950): the rows of a window or tree over the
// batch's shared prefix, their sequence's cached context and their own
// ancestors.
//
// The keys of a row are split among work items: the prefix into ranges that
// all rows of a kv head share (so its keys and values are read once per tile
// of rows of the whole batch, not once per sequence), and each sequence's
// cache, the step's own keys at its end, into ranges by its length.  An
// item runs one pass over its range with a running maximum and sum and leaves
// an unnormalised float32 output with (maximum, sum); k_attend_combine joins
// the items of a row in a fixed order.
//
// Matrix layout (v_mfma_f32_32x32x16): scores are formed transposed, S^T = K
// Q^T, so that a lane holds 16 keys of one row (column l % 32; keys 8 (r / 4) +
// 4 (l / 32) + r % 4): maxima and sums stay in the lane up to one exchange with
// lane l ^ 32, and the exponentials are already the operand of O^T = V^T P^T,
// whose k order may be any as long as both operands share it.  V^T is read
// from row-major LDS by the transposing LDS read (each 16 lanes take a 4 x 16
// block and get its columns).
//
// Rows of a group of query heads that share a kv head are stacked into one
// tile.  A workgroup's four waves split the tile's rows (WQ = 4: 128 rows, for
// the prefix of a batch), the keys of a tile (WQ = 1: 32 rows, for the few rows
// of one sequence, where cache bandwidth is the bound), or both (WQ = 2: 64).
// Two workgroups share a CU: 220 registers per lane, up to 81 KB of LDS.
//
// Measured (bf16, 32 query heads on 8 kv heads of 128):
// - 128 single tokens over own caches of 1000 to 4000 tokens and a prefix of
//   2048 (1.34 GB): 229 us + 7 us for the join, 5.7 TB/s.  Bound: memory and the
//   start and end of each range; ranges of 512 to 2048 keys differ by 5%.
// - 64 windows of 9 rows, prefix 8192, own caches of 256 to 1024 (84 GFLOP):
//   122 + 13 us, 620 TFLOP/s.  Bound: the loads and their way through LDS (108 us
//   alone when the whole took 150), then the vector work of the exponentials.
// - one token over 333 + 700 keys: 9 + 4 us; bound: two launches, the trips to
//   memory of one range, and those of the join, two for each range in turn.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_attend.h"

namespace sv {

// What one work item computes: rows [row0, row0 + rows) of a stack of rows
// (stack row i is query row base_row + i / n, head kvh n + i % n) over keys
// [k0, k1) at k / v; keys from `draft` on are the step's own and follow the
// ancestor sets (s_anc), the others are seen by every row.
struct Item {
  const uint16_t *k, *v;
  int64_t tok_stride;
  int64_t base_row;  // query row (b * R + r) of stack row 0
  int row0, rows;
  int kvh;
  int k0, k1, draft;
  int part;
};

// LDS rows in elements.  The 128 bytes that one cycle serves are 8 lanes of 16
// bytes in consecutive key rows (16 bytes of padding put them side by side),
// or the 4 value rows of 32 bytes of a transposing read (32 bytes of padding).
template <int D> constexpr int at_key_row() { return D + 8; }
template <int D> constexpr int at_value_row() { return D + 16; }
template <int D, int WQ> constexpr int at_tile_keys() { return WQ == 1 ? 128 : 64; }
template <int D, int WQ> constexpr size_t at_tile_bytes() {
  const size_t kv = static_cast<size_t>(at_tile_keys<D, WQ>()) * (at_key_row<D>() + at_value_row<D>()) * 2;
  const size_t merge = WQ < 4 ? 4 * 32 * static_cast<size_t>(D + 4) * 4 : 0;
  return kv > merge ? kv : merge;
}

// a (values d .. d + 3 of a row with ancestor set anc) plus the infinities and
// NaN among the row's own keys' values.
template <int DT> __device__ float4 add_odd(const Item &it, const uint32_t *anc, int d, float4 a) {
  for (int key = max(it.k0, it.draft); key < it.k1; ++key) {
    const int own = key - it.draft;
    if (!((anc[own >> 5] >> (own & 31)) & 1)) continue;
    const uint2 w = *reinterpret_cast<const uint2 *>(it.v + key * it.tok_stride + d);
    const uint32_t b[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
    float *x = &a.x;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((b[k] & AtElt<DT>::kExp) == AtElt<DT>::kExp) x[k] += Elt<DT>::dec(b[k]);
  }
  return a;
}

template <int DT, int D, int WQ>
__device__ __forceinline__ void attend_item(const AttendArgs &A, const Item &it, char *lds, const uint32_t (*s_anc)[8],
                                            float2 *s_ml) {
  using T = AtElt<DT>;
  constexpr int WK = 4 / WQ;
  constexpr int KT = at_tile_keys<D, WQ>();
  constexpr int SB = KT / (32 * WK);      // 32-key blocks per wave and tile
  constexpr int kRow = at_key_row<D>(), kVRow = at_value_row<D>();
  constexpr int kChunks = D / 8;          // 16-byte pieces per row
  constexpr int kLoads = KT * kChunks / kAtThreads;
  uint16_t *s_k = reinterpret_cast<uint16_t *>(lds);
  uint16_t *s_v = s_k + KT * kRow;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wq = wave % WQ, wk = wave / WQ;
  const int q32 = lane & 31, half = lane >> 5;

  // this lane's row, its query fragments: d = 16 s + 8 half ..
  const int i = it.row0 + wq * 32 + q32;
  const int ic = min(i, it.rows - 1);
  const int64_t qrow = it.base_row + ic / A.n;
  const int head = it.kvh * A.n + ic % A.n;
  uint4 qf[D / 16];
  {
    const uint16_t *p = A.q + qrow * A.q_row_stride + head * D + half * 8;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      qf[s] = load_vec(p + s * 16);
      // a negative scale acts on the queries' signs, so that larger products are larger scores
      if (A.negate) qf[s] = make_uint4(qf[s].x ^ 0x80008000u, qf[s].y ^ 0x80008000u, qf[s].z ^ 0x80008000u, qf[s].w ^ 0x80008000u);
    }
  }
  const int r = static_cast<int>(qrow % A.R);

  at_f32x16_t o[D / 32];
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[t][e] = 0.0f;
  float m = kNegInf, l = 0.0f;  // l: this half's keys only

  uint4 rk[kLoads], rv[kLoads];
  // WQ = 1: every wave fills its own 32 keys of the tile and reads only those,
  // so the waves run apart until the end; else the workgroup fills the tile.
  constexpr bool kApart = WQ == 1;
  constexpr int kRowsPerPass = (kApart ? 64 : kAtThreads) / kChunks;
  const int piece = tid % kChunks, first = kApart ? wave * 32 + lane / kChunks : tid / kChunks;
  // one sequence's cache is read once: streamed
  auto fetch = [&](const uint16_t *p) { return kApart ? load_stream(reinterpret_cast<const uint4 *>(p)) : load_vec(p); };
  const bool near = it.tok_stride < (1 << 22);  // a tile's offsets fit 32 bits
  const uint32_t lane_off = static_cast<uint32_t>(first) * static_cast<uint32_t>(it.tok_stride) + piece * 8;
  auto load = [&](int t0) {
    if (near && t0 + KT <= it.k1) {
      // whole tiles: one offset per lane, everything else scalar
      const uint16_t *pk = it.k + t0 * it.tok_stride, *pv = it.v + t0 * it.tok_stride;
      const int64_t pass = kRowsPerPass * it.tok_stride;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        rk[j] = fetch(pk + j * pass + lane_off);
        rv[j] = fetch(pv + j * pass + lane_off);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int64_t key = min(t0 + first + j * kRowsPerPass, it.k1 - 1);
        rk[j] = fetch(it.k + key * it.tok_stride + piece * 8);
        rv[j] = fetch(it.v + key * it.tok_stride + piece * 8);
      }
    }
  };
  auto tile_barrier = [&]() {
    if (kApart) __builtin_amdgcn_wave_barrier();
    else __syncthreads();
  };
  bool odd = false;
  load(it.k0);
  for (int t0 = it.k0; t0 < it.k1; t0 += KT) {
    // Keys past the range get zero values: their exponentials are zero, but
    // zero times what a cache holds behind its end need not be.
    // Infinities and NaN among the step's own values, which must reach only the
    // rows that see them, are left out here and added at the end.
    const bool masked = t0 + KT > it.draft;
    tile_barrier();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int row = first + j * kRowsPerPass;
      uint4 v = rv[j];
      if (t0 + KT > it.k1 && t0 + row >= it.k1) v = make_uint4(0, 0, 0, 0);
      if (masked && t0 + row >= it.draft && t0 + row < it.k1) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if ((w[k] & T::kExp) == T::kExp) w[k] &= 0xFFFF0000u, odd = true;
          if (((w[k] >> 16) & T::kExp) == T::kExp) w[k] &= 0xFFFFu, odd = true;
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4 *>(s_k + row * kRow + piece * 8) = rk[j];
      *reinterpret_cast<uint4 *>(s_v + row * kVRow + piece * 8) = v;
    }
    tile_barrier();
    if (t0 + KT < it.k1) load(t0 + KT);
    if (t0 + wk * SB * 32 >= it.k1) continue;  // nothing of this tile for this wave
    // raw products of the wave's blocks of 32 keys
    at_f32x16_t s[SB];
#pragma unroll
    for (int sb = 0; sb < SB; ++sb) {
#pragma unroll
      for (int e = 0; e < 16; ++e) s[sb][e] = 0.0f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
        s[sb] = T::mma(*reinterpret_cast<const uint4 *>(s_k + ((wk * SB + sb) * 32 + q32) * kRow + d * 16 + half * 8), qf[d], s[sb]);
    }
    if (masked || t0 + KT > it.k1) {
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int key = t0 + (wk * SB + sb) * 32 + 8 * (e >> 2) + 4 * half + (e & 3);
          const int own = key - it.draft;
          const bool ok = key < it.k1 && (own < 0 || ((s_anc[r][(own & 255) >> 5] >> (own & 31)) & 1));
          s[sb][e] = ok ? s[sb][e] : kNegInf;
        }
    }
    float top = kNegInf;
#pragma unroll
    for (int sb = 0; sb < SB; ++sb)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[sb][e]);
    const float2 tops = both_halves(top);
    const float mn = fmaxf(m, fmaxf(tops.x, tops.y));
    // Outputs are rescaled only when some row's maximum rose: 1 is exact.
    if (__any(mn > m)) {
      const float alpha = m == kNegInf ? 0.0f : exp2_fast((m - mn) * A.scale_log2);
      l *= alpha;
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[t][e] *= alpha;
      m = mn;
    }
    // The lifted exponent is taken from the difference to the maximum, so that
    // the largest is 2^15 exactly however far the scores are (65504 ends the
    // type); unlifted, one multiply-add does.
    const float top_s = m == kNegInf ? 0.0f : m, mu = top_s * A.scale_log2;
    float sum = 0.0f;
#pragma unroll
    for (int sb = 0; sb < SB; ++sb)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[sb][e] = exp2_fast(T::kLift > 0 ? __builtin_fmaf(s[sb][e] - top_s, A.scale_log2, T::kLift)
                                          : __builtin_fmaf(s[sb][e], A.scale_log2, -mu));
        sum += s[sb][e];
      }
    l += sum;
#pragma unroll
    for (int sb = 0; sb < SB; ++sb) {
      const int kb = (wk * SB + sb) * 32;  // this block's first key in the tile
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const uint4 p = make_uint4(T::pack(s[sb][8 * ks], s[sb][8 * ks + 1]), T::pack(s[sb][8 * ks + 2], s[sb][8 * ks + 3]),
                                   T::pack(s[sb][8 * ks + 4], s[sb][8 * ks + 5]), T::pack(s[sb][8 * ks + 6], s[sb][8 * ks + 7]));
        // lane l: block of 4 keys x 16 values; its address is row (l % 16) / 4, values 4 (l % 4)
        const uint16_t *base = s_v + (kb + ks * 16 + 4 * half + ((lane & 15) >> 2)) * kVRow + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
#pragma unroll
        for (int t = 0; t < D / 32; ++t) {
          const at_i16x4_t a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(base + t * 32));
          const at_i16x4_t a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(base + t * 32 + 8 * kVRow));
          const uint2 u0 = __builtin_bit_cast(uint2, a0), u1 = __builtin_bit_cast(uint2, a1);
          o[t] = T::mma(make_uint4(u0.x, u0.y, u1.x, u1.y), p, o[t]);
        }
      }
    }
  }
  // (also: every wave is done with the tiles)
  const bool any_odd = it.k1 > it.draft ? __syncthreads_or(odd) : (__syncthreads(), false);
  const float2 ls = both_halves(l);
  l = ls.x + ls.y;

  const int64_t rows_all = static_cast<int64_t>(A.B) * A.R * A.Hq;
  if (WQ == 4) {
    if (i < it.rows) {
      const int64_t at = it.part * rows_all + qrow * A.Hq + head;
      float *po = A.part_o + at * D;
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          float4 a = make_float4(o[t][4 * f], o[t][4 * f + 1], o[t][4 * f + 2], o[t][4 * f + 3]);
          const int d = t * 32 + 8 * f + 4 * half;
          if (any_odd) a = add_odd<DT>(it, s_anc[r], d, a);
          *reinterpret_cast<float4 *>(po + d) = a;
        }
      if (half == 0) A.part_ml[at] = make_float2(m, l);
    }
    return;
  }
  // WK waves hold the same rows over different keys: joined in wave order.
  constexpr int kRows = 32 * WQ;
  float *s_o = reinterpret_cast<float *>(lds);
  const int row = wq * 32 + q32;
  const int live = min(kRows, it.rows - it.row0);
  if (half == 0) s_ml[wk * kRows + row] = make_float2(m, l);
  __syncthreads();
  float M = kNegInf;
#pragma unroll
  for (int w = 0; w < WK; ++w) M = fmaxf(M, s_ml[w * kRows + row].x);
  const float f = m == kNegInf ? 0.0f : exp2_fast((m - M) * A.scale_log2);
  if (row < live)
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4 *>(s_o + (wk * kRows + row) * (D + 4) + t * 32 + 8 * g + 4 * half) =
          make_float4(o[t][4 * g] * f, o[t][4 * g + 1] * f, o[t][4 * g + 2] * f, o[t][4 * g + 3] * f);
  __syncthreads();
  for (int z = tid; z < live * (D / 4); z += kAtThreads) {
    const int q = z / (D / 4), c = z % (D / 4);
    const int qi = it.row0 + q;
    float4 a = *reinterpret_cast<const float4 *>(s_o + q * (D + 4) + c * 4);
#pragma unroll
    for (int w = 1; w < WK; ++w) {
      const float4 b = *reinterpret_cast<const float4 *>(s_o + (w * kRows + q) * (D + 4) + c * 4);
      a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
    }
    if (any_odd) a = add_odd<DT>(it, s_anc[qi / A.n], c * 4, a);
    const int64_t at = it.part * rows_all + (it.base_row + qi / A.n) * A.Hq + it.kvh * A.n + qi % A.n;
    *reinterpret_cast<float4 *>(A.part_o + at * D + c * 4) = a;
    if (c == 0) {
      float Mq = kNegInf, L = 0.0f;
#pragma unroll
      for (int w = 0; w < WK; ++w) Mq = fmaxf(Mq, s_ml[w * kRows + q].x);
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const float2 v = s_ml[w * kRows + q];
        L += v.x == kNegInf ? v.y : v.y * exp2_fast((v.x - Mq) * A.scale_log2);  // (no maximum: zero, or NaN)
      }
      A.part_ml[at] = make_float2(Mq, L);
    }
  }
}

// tree: nothing for a window, or the TreeParents.
template <int DT, int D, int WQP, int WQO, class... Tree>
__global__ void __launch_bounds__(kAtThreads, 2) k_attend(AttendArgs A, Tree... tree) {
  constexpr size_t kBytes = at_tile_bytes<D, WQP>() > at_tile_bytes<D, WQO>() ? at_tile_bytes<D, WQP>() : at_tile_bytes<D, WQO>();
  __shared__ uint4 s_tile[kBytes / sizeof(uint4)];
  __shared__ uint32_t s_anc[kTreeMaxNodes][8];
  __shared__ uint8_t s_parent[kTreeMaxNodes];
  __shared__ float2 s_ml[128];  // [waves on the same rows][rows]
  char *lds = reinterpret_cast<char *>(s_tile);
  Item it{};
  int id = blockIdx.x;
  if (id < A.prefix_items) {
    // row tiles of one (kv head, range) are Hkv * parts apart: a multiple of 8
    // of those keeps them on one XCD
    const int pairs = A.Hkv * A.prefix_parts;
    const int pair = id % pairs;
    it.kvh = pair % A.Hkv;
    it.part = pair / A.Hkv;
    it.row0 = id / pairs * (32 * WQP);
    it.rows = A.B * A.R * A.n;
    it.base_row = 0;
    it.k = A.prefix_k + it.kvh * D;
    it.v = A.prefix_v + it.kvh * D;
    it.tok_stride = A.prefix_tok_stride;
    it.k0 = it.part * A.prefix_chunk;
    it.k1 = min(it.k0 + A.prefix_chunk, A.P);
    it.draft = it.k1 + (1 << 30);
    if (A.P - it.k0 <= 0) return;
    attend_item<DT, D, WQP>(A, it, lds, s_anc, s_ml);
    return;
  }
  id -= A.prefix_items;
  // All heads and row tiles of a range of one sequence's tokens follow each
  // other on one XCD (8 blocks apart): together they read whole tokens.  With
  // a head per XCD instead, every XCD reads the same eighth of the memory
  // channels.
  const int per = A.Hkv * A.own_tiles;
  const int j = id / 8;
  const int range = j / per * 8 + id % 8;
  if (range >= A.B * A.own_parts) return;
  const int tile = j % per % A.own_tiles;
  it.kvh = j % per / A.own_tiles;
  const int split = range / A.B;  // every sequence's first range, then the second ..: full ones go first
  // moved on from split to split: where B is a multiple of 8, all ranges of a
  // long sequence would lie on one XCD (one of 60000 keys among 31 of 500 took
  // 235 us, 122 spread out)
  int b = range - split * A.B;
  if (A.B >= 8) {
    b += split & 7;
    if (b >= A.B) b -= A.B;
  }
  const int len = A.ctx_len[b];
  const int live = live_rows(A, b);
  if (bad_len(A, len) || live == 0) return;
  const int keys = __builtin_amdgcn_readfirstlane(len + live);  // (the same for the workgroup: scalar from here)
  const int own = attend_own_range(A.split, keys);
  it.row0 = tile * (32 * WQO);
  it.rows = live * A.n;
  if (static_cast<int64_t>(split) * own >= keys || it.row0 >= it.rows) return;
  it.k0 = split * own;
  it.k1 = min(it.k0 + own, keys);
  it.draft = len;
  it.part = A.prefix_parts + split;
  it.base_row = static_cast<int64_t>(b) * A.R;
  it.k = A.k + b * A.seq_stride + it.kvh * D;
  it.v = A.v + b * A.seq_stride + it.kvh * D;
  it.tok_stride = A.tok_stride;
  if (it.k1 > len) ancestor_sets(A.R, s_anc, s_parent, tree...);
  __syncthreads();
  attend_item<DT, D, WQO>(A, it, lds, s_anc, s_ml);
}

// One wave per (row, head): the row's items in order, weighted by their
// maxima; a sequence whose length is out of range gets NaN.
template <int DT, int D>
__global__ void __launch_bounds__(256) k_attend_combine(AttendJoin A) {
  constexpr int E = D / 64;
  const int rows = A.B * A.R * A.Hq;  // at most 2^30
  const int row = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // scalar: the same for the wave
  const int lane = threadIdx.x & 63;
  if (row >= rows) return;  // (bound: the partial outputs, 4 D bytes a row and range, written and read once)
  const int br = row / A.Hq, b = br / A.R, r = br % A.R;
  const int live = live_rows(A, b);
  if (r >= live) return;
  const int len = A.ctx_len[b];
  float acc[E] = {};
  float M = kNegInf, L = 0.0f;
  if (bad_len(A, len)) {
    M = L = __builtin_nanf("");
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = L;
  } else {
    const int keys = len + live, own = attend_own_range(A.split, keys);
    int parts = A.prefix_parts;
    for (int k0 = 0; k0 < keys; k0 += own) ++parts;
    for (int p = 0; p < parts; ++p) M = fmaxf(M, A.part_ml[static_cast<int64_t>(p) * rows + row].x);
    for (int p = 0; p < parts; ++p) {
      const int64_t at = static_cast<int64_t>(p) * rows + row;
      const float2 ml = A.part_ml[at];
      const float f = ml.x == kNegInf ? 0.0f : exp2_fast((ml.x - M) * A.scale_log2);
      L += f * ml.y;
      const float *po = A.part_o + at * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f * po[e];
    }
  }
  uint16_t *out = A.out + static_cast<int64_t>(row) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = AtElt<DT>::bits(acc[e] / L);
  if (A.lse && lane == 0) A.lse[row] = (M * A.scale_log2 + log2f(L * (AtElt<DT>::kLift > 0 ? 0x1p-15f : 1.0f))) * 0.6931471805599453f;
}

namespace {

template <int DT, int D, int WQP, int WQO>
void launch_shape(const AttendArgs &A, const TreeParents *parents, dim3 grid, hipStream_t st) {
  if (parents)
    hipLaunchKernelGGL((k_attend<DT, D, WQP, WQO, TreeParents>), grid, dim3(kAtThreads), 0, st, A, *parents);
  else
    hipLaunchKernelGGL((k_attend<DT, D, WQP, WQO>), grid, dim3(kAtThreads), 0, st, A);
}

template <int DT, int D, int WQP>
void launch_own(const AttendArgs &A, const TreeParents *parents, const AttendPlan &P, dim3 grid, hipStream_t st) {
  // (a sequence's rows are no more than the batch's: 4 waves on them mean 4 on the prefix)
  if (WQP == 4 && P.own_waves == 4)
    launch_shape<DT, D, 4, 4>(A, parents, grid, st);
  else if (P.own_waves == 2)
    launch_shape<DT, D, WQP, 2>(A, parents, grid, st);
  else
    launch_shape<DT, D, WQP, 1>(A, parents, grid, st);
}

template <int DT, int D>
void launch_type(const AttendArgs &A, const TreeParents *parents, const AttendPlan &P, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(P.prefix_items + P.own_blocks));
  if (P.prefix_waves == 4)
    launch_own<DT, D, 4>(A, parents, P, grid, st);
  else
    launch_own<DT, D, 1>(A, parents, P, grid, st);
  const int64_t rows = static_cast<int64_t>(A.B) * A.R * A.Hq;
  hipLaunchKernelGGL((k_attend_combine<DT, D>), dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, st,
                     static_cast<const AttendJoin &>(A));
}

}  // namespace

void launch_attend(int dtype, int D, const AttendArgs &A, const TreeParents *parents, const AttendPlan &P, hipStream_t st) {
  if (dtype == DT_BF16) {
    if (D == 64) launch_type<DT_BF16, 64>(A, parents, P, st);
    else launch_type<DT_BF16, 128>(A, parents, P, st);
  } else {
    if (D == 64) launch_type<DT_F16, 64>(A, parents, P, st);
    else launch_type<DT_F16, 128>(A, parents, P, st);
  }
}

}  // namespace sv
