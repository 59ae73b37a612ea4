// Attention of a step's rows over paged caches (gfx950): sv_attention's work
// items, ranges and join, with keys and values found through page tables and
// held in 16 bits, or in 8 with a scale for each block of tokens and head.
//
// Pages.  Ranges begin at multiples of 128 tokens and pages hold 16 at least, so
// 16 aligned tokens (a strip) lie in one page and under one scale.  Each lane of
// a wave looks up one strip of the next 1024 tokens (page, key scale, value
// scale): one trip for the table and one for the scales, after which a strip's
// page is a lane read, and its rows are read whole: rows past the range are
// inside the page.
//
// Scales.  A score is its product times the key scale, one multiplication; the
// value scale multiplies the exponential.  Both are wave-uniform per strip.  In
// float16 exponentials are held 2^15 times larger and the value scales relative
// to the largest so far, as either alone could leave the type.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_attend.h"

namespace sv {

namespace {

constexpr int kStrip = 16;               // tokens that share page and scale
constexpr int kLookup = 64 * kStrip;     // tokens of one look-up

// Rows [row0, row0 + rows) of a stack (see sv_attention.hip's Item) over tokens
// [k0, k1) of a page table.
struct PagedItem {
  const int32_t *table;
  int64_t base_row;
  int row0, rows;
  int kvh;
  int k0, k1, draft;
  int part;
};

template <int D> constexpr int pg_key_row() { return D + 8; }
template <int D> constexpr int pg_value_row() { return D + 16; }
template <int WQ> constexpr int pg_tile_keys() { return WQ == 1 ? 128 : 64; }
template <int D, int WQ> constexpr size_t pg_tile_bytes() {
  const size_t kv = static_cast<size_t>(pg_tile_keys<WQ>()) * (pg_key_row<D>() + pg_value_row<D>()) * 2;
  const size_t merge = WQ < 4 ? 4 * 32 * static_cast<size_t>(D + 4) * 4 : 0;
  return kv > merge ? kv : merge;
}

// 16 bytes as 16 values of the storage type (exact).
template <int DT> __device__ __forceinline__ void widen(uint4 raw, uint4 *lo, uint4 *hi) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DT_BF16) {
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true));
    } else {
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.0f, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.0f, true));
    }
  }
  *lo = make_uint4(o[0], o[1], o[2], o[3]);
  *hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// What is no finite number among 16 bytes of values, as zeros.
template <int DT, bool F8> __device__ __forceinline__ uint4 drop_odd(uint4 v, bool *odd) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (F8) {
      const uint32_t nan = ((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
      if (nan) w[k] &= ~((nan >> 7) * 0xFFu), *odd = true;
    } else {
      if ((w[k] & AtElt<DT>::kExp) == AtElt<DT>::kExp) w[k] &= 0xFFFF0000u, *odd = true;
      if (((w[k] >> 16) & AtElt<DT>::kExp) == AtElt<DT>::kExp) w[k] &= 0xFFFFu, *odd = true;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// a (values d .. d + 3 of a row with ancestor set anc) plus the infinities and
// NaN among the row's own keys' values.
template <int DT, bool F8>
__device__ float4 add_odd_paged(const PagedAttendArgs &A, const PagedItem &it, const uint32_t *anc, int d, float4 a) {
  for (int key = max(it.k0, it.draft); key < it.k1; ++key) {
    const int own = key - it.draft;
    if (!((anc[own >> 5] >> (own & 31)) & 1)) continue;
    const int page = it.table[key >> A.pool.page_shift];
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(A.pool.num_pages)) continue;
    const uint8_t *v = A.pool.v + page * A.pool.page_bytes + (key & ((1 << A.pool.page_shift) - 1)) * A.pool.token_bytes +
                       it.kvh * A.pool.head_bytes;
    float *x = &a.x;
    if constexpr (F8) {
      const uint32_t w = *reinterpret_cast<const uint32_t *>(v + d);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (((w >> (8 * k)) & 0x7F) == 0x7F) x[k] = __builtin_nanf("");
    } else {
      const uint2 w = *reinterpret_cast<const uint2 *>(v + 2 * d);
      const uint32_t b[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((b[k] & AtElt<DT>::kExp) == AtElt<DT>::kExp) x[k] += Elt<DT>::dec(b[k]);
    }
  }
  return a;
}

}  // namespace

template <int DT, bool F8, int D, int WQ>
__device__ __forceinline__ void paged_item(const PagedAttendArgs &A, const PagedItem &it, char *lds, const uint32_t (*s_anc)[8],
                                           float2 *s_ml) {
  using T = AtElt<DT>;
  constexpr int WK = 4 / WQ;
  constexpr int KT = pg_tile_keys<WQ>();
  constexpr int SB = KT / (32 * WK);  // 32-key blocks per wave and tile
  constexpr int kRow = pg_key_row<D>(), kVRow = pg_value_row<D>();
  constexpr int kBytes = F8 ? 1 : 2;
  constexpr int kChunks = D * kBytes / 16;   // 16-byte pieces of a row
  constexpr int kWaveRows = 64 / kChunks;    // rows of one load of a wave: within a strip
  constexpr bool kApart = WQ == 1;
  constexpr int kLoads = KT * kChunks / kAtThreads;
  constexpr bool kRelative = F8 && T::kLift > 0;
  uint16_t *s_k = reinterpret_cast<uint16_t *>(lds);
  uint16_t *s_v = s_k + KT * kRow;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
  float ref = kRelative ? 0.0f : 1.0f;

  // the strips of the look-up that begins at token c0, one per lane
  int c0 = it.k0, pages = 0;
  float kscale = 1.0f, vscale = 1.0f;
  bool bad = false;
  const int last = (it.k1 - 1) & -kStrip;
  auto look_up = [&](int at) {
    c0 = at;
    const int key = min(at + lane * kStrip, last);
    pages = it.table[key >> A.pool.page_shift];
    if (static_cast<uint32_t>(pages) >= static_cast<uint32_t>(A.pool.num_pages)) pages = 0, bad = true;
    if (F8) {
      const int in_page = key & ((1 << A.pool.page_shift) - 1);
      const int64_t s = ((static_cast<int64_t>(pages) << (A.pool.page_shift - A.pool.block_shift)) + (in_page >> A.pool.block_shift)) * A.pool.Hkv + it.kvh;
      kscale = A.pool.k_scale[s];
      vscale = A.pool.v_scale[s];
    }
  };
  look_up(it.k0);

  uint4 rk[kLoads], rv[kLoads];
  float ks[2 * SB], vs[2 * SB], ks_next[2 * SB], vs_next[2 * SB];  // scales of this wave's strips, of the tile and of the one loaded
  const int piece = lane % kChunks;
  constexpr int kStep = kApart ? kWaveRows : 4 * kWaveRows;
  const int row0 = kApart ? wave * 32 : wave * kWaveRows;  // of this wave's first load
  const int row_lane = lane / kChunks;
  const uint32_t lane_off = static_cast<uint32_t>(row_lane) * static_cast<uint32_t>(A.pool.token_bytes) + piece * 16;
  const int page_mask = (1 << A.pool.page_shift) - 1;
  // one sequence's pages are read once: streamed
  auto fetch = [&](const uint8_t *p) { return kApart ? load_stream(reinterpret_cast<const uint4 *>(p)) : load_vec(p); };
  auto load = [&](int t0) {
    if (t0 - c0 >= kLookup) look_up(t0);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int key = t0 + row0 + j * kStep;  // (the wave's first row: rows follow within a strip)
      const int strip = min(key, last + (key & (kStrip - 1))) ;
      const int page = __builtin_amdgcn_readlane(pages, (strip - c0) / kStrip);
      const int64_t off = page * A.pool.page_bytes + (strip & page_mask) * A.pool.token_bytes + it.kvh * A.pool.head_bytes;
      rk[j] = fetch(A.pool.k + off + lane_off);
      rv[j] = fetch(A.pool.v + off + lane_off);
    }
    if (F8)
#pragma unroll
      for (int g = 0; g < 2 * SB; ++g) {
        const int at = (min(t0 + wk * SB * 32 + g * kStrip, last) - c0) / kStrip;
        ks_next[g] = read_lane_f32(kscale, at);
        vs_next[g] = read_lane_f32(vscale, at);
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
    // zero times what a page holds behind the last token need not be.
    // Infinities and NaN among the step's own values, which must reach only the
    // rows that see them, are left out here and added at the end.
    const bool masked = t0 + KT > it.draft;
    tile_barrier();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int row = row0 + j * kStep + row_lane;
      uint4 v = rv[j];
      if (t0 + KT > it.k1 && t0 + row >= it.k1) v = make_uint4(0, 0, 0, 0);
      if (masked && t0 + row >= it.draft && t0 + row < it.k1) v = drop_odd<DT, F8>(v, &odd);
      if constexpr (F8) {
        uint4 lo, hi;
        widen<DT>(rk[j], &lo, &hi);
        *reinterpret_cast<uint4 *>(s_k + row * kRow + piece * 16) = lo;
        *reinterpret_cast<uint4 *>(s_k + row * kRow + piece * 16 + 8) = hi;
        widen<DT>(v, &lo, &hi);
        *reinterpret_cast<uint4 *>(s_v + row * kVRow + piece * 16) = lo;
        *reinterpret_cast<uint4 *>(s_v + row * kVRow + piece * 16 + 8) = hi;
      } else {
        *reinterpret_cast<uint4 *>(s_k + row * kRow + piece * 8) = rk[j];
        *reinterpret_cast<uint4 *>(s_v + row * kVRow + piece * 8) = v;
      }
    }
#pragma unroll
    for (int g = 0; g < 2 * SB; ++g) ks[g] = ks_next[g], vs[g] = vs_next[g];
    tile_barrier();
    if (t0 + KT < it.k1) load(t0 + KT);
    if (t0 + wk * SB * 32 >= it.k1) continue;  // nothing of this tile for this wave
    // products of the wave's blocks of 32 keys
    at_f32x16_t s[SB];
#pragma unroll
    for (int sb = 0; sb < SB; ++sb) {
#pragma unroll
      for (int e = 0; e < 16; ++e) s[sb][e] = 0.0f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
        s[sb] = T::mma(*reinterpret_cast<const uint4 *>(s_k + ((wk * SB + sb) * 32 + q32) * kRow + d * 16 + half * 8), qf[d], s[sb]);
      if (F8)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[sb][e] *= ks[2 * sb + (e >> 3)];
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
    float wt[2 * SB];
    if (F8) {
      if (kRelative) {
        float most = vs[0];
#pragma unroll
        for (int g = 1; g < 2 * SB; ++g) most = fmaxf(most, vs[g]);
        if (most > ref) {
          const float down = ref / most;
#pragma unroll
          for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[t][e] *= down;
          ref = most;
        }
      }
#pragma unroll
      for (int g = 0; g < 2 * SB; ++g) wt[g] = kRelative ? vs[g] / ref : vs[g];
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
        if (F8) s[sb][e] *= wt[2 * sb + (e >> 3)];
      }
    l += sum;
#pragma unroll
    for (int sb = 0; sb < SB; ++sb) {
      const int kb = (wk * SB + sb) * 32;  // this block's first key in the tile
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        const uint4 p = make_uint4(T::pack(s[sb][8 * kp], s[sb][8 * kp + 1]), T::pack(s[sb][8 * kp + 2], s[sb][8 * kp + 3]),
                                   T::pack(s[sb][8 * kp + 4], s[sb][8 * kp + 5]), T::pack(s[sb][8 * kp + 6], s[sb][8 * kp + 7]));
        // lane l: block of 4 keys x 16 values; its address is row (l % 16) / 4, values 4 (l % 4)
        const uint16_t *base = s_v + (kb + kp * 16 + 4 * half + ((lane & 15) >> 2)) * kVRow + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
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
  if (__any(bad)) l = __builtin_nanf("");  // a page that is none: the rows are no numbers

  const int64_t rows_all = static_cast<int64_t>(A.B) * A.R * A.Hq;
  if (WQ == 4) {
    if (i < it.rows) {
      const int64_t at = it.part * rows_all + qrow * A.Hq + head;
      float *po = A.part_o + at * D;
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          float4 a = make_float4(o[t][4 * f] * ref, o[t][4 * f + 1] * ref, o[t][4 * f + 2] * ref, o[t][4 * f + 3] * ref);
          const int d = t * 32 + 8 * f + 4 * half;
          if (any_odd) a = add_odd_paged<DT, F8>(A, it, s_anc[r], d, a);
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
  const float f = m == kNegInf ? 0.0f : exp2_fast((m - M) * A.scale_log2) * ref;
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
    if (any_odd) a = add_odd_paged<DT, F8>(A, it, s_anc[qi / A.n], c * 4, a);
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
template <int DT, bool F8, int D, int WQP, int WQO, class... Tree>
__global__ void __launch_bounds__(kAtThreads, 2) k_paged_attend(PagedAttendArgs A, Tree... tree) {
  constexpr size_t kBytes = pg_tile_bytes<D, WQP>() > pg_tile_bytes<D, WQO>() ? pg_tile_bytes<D, WQP>() : pg_tile_bytes<D, WQO>();
  __shared__ uint4 s_tile[kBytes / sizeof(uint4)];
  __shared__ uint32_t s_anc[kTreeMaxNodes][8];
  __shared__ uint8_t s_parent[kTreeMaxNodes];
  __shared__ float2 s_ml[128];  // [waves on the same rows][rows]
  char *lds = reinterpret_cast<char *>(s_tile);
  PagedItem it{};
  const int heads = A.pool.Hkv;
  int id = blockIdx.x;
  if (id < A.prefix_items) {
    // row tiles of one (kv head, range) are Hkv * parts apart: a multiple of 8
    // of those keeps them on one XCD
    const int pairs = heads * A.prefix_parts;
    const int pair = id % pairs;
    it.kvh = pair % heads;
    it.part = pair / heads;
    it.row0 = id / pairs * (32 * WQP);
    it.rows = A.B * A.R * A.n;
    it.base_row = 0;
    it.table = A.prefix_table;
    it.k0 = it.part * A.prefix_chunk;
    it.k1 = min(it.k0 + A.prefix_chunk, A.P);
    it.draft = it.k1 + (1 << 30);
    if (A.P - it.k0 <= 0) return;
    paged_item<DT, F8, D, WQP>(A, it, lds, s_anc, s_ml);
    return;
  }
  id -= A.prefix_items;
  // All heads and row tiles of a range of one sequence's tokens follow each
  // other on one XCD (8 blocks apart), every sequence's first range first, the
  // next moved on by one: see k_attend.
  const int per = heads * A.own_tiles;
  const int j = id / 8;
  const int range = j / per * 8 + id % 8;
  if (range >= A.B * A.own_parts) return;
  const int tile = j % per % A.own_tiles;
  it.kvh = j % per / A.own_tiles;
  const int split = range / A.B;
  int b = range - split * A.B;
  if (A.B >= 8) {
    b += split & 7;
    if (b >= A.B) b -= A.B;
  }
  const int len = A.ctx_len[b];
  const int live = live_rows(A, b);
  if (bad_len(A, len) || live == 0) return;
  const int keys = __builtin_amdgcn_readfirstlane(len + live);
  const int own = attend_own_range(A.split, keys);
  it.row0 = tile * (32 * WQO);
  it.rows = live * A.n;
  if (static_cast<int64_t>(split) * own >= keys || it.row0 >= it.rows) return;
  it.k0 = split * own;
  it.k1 = min(it.k0 + own, keys);
  it.draft = len;
  it.part = A.prefix_parts + split;
  it.base_row = static_cast<int64_t>(b) * A.R;
  it.table = A.table + b * A.table_stride;
  if (it.k1 > len) ancestor_sets(A.R, s_anc, s_parent, tree...);
  __syncthreads();
  paged_item<DT, F8, D, WQO>(A, it, lds, s_anc, s_ml);
}

namespace {

template <int DT, bool F8, int D, int WQP, int WQO>
void launch_shape(const PagedAttendArgs &A, const TreeParents *parents, dim3 grid, hipStream_t st) {
  if (parents)
    hipLaunchKernelGGL((k_paged_attend<DT, F8, D, WQP, WQO, TreeParents>), grid, dim3(kAtThreads), 0, st, A, *parents);
  else
    hipLaunchKernelGGL((k_paged_attend<DT, F8, D, WQP, WQO>), grid, dim3(kAtThreads), 0, st, A);
}

template <int DT, bool F8, int D, int WQP>
void launch_own(const PagedAttendArgs &A, const TreeParents *parents, const AttendPlan &P, dim3 grid, hipStream_t st) {
  // (a sequence's rows are no more than the batch's: 4 waves on them mean 4 on the prefix)
  if (WQP == 4 && P.own_waves == 4)
    launch_shape<DT, F8, D, 4, 4>(A, parents, grid, st);
  else if (P.own_waves == 2)
    launch_shape<DT, F8, D, WQP, 2>(A, parents, grid, st);
  else
    launch_shape<DT, F8, D, WQP, 1>(A, parents, grid, st);
}

template <int DT, bool F8, int D>
void launch_dim(const PagedAttendArgs &A, const TreeParents *parents, const AttendPlan &P, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(P.prefix_items + P.own_blocks));
  if (P.prefix_waves == 4)
    launch_own<DT, F8, D, 4>(A, parents, P, grid, st);
  else
    launch_own<DT, F8, D, 1>(A, parents, P, grid, st);
  launch_attend_join(DT, D, A, st);
}

template <int DT, bool F8>
void launch_cache(int D, const PagedAttendArgs &A, const TreeParents *parents, const AttendPlan &P, hipStream_t st) {
  if (D == 64) launch_dim<DT, F8, 64>(A, parents, P, st);
  else launch_dim<DT, F8, 128>(A, parents, P, st);
}

}  // namespace

void launch_paged_attend(int dtype, bool f8, int D, const PagedAttendArgs &A, const TreeParents *parents, const AttendPlan &P, hipStream_t st) {
  if (dtype == DT_BF16) {
    if (f8) launch_cache<DT_BF16, true>(D, A, parents, P, st);
    else launch_cache<DT_BF16, false>(D, A, parents, P, st);
  } else {
    if (f8) launch_cache<DT_F16, true>(D, A, parents, P, st);
    else launch_cache<DT_F16, false>(D, A, parents, P, st);
  }
}

}  // namespace sv
