// Attention of a step's rows over paged caches (gfx950): sv_attention's work
// items, ranges and join, with keys and values found through page tables and
// held in 16 bits, or in 8 with a scale for each block of tokens and head.
//
// Pages.  Ranges begin at multiples of 128 tokens and pages hold 16 at least, so
// 16 aligned tokens (a strip) lie in one page and under one scale.  Each lane of
// a wave looks up one strip of the next 1024 tokens (address, key scale, value
// scale): one trip for the table and one for the scales, after which a strip's
// address is two lane reads, and its rows are read whole: rows past the range
// are inside the page.
//
// Scales.  A score is its product times the key scale, one multiplication; the
// value scale multiplies the exponential, and the product is rounded to the
// rows' type once, as 16-bit pages' exponentials are.  Both are wave-uniform per
// strip.  In float16 exponentials are held 2^15 times larger and the value
// scales relative to the largest so far, as either alone could leave the type.
//
// 8-bit products (keys against queries rounded to sums of 8-bit numbers) were
// not taken: the scaled 8-bit matrix instruction's sums are off by up to 1.4e-4 of the
// sum of the products' magnitudes.
//
// Bounds.  Few rows are the pages' traffic: a copy reaches 4.9 TB/s here, reads
// alone 7.0.  Single tokens of 128 sequences with 4000 keys of 8 heads of 128: 1.05
// GB of 8-bit pages in 178 us (5.9 TB/s), 2.1 GB of bf16 pages in 337 us (6.2 TB/s).
// Behind a shared prefix it is matrix and vector work on the same tiles: 18432
// stacked rows over 8192 keys, 8-bit, are 77 GFLOP in 112 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sv_attend.h"

namespace sv {

namespace {

constexpr int kFewWaves = kAtThreads / 64;
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
constexpr int kPgTileKeys = 64;
template <int D, int WQ> constexpr size_t pg_tile_bytes() {
  const size_t kv = static_cast<size_t>(kPgTileKeys) * (pg_key_row<D>() + pg_value_row<D>()) * 2;
  const size_t merge = WQ < 4 ? 4 * 32 * static_cast<size_t>(D + 4) * 4 : 0;
  return kv > merge ? kv : merge;
}

// Bytes from the pools' start to a strip's first row (page, token in it, head), and
// the offset that lane `at` holds.
__device__ __forceinline__ int2 strip_offset(const PagedAttendArgs &A, int page, int in_page, int kvh) {
  const int64_t off = page * A.pool.page_bytes + in_page * A.pool.token_bytes + kvh * A.pool.head_bytes;
  return make_int2(static_cast<int>(off), static_cast<int>(off >> 32));
}
__device__ __forceinline__ int64_t strip_at(int2 strips, int at) {
  return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(strips.y, at))) << 32 |
                              static_cast<uint32_t>(__builtin_amdgcn_readlane(strips.x, at)));
}

// 16 bytes as 16 values of the storage type, times a power of two (exact).
template <int DT> __device__ __forceinline__ void widen(uint4 raw, float scale, uint4 *lo, uint4 *hi) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DT_BF16) {
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, true));
    } else {
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], scale, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], scale, true));
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

typedef float pg_f32x4_t __attribute__((ext_vector_type(4)));
typedef int pg_i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) pg_i32x2_t *lds_i32x2_t;

namespace {

// 8 bytes as an operand of 8 values (exact).
template <int DT> __device__ __forceinline__ uint4 widen8(uint2 raw) {
  if constexpr (DT == DT_BF16)
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw.x, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw.x, 1.0f, true)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw.y, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw.y, 1.0f, true)));
  else
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw.x, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw.x, 1.0f, true)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw.y, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw.y, 1.0f, true)));
}

template <int DT> __device__ __forceinline__ pg_f32x4_t mma16(uint4 a, uint4 b, pg_f32x4_t c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(at_bf16x8_t, a), __builtin_bit_cast(at_bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(at_f16x8_t, a), __builtin_bit_cast(at_f16x8_t, b), c, 0, 0, 0);
}

// The maximum and the sum over the lanes that hold one row: l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float row_max(float x) {
  const float2 h = both_halves(x);
  x = fmaxf(h.x, h.y);
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float row_sum(float x) {
  const float2 h = both_halves(x);
  x = h.x + h.y;
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Bytes between rows of LDS.  Key rows of 16 bytes more put the rows that 8 lanes
// read 16 bytes of side by side; a transposing read takes 8 rows of 16 bytes (8
// bits: 16 bytes more) or 4 of 32 (16 bits: 32 bytes more).
template <bool F8, int D> constexpr int few_key_pitch() { return F8 ? D + 16 : 2 * D + 16; }
template <bool F8, int D> constexpr int few_value_pitch() { return F8 ? D + 16 : 2 * D + 32; }
template <bool F8, int D, int NC> constexpr size_t few_bytes() {
  const size_t tile = static_cast<size_t>(32 * kFewWaves) * (few_key_pitch<F8, D>() + few_value_pitch<F8, D>());
  const size_t merge = static_cast<size_t>(kFewWaves) * 16 * NC * (64 + 4) * 4;
  return tile > merge ? tile : merge;
}

}  // namespace

// What a wave's lanes wrote to LDS is there for all of them: its LDS operations
// run in order, this keeps the compiler from moving them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Few rows: NC tiles of 16 stacked rows.  Keys and values lie in LDS as the pages
// hold them and become operands in registers, once for all tiles.  Every wave has
// blocks of 32 keys of its own for the same rows, so the waves run without
// barriers until the end.
//
// The k order of a product may be any that both operands share, and so may the
// keys' order in the score tile.  Keys are placed in LDS such that a lane's
// exponentials belong to 8 consecutive keys: the operand of the second product as
// they are, under one scale, against values whose transposing read takes 8
// consecutive rows (no bank conflicts).
//
// Bound: memory.  128 single tokens of 32 / 8 heads of 128 over 4000 keys, 8-bit:
// 178 to 182 us, 5.9 TB/s; over 1000 to 4000 behind 2048 shared ones 127 to 130.  Rows
// of a sequence in tiles of 16 rows of 16x16x32 products hold half the registers of
// tiles of 32: of 16 rows four workgroups are on a CU (two with 16-bit heads of 128,
// whose tiles are 71 KB of LDS, or where a batch's prefix is in the same kernel).
// One sequence: trips to memory, 6.3 to 6.9 us over 100 keys, 10 over 1033, 12 over 4000,
// 21 over 30000 (with the join).
// Tried: 16 waves a workgroup (slower but for 32 sequences of 1000), two tiles in flight
// (144 to 141 us at two waves a SIMD; the registers hold two more waves instead).
template <int DT, bool F8, int D, int NC>
__device__ __forceinline__ void few_item(const PagedAttendArgs &A, const PagedItem &it, char *lds, const uint32_t (*s_anc)[8],
                                         float2 *s_ml, bool direct) {
  using T = AtElt<DT>;
  constexpr int ROWS = 16 * NC;
  constexpr int KT = 32 * kFewWaves;                   // keys of a tile, 32 of them a wave's
  constexpr int kBytes = F8 ? 1 : 2;
  constexpr int kChunks = D * kBytes / 16;             // 16-byte pieces of a row
  constexpr int kWaveRows = 64 / kChunks;              // rows of one load of a wave: within a strip
  constexpr int kLoads = 32 / kWaveRows;
  constexpr int kKP = few_key_pitch<F8, D>(), kVP = few_value_pitch<F8, D>();
  constexpr bool kRelative = F8 && T::kLift > 0;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, grp = lane >> 4;
  char *s_k = lds + wave * 32 * (kKP + kVP), *s_v = s_k + 32 * kKP;

  // this lane's rows (col of each tile), their query fragments
  constexpr int kSteps = D / 32;                       // matrix steps of a score
  uint4 qf[NC][kSteps];
  int rows[NC];                                        // rows of the step, for their ancestors
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int ic = min(it.row0 + 16 * c + col, it.rows - 1);
    const int64_t qrow = it.base_row + ic / A.n;
    const uint16_t *p = A.q + qrow * A.q_row_stride + (it.kvh * A.n + ic % A.n) * D;
    rows[c] = static_cast<int>(qrow % A.R);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      // 8 bits: a 16-byte read of keys is two steps' operands
      qf[c][s] = load_vec(p + (F8 ? (s >> 1) * 64 + 16 * grp + 8 * (s & 1) : s * 32 + 8 * grp));
      // a negative scale acts on the queries' signs, so that larger products are larger scores
      if (A.negate) qf[c][s] = make_uint4(qf[c][s].x ^ 0x80008000u, qf[c][s].y ^ 0x80008000u, qf[c][s].z ^ 0x80008000u, qf[c][s].w ^ 0x80008000u);
    }
  }

  constexpr int kTiles = D / 16;  // output tiles: values 16 t + 4 grp .. + 3 of a row
  pg_f32x4_t o[NC][kTiles];
  float m[NC], l[NC];             // l: this lane's keys only
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    m[c] = kNegInf, l[c] = 0.0f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) o[c][t] = pg_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  float ref = kRelative ? 0.0f : 1.0f;
  auto rescale_all = [&](const float (&f)[NC]) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][t][e] *= f[c];
  };

  // the strips of the look-up that begins at token c0, one per lane
  int c0 = it.k0;
  int2 strips{};
  float kscale = 1.0f, vscale = 1.0f;
  bool bad = false;
  const int last = (it.k1 - 1) & -kStrip;
  auto look_up = [&](int at) {
    c0 = at;
    const int key = min(at + lane * kStrip, last), in_page = key & ((1 << A.pool.page_shift) - 1);
    int page = it.table[key >> A.pool.page_shift];
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(A.pool.num_pages)) page = 0, bad = true;
    strips = strip_offset(A, page, in_page, it.kvh);
    if (F8) {
      const int64_t s = ((static_cast<int64_t>(page) << (A.pool.page_shift - A.pool.block_shift)) + (in_page >> A.pool.block_shift)) * A.pool.Hkv + it.kvh;
      kscale = A.pool.k_scale[s];
      vscale = A.pool.v_scale[s];
    }
  };
  look_up(it.k0);

  uint4 rk[kLoads], rv[kLoads];
  float ks[2], vs[2], ks_next[2], vs_next[2];  // scales of this wave's strips, of the tile and of the one loaded
  const int piece = lane % kChunks, row_lane = lane / kChunks;
  const uint32_t lane_off = static_cast<uint32_t>(row_lane) * static_cast<uint32_t>(A.pool.token_bytes) + piece * 16;
  // one sequence's pages are read once: streamed
  auto fetch = [&](const uint8_t *p) { return load_stream(reinterpret_cast<const uint4 *>(p)); };
  auto load = [&](int t0) {
    if (t0 - c0 >= kLookup) look_up(t0);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int64_t off = strip_at(strips, (min(t0 + wave * 32 + g * kStrip, last) - c0) / kStrip);
#pragma unroll
      for (int x = 0; x < kStrip / kWaveRows; ++x) {
        const int j = g * (kStrip / kWaveRows) + x;
        rk[j] = fetch(A.pool.k + off + x * kWaveRows * A.pool.token_bytes + lane_off);
        rv[j] = fetch(A.pool.v + off + x * kWaveRows * A.pool.token_bytes + lane_off);
      }
    }
    if (F8)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int at = (min(t0 + wave * 32 + g * kStrip, last) - c0) / kStrip;
        ks_next[g] = read_lane_f32(kscale, at);
        vs_next[g] = read_lane_f32(vscale, at);
      }
  };
  // LDS row of a key of the wave's: see above
  auto key_row = [](int key) { return 16 * ((key >> 2) & 1) + 4 * (key >> 3) + (key & 3); };
  bool odd = false;
  load(it.k0);
  for (int t0 = it.k0; t0 < it.k1; t0 += KT) {
    const int w0 = t0 + wave * 32;  // the wave's first key
    // Keys past the range get zero values: their exponentials are zero, but
    // zero times what a page holds behind the last token need not be.
    // Infinities and NaN among the step's own values, which must reach only the
    // rows that see them, are left out here and added at the end.
    const bool plain = t0 + KT <= it.draft && t0 + KT <= it.k1;
    wave_sync();
    if (!plain) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int key = w0 + j * kWaveRows + row_lane;
        if (key >= it.k1) rv[j] = make_uint4(0, 0, 0, 0);
        else if (key >= it.draft) rv[j] = drop_odd<DT, F8>(rv[j], &odd);
      }
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int at = j * kWaveRows + row_lane;
      *reinterpret_cast<uint4 *>(s_k + key_row(at) * kKP + piece * 16) = rk[j];
      *reinterpret_cast<uint4 *>(s_v + at * kVP + piece * 16) = rv[j];
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) ks[g] = ks_next[g], vs[g] = vs_next[g];
    wave_sync();
    if (t0 + KT < it.k1) load(t0 + KT);
    if (w0 >= it.k1) continue;  // nothing of this tile for this wave
    // products: element e of a lane is key 8 grp + e
    float s[NC][8];
    {
      pg_f32x4_t acc[2][NC];
#pragma unroll
      for (int tau = 0; tau < 2; ++tau)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[tau][c] = pg_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < (F8 ? D / 64 : D / 32); ++x)
#pragma unroll
        for (int tau = 0; tau < 2; ++tau) {
          const uint4 w = *reinterpret_cast<const uint4 *>(s_k + (tau * 16 + col) * kKP + grp * 16 + x * 64);
          if constexpr (F8) {
            const uint4 k0 = widen8<DT>(make_uint2(w.x, w.y)), k1 = widen8<DT>(make_uint2(w.z, w.w));
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[tau][c] = mma16<DT>(k0, qf[c][2 * x], acc[tau][c]);
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[tau][c] = mma16<DT>(k1, qf[c][2 * x + 1], acc[tau][c]);
          } else {
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[tau][c] = mma16<DT>(w, qf[c][x], acc[tau][c]);
          }
        }
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[c][e] = acc[e >> 2][c][e & 3];
    }
    if (!plain) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = w0 + 8 * grp + e;
          const int own = key - it.draft;
          const bool ok = key < it.k1 && (own < 0 || ((s_anc[rows[c]][(own & 255) >> 5] >> (own & 31)) & 1));
          s[c][e] = ok ? s[c][e] : kNegInf;
        }
    }
    // the scales of a lane's 8 keys
    const float kf = !F8 ? 1.0f : grp < 2 ? ks[0] : ks[1];
    float vf = !F8 ? 1.0f : grp < 2 ? vs[0] : vs[1];
    // Outputs are rescaled only when some row's maximum rose: 1 is exact.
    float mn[NC];
    bool rose = false;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float top = s[c][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, s[c][e]);
      mn[c] = fmaxf(m[c], row_max(F8 ? top * kf : top));
      rose |= mn[c] > m[c];
    }
    if (__any(rose)) {
      float alpha[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        alpha[c] = m[c] == kNegInf ? 0.0f : exp2_fast((m[c] - mn[c]) * A.scale_log2);
        l[c] *= alpha[c];
        m[c] = mn[c];
      }
      rescale_all(alpha);
    }
    if (kRelative) {
      const float most = fmaxf(vs[0], vs[1]);
      if (most > ref) {
        float down[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) down[c] = ref / most;
        rescale_all(down);
        ref = most;
      }
      vf = ref > 0.0f ? vf / ref : 0.0f;  // (scales of zero alone so far)
    }
    // bf16: one multiply-add per exponent, the key scale in its factor (never
    // zero: masked products are -inf).  In float16 the exponent is taken from the
    // difference to the maximum, so that the largest is 2^15 exactly however far
    // the scores are (65504 ends the type).
    const float kq = F8 ? fmaxf(kf, __FLT_MIN__) : 1.0f;
    const float factor = F8 ? fmaxf(A.scale_log2 * kf, __FLT_MIN__) : A.scale_log2;
    uint4 p[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float top_s = m[c] == kNegInf ? 0.0f : m[c], mu = top_s * A.scale_log2;
      float *e = s[c], sum = 0.0f;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
#pragma clang fp contract(off)  // (the product is rounded as the maximum's was: no difference is above zero)
        e[x] = exp2_fast(T::kLift > 0 ? __builtin_fmaf((F8 ? e[x] * kq : e[x]) - top_s, A.scale_log2, T::kLift)
                                      : __builtin_fmaf(e[x], factor, -mu));
        sum += e[x];
        if (F8) e[x] *= vf;
      }
      l[c] += sum;
      p[c] = make_uint4(T::pack(e[0], e[1]), T::pack(e[2], e[3]), T::pack(e[4], e[5]), T::pack(e[6], e[7]));
    }
    // values of keys 8 grp .. + 7
    const char *row = s_v + (8 * grp + ((lane & 15) >> (F8 ? 1 : 2))) * kVP + (F8 ? (lane & 1) * 8 : (lane & 3) * 8);
    uint2 w[kTiles][F8 ? 1 : 2];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if constexpr (F8) {
        w[t][0] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2_t)(row + t * 16)));
      } else {
        w[t][0] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(row + t * 32)));
        w[t][F8 ? 0 : 1] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(row + t * 32 + 4 * kVP)));
      }
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const uint4 v = F8 ? widen8<DT>(w[t][0]) : make_uint4(w[t][0].x, w[t][0].y, w[t][F8 ? 0 : 1].x, w[t][F8 ? 0 : 1].y);
#pragma unroll
      for (int c = 0; c < NC; ++c) o[c][t] = mma16<DT>(v, p[c], o[c][t]);
    }
  }
  // (also: every wave is done with the tiles)
  const bool any_odd = it.k1 > it.draft ? __syncthreads_or(odd) : (__syncthreads(), false);
  const bool any_bad = __any(bad);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    l[c] = row_sum(l[c]);
    if (any_bad) l[c] = __builtin_nanf("");  // a page that is none: the rows are no numbers
  }

  const int64_t rows_all = static_cast<int64_t>(A.B) * A.R * A.Hq;
  // The waves hold the same rows over different keys: joined in wave order, 64
  // values of a row at a time.
  float *s_o = reinterpret_cast<float *>(lds);
  const int live = min(ROWS, it.rows - it.row0);
  if (grp == 0)
#pragma unroll
    for (int c = 0; c < NC; ++c) s_ml[wave * ROWS + 16 * c + col] = make_float2(m[c], l[c]);
  __syncthreads();
  float f[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float M = kNegInf;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) M = fmaxf(M, s_ml[w * ROWS + 16 * c + col].x);
    f[c] = m[c] == kNegInf ? 0.0f : exp2_fast((m[c] - M) * A.scale_log2) * ref;
  }
#pragma unroll
  for (int part = 0; part < D / 64; ++part) {
    if (part > 0) __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (16 * c + col < live)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const pg_f32x4_t a = o[c][part * 4 + t];
          *reinterpret_cast<float4 *>(s_o + (wave * ROWS + 16 * c + col) * (64 + 4) + t * 16 + 4 * grp) =
            make_float4(a[0] * f[c], a[1] * f[c], a[2] * f[c], a[3] * f[c]);
        }
    __syncthreads();
    for (int z = tid; z < live * 16; z += kAtThreads) {
      const int q = z / 16, c = z % 16, d = part * 64 + c * 4;
      const int qi = it.row0 + q;
      float4 a = *reinterpret_cast<const float4 *>(s_o + q * (64 + 4) + c * 4);
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) {
        const float4 b = *reinterpret_cast<const float4 *>(s_o + (w * ROWS + q) * (64 + 4) + c * 4);
        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
      }
      if (any_odd) a = add_odd_paged<DT, F8>(A, it, s_anc[qi / A.n], d, a);
      float Mq = kNegInf, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) Mq = fmaxf(Mq, s_ml[w * ROWS + q].x);
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) {
        const float2 v = s_ml[w * ROWS + q];
        L += v.x == kNegInf ? v.y : v.y * exp2_fast((v.x - Mq) * A.scale_log2);  // (no maximum: zero, or NaN)
      }
      const int64_t row = (it.base_row + qi / A.n) * A.Hq + it.kvh * A.n + qi % A.n;
      if (direct) {
        const uint32_t lo = T::bits(a.x / L) | static_cast<uint32_t>(T::bits(a.y / L)) << 16;
        const uint32_t hi = T::bits(a.z / L) | static_cast<uint32_t>(T::bits(a.w / L)) << 16;
        *reinterpret_cast<uint2 *>(A.out + row * D + d) = make_uint2(lo, hi);
        if (A.lse && d == 0) A.lse[row] = (Mq * A.scale_log2 + log2f(L * (T::kLift > 0 ? 0x1p-15f : 1.0f))) * 0.6931471805599453f;
      } else {
        const int64_t at = it.part * rows_all + row;
        *reinterpret_cast<float4 *>(A.part_o + at * D + d) = a;
        if (d == 0) A.part_ml[at] = make_float2(Mq, L);
      }
    }
  }
}

// Many rows: 32 of them on each of WQ waves, whose 4 / WQ groups take the keys of a
// tile in turn.  Keys and values are widened once, on their way to LDS, for all
// waves: tiles of 64 keys, requested one tile ahead.  Scores are formed transposed,
// as k_attend does it: a lane's exponentials are the operand of the second product.
//
// Bound: 2304 rows of each of 8 kv heads over 8192 8-bit keys are 77 GFLOP, 53 us at
// the rate of a large product; they take 112 (the matrix pipes are busy for 28 percent
// of the cycles, the vector units for 42, both at once for 9).  With the join 123, in
// float16, whose scales are products of their own, 139; 16-bit pages 118 and 124.
// Without its parts one by one: loads -18, values' products -13, exponentials -8,
// widening -8 us.
// Tried: two LDS buffers and one barrier (122 us for 124 alone, 149 for 136 beside
// the sequences' own keys), the next tile's scores beside the softmax (129.5 for 130.5),
// steps of 32 keys (136 for 124), three waves a SIMD (160), tiles of 16 and 48 rows (139 for 132).
template <int DT, bool F8, int D, int WQ>
__device__ __forceinline__ void paged_item(const PagedAttendArgs &A, const PagedItem &it, char *lds, const uint32_t (*s_anc)[8],
                                           float2 *s_ml) {
  using T = AtElt<DT>;
  constexpr int WK = 4 / WQ;
  constexpr int KT = kPgTileKeys;
  constexpr int SB = KT / (32 * WK);  // 32-key blocks per wave and tile
  constexpr int kRow = pg_key_row<D>(), kVRow = pg_value_row<D>();
  constexpr int kBytes = F8 ? 1 : 2;
  constexpr int kChunks = D * kBytes / 16;   // 16-byte pieces of a row
  constexpr int kWaveRows = 64 / kChunks;    // rows of one load of a wave: within a strip
  constexpr int kLoads = KT * kChunks / kAtThreads;
  constexpr bool kRelative = F8 && T::kLift > 0;
  constexpr bool kFolded = F8 && DT == DT_BF16;  // scales' powers of two enter as values are widened (bf16 holds them all)
  uint16_t *s_k = reinterpret_cast<uint16_t *>(lds);
  uint16_t *s_v = s_k + KT * kRow;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave % WQ, wk = wave / WQ;
  const int q32 = lane & 31, half = lane >> 5;

  // A row's 16-byte pieces in LDS: those of 8-bit pages widen to two, the first
  // ones side by side and the second ones behind them, so that 8 lanes write 128
  // bytes.  Place x of a row (8 values) holds d = place_d(x) ..
  auto place_d = [](int x) { return F8 ? 16 * (x % kChunks) + 8 * (x / kChunks) : 8 * x; };
  // this lane's row, its query fragments: places 2 s + half
  const int i = it.row0 + wq * 32 + q32;
  const int ic = min(i, it.rows - 1);
  const int64_t qrow = it.base_row + ic / A.n;
  const int head = it.kvh * A.n + ic % A.n;
  uint4 qf[D / 16];
  {
    const uint16_t *p = A.q + qrow * A.q_row_stride + head * D;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      qf[s] = load_vec(p + place_d(2 * s + half));
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
  int c0 = it.k0;
  int2 strips{};
  float kscale = 1.0f, vscale = 1.0f;
  bool bad = false, whole = true;
  const int last = (it.k1 - 1) & -kStrip;
  auto look_up = [&](int at) {
    c0 = at;
    const int key = min(at + lane * kStrip, last), in_page = key & ((1 << A.pool.page_shift) - 1);
    int page = it.table[key >> A.pool.page_shift];
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(A.pool.num_pages)) page = 0, bad = true;
    strips = strip_offset(A, page, in_page, it.kvh);
    if (F8) {
      const int64_t s = ((static_cast<int64_t>(page) << (A.pool.page_shift - A.pool.block_shift)) + (in_page >> A.pool.block_shift)) * A.pool.Hkv + it.kvh;
      kscale = A.pool.k_scale[s];
      vscale = A.pool.v_scale[s];
      // powers of two alone, as cache_append leaves them, need no products
      if (kFolded) whole = __all(((__float_as_uint(kscale) | __float_as_uint(vscale)) & 0x7FFFFFu) == 0);
    }
  };
  auto power = [](float x) { return __uint_as_float(__float_as_uint(x) & 0x7F800000u); };
  auto rest = [](float x) { return __uint_as_float((__float_as_uint(x) & 0x7FFFFFu) | 0x3F800000u); };
  look_up(it.k0);

  uint4 rk[kLoads], rv[kLoads];
  // scales: of this wave's strips to compute with, of the tile and of the one
  // loaded; of its strips to widen, of the one loaded; whether those of the tile are all powers of two
  float ks[2 * SB], vs[2 * SB], ks_next[2 * SB], vs_next[2 * SB], kw[kLoads], vw[kLoads];
  bool plain_scales = true, plain_next = true;
  const int piece = lane % kChunks;
  constexpr int kStep = 4 * kWaveRows;
  const int row0 = wave * kWaveRows;  // of this wave's first load
  const int row_lane = lane / kChunks;
  static_assert(kStep % kStrip == 0, "a wave's rows have one place in their strips");
  const uint32_t lane_off = static_cast<uint32_t>(row0 % kStrip + row_lane) * static_cast<uint32_t>(A.pool.token_bytes) + piece * 16;
  auto load = [&](int t0) {
    if (t0 - c0 >= kLookup) look_up(t0);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      // (the wave's first row's strip: its rows follow within it)
      const int64_t off = strip_at(strips, (min(t0 + (row0 & -kStrip) + j * kStep, last) - c0) / kStrip);
      rk[j] = load_vec(A.pool.k + off + lane_off);
      rv[j] = load_vec(A.pool.v + off + lane_off);
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int at = (min(t0 + row0 + j * kStep, last) - c0) / kStrip;
      kw[j] = kFolded ? power(read_lane_f32(kscale, at)) : 1.0f;
      vw[j] = kFolded ? power(read_lane_f32(vscale, at)) : 1.0f;
    }
    plain_next = whole;
    if (F8 && !(kFolded && whole))
#pragma unroll
      for (int g = 0; g < 2 * SB; ++g) {
        const int at = (min(t0 + wk * SB * 32 + g * kStrip, last) - c0) / kStrip;
        ks_next[g] = kFolded ? rest(read_lane_f32(kscale, at)) : read_lane_f32(kscale, at);
        vs_next[g] = kFolded ? rest(read_lane_f32(vscale, at)) : read_lane_f32(vscale, at);
      }
  };
  bool odd = false;
  load(it.k0);
  for (int t0 = it.k0; t0 < it.k1; t0 += KT) {
    // Keys past the range get zero values: their exponentials are zero, but
    // zero times what a page holds behind the last token need not be.
    // Infinities and NaN among the step's own values, which must reach only the
    // rows that see them, are left out here and added at the end.
    const bool masked = t0 + KT > it.draft;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int row = row0 + j * kStep + row_lane;
      uint4 v = rv[j];
      if (t0 + KT > it.k1 && t0 + row >= it.k1) v = make_uint4(0, 0, 0, 0);
      if (masked && t0 + row >= it.draft && t0 + row < it.k1) v = drop_odd<DT, F8>(v, &odd);
      if constexpr (F8) {
        uint4 lo, hi;
        widen<DT>(rk[j], kw[j], &lo, &hi);
        *reinterpret_cast<uint4 *>(s_k + row * kRow + piece * 8) = lo;
        *reinterpret_cast<uint4 *>(s_k + row * kRow + (kChunks + piece) * 8) = hi;
        widen<DT>(v, vw[j], &lo, &hi);
        *reinterpret_cast<uint4 *>(s_v + row * kVRow + piece * 8) = lo;
        *reinterpret_cast<uint4 *>(s_v + row * kVRow + (kChunks + piece) * 8) = hi;
      } else {
        *reinterpret_cast<uint4 *>(s_k + row * kRow + piece * 8) = rk[j];
        *reinterpret_cast<uint4 *>(s_v + row * kVRow + piece * 8) = v;
      }
    }
#pragma unroll
    for (int g = 0; g < 2 * SB; ++g) ks[g] = ks_next[g], vs[g] = vs_next[g];
    plain_scales = plain_next;
    __syncthreads();
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
    }
    if (F8 && !(kFolded && plain_scales))
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[sb][e] *= ks[2 * sb + (e >> 3)];
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
      for (int g = 0; g < 2 * SB; ++g) wt[g] = !kRelative ? vs[g] : ref > 0.0f ? vs[g] / ref : 0.0f;  // (scales of zero alone so far)
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
    if (F8 && !(kFolded && plain_scales))
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[sb][e] *= wt[2 * sb + (e >> 3)];
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
          const int d = place_d(t * 4 + f) + 4 * half;
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
        *reinterpret_cast<float4 *>(s_o + (wk * kRows + row) * (D + 4) + place_d(t * 4 + g) + 4 * half) =
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

// A sequence whose length is out of range: its rows of this head are no numbers
// (calls without a join; else the join says so).
template <int DT, int D>
__device__ void no_numbers(const PagedAttendArgs &A, int b, int live, int kvh) {
  for (int z = threadIdx.x; z < live * A.n * (D / 4); z += blockDim.x) {
    const int q = z / (D / 4), c = z % (D / 4);
    const int64_t row = (static_cast<int64_t>(b) * A.R + q / A.n) * A.Hq + kvh * A.n + q % A.n;
    const uint32_t nan2 = DT == DT_BF16 ? 0x7FC07FC0u : 0x7E007E00u;
    *reinterpret_cast<uint2 *>(A.out + row * D + c * 4) = make_uint2(nan2, nan2);
    if (A.lse && c == 0) A.lse[row] = __builtin_nanf("");
  }
}

// The own item of block `id`: false where there is none.  All heads and row
// tiles of a range of one sequence's tokens follow each other on one XCD (8
// blocks apart), every sequence's first range first, the next moved on by one:
// see k_attend.
template <int DT, int D>
__device__ __forceinline__ bool own_item(const PagedAttendArgs &A, int id, int tile_rows, PagedItem *it, bool *direct) {
  const int heads = A.pool.Hkv;
  const int per = heads * A.own_tiles;
  const int j = id / 8;
  const int range = j / per * 8 + id % 8;
  if (range >= A.B * A.own_parts) return false;
  const int tile = j % per % A.own_tiles;
  it->kvh = j % per / A.own_tiles;
  const int split = range / A.B;
  int b = range - split * A.B;
  if (A.B >= 8) {
    b += split & 7;
    if (b >= A.B) b -= A.B;
  }
  const int len = A.ctx_len[b];
  const int live = live_rows(A, b);
  if (live == 0) return false;
  if (bad_len(A, len)) {
    if (A.direct && split == 0 && tile == 0) no_numbers<DT, D>(A, b, live, it->kvh);
    return false;
  }
  const int keys = __builtin_amdgcn_readfirstlane(len + live);
  const int own = attend_own_range(A.split, keys);
  it->row0 = tile * tile_rows;
  it->rows = live * A.n;
  if (static_cast<int64_t>(split) * own >= keys || it->row0 >= it->rows) return false;
  *direct = A.direct && own >= keys;
  it->k0 = split * own;
  it->k1 = min(it->k0 + own, keys);
  it->draft = len;
  it->part = A.prefix_parts + split;
  it->base_row = static_cast<int64_t>(b) * A.R;
  it->table = A.table + b * A.table_stride;
  return true;
}

__device__ __forceinline__ void prefix_item(const PagedAttendArgs &A, int id, int tile_rows, PagedItem *it) {
  // row tiles of one (kv head, range) are Hkv * parts apart: a multiple of 8
  // of those keeps them on one XCD
  const int heads = A.pool.Hkv, pairs = heads * A.prefix_parts;
  const int pair = id % pairs;
  it->kvh = pair % heads;
  it->part = pair / heads;
  it->row0 = id / pairs * tile_rows;
  it->rows = A.B * A.R * A.n;
  it->base_row = 0;
  it->table = A.prefix_table;
  it->k0 = it->part * A.prefix_chunk;
  it->k1 = min(it->k0 + A.prefix_chunk, A.P);
  it->draft = it->k1 + (1 << 30);
}

// Up to 16 NC stacked rows of a sequence.  MANY: the prefix has the rows of a
// batch, in tiles of 128 on four waves; else tiles of 16 NC, if there is a prefix.
// tree: nothing for a window, or the TreeParents.
template <int DT, bool F8, int D, int NC, bool MANY, class... Tree>
__global__ void __launch_bounds__(kAtThreads, F8 && NC == 1 && !MANY ? 4 : 2) k_paged_few(PagedAttendArgs A, Tree... tree) {
  constexpr size_t kOwn = few_bytes<F8, D, NC>(), kPrefix = MANY ? pg_tile_bytes<D, 4>() : 0;
  __shared__ uint4 s_tile[(kOwn > kPrefix ? kOwn : kPrefix) / sizeof(uint4)];
  __shared__ uint32_t s_anc[16 * NC][8];  // (16 stacked rows are 16 rows at most)
  __shared__ uint8_t s_parent[16 * NC];
  __shared__ float2 s_ml[16 * NC * kFewWaves];
  char *lds = reinterpret_cast<char *>(s_tile);
  PagedItem it{};
  if (static_cast<int>(blockIdx.x) < A.prefix_items) {
    prefix_item(A, blockIdx.x, MANY ? 128 : 16 * NC, &it);
    if constexpr (MANY) paged_item<DT, F8, D, 4>(A, it, lds, s_anc, s_ml);
    else few_item<DT, F8, D, NC>(A, it, lds, s_anc, s_ml, false);
    return;
  }
  bool direct = false;
  if (!own_item<DT, D>(A, blockIdx.x - A.prefix_items, 16 * NC, &it, &direct)) return;
  if (it.k1 > it.draft) ancestor_sets(A.R, s_anc, s_parent, tree...);
  __syncthreads();
  few_item<DT, F8, D, NC>(A, it, lds, s_anc, s_ml, direct);
}

// More rows: tiles of 64 or 128 stacked rows of a sequence on 2 or 4 waves (WQO),
// of the prefix 32 or 128 (WQP waves).
template <int DT, bool F8, int D, int WQP, int WQO, class... Tree>
__global__ void __launch_bounds__(kAtThreads, 2) k_paged_attend(PagedAttendArgs A, Tree... tree) {
  constexpr size_t kP = WQP == 1 ? few_bytes<F8, D, 2>() : pg_tile_bytes<D, WQP>();
  constexpr size_t kO = pg_tile_bytes<D, WQO>();
  __shared__ uint4 s_tile[(kP > kO ? kP : kO) / sizeof(uint4)];
  __shared__ uint32_t s_anc[kTreeMaxNodes][8];
  __shared__ uint8_t s_parent[kTreeMaxNodes];
  __shared__ float2 s_ml[128];  // [waves on the same rows][rows]
  char *lds = reinterpret_cast<char *>(s_tile);
  PagedItem it{};
  if (static_cast<int>(blockIdx.x) < A.prefix_items) {
    prefix_item(A, blockIdx.x, 32 * WQP, &it);
    if constexpr (WQP == 1) few_item<DT, F8, D, 2>(A, it, lds, s_anc, s_ml, false);
    else paged_item<DT, F8, D, WQP>(A, it, lds, s_anc, s_ml);
    return;
  }
  bool direct = false;
  if (!own_item<DT, D>(A, blockIdx.x - A.prefix_items, 32 * WQO, &it, &direct)) return;
  if (it.k1 > it.draft) ancestor_sets(A.R, s_anc, s_parent, tree...);
  __syncthreads();
  paged_item<DT, F8, D, WQO>(A, it, lds, s_anc, s_ml);
}

// One wave per (row, head): the row's items joined.  Their maxima and sums are
// read by the lanes, one each, and the outputs 8 at a time, all of them in
// flight; the sums' order is the items'.  18432 rows of 128 with 4 ranges: 12 us
// (38 MB of partial outputs); one token's 32 rows 3.
template <int DT, int D>
__global__ void __launch_bounds__(256) k_paged_join(AttendJoin A, int direct) {
  constexpr int E = D / 64;
  const int rows = A.B * A.R * A.Hq;  // at most 2^30
  const int row = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= rows) return;
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
    const int parts = A.prefix_parts + (keys + own - 1) / own;
    if (direct && parts == 1) return;
    for (int p0 = 0; p0 < parts; p0 += 64) {
      const int n = min(64, parts - p0);
      const float2 ml = lane < n ? A.part_ml[static_cast<int64_t>(p0 + lane) * rows + row] : make_float2(kNegInf, 0.0f);
      float top = ml.x;
#pragma unroll
      for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
      const float mn = fmaxf(M, top);
      const float alpha = M == kNegInf ? 0.0f : exp2_fast((M - mn) * A.scale_log2);
      M = mn;
      L *= alpha;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= alpha;
      const float f = ml.x == kNegInf ? 0.0f : exp2_fast((ml.x - M) * A.scale_log2);
      // (no maximum: the sum is zero, or NaN, which stays)
      L += wave_sum(ml.x == kNegInf ? ml.y : f * ml.y);
      const float *po = A.part_o + (static_cast<int64_t>(p0) * rows + row) * D + lane * E;
      const int64_t step = static_cast<int64_t>(rows) * D;
      for (int p = 0; p < n; p += 8) {
        float v[8][E];
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int e = 0; e < E; ++e) v[x][e] = p + x < n ? po[(p + x) * step + e] : 0.0f;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float w = read_lane_f32(f, min(p + x, 63));
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(w, v[x][e], acc[e]);
        }
      }
    }
  }
  uint16_t *out = A.out + static_cast<int64_t>(row) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = AtElt<DT>::bits(acc[e] / L);
  if (A.lse && lane == 0) A.lse[row] = (M * A.scale_log2 + log2f(L * (AtElt<DT>::kLift > 0 ? 0x1p-15f : 1.0f))) * 0.6931471805599453f;
}

namespace {

// kernel(A) or kernel(A, parents).
template <class Plain, class Tree>
void launch(Plain plain, Tree tree, const PagedAttendArgs &A, const TreeParents *parents, const PagedPlan &P, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(P.prefix_items + P.own_blocks)), threads(kAtThreads);
  if (parents) hipLaunchKernelGGL(tree, grid, threads, 0, st, A, *parents);
  else hipLaunchKernelGGL(plain, grid, threads, 0, st, A);
}

template <int DT, bool F8, int D, int NC>
void launch_few(const PagedAttendArgs &A, const TreeParents *parents, const PagedPlan &P, hipStream_t st) {
  using T = TreeParents;
  if (P.prefix_items > 0 && P.prefix_waves == 4) launch(k_paged_few<DT, F8, D, NC, true>, k_paged_few<DT, F8, D, NC, true, T>, A, parents, P, st);
  else launch(k_paged_few<DT, F8, D, NC, false>, k_paged_few<DT, F8, D, NC, false, T>, A, parents, P, st);
}

template <int DT, bool F8, int D>
void launch_dim(const PagedAttendArgs &A, const TreeParents *parents, const PagedPlan &P, hipStream_t st) {
  using T = TreeParents;
  if (P.few == 16) {
    launch_few<DT, F8, D, 1>(A, parents, P, st);
  } else if (P.few == 32) {
    launch_few<DT, F8, D, 2>(A, parents, P, st);
  } else if (P.few == 48) {
    if constexpr (paged_few_rows(F8) == 48) launch_few<DT, F8, D, 3>(A, parents, P, st);
  } else if (P.prefix_waves == 4) {
    // (a sequence's rows are no more than the batch's: 4 waves on them mean 4 on the prefix)
    if (P.own_waves == 4) launch(k_paged_attend<DT, F8, D, 4, 4>, k_paged_attend<DT, F8, D, 4, 4, T>, A, parents, P, st);
    else launch(k_paged_attend<DT, F8, D, 4, 2>, k_paged_attend<DT, F8, D, 4, 2, T>, A, parents, P, st);
  } else {
    launch(k_paged_attend<DT, F8, D, 1, 2>, k_paged_attend<DT, F8, D, 1, 2, T>, A, parents, P, st);
  }
  if (P.direct && P.own_parts == 1) return;
  const int64_t rows = static_cast<int64_t>(A.B) * A.R * A.Hq;
  hipLaunchKernelGGL((k_paged_join<DT, D>), dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, st,
                     static_cast<const AttendJoin &>(A), A.direct);
}

template <int DT, bool F8>
void launch_cache(int D, const PagedAttendArgs &A, const TreeParents *parents, const PagedPlan &P, hipStream_t st) {
  if (D == 64) launch_dim<DT, F8, 64>(A, parents, P, st);
  else launch_dim<DT, F8, 128>(A, parents, P, st);
}

}  // namespace

void launch_paged_attend(int dtype, bool f8, int D, const PagedAttendArgs &A, const TreeParents *parents, const PagedPlan &P, hipStream_t st) {
  if (dtype == DT_BF16) {
    if (f8) launch_cache<DT_BF16, true>(D, A, parents, P, st);
    else launch_cache<DT_BF16, false>(D, A, parents, P, st);
  } else {
    if (f8) launch_cache<DT_F16, true>(D, A, parents, P, st);
    else launch_cache<DT_F16, false>(D, A, parents, P, st);
  }
}

}  // namespace sv
