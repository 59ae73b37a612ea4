// LM head on 4-bit weights with group scales (gfx950).
//
//   logits[m][v] = sum_g s[v][g] sum_{k in g} h[m][k] (q[v][k] - z[v][g])
//
// The nibbles go to the matrix cores as exact numbers: OR-ing one into the
// mantissa of 16.0 gives 16 + q in bf16 and f16, two per instruction.  The
// group's sum of h (16 + q) then accumulates in float32 from the start value
// -(16 + z) sum(h), and is scaled by s in float32 into the total, so no weight
// is rounded and the only errors are those of float32 sums (the 16 costs a
// factor of about 5 in their size; the 128 of an unshifted bf16 mantissa
// would cost 27).
//
// v_mfma_f32_16x16x32: lane l supplies A[l % 16][8 (l / 16) + j] and the same
// of B's column l % 16; accumulator register r of lane l is
// C[4 (l / 16) + r][l % 16].  Weight rows are loaded 128 bytes at a time (8
// lanes a row: whole cache lines; 16 rows of 64 bytes ran a third slower), and
// pass through a piece of LDS of their wave's own to the lanes that multiply
// them.  Within 8 values the order is 0 4 1 5 2 6 3 7 (the nibble pairs of a
// dword), and the hidden rows are stored to LDS in that order, with the sums of
// their groups.
//
// Measured at K = 4096, groups of 128: V = 128256 (263 MB of weights), M = 8: 54
// us, 5.1 TB/s; M = 72: 121 us, where vector work (39%), matrix work (29%) and
// LDS (32%) take turns, as registers leave room for two waves per SIMD; M =
// 576: 823 to 850 us, 710 to 736 TFLOP/s, as every 64 rows unpack the weights
// again; V = 50257, M = 256: 160 us, 650 TFLOP/s, and 235 us with groups of
// 32, whose scaling is four times the vector work.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_device.h"
#include "sv_launch.h"
#include "sv_plan.h"

namespace sv {

typedef __bf16 q_bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 q_f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 q_bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 q_f16x2_t __attribute__((ext_vector_type(2)));
typedef float q_f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kQStep = 128;               // K values per step: 16 bytes of weights per lane
constexpr int kQThreads = kLmQuantThreads;
constexpr int kQWaves = kQThreads / 64;

template <int DT> struct QuantElt;
template <> struct QuantElt<DT_BF16> {
  static constexpr uint32_t kOne = 0x41804180u, kMask = 0x00780078u;  // 16.0 twice; the nibble's mantissa bits
  static constexpr int kShift = 3;
  // c + the two values of a, in float32
  __device__ static __forceinline__ float sum2(uint32_t a, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(q_bf16x2_t, a), __builtin_bit_cast(q_bf16x2_t, 0x3F803F80u), c, false);
  }
  __device__ static __forceinline__ q_f32x4_t mma(uint4 a, uint4 b, q_f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(q_bf16x8_t, a), __builtin_bit_cast(q_bf16x8_t, b), c, 0, 0, 0);
  }
};
template <> struct QuantElt<DT_F16> {
  static constexpr uint32_t kOne = 0x4C004C00u, kMask = 0x03C003C0u;
  static constexpr int kShift = 6;
  __device__ static __forceinline__ float sum2(uint32_t a, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(q_f16x2_t, a), __builtin_bit_cast(q_f16x2_t, 0x3C003C00u), c, false);
  }
  __device__ static __forceinline__ q_f32x4_t mma(uint4 a, uint4 b, q_f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(q_f16x8_t, a), __builtin_bit_cast(q_f16x8_t, b), c, 0, 0, 0);
  }
};

// The 8 values 16 + q of a dword of nibbles, in the order 0 4 1 5 2 6 3 7.  The
// two constants come in registers, one of them scalar: only then do AND and OR
// become one instruction.
template <int DT> __device__ __forceinline__ uint4 unpack8(uint32_t w, uint32_t mask, uint32_t one) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int sh = QuantElt<DT>::kShift - 4 * i;
    o[i] = ((sh >= 0 ? w << (sh >= 0 ? sh : 0) : w >> (sh >= 0 ? 0 : -sh)) & mask) | one;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight hidden values in the order of unpack8, and their sum.
__device__ __forceinline__ uint4 permute8(uint4 v) {
  return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                    __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
}
template <int DT> __device__ __forceinline__ float sum8(uint4 v) {
  using Q = QuantElt<DT>;
  return Q::sum2(v.x, Q::sum2(v.y, Q::sum2(v.z, Q::sum2(v.w, 0.0f))));
}
// Sum over the lanes (8 values each) that hold one group, in every one of them.
template <int kGroup> __device__ __forceinline__ float group_sum(float s) {
  s += dpp_f32<0xB1>(s);
  s += dpp_f32<0x4E>(s);
  if (kGroup >= 64) s += dpp_f32<0x141>(s);   // the other half of 8 lanes
  if (kGroup >= 128) s += dpp_f32<0x140>(s);  // the other half of 16 lanes
  return s;
}

// Rows of 16 lanes (quads) hold the 16-byte blocks b0..b3 of a step, 32 values
// each.  One MFMA multiplies one register of all four, so dwords are exchanged
// between the quads until a register holds values of one group only: not at
// all for groups of 128, between the halves of the wave for 64, and a full 4 x
// 4 exchange for 32.  step_at() is where register s of a quad then lies.
template <int kGroup> __device__ __forceinline__ void exchange(uint32_t (&r)[4]) {
  if (kGroup <= 64)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto p = __builtin_amdgcn_permlane32_swap(r[i], r[i + 2], false, false);
      r[i] = p[0];
      r[i + 2] = p[1];
    }
  if (kGroup <= 32)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const auto p = __builtin_amdgcn_permlane16_swap(r[i], r[i + 1], false, false);
      r[i] = p[0];
      r[i + 1] = p[1];
    }
}
template <int kGroup> __device__ __forceinline__ int step_at(int s, int quad) {
  if (kGroup == 32) return s * 32 + quad * 8;
  if (kGroup == 64) return ((s & 2) + (quad & 1)) * 32 + ((quad & 2) + (s & 1)) * 8;
  return quad * 32 + s * 8;
}

// Where the 16-byte piece p of a hidden row lies in its LDS row: exclusive-ored
// with the row, so that the 16 lanes one cycle pair serves (rows 0-3 and 12-15
// of one quad, 4-11 of the next) meet 16 different bank groups.  Neighbouring
// quads' pieces differ in bit 2 (bit 0 for groups of 32), which rows 4-11 undo.
template <int kGroup> __device__ __forceinline__ int a_slot(int p, int row) {
  const int f = (row & 15) ^ (kGroup == 32 ? 0 : 4 * ((row >> 2 ^ row >> 3) & 1));
  return p ^ f;
}

// A workgroup barrier that orders LDS only: global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <int DT> __device__ __forceinline__ void store_logit(const LmQuantArgs &A, int64_t at, float x) {
  if (A.out_f32) static_cast<float *>(A.out)[at] = x;
  else if (DT == DT_BF16) static_cast<__bf16 *>(A.out)[at] = static_cast<__bf16>(x);
  else static_cast<_Float16 *>(A.out)[at] = static_cast<_Float16>(x);
}

// Hidden rows of a call with many of them, laid out once: permuted as the tiles
// want them, zeros up to a whole chunk, and the sums of their groups
// ([group][row]).  The product's workgroups then copy them as they are; doing
// this in each of them took a third of their vector instructions.
template <int DT>
__global__ void __launch_bounds__(256) k_lm_prepare(LmQuantArgs A) {
  const int piece = blockIdx.x * 256 + threadIdx.x, row = blockIdx.y;
  const int pieces = A.padded / 8;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (piece * 8 < A.K) v = load_vec(A.h + row * A.lda + piece * 8);
  const float s8 = sum8<DT>(v);
  const float s32 = group_sum<32>(s8), s64 = group_sum<64>(s8), s128 = group_sum<128>(s8);
  if (piece >= pieces) return;
  const int per = A.group / 8;
  if (piece % per == 0) A.sums[static_cast<int64_t>(piece / per) * A.M + row] = A.group == 32 ? s32 : A.group == 64 ? s64 : s128;
  *reinterpret_cast<uint4 *>(A.prepared + static_cast<int64_t>(row) * A.padded + piece * 8) = permute8(v);
}

// MT x NT tiles of 16 x 16 per wave; the waves of a team lie side by side along
// V and share the hidden rows, scales and zero points of kChunk values of K in
// LDS.  kGroup: values per scale.  Weights go from memory to registers a chunk
// ahead and stay in flight across the barriers.  kSplit = 1: the workgroup is
// one team.  kSplit = 4 (problems with too few columns to fill the chip): every
// wave is a team of its own on the same columns, takes every fourth chunk of K
// without any barrier, and the four sums are added in wave order at the end.
// kPrepared: the hidden rows come from k_lm_prepare.
template <int DT, int MT, int NT, int kGroup, int kChunk, int kSplit, bool kPrepared>
__global__ void __launch_bounds__(kQThreads, MT * NT <= 2 && kSplit == 1 ? 4 : MT == 2 && kSplit == 4 ? 1 : 2) k_lm_quant(LmQuantArgs A) {
  using E = Elt<DT>;
  using Q = QuantElt<DT>;
  constexpr int kTeamWaves = kQWaves / kSplit, kTeamThreads = kQThreads / kSplit;
  constexpr int kRows = 16 * MT, kCols = 16 * NT * kTeamWaves;
  constexpr int kSteps = kChunk / kQStep;
  constexpr int kG = kQStep / kGroup, kGC = kChunk / kGroup;  // groups per step and chunk
  constexpr int kSub = kGroup / 32;                           // MFMAs per group and tile
  constexpr int kPieces = kChunk / 8;                         // 16-byte pieces per row of a chunk
  constexpr int kRowsPerPass = kTeamThreads / kPieces;
  constexpr int kLoads = kRows / kRowsPerPass;
  constexpr int kScales = (kGC * kCols + kTeamThreads - 1) / kTeamThreads;
  static_assert(kRows % kRowsPerPass == 0, "whole passes");
  static_assert(kSplit == 1 || kSplit == kQWaves, "teams are the workgroup or its waves");
  __shared__ uint16_t s_as[kSplit][kRows * kChunk];
  __shared__ uint4 s_w[kQWaves][NT][128];  // a step's weights on their way to the lanes that multiply them
  __shared__ float s_sums[kSplit][kGC][kRows];    // sums of the hidden values per group
  __shared__ float2 s_scales[kSplit][kGC][kCols];  // scale, -(16 + zero)
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int team = kSplit > 1 ? wave : 0, team_wave = kSplit > 1 ? 0 : wave;
  const int tid = kSplit > 1 ? lane : threadIdx.x;  // within the team
  uint16_t *s_a = s_as[team];
  float(*s_sum)[kRows] = s_sums[team];
  float2(*s_scale)[kCols] = s_scales[team];
  const int c16 = lane & 15, quad = lane >> 4;
  // column tiles round the XCDs, the row blocks of one column tile on one XCD
  const int ct = blockIdx.x / (8 * A.row_blocks) * 8 + blockIdx.x % 8;
  const int row0 = blockIdx.x / 8 % A.row_blocks * kRows;
  const int col0 = ct * kCols;
  if (col0 >= A.V) return;
  const int chunks_all = (A.K + kChunk - 1) / kChunk;
  const int groups = A.K / kGroup, blocks = A.K / 32;
  // this workgroup's chunks of K: all, or (prepared rows) blockIdx.y's share
  const int begin = kPrepared ? blockIdx.y * A.split_chunks : 0;
  const int chunks = kPrepared ? min(begin + A.split_chunks, chunks_all) : chunks_all;

  uint4 ra[kLoads];
  const int piece = tid % kPieces, first = tid / kPieces;
  // prepared rows: offsets from the tile's first (past M: the last row again, whose products are not stored)
  constexpr int kSums = (kGC * kRows + kTeamThreads - 1) / kTeamThreads;
  float rsum[kSums];
  uint32_t aoff[kLoads];
  const uint16_t *atile = A.prepared + static_cast<int64_t>(row0) * A.padded;
  if constexpr (kPrepared)
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      aoff[j] = static_cast<uint32_t>(min(first + j * kRowsPerPass, A.M - 1 - row0)) * A.padded + piece * 8;
  auto load_a = [&](int chunk) {
    if constexpr (kPrepared) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) ra[j] = load_vec(atile + chunk * kChunk + aoff[j]);
#pragma unroll
      for (int j = 0; j < kSums; ++j) {
        const int x = min(tid + j * kTeamThreads, kGC * kRows - 1);
        rsum[j] = as_global<float>(A.sums)[static_cast<int64_t>(chunk * kGC + x / kRows) * A.M + min(row0 + x % kRows, A.M - 1)];
      }
    } else {
      const bool in = chunk * kChunk + piece * 8 < A.K;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = row0 + first + j * kRowsPerPass;
        ra[j] = make_uint4(0, 0, 0, 0);
        if (in && r < A.M) ra[j] = load_vec(A.h + r * A.lda + chunk * kChunk + piece * 8);
      }
    }
  };
  auto store_a = [&]() {
    if constexpr (kPrepared) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        *reinterpret_cast<uint4 *>(&s_a[(first + j * kRowsPerPass) * kChunk + a_slot<kGroup>(piece, first + j * kRowsPerPass) * 8]) = ra[j];
#pragma unroll
      for (int j = 0; j < kSums; ++j) {
        const int x = tid + j * kTeamThreads;
        if (x < kGC * kRows) s_sum[x / kRows][x % kRows] = rsum[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = first + j * kRowsPerPass;
        if (row0 + r >= A.M) continue;  // these rows were zeroed once
        const float s = group_sum<kGroup>(sum8<DT>(ra[j]));
        if (piece % (kGroup / 8) == 0) s_sum[piece / (kGroup / 8)][r] = s;
        *reinterpret_cast<uint4 *>(&s_a[r * kChunk + a_slot<kGroup>(piece, r) * 8]) = permute8(ra[j]);
      }
    }
  };
  uint32_t rs[kScales], rz[kScales];
  auto load_scales = [&](int chunk) {
#pragma unroll
    for (int j = 0; j < kScales; ++j) {
      const int x = tid + j * kTeamThreads;
      const int64_t v = min(col0 + x / kGC, A.V - 1);
      const int g = min(chunk * kGC + x % kGC, groups - 1);
      rs[j] = E::raw(A.scales, v * groups + g);
      rz[j] = A.zeros ? as_global<uint8_t>(A.zeros)[v * groups + g] : 8u;
    }
  };
  auto store_scales = [&]() {
#pragma unroll
    for (int j = 0; j < kScales; ++j) {
      const int x = tid + j * kTeamThreads;
      if (x < kGC * kCols) s_scale[x % kGC][x / kGC] = make_float2(E::dec(rs[j]), -16.0f - static_cast<float>(rz[j]));
    }
  };
  // Weights arrive two steps at a time: one load takes 8 rows of 128 bytes (a
  // cache line each), two loads the 16 rows of a tile.  Rows past V: the last
  // row, never stored.  Where K ends inside the two steps, blocks past it meet
  // zero hidden values, and the row's last block stands in for them.
  const uint8_t *wtile = A.w + col0 * static_cast<int64_t>(A.K / 2);
  const int last = (A.K - 1) / (2 * kQStep);
  uint32_t woff[NT][2], wtail[NT][2];
  uint4 rw[kSteps][NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = i * 8 + (lane >> 3), block = (lane & 7) ^ (n & 7);
      woff[t][i] = static_cast<uint32_t>(min(team_wave * NT * 16 + t * 16 + n, A.V - 1 - col0)) * (A.K / 2) + block * 16;
      wtail[t][i] = woff[t][i] - max(last * 8 + block - (blocks - 1), 0) * 16;
    }
  auto load_w = [&](int slot, int pair) {
    const int at = min(pair, last);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        rw[slot + i][t] = load_stream(reinterpret_cast<const uint4 *>(wtile + at * 128 + (at == last ? wtail[t][i] : woff[t][i])));
  };
  uint32_t mask, one;
  asm("s_mov_b32 %0, %1" : "=s"(mask) : "i"(Q::kMask));
  asm("v_mov_b32 %0, %1" : "=v"(one) : "i"(Q::kOne));

  q_f32x4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = q_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  auto team_barrier = [&]() {
    if (kSplit > 1) __builtin_amdgcn_wave_barrier();
    else lds_barrier();
  };
  load_a(min(begin + team, chunks - 1));
  load_scales(min(begin + team, chunks - 1));
#pragma unroll
  for (int u = 0; u < kSteps; u += 2) load_w(u, ((begin + team) * kSteps + u) / 2);
  for (int r = A.M - row0 + team_wave; !kPrepared && r < kRows; r += kTeamWaves) {
    for (int x = lane; x < kPieces; x += 64) *reinterpret_cast<uint4 *>(&s_a[r * kChunk + x * 8]) = make_uint4(0, 0, 0, 0);
    if (lane < kGC) s_sum[lane][r] = 0.0f;
  }
  for (int c = begin + team; c < chunks; c += kSplit) {
    if (c >= begin + kSplit) team_barrier();  // every wave is done with the previous chunk
    store_a();
    store_scales();
    load_a(min(c + kSplit, chunks - 1));
    load_scales(min(c + kSplit, chunks - 1));
    team_barrier();
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      uint32_t w[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (u % 2 == 0) {
          s_w[wave][t][lane] = rw[u][t];
          s_w[wave][t][64 + lane] = rw[u + 1][t];
        }
        const uint4 x = s_w[wave][t][c16 * 8 + ((u % 2 * 4 + quad) ^ (c16 & 7))];
        w[t][0] = x.x;
        w[t][1] = x.y;
        w[t][2] = x.z;
        w[t][3] = x.w;
        exchange<kGroup>(w[t]);
      }
      if (u % 2 == 0) load_w(u, ((c + kSplit) * kSteps + u) / 2);  // past the end: the last steps again, unused
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        q_f32x4_t part[MT][NT];
        float2 sc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) sc[t] = s_scale[u * kG + g][(team_wave * NT + t) * 16 + c16];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float4 hs = *reinterpret_cast<const float4 *>(&s_sum[u * kG + g][m * 16 + quad * 4]);
#pragma unroll
          for (int t = 0; t < NT; ++t) part[m][t] = q_f32x4_t{sc[t].y * hs.x, sc[t].y * hs.y, sc[t].y * hs.z, sc[t].y * hs.w};
        }
#pragma unroll
        for (int s = g * kSub; s < (g + 1) * kSub; ++s) {
          uint4 b[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) b[t] = unpack8<DT>(w[t][s], mask, one);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 a = *reinterpret_cast<const uint4 *>(&s_a[(m * 16 + c16) * kChunk + a_slot<kGroup>(u * (kQStep / 8) + step_at<kGroup>(s, quad) / 8, c16) * 8]);
#pragma unroll
            for (int t = 0; t < NT; ++t) part[m][t] = Q::mma(a, b[t], part[m][t]);
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][t][e] = __builtin_fmaf(sc[t].x, part[m][t][e], acc[m][t][e]);
        // one group's partial sums at a time: interleaving several would spill
        if (MT * NT > 2) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (kSplit > 1) {
    // wave order: each adds its sums to those before it
    __shared__ float4 s_acc[MT][NT][64];
    for (int z = 0; z < kSplit; ++z) {
      __syncthreads();
      if (z != wave) continue;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (z > 0) {
            const float4 x = s_acc[m][t][lane];
            acc[m][t] = q_f32x4_t{x.x + acc[m][t][0], x.y + acc[m][t][1], x.z + acc[m][t][2], x.w + acc[m][t][3]};
          }
          s_acc[m][t][lane] = make_float4(acc[m][t][0], acc[m][t][1], acc[m][t][2], acc[m][t][3]);
        }
    }
    if (wave != kSplit - 1) return;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int v = col0 + (team_wave * NT + t) * 16 + c16;
    if (v >= A.V) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = row0 + m * 16 + quad * 4 + e;
        if (r >= A.M) continue;
        if (kPrepared && A.splits > 1)
          A.partial[(static_cast<int64_t>(blockIdx.y) * A.M + r) * A.V + v] = acc[m][t][e];
        else
          store_logit<DT>(A, r * A.out_stride + v, acc[m][t][e]);
      }
  }
}

// The shares of K of every logit, added in order.
template <int DT>
__global__ void __launch_bounds__(256) k_lm_join(LmQuantArgs A) {
  const int v = blockIdx.x * 256 + threadIdx.x, r = blockIdx.y;
  if (v >= A.V) return;
  const float *p = A.partial + static_cast<int64_t>(r) * A.V + v;
  float x = p[0];
  for (int s = 1; s < A.splits; ++s) x += p[static_cast<int64_t>(s) * A.M * A.V];
  store_logit<DT>(A, r * A.out_stride + v, x);
}

namespace {

template <int DT, int MT, int NT, int kChunk, int kSplit = 1, bool kPrepared = false>
void launch_tiles(LmQuantArgs A, hipStream_t st) {
  const int cols = 16 * NT * kQWaves / kSplit;
  A.row_blocks = (A.M + 16 * MT - 1) / (16 * MT);
  dim3 grid(static_cast<unsigned>((A.V + cols - 1) / cols + 7) / 8 * 8 * A.row_blocks);
  grid.y = kPrepared ? A.splits : 1;
  if (kPrepared)
    hipLaunchKernelGGL(k_lm_prepare<DT>, dim3((A.padded / 8 + 255) / 256, A.M), dim3(256), 0, st, A);
  if (A.group == 32)
    hipLaunchKernelGGL((k_lm_quant<DT, MT, NT, 32, kChunk, kSplit, kPrepared>), grid, dim3(kQThreads), 0, st, A);
  else if (A.group == 64)
    hipLaunchKernelGGL((k_lm_quant<DT, MT, NT, 64, kChunk, kSplit, kPrepared>), grid, dim3(kQThreads), 0, st, A);
  else
    hipLaunchKernelGGL((k_lm_quant<DT, MT, NT, 128, kChunk, kSplit, kPrepared>), grid, dim3(kQThreads), 0, st, A);
  if (kPrepared && A.splits > 1)
    hipLaunchKernelGGL(k_lm_join<DT>, dim3((A.V + 255) / 256, A.M), dim3(256), 0, st, A);
}

// Tiles by rows: the fewest 16-row tiles that hold them, as weights are
// unpacked once per row block; past 32 rows in blocks of 64 or 80.  Small
// vocabularies share K out: among a workgroup's waves up to 32 rows, while
// 16-column workgroups fill the chip about twice at most (us at K = 4096: M = 4,
// V = 8000 11, not shared 18; M = 16, V = 16000 20 and 14; M = 24, V = 8000 16 and
// 39), among workgroups beyond (M = 64, V = 8000 25 and 42; M = 200, V = 4000 35
// and 52), see lm_quant_layout.
template <int DT>
void launch_type(const LmQuantArgs &A, hipStream_t st) {
  const int64_t M = A.M, tiles = (A.V + 15) / 16;
  if (M <= 16 && tiles <= 640)
    launch_tiles<DT, 1, 1, 256, 4>(A, st);
  else if (M <= 16 && A.V < 512 * 128)
    launch_tiles<DT, 1, 1, 512>(A, st);  // 64 columns: 128 would leave CUs idle (V = 32000: 11 us, 13 with 128)
  else if (M <= 16)
    launch_tiles<DT, 1, 2, 256>(A, st);  // (V = 128256, M = 8: 55 us, 65 with 64 columns)
  else if (M <= kLmQuantDirectRows && tiles <= 1024)
    launch_tiles<DT, 2, 1, 256, 4>(A, st);
  else if (M <= kLmQuantDirectRows)
    launch_tiles<DT, 2, 2, 256>(A, st);
  else if (lm_quant_rows(M) == 64)
    launch_tiles<DT, 4, 2, 256, 1, true>(A, st);
  else
    launch_tiles<DT, 5, 2, 256, 1, true>(A, st);
}

}  // namespace

void launch_lm_quant(int dtype, const LmQuantArgs &A, hipStream_t st) {
  if (dtype == DT_BF16) launch_type<DT_BF16>(A, st);
  else launch_type<DT_F16>(A, st);
}

}  // namespace sv
