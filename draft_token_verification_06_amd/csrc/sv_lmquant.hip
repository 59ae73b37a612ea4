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
// C[4 (l / 16) + r][l % 16].  A lane loads 16 bytes (32 values) of one weight
// row, four lanes 64 contiguous bytes; a 4 x 4 exchange of dwords between
// those four lanes (two lane-swap instructions per pair) gives every lane the
// 8 values of each 32-value step, in the rows' own layout.  Within 8 values
// the order is 0 4 1 5 2 6 3 7 (the nibble pairs of a dword), and the hidden
// rows are stored to LDS in that order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_device.h"
#include "sv_launch.h"
#include "sv_plan.h"

namespace sv {

typedef __bf16 q_bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 q_f16x8_t __attribute__((ext_vector_type(8)));
typedef float q_f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kQStep = 128;               // K values per step: 16 bytes of weights per lane
constexpr int kQRow = kQStep + 8;         // LDS row of a step: 16 bytes of padding spread the banks
constexpr int kQThreads = kLmQuantThreads;
constexpr int kQWaves = kQThreads / 64;

template <int DT> struct QuantElt;
template <> struct QuantElt<DT_BF16> {
  static constexpr uint32_t kOne = 0x41804180u, kMask = 0x00780078u;  // 16.0 twice; the nibble's mantissa bits
  static constexpr int kShift = 3;
  __device__ static __forceinline__ q_f32x4_t mma(uint4 a, uint4 b, q_f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(q_bf16x8_t, a), __builtin_bit_cast(q_bf16x8_t, b), c, 0, 0, 0);
  }
};
template <> struct QuantElt<DT_F16> {
  static constexpr uint32_t kOne = 0x4C004C00u, kMask = 0x03C003C0u;
  static constexpr int kShift = 6;
  __device__ static __forceinline__ q_f32x4_t mma(uint4 a, uint4 b, q_f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(q_f16x8_t, a), __builtin_bit_cast(q_f16x8_t, b), c, 0, 0, 0);
  }
};

// The 8 values 16 + q of a dword of nibbles, in the order 0 4 1 5 2 6 3 7.
template <int DT> __device__ __forceinline__ uint4 unpack8(uint32_t w) {
  using Q = QuantElt<DT>;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int sh = Q::kShift - 4 * i;
    o[i] = ((sh >= 0 ? w << (sh >= 0 ? sh : 0) : w >> (sh >= 0 ? 0 : -sh)) & Q::kMask) | Q::kOne;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Rows of 16 lanes hold 16-byte blocks b0..b3 of 64 bytes; afterwards register
// s of the row g holds dword g of block s.
__device__ __forceinline__ void exchange4(uint32_t (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto p = __builtin_amdgcn_permlane32_swap(r[i], r[i + 2], false, false);
    r[i] = p[0];
    r[i + 2] = p[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const auto p = __builtin_amdgcn_permlane16_swap(r[i], r[i + 1], false, false);
    r[i] = p[0];
    r[i + 1] = p[1];
  }
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

// MT x NT tiles of 16 x 16 per wave; the waves of a workgroup lie side by
// side along V.  kGroup: values per scale.
template <int DT, int MT, int NT, int kGroup, int PF>
__global__ void __launch_bounds__(kQThreads) k_lm_quant(LmQuantArgs A) {
  using E = Elt<DT>;
  using Q = QuantElt<DT>;
  constexpr int kRows = 16 * MT;
  constexpr int kG = kQStep / kGroup;              // groups per step
  constexpr int kSub = kGroup / 32;                // MFMA steps per group
  constexpr int kLoads = kRows * (kQStep / 8) / kQThreads;  // 16-byte loads of a step's hidden rows per thread
  __shared__ uint16_t s_a[2][kRows * kQRow];
  __shared__ float s_sum[2][kG][kRows];  // sums of the hidden values per group
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c16 = lane & 15, quad = lane >> 4;
  const int row0 = blockIdx.y * kRows;
  const int col0 = (blockIdx.x * kQWaves + wave) * (16 * NT);
  const int steps = (A.K + kQStep - 1) / kQStep;
  const int groups = A.K / kGroup;

  // hidden rows of a step: thread -> row (tid / 16) + 16 j, 16-byte piece tid % 16
  uint4 ra[kLoads];
  const int piece = tid & 15;
  const uint16_t *hrow[kLoads];
  bool live[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = row0 + (tid >> 4) + 16 * j;
    live[j] = r < A.M;
    hrow[j] = A.h + (live[j] ? r : 0) * A.lda + piece * 8;
  }
  auto load_a = [&](int step) {
    const bool in = step * kQStep + piece * 8 < A.K;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      ra[j] = in && live[j] ? load_vec(hrow[j] + step * kQStep) : make_uint4(0, 0, 0, 0);
  };
  auto store_a = [&](int buf) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      float x[8];
      E::vec(ra[j], x);
      float s = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
      s += dpp_f32<0xB1>(s);
      s += dpp_f32<0x4E>(s);
      if (kGroup >= 64) s += dpp_f32<0x141>(s);   // the other half of 8 lanes
      if (kGroup >= 128) s += dpp_f32<0x140>(s);  // the other half of 16 lanes
      const int r = (tid >> 4) + 16 * j;
      if (piece % (kGroup / 8) == 0) s_sum[buf][piece / (kGroup / 8)][r] = s;
      const uint4 v = ra[j];
      const uint4 p = make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                                 __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
      *reinterpret_cast<uint4 *>(&s_a[buf][r * kQRow + piece * 8]) = p;
    }
  };

  // weight rows of this lane's columns (past V: the last row, never stored)
  const uint8_t *wrow[NT];
  const uint16_t *srow[NT];
  const uint8_t *zrow[NT];
  uint4 rw[PF][NT];
  uint32_t rs[PF][NT][kG], rz[PF][NT][kG];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t v = min(col0 + t * 16 + c16, A.V - 1);
    wrow[t] = A.w + v * (A.K / 2);
    srow[t] = A.scales + v * groups;
    zrow[t] = A.zeros ? A.zeros + v * groups : nullptr;
  }
  auto load_w = [&](int slot, int step) {
    // blocks and groups past the end meet zero hidden values: any in-bounds data will do
    const int block = min(step * 4 + quad, A.K / 32 - 1);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      rw[slot][t] = load_vec(wrow[t] + block * 16);
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const int at = min(step * kG + g, groups - 1);
        rs[slot][t][g] = E::raw(srow[t], at);
        rz[slot][t][g] = A.zeros ? as_global<uint8_t>(zrow[t])[at] : 8u;
      }
    }
  };

  q_f32x4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = q_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  load_a(0);
#pragma unroll
  for (int u = 0; u < PF; ++u) load_w(u, min(u, steps - 1));
  store_a(0);
  load_a(min(1, steps - 1));
  lds_barrier();
  for (int i0 = 0; i0 < steps; i0 += PF) {
#pragma unroll
    for (int u = 0; u < PF; ++u) {
      const int i = i0 + u;
      if (i >= steps) break;
      const int buf = i & 1;
      // Stage the next step while this one multiplies: the buffer it goes to
      // was last read before the barrier that ended the previous step.
      store_a(buf ^ 1);
      load_a(min(i + 2, steps - 1));
      uint32_t w[NT][4];
      float sc[NT][kG], zp[NT][kG];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        w[t][0] = rw[u][t].x;
        w[t][1] = rw[u][t].y;
        w[t][2] = rw[u][t].z;
        w[t][3] = rw[u][t].w;
        exchange4(w[t]);
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          sc[t][g] = E::dec(rs[u][t][g]);
          zp[t][g] = -16.0f - static_cast<float>(rz[u][t][g]);
        }
      }
      load_w(u, min(i + PF, steps - 1));
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        q_f32x4_t part[MT][NT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float4 hs = *reinterpret_cast<const float4 *>(&s_sum[buf][g][m * 16 + quad * 4]);
#pragma unroll
          for (int t = 0; t < NT; ++t) part[m][t] = q_f32x4_t{zp[t][g] * hs.x, zp[t][g] * hs.y, zp[t][g] * hs.z, zp[t][g] * hs.w};
        }
#pragma unroll
        for (int s = g * kSub; s < (g + 1) * kSub; ++s) {
          uint4 b[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) b[t] = unpack8<DT>(w[t][s]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 a = *reinterpret_cast<const uint4 *>(&s_a[buf][(m * 16 + c16) * kQRow + s * 32 + quad * 8]);
#pragma unroll
            for (int t = 0; t < NT; ++t) part[m][t] = Q::mma(a, b[t], part[m][t]);
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][t][e] = __builtin_fmaf(sc[t][g], part[m][t][e], acc[m][t][e]);
      }
      lds_barrier();
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int v = col0 + t * 16 + c16;
    if (v >= A.V) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = row0 + m * 16 + quad * 4 + e;
        if (r < A.M) store_logit<DT>(A, r * A.out_stride + v, acc[m][t][e]);
      }
  }
}

namespace {

template <int DT, int MT, int NT, int PF>
void launch_tiles(const LmQuantArgs &A, hipStream_t st) {
  const dim3 grid((A.V + 16 * NT * kQWaves - 1) / (16 * NT * kQWaves), (A.M + 16 * MT - 1) / (16 * MT));
  if (A.group == 32)
    hipLaunchKernelGGL((k_lm_quant<DT, MT, NT, 32, PF>), grid, dim3(kQThreads), 0, st, A);
  else if (A.group == 64)
    hipLaunchKernelGGL((k_lm_quant<DT, MT, NT, 64, PF>), grid, dim3(kQThreads), 0, st, A);
  else
    hipLaunchKernelGGL((k_lm_quant<DT, MT, NT, 128, PF>), grid, dim3(kQThreads), 0, st, A);
}

template <int DT>
void launch_type(const LmQuantArgs &A, hipStream_t st) {
  if (A.M <= 16)
    launch_tiles<DT, 1, 1, 4>(A, st);
  else if (A.M <= 32)
    launch_tiles<DT, 2, 1, 4>(A, st);
  else
    launch_tiles<DT, 4, 2, 2>(A, st);
}

}  // namespace

void launch_lm_quant(int dtype, const LmQuantArgs &A, hipStream_t st) {
  if (dtype == DT_BF16) launch_type<DT_BF16>(A, st);
  else launch_type<DT_F16>(A, st);
}

}  // namespace sv
