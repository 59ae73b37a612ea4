// What the attention kernels share (gfx950): matrix products of the storage
// types, the rows' ancestor sets, and a sequence's length and live rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_device.h"
#include "sv_launch.h"
#include "sv_plan.h"

namespace sv {

typedef __bf16 at_bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 at_f16x8_t __attribute__((ext_vector_type(8)));
typedef float at_f32x16_t __attribute__((ext_vector_type(16)));
typedef short at_i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) at_i16x4_t *lds_i16x4_t;

constexpr int kAtThreads = kAttendThreads;

template <int DT> struct AtElt;
template <> struct AtElt<DT_BF16> {
  static constexpr uint32_t kExp = 0x7F80u;  // exponent of infinities and NaN
  static constexpr float kLift = 0.0f;
  __device__ static __forceinline__ at_f32x16_t mma(uint4 a, uint4 b, at_f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(at_bf16x8_t, a), __builtin_bit_cast(at_bf16x8_t, b), c, 0, 0, 0);
  }
  // Two exponentials to the storage type, rounded to nearest: the matrix units
  // take two operands of one type, and the values come in that type.  It costs
  // half a step of each weight (2^-8 in bfloat16), as much as rounding the
  // output does; a second product for what the rounding leaves would double
  // the matrix work of the values.
  __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
  }
  __device__ static __forceinline__ uint16_t bits(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
};
template <> struct AtElt<DT_F16> {
  static constexpr uint32_t kExp = 0x7C00u;
  // Exponentials of rows in float16 are held 2^15 times larger, sums and
  // outputs with them: weights down to 2^-29 of the largest stay normal
  // numbers (down to 2^-14 otherwise, and thousands of smaller ones add up).
  static constexpr float kLift = 15.0f;
  __device__ static __forceinline__ at_f32x16_t mma(uint4 a, uint4 b, at_f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(at_f16x8_t, a), __builtin_bit_cast(at_f16x8_t, b), c, 0, 0, 0);
  }
  __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2{static_cast<_Float16>(lo), static_cast<_Float16>(hi)});
  }
  __device__ static __forceinline__ uint16_t bits(float x) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x)); }
};

// The values of lanes l and l ^ 32 (in either order): one lane-swap instruction.
__device__ __forceinline__ float2 both_halves(float x) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return make_float2(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

__device__ __forceinline__ bool bad_len(const AttendJoin &A, int len) { return len < 0 || len > A.max_ctx; }
__device__ __forceinline__ int live_rows(const AttendJoin &A, int b) {
  return A.row_count ? min(max(A.row_count[b], 0), A.R) : A.R;
}

// Ancestor sets of the rows, one row per thread; parents go to LDS first, as a
// walk through the argument block would cost a trip to memory a step.  (A
// barrier follows at the caller's.)  tree: nothing for a window, or the TreeParents.
template <class... Tree>
__device__ __forceinline__ void ancestor_sets(int R, uint32_t (*s_anc)[8], uint8_t *s_parent, const Tree &...tree) {
  constexpr bool kTree = sizeof...(Tree) > 0;
  if constexpr (kTree) {
    for (int v = threadIdx.x; v < R; v += kAtThreads) s_parent[v] = (tree.parent[v], ...);
    __syncthreads();
  }
  for (int v = threadIdx.x; v < R; v += kAtThreads) {
    uint32_t w[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) w[x] = 0;
    if constexpr (kTree) {
      for (int u = v; u > 0; u = s_parent[u])
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x] |= x == (u >> 5) ? 1u << (u & 31) : 0u;
      w[0] |= 1u;  // the root
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int n = v + 1 - 32 * x;
        w[x] = n >= 32 ? ~0u : n > 0 ? (1u << n) - 1 : 0u;
      }
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) s_anc[v][x] = w[x];
  }
}

}  // namespace sv
