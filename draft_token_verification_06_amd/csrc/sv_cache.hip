// The paged cache of a verification step (gfx950): rotary positions, appending a
// step's rows to the pages, and moving a tree's accepted path behind the context.
//
// Angles.  A frequency is held as the fraction of a turn per position in units
// of 2^-64; times the position, modulo 2^64, it is the angle without loss (a
// float32 product at position 10^6 is off by a sixteenth of a radian).  The two
// top bits choose the quadrant, the rest is within pi/4 and goes through the
// sine's and cosine's power series in float64: up to x^15 and x^16, whose next
// terms are below 5e-17.  A workgroup does this once per (row, frequency) and
// keeps the results in LDS for all heads.
//
// 8-bit pages.  One wave owns a block of tokens of one head (its rows, its
// scale, its earlier tokens), so nothing is shared and no order matters.  Keys
// are turned in float64 and rounded to odd in float32: rounding that once more,
// to 8 bits, gives the nearest number, and comparisons with 448 2^k are exact.
// Quotients by other scales than powers of two are rounded to odd likewise.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "sv_device.h"
#include "sv_launch.h"
#include "sv_plan.h"

namespace sv {

namespace {

constexpr float kF8Max = 448.0f;
constexpr float kF8LeastScale = 0x1p-100f;

// 16-bit values of the storage types from float32, to nearest.
template <int DT> __device__ __forceinline__ uint16_t half_bits(float x) {
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}
template <int DT> __device__ __forceinline__ uint4 pack8(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = half_bits<DT>(x[2 * i]) | static_cast<uint32_t>(half_bits<DT>(x[2 * i + 1])) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// Four 8-bit numbers of float32 values within +-448, to nearest, ties to even;
// infinities become NaN (inf * 0 + inf), finite values keep their bits.
__device__ __forceinline__ uint32_t pack_f8(float a, float b, float c, float d) {
  a = __builtin_fmaf(a, 0.0f, a), b = __builtin_fmaf(b, 0.0f, b), c = __builtin_fmaf(c, 0.0f, c), d = __builtin_fmaf(d, 0.0f, d);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}
__device__ __forceinline__ void unpack_f8(uint32_t w, float *x) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  x[0] = lo[0], x[1] = lo[1], x[2] = hi[0], x[3] = hi[1];
}

// d in float32, an inexact result with its last bit set.
__device__ __forceinline__ float round_to_odd(double d) {
  const float f = static_cast<float>(d);
  const double rest = d - static_cast<double>(f);  // (NaN and infinities: not a number, left alone)
  const uint32_t bits = __float_as_uint(f);
  const bool even = !(bits & 1) && finite(f);
  if (even && rest > 0) return __uint_as_float(bits + (f < 0 || bits == 0x80000000u ? -1 : 1));
  if (even && rest < 0) return __uint_as_float(bits + (f < 0 || bits == 0x80000000u ? 1 : -1));
  return f;
}

// y / n in float32, an inexact result with its last bit set (but for those below
// 2^-60); n in [1/2, 1), about = 1 / n to a unit or so.  One step of refinement
// leaves one of the two numbers beside the quotient, whose remainder float32 holds.
__device__ __forceinline__ float odd_quotient(float y, float n, float about) {
  const float g = y * about, f = __builtin_fmaf(__builtin_fmaf(-g, n, y), about, g);
  const float rest = __builtin_fmaf(-f, n, y);
  const uint32_t bits = __float_as_uint(f);
  const int away = (__float_as_uint(rest) ^ bits) >> 31 ? -1 : 1;
  return !(bits & 1) && fabsf(f) > 0x1p-60f && rest != 0.0f ? __uint_as_float(bits + away) : f;
}

// Sine and cosine of `phase` 2^-64 turns.
__device__ __forceinline__ void turn_sincos(uint64_t phase, double *sine, double *cosine) {
  const uint64_t quarter = (phase + (1ull << 61)) >> 62;
  const double x = static_cast<double>(static_cast<int64_t>(phase - (quarter << 62))) * (6.283185307179586477 * 0x1p-64);
  const double z = x * x;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;
  s = fma(s, z, 1.0 / 6227020800.0), c = fma(c, z, -1.0 / 87178291200.0);
  s = fma(s, z, -1.0 / 39916800.0), c = fma(c, z, 1.0 / 479001600.0);
  s = fma(s, z, 1.0 / 362880.0), c = fma(c, z, -1.0 / 3628800.0);
  s = fma(s, z, -1.0 / 5040.0), c = fma(c, z, 1.0 / 40320.0);
  s = fma(s, z, 1.0 / 120.0), c = fma(c, z, -1.0 / 720.0);
  s = fma(s, z, -1.0 / 6.0), c = fma(c, z, 1.0 / 24.0);
  s = fma(s * z, x, x), c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  const bool swap = quarter & 1;
  const double a = swap ? c : s, b = swap ? s : c;
  *sine = quarter & 2 ? -a : a;
  *cosine = (quarter + 1) & 2 ? -b : b;
}

// (cosine, sine) of row `pos` at a frequency (A.turns), times the magnitude; lo:
// what float32 leaves of them.
__device__ __forceinline__ void angle(const Rotation &A, uint64_t frequency, int64_t pos, float2 *hi, float2 *lo) {
  double s, c;
  const uint64_t phase = static_cast<uint64_t>(pos) * frequency;
  turn_sincos(A.inverse ? 0 - phase : phase, &s, &c);
  s *= A.magnitude, c *= A.magnitude;
  *hi = make_float2(static_cast<float>(c), static_cast<float>(s));
  *lo = make_float2(static_cast<float>(c - hi->x), static_cast<float>(s - hi->y));
}

// A head's row is handled in units of 16 values by D / 16 lanes.  Unit j takes
// two pieces of 8 values that hold 8 whole pairs, of angles 8 j .. 8 j + 7
// (pieces j and j + rot / 16 where pairs are rot / 2 apart), or two pieces
// behind the turned ones.
__device__ __forceinline__ int2 unit_pieces(const Rotation &A, int j) {
  return !A.interleaved && j < A.rot / 16 ? make_int2(j, j + A.rot / 16) : make_int2(2 * j, 2 * j + 1);
}

// Values a, b of a unit turned in float32; cs: its 8 (cosine, sine) pairs.
__device__ __forceinline__ void turn_unit(bool interleaved, const float2 *cs, float *a, float *b) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 w = cs[i];
      const float x = a[i], y = b[i];
      a[i] = __builtin_fmaf(x, w.x, -(y * w.y));
      b[i] = __builtin_fmaf(y, w.x, x * w.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float *p = i < 4 ? a + 2 * i : b + 2 * (i - 4);
      const float2 w = cs[i];
      const float x = p[0], y = p[1];
      p[0] = __builtin_fmaf(x, w.x, -(y * w.y));
      p[1] = __builtin_fmaf(y, w.x, x * w.y);
    }
  }
}
// The same in float64, rounded to odd.
__device__ __forceinline__ void turn_unit_odd(bool interleaved, const float2 *hi, const float2 *lo, float *a, float *b) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float *p = !interleaved ? a + i : i < 4 ? a + 2 * i : b + 2 * (i - 4);
    float *r = !interleaved ? b + i : p + 1;
    const double c = static_cast<double>(hi[i].x) + lo[i].x, s = static_cast<double>(hi[i].y) + lo[i].y;
    const double x = *p, y = *r;
    *p = round_to_odd(fma(x, c, -(y * s)));
    *r = round_to_odd(fma(y, c, x * s));
  }
}

template <class... Tree> __device__ __forceinline__ int row_depth(int r, const Tree &...tree) {
  if constexpr (sizeof...(Tree) > 0) return (tree.depth[r], ...);
  else return r;
}

}  // namespace

// ---------------------------------------------------------------------------
// Rotary positions alone.  Bound: memory (each value read and written once): 4
// times 8191 rows of 32 heads of 128 in 16 bits take 114 us, 4.7 TB/s of the 4.9
// that a copy reaches, half of the rows in float32, as many bytes, 133 us, 4.0 TB/s;
// 72 rows 3.1 to 3.6 us, a launch and two trips to memory.
// ---------------------------------------------------------------------------
namespace {

// The (cosine, sine) pairs [rows][rot / 2] of a workgroup's rows; returns their number.
template <class... Tree>
__device__ __forceinline__ int rotary_angles(const RotaryArgs &A, int64_t row0, float2 *s_cs, const Tree &...tree) {
  const Rotation &T = A.rotation;
  const int rows = static_cast<int>(min(static_cast<int64_t>(A.group), A.rows - row0));
  const int half = T.rot / 2;
  for (int e = threadIdx.x; e < rows * half; e += kRotaryThreads) {
    const int64_t row = row0 + e / half;
    const int64_t b = row / A.R;
    const int64_t pos = (T.base_pos ? T.base_pos[b] : 0) + row_depth(static_cast<int>(row - b * A.R), tree...);
    float2 lo;
    angle(T, T.turns[e % half], pos, &s_cs[e], &lo);
  }
  __syncthreads();
  return rows;
}

template <int DT> __device__ __forceinline__ void store_raw(char *row, int i, uint32_t bits) {
  if constexpr (DT == DT_F32) reinterpret_cast<uint32_t *>(row)[i] = bits;
  else reinterpret_cast<uint16_t *>(row)[i] = static_cast<uint16_t>(bits);
}
template <int DT> __device__ __forceinline__ void store_value(char *row, int i, float x) {
  if constexpr (DT == DT_F32) reinterpret_cast<float *>(row)[i] = x;
  else reinterpret_cast<uint16_t *>(row)[i] = half_bits<DT>(x);
}

}  // namespace

template <int DT, class... Tree>
__global__ void __launch_bounds__(kRotaryThreads) k_rotary(RotaryArgs A, Tree... tree) {
  extern __shared__ float2 s_cs[];  // [group][rot / 2]
  const Rotation &T = A.rotation;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * A.group;
  const int rows = rotary_angles(A, row0, s_cs, tree...);
  const int half = T.rot / 2;
  constexpr int EB = Elt<DT>::kBytes, EPV = Elt<DT>::kEPV;
  // in place only the turned values are touched
  const int units = A.in_place ? T.rot / 16 : A.D / 16;
  const int all = rows * A.H * units;
  for (int e = threadIdx.x; e < all; e += kRotaryThreads) {
    const int j = e % units, h = e / units % A.H, t = e / units / A.H;
    const int64_t row = row0 + t;
    if (A.row_count) {
      const int64_t b = row / A.R;
      if (row - b * A.R >= A.row_count[b]) continue;
    }
    const int2 piece = unit_pieces(T, j);
    const char *x = A.x + (row * A.x_stride + static_cast<int64_t>(h) * A.D) * EB;
    char *y = A.out + (row * A.out_stride + static_cast<int64_t>(h) * A.D) * EB;
    uint4 raw[16 / EPV];
#pragma unroll
    for (int i = 0; i < 8 / EPV; ++i) {
      raw[i] = load_vec(x + piece.x * 8 * EB + i * 16);
      raw[8 / EPV + i] = load_vec(x + piece.y * 8 * EB + i * 16);
    }
    if (j < T.rot / 16) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16 / EPV; ++i) Elt<DT>::vec(raw[i], v + i * EPV);
      turn_unit(T.interleaved, s_cs + t * half + j * 8, v, v + 8);
      if constexpr (DT == DT_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          raw[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
      } else {
        raw[0] = pack8<DT>(v);
        raw[1] = pack8<DT>(v + 8);
      }
    }
#pragma unroll
    for (int i = 0; i < 8 / EPV; ++i) {
      *reinterpret_cast<uint4 *>(y + piece.x * 8 * EB + i * 16) = raw[i];
      *reinterpret_cast<uint4 *>(y + piece.y * 8 * EB + i * 16) = raw[8 / EPV + i];
    }
  }
}

// Any even number of turned values: a thread per pair (and per two values
// behind them), 2 or 4 bytes at a time.  Only for what units of 16 do not cover:
// the same bytes take 240 us in 16 bits (2.2 TB/s) and 180 in float32 (3.0), bound by
// the number of loads and stores; 72 rows 6.5 us.
template <int DT, class... Tree>
__global__ void __launch_bounds__(kRotaryThreads) k_rotary_pairs(RotaryArgs A, Tree... tree) {
  extern __shared__ float2 s_cs[];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * A.group;
  const int rows = rotary_angles(A, row0, s_cs, tree...);
  constexpr int EB = Elt<DT>::kBytes;
  const int half = A.rotation.rot / 2, pairs = A.in_place ? half : A.D / 2;
  for (int e = threadIdx.x; e < rows * A.H * pairs; e += kRotaryThreads) {
    const int j = e % pairs, h = e / pairs % A.H, t = e / pairs / A.H;
    const int64_t row = row0 + t;
    if (A.row_count && row % A.R >= A.row_count[row / A.R]) continue;
    const char *x = A.x + (row * A.x_stride + static_cast<int64_t>(h) * A.D) * EB;
    char *y = A.out + (row * A.out_stride + static_cast<int64_t>(h) * A.D) * EB;
    const bool turned = j < half;
    const int a = turned && !A.rotation.interleaved ? j : 2 * j, b = turned && !A.rotation.interleaved ? j + half : 2 * j + 1;
    const uint32_t ra = Elt<DT>::raw(x, a), rb = Elt<DT>::raw(x, b);
    if (!turned) {
      store_raw<DT>(y, a, ra);
      store_raw<DT>(y, b, rb);
      continue;
    }
    const float2 w = s_cs[t * half + j];
    const float u = Elt<DT>::dec(ra), v = Elt<DT>::dec(rb);
    store_value<DT>(y, a, __builtin_fmaf(u, w.x, -(v * w.y)));
    store_value<DT>(y, b, __builtin_fmaf(v, w.x, u * w.y));
  }
}

// ---------------------------------------------------------------------------
// Storing rows in a block of 8-bit tokens.
// ---------------------------------------------------------------------------
namespace {

// Lanes of a wave on a block: D / 16 lanes per token, so many tokens a pass.
// Kernels are built for 1, 2, 4 or 8 passes (registers are what a wave holds).
template <int D> constexpr int kUnits = D / 16;
template <int D> constexpr int kPassTokens = 64 / kUnits<D>;

// The largest of the wave's (non-negative) values, in every lane.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x124>(v));
  v = fmaxf(v, dpp_f32<0x128>(v));
  return fmaxf(fmaxf(read_lane_f32(v, 0), read_lane_f32(v, 16)), fmaxf(read_lane_f32(v, 32), read_lane_f32(v, 48)));
}

// The wave's values y (pass p, token p T + lane / units, 16 of it) whose bit in
// `live` is set, to the block at `block` (token 0, this head): token u goes to
// place u + shift.  Places below `first` hold earlier tokens, scaled by held (the
// value at `scale`, which the caller has asked for with the rows).
template <int D, int kP>
__device__ __forceinline__ void store_f8(const float (&y)[kP][16], uint32_t live, int shift, int first, uint8_t *block,
                                         int64_t token_bytes, float *scale, float held, int2 piece) {
  const int lane = threadIdx.x & 63, t_lane = lane / kUnits<D>;
  float a = 0.0f;
#pragma unroll
  for (int p = 0; p < kP; ++p)
    if (live >> p & 1)
#pragma unroll
      for (int i = 0; i < 16; ++i) a = fmaxf(a, finite(y[p][i]) ? fabsf(y[p][i]) : 0.0f);
  a = wave_max(a);
  float base = kF8LeastScale;
  bool earlier = false;
  if (first > 0) {
    const float s0 = read_lane_f32(held, 0);  // (the same in every lane: decisions on it are scalar)
    earlier = s0 > 0.0f && finite(s0);
    if (earlier) base = s0;
  }
  // the least j >= 0 with a <= 448 base 2^j (these products are exact in float64)
  int j = 0;
  const double top = a, limit = static_cast<double>(kF8Max) * base;
  if (top > limit) {
    j = max(0, ilogb(top) - ilogb(limit));
    if (top > ldexp(limit, j)) ++j;
  }
  const float now = ldexpf(base, j);
  if (earlier && j > 0) {
    const float down = ldexpf(1.0f, -j);
    for (int e = lane; e < first * (D / 16); e += 64) {
      uint4 *at = reinterpret_cast<uint4 *>(block + e / (D / 16) * token_bytes + e % (D / 16) * 16);
      const uint4 w = *at;
      const uint32_t in[4] = {w.x, w.y, w.z, w.w};
      uint32_t out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
        unpack_f8(in[i], x);
        out[i] = pack_f8(x[0] * down, x[1] * down, x[2] * down, x[3] * down);
      }
      *at = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
  if (lane == 0 && (!earlier || j > 0)) *scale = now;
  // A power of two (anything but a scale of the caller's own) divides exactly as
  // its inverse.  Other quotients are formed one by one and rounded to odd.
  const bool exact = __builtin_amdgcn_readfirstlane((__float_as_uint(now) & 0x7FFFFF) == 0 && now >= 0x1p-126f);
  const float inverse = 1.0f / now;
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    if (!(live >> p & 1)) continue;
    float x[16];
    if (exact) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = y[p][i] * inverse;
    } else {
      const float part = __builtin_amdgcn_frexp_mantf(now), about = __builtin_amdgcn_rcpf(part);
      const int e = __builtin_amdgcn_frexp_expf(now);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] = odd_quotient(__builtin_amdgcn_ldexpf(y[p][i], -e), part, about);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_f8(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    uint8_t *at = block + (p * kPassTokens<D> + t_lane + shift) * token_bytes;
    *reinterpret_cast<uint2 *>(at + piece.x * 8) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(at + piece.y * 8) = make_uint2(w[2], w[3]);
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// Appending.  A workgroup takes the rows that fall into one block of one
// sequence; its waves take heads in turn: keys, values, queries.  Every row is read
// once, into registers, where 8-bit pages find their scale.
//
// Bound: memory for prompts.  4 times 4096 rows of 32 + 2 * 8 heads of 128, half
// of each turned: 369 MB in 84 us in 8-bit blocks of 16 (4.4 TB/s), 95 in blocks of 32
// and 112 in blocks of 64, where float64 products and conversions take turns with
// the memory and 4 and 8 passes leave three and two waves a SIMD; 403 MB in 95 us
// (4.2 TB/s) in 16 bits.  Whole heads turned cost up to 3 us more.  One prompt of 512
// rows has few workgroups: 9.6, 15 and 26 us in blocks of 16, 32 and 64, 9.4 in 16 bits.
// Steps are trips to memory after each other (length, page, rows, store): one
// token 6.5 to 7.3 us, 64 windows of 9 rows 11, 128 single tokens 6.6 to 7.1; in 16
// bits 4.1, 8.9 and 5.7.
// Keys in float32, with a bound on the error and only passes with an open byte
// once more in float64, were slower (11776 rows of four prompts in blocks of 32 107
// us for 77, windows 13.1 for 11.5): the test costs more than the products.
// ---------------------------------------------------------------------------
namespace {
// Angles of a row in LDS: two more than there are, so that rows begin 16 bytes
// apart in the banks and the lanes of a pass, 64 bytes apart, do not meet.
__host__ __device__ constexpr int append_row_angles(int rot) { return rot / 2 + 2; }
}  // namespace

template <int DT, bool F8, int D, int kP, class... Tree>
__global__ void __launch_bounds__(kAppendThreads, kP == 8 ? 2 : kP == 4 ? 3 : 4) k_append(AppendArgs A, Tree... tree) {
  // [tokens][row_angles], then what float32 leaves of them (8-bit pages)
  extern __shared__ __attribute__((aligned(16))) float2 s_cs[];
  const Rotation &T = A.rotation;
  const int b = blockIdx.x / A.blocks;
  const int ctx = A.ctx_len[b];
  const int rows = A.row_count ? min(max(A.row_count[b], 0), A.R) : A.R;
  const int64_t end = static_cast<int64_t>(ctx) + rows;
  if (ctx < 0 || end > static_cast<int64_t>(A.table_pages) << A.pool.page_shift) return;
  const int block = 1 << A.pool.block_shift;
  const int64_t slot0 = (static_cast<int64_t>(ctx >> A.pool.block_shift) + blockIdx.x % A.blocks) << A.pool.block_shift;
  const int t0 = static_cast<int>(max(ctx - slot0, int64_t{0})), t1 = static_cast<int>(min(end - slot0, static_cast<int64_t>(block)));
  if (t0 >= t1) return;
  const int row0 = static_cast<int>(slot0 - ctx);  // row of the block's first token (negative where it is an earlier one)
  const int page = A.table[b * A.table_stride + (slot0 >> A.pool.page_shift)];
  const int half = T.rot / 2;
  const int row_angles = append_row_angles(T.rot);
  float2 *s_lo = s_cs + min(A.R, block) * row_angles;
  constexpr int kU = kUnits<D>, kT = kPassTokens<D>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = lane % kU, t_lane = t0 + lane / kU;  // (passes begin at the first row)
  const int2 piece = unit_pieces(T, j);
  const bool turned = j < T.rot / 16;
  const int heads = A.pool.Hkv;
  const bool stored = static_cast<uint32_t>(page) < static_cast<uint32_t>(A.pool.num_pages);
  const int64_t seq_row = static_cast<int64_t>(b) * A.R + row0;
  const int in_page = static_cast<int>(slot0) & ((1 << A.pool.page_shift) - 1);
  // Rows of a task (kG passes of them are asked for together; behind the last
  // row the last one again, so that the loads stand in a known order).  The first
  // task's are on their way while the angles are formed: those only wait for
  // their own frequency, which a lane keeps.
  constexpr int kG = kP < 4 ? kP : 4;
  uint4 ra[kG], rb[kG];
  auto fetch = [&](int task, int p0) {
    const bool query = task >= 2 * heads, value = !query && task >= heads;
    const int h = query ? task - 2 * heads : value ? task - heads : task;
    const uint16_t *x = query ? A.q : value ? A.v : A.k;
    const int64_t stride = query ? A.q_stride : value ? A.v_stride : A.k_stride;
#pragma unroll
    for (int p = 0; p < kG; ++p) {
      const uint16_t *row = x + (seq_row + min((p0 + p) * kT + t_lane, t1 - 1)) * stride + h * D;
      ra[p] = load_vec(row + piece.x * 8);
      rb[p] = load_vec(row + piece.y * 8);
    }
  };
  const int task0 = blockIdx.y * (kAppendThreads / 64) + wave, tasks = 2 * heads + A.Hq;
  const int64_t pos0 = T.base_pos ? T.base_pos[b] : ctx;
  const int shift = half > 1 ? 32 - __builtin_clz(half - 1) : 0, i = lane & ((1 << shift) - 1);  // lanes of a token (half <= 64), without divisions
  const uint64_t frequency = i < half ? T.turns[i] : 0;
  __builtin_amdgcn_sched_barrier(0);
  constexpr bool kEarly = kP >= 4;
  if (kEarly) fetch(min(task0, tasks - 1), 0);
  __builtin_amdgcn_sched_barrier(0);
  if (i < half)
    for (int t = threadIdx.x >> shift; t < t1 - t0; t += kAppendThreads >> shift) {
      float2 lo;
      const int at = t * row_angles + i;
      angle(T, frequency, pos0 + row_depth(row0 + t0 + t, tree...), &s_cs[at], &lo);
      if (F8) s_lo[at] = lo;
    }
  __syncthreads();

  for (int task = task0; task < tasks; task += gridDim.y * (kAppendThreads / 64)) {
    const bool query = task >= 2 * heads, value = !query && task >= heads;
    if (!query && !stored) continue;
    const int h = query ? task - 2 * heads : value ? task - heads : task;
    if (F8 && !query) {
      const int64_t at = ((static_cast<int64_t>(page) << (A.pool.page_shift - A.pool.block_shift)) + (in_page >> A.pool.block_shift)) * heads + h;
      float *scale = (value ? A.pool.v_scale : A.pool.k_scale) + at;
      const float held = t0 > 0 ? *scale : 0.0f;
      float y[kP][16];
      uint32_t live = 0;
#pragma unroll
      for (int p0 = 0; p0 < kP; p0 += kG) {
        if (!kEarly || task != task0 || p0 > 0) fetch(task, p0);
#pragma unroll
        for (int p = p0; p < p0 + kG; ++p) {
          const int t = p * kT + t_lane;
          if (t < t1) {
            live |= 1u << p;
            Elt<DT>::vec(ra[p - p0], y[p]);
            Elt<DT>::vec(rb[p - p0], y[p] + 8);
            const int at = (t - t0) * row_angles + j * 8;
            if (!value && turned) turn_unit_odd(T.interleaved, s_cs + at, s_lo + at, y[p], y[p] + 8);
          }
          __builtin_amdgcn_sched_barrier(0);  // one pass's float64 values at a time
        }
      }
      uint8_t *dst = (value ? A.pool.v : A.pool.k) + page * A.pool.page_bytes + in_page * A.pool.token_bytes + h * A.pool.head_bytes;
      store_f8<D, kP>(y, live, t0, t0, dst, A.pool.token_bytes, scale, held, piece);
      continue;
    }
#pragma unroll
    for (int p0 = 0; p0 < kP; p0 += kG) {
      if (!kEarly || task != task0 || p0 > 0) fetch(task, p0);
#pragma unroll
      for (int p = 0; p < kG; ++p) {
        const int t = (p0 + p) * kT + t_lane;
        if (t >= t1) continue;
        if (!value && turned) {
          float v[16];
          Elt<DT>::vec(ra[p], v);
          Elt<DT>::vec(rb[p], v + 8);
          turn_unit(T.interleaved, s_cs + (t - t0) * row_angles + j * 8, v, v + 8);
          ra[p] = pack8<DT>(v);
          rb[p] = pack8<DT>(v + 8);
        }
        uint16_t *out;
        if (query) {
          out = A.q_out + (seq_row + t) * A.q_out_stride + h * D;
        } else {
          uint8_t *dst = (value ? A.pool.v : A.pool.k) + page * A.pool.page_bytes + (in_page + t) * A.pool.token_bytes + h * A.pool.head_bytes;
          out = reinterpret_cast<uint16_t *>(dst);
        }
        *reinterpret_cast<uint4 *>(out + piece.x * 8) = ra[p];
        *reinterpret_cast<uint4 *>(out + piece.y * 8) = rb[p];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Keeping an accepted path.  One wave per (layer, sequence, head, keys or
// values): it holds the path's rows in registers before it stores the first.
// Bound: trips to memory after each other (path, pages, rows and scales, store):
// 2.9 to 3.3 us for 4 trees of one layer.  64 trees of 32 layers take 18 us, of which
// the 12.6 MB alone would be 2.6: rows of 128 bytes over gigabytes of pages.  Paths of
// three nodes each are 25 MB, 21 us, in 16-bit pages 50 MB, 14 us (3.5 TB/s).
// ---------------------------------------------------------------------------
namespace {

// Nodes that sequence b's accepted path may have; -1: the sequence is left alone.
// (R - 1 at most, also where nodes repeat: the rows' own places are what the
// table has room for.)
__device__ __forceinline__ int path_most(const CommitArgs &A, int b, int ctx) {
  if (ctx < 0 || static_cast<int64_t>(ctx) + A.R > static_cast<int64_t>(A.table_pages) << A.pool.page_shift) return -1;
  return min(max(A.n_accepted[b], 0), A.nodes ? min(A.max_nodes, A.R - 1) : A.R - 1);
}
__device__ __forceinline__ bool on_path(const CommitArgs &A, int node) { return static_cast<uint32_t>(node - 1) < static_cast<uint32_t>(A.R - 1); }

}  // namespace

template <bool F8, int D, int kP>
__global__ void __launch_bounds__(kCommitThreads) k_commit(CommitArgs A) {
  constexpr int kU = kUnits<D>, kT = kPassTokens<D>;
  const int lane = threadIdx.x & 63;
  const int j = lane % kU, t_lane = lane / kU;
  const int heads = A.pool.Hkv;
  const int groups = (2 * heads + kCommitThreads / 64 - 1) / (kCommitThreads / 64);
  const int task = blockIdx.x % groups * (kCommitThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x / groups % A.B, layer = blockIdx.x / groups / A.B;
  if (task >= 2 * heads) return;
  // (what the path does not reach is read with the rest: one trip to memory, not one per node)
  const int ctx = A.ctx_len[b];
  const int32_t *nodes = A.nodes + b * A.nodes_stride;
  const int mine = lane < A.max_nodes ? nodes[lane] : 0;
  int node[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) node[p] = p * kT + t_lane < A.max_nodes ? nodes[p * kT + t_lane] : 0;
  const int most = path_most(A, b, ctx);
  const uint64_t off = ~__ballot(lane < most && on_path(A, mine));
  const int n = most < 0 ? -1 : off ? __builtin_ctzll(off) : 64;
  if (A.new_len && layer == 0 && task == 0 && lane == 0) A.new_len[b] = n < 0 ? ctx : ctx + 1 + n;
  if (n <= 0) return;
  const bool value = task >= heads;
  const int h = value ? task - heads : task;
  const int page_mask = (1 << A.pool.page_shift) - 1, scale_shift = A.pool.page_shift - A.pool.block_shift;
  uint8_t *pages = (value ? A.pool.v : A.pool.k) + layer * A.layer_bytes + h * A.pool.head_bytes;
  float *scales = F8 ? (value ? A.pool.v_scale : A.pool.k_scale) + layer * A.layer_scales : nullptr;
  const int32_t *table = A.table + b * A.table_stride;
  auto home = [&](int slot) { return table[slot >> A.pool.page_shift]; };
  auto token = [&](int page, int slot) { return pages + page * A.pool.page_bytes + (slot & page_mask) * A.pool.token_bytes; };
  auto scale_at = [&](int page, int slot) {
    return scales + ((static_cast<int64_t>(page) << scale_shift) + ((slot & page_mask) >> A.pool.block_shift)) * heads + h;
  };
  const int first = ctx + 1;
  uint32_t live = 0;
  uint4 raw[kP], raw2[F8 ? 1 : kP];
  float factor[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    const int u = p * kT + t_lane;
    if (u >= n) continue;
    const int slot = ctx + node[p];
    const int from = home(slot);
    if (static_cast<uint32_t>(from) >= static_cast<uint32_t>(A.pool.num_pages)) continue;
    live |= 1u << p;
    if (F8) {
      raw[p] = load_vec(token(from, slot) + j * 16);
      factor[p] = *scale_at(from, slot);
    } else {
      raw[p] = load_vec(token(from, slot) + j * 32);
      raw2[F8 ? 0 : p] = load_vec(token(from, slot) + j * 32 + 16);
    }
  }
  const int block = F8 ? 1 << A.pool.block_shift : 1;
  int slot0 = first & -block, to = __builtin_amdgcn_readfirstlane(home(slot0));  // the first block that takes rows
  float held = F8 && static_cast<uint32_t>(to) < static_cast<uint32_t>(A.pool.num_pages) ? *scale_at(to, slot0) : 0.0f;
  // every row is in registers before the first store: a path's rows may lie
  // where others of it go
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
  if constexpr (!F8) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      if (!(live >> p & 1)) continue;
      const int slot = first + p * kT + t_lane;
      const int to = home(slot);
      if (static_cast<uint32_t>(to) >= static_cast<uint32_t>(A.pool.num_pages)) continue;
      uint4 *at = reinterpret_cast<uint4 *>(token(to, slot) + j * 32);
      at[0] = raw[p];
      at[1] = raw2[p];
    }
  } else {
    float y[kP][16];
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      if (!(live >> p & 1)) continue;
      const uint32_t w[4] = {raw[p].x, raw[p].y, raw[p].z, raw[p].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unpack_f8(w[i], &y[p][4 * i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) y[p][4 * i + k] *= factor[p];
      }
    }
    for (;;) {
      uint32_t here = 0;
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        const int t = first + p * kT + t_lane - slot0;
        if (t >= 0 && t < block) here |= live & 1u << p;
      }
      if (static_cast<uint32_t>(to) < static_cast<uint32_t>(A.pool.num_pages) && __any(here != 0))
        store_f8<D, kP>(y, here, first - slot0, max(first - slot0, 0), token(to, slot0), A.pool.token_bytes, scale_at(to, slot0), held,
                        make_int2(2 * j, 2 * j + 1));
      slot0 += block;
      if (slot0 >= first + n) break;
      to = __builtin_amdgcn_readfirstlane(home(slot0));
      if (static_cast<uint32_t>(to) < static_cast<uint32_t>(A.pool.num_pages)) held = *scale_at(to, slot0);
    }
  }
}

// The lengths alone: where new_len is ctx_len itself, after the rows have moved.
__global__ void __launch_bounds__(64) k_advance(CommitArgs A) {
  const int b = blockIdx.x * 64 + threadIdx.x;
  if (b >= A.B) return;
  const int ctx = A.ctx_len[b], most = path_most(A, b, ctx);
  int n = A.nodes ? 0 : most;
  if (A.nodes)
    while (n < most && on_path(A, A.nodes[b * A.nodes_stride + n])) ++n;
  if (most < 0) n = -1;
  A.new_len[b] = n < 0 ? ctx : ctx + 1 + n;
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
void launch_rotary(int dtype, RotaryArgs A, const TreeDepths *depths, hipStream_t st) {
  // few rows: a workgroup each, as long as that fills no more than the chip
  A.group = kRotaryTokens;
  while (A.group > 1 && A.rows / A.group < 1024) A.group /= 2;
  const dim3 grid(static_cast<unsigned>((A.rows + A.group - 1) / A.group)), threads(kRotaryThreads);
  const unsigned lds = A.group * (A.rotation.rot / 2) * sizeof(float2);
  auto go = [&](auto plain, auto tree) {
    if (depths) hipLaunchKernelGGL(tree, grid, threads, lds, st, A, *depths);
    else hipLaunchKernelGGL(plain, grid, threads, lds, st, A);
  };
  if (A.rotation.rot % 16 == 0) {
    if (dtype == DT_F32) go(k_rotary<DT_F32>, k_rotary<DT_F32, TreeDepths>);
    else if (dtype == DT_BF16) go(k_rotary<DT_BF16>, k_rotary<DT_BF16, TreeDepths>);
    else go(k_rotary<DT_F16>, k_rotary<DT_F16, TreeDepths>);
  } else {
    if (dtype == DT_F32) go(k_rotary_pairs<DT_F32>, k_rotary_pairs<DT_F32, TreeDepths>);
    else if (dtype == DT_BF16) go(k_rotary_pairs<DT_BF16>, k_rotary_pairs<DT_BF16, TreeDepths>);
    else go(k_rotary_pairs<DT_F16>, k_rotary_pairs<DT_F16, TreeDepths>);
  }
}

namespace {

template <int DT, bool F8, int D, int kP>
void launch_append_passes(const AppendArgs &A, const TreeDepths *depths, hipStream_t st) {
  const int64_t x = static_cast<int64_t>(A.B) * A.blocks;
  const int64_t tasks = (2 * A.pool.Hkv + A.Hq + kAppendThreads / 64 - 1) / (kAppendThreads / 64);
  // Blocks that do not fill the chip: their heads are spread over workgroups, each
  // of which forms the block's angles again.  Up to 4096 of them: prompts of 4 times
  // 4096 rows, half of each head turned, take 84, 95 and 112 us in blocks of 16, 32
  // and 64; with up to 1024 88, 113 and 124, 2048 88, 94 and 112, 8192 83, 104 and 112
  // (16 bits 95, 93, 96 and 95).
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(tasks, 4096 / x));
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y)), threads(kAppendThreads);
  const unsigned lds = std::min(A.R, 1 << A.pool.block_shift) * append_row_angles(A.rotation.rot) * sizeof(float2) * (F8 ? 2 : 1);
  if (depths) hipLaunchKernelGGL((k_append<DT, F8, D, kP, TreeDepths>), grid, threads, lds, st, A, *depths);
  else hipLaunchKernelGGL((k_append<DT, F8, D, kP>), grid, threads, lds, st, A);
}

// Passes over what a block can hold of a call's rows.
template <int DT, bool F8, int D>
void launch_append_shape(const AppendArgs &A, const TreeDepths *depths, hipStream_t st) {
  const int tokens = std::min(A.R, 1 << A.pool.block_shift);
  if (tokens <= kPassTokens<D>) launch_append_passes<DT, F8, D, 1>(A, depths, st);
  else if (tokens <= 2 * kPassTokens<D>) launch_append_passes<DT, F8, D, 2>(A, depths, st);
  else if (D == 64 || tokens <= 4 * kPassTokens<D>) launch_append_passes<DT, F8, D, 4>(A, depths, st);
  else launch_append_passes<DT, F8, D, D == 64 ? 4 : 8>(A, depths, st);
}

template <int DT, bool F8>
void launch_append_dim(const AppendArgs &A, const TreeDepths *depths, hipStream_t st) {
  if (A.D == 64) launch_append_shape<DT, F8, 64>(A, depths, st);
  else launch_append_shape<DT, F8, 128>(A, depths, st);
}

}  // namespace

void launch_append(int dtype, bool f8, const AppendArgs &A, const TreeDepths *depths, hipStream_t st) {
  if (dtype == DT_BF16) {
    if (f8) launch_append_dim<DT_BF16, true>(A, depths, st);
    else launch_append_dim<DT_BF16, false>(A, depths, st);
  } else {
    if (f8) launch_append_dim<DT_F16, true>(A, depths, st);
    else launch_append_dim<DT_F16, false>(A, depths, st);
  }
}

namespace {

template <bool F8, int D, int kP>
void launch_commit_passes(const CommitArgs &A, hipStream_t st) {
  const int64_t groups = (2 * A.pool.Hkv + kCommitThreads / 64 - 1) / (kCommitThreads / 64);
  hipLaunchKernelGGL((k_commit<F8, D, kP>), dim3(static_cast<unsigned>(groups * A.B * A.layers)), dim3(kCommitThreads), 0, st, A);
}

template <bool F8, int D>
void launch_commit_shape(const CommitArgs &A, hipStream_t st) {
  if (A.max_nodes <= kPassTokens<D>) launch_commit_passes<F8, D, 1>(A, st);
  else if (A.max_nodes <= 2 * kPassTokens<D>) launch_commit_passes<F8, D, 2>(A, st);
  else launch_commit_passes<F8, D, D == 64 ? 4 : 8>(A, st);
}

}  // namespace

void launch_commit(bool f8, const CommitArgs &A, hipStream_t st) {
  const bool in_place = A.new_len == A.ctx_len;
  if (A.nodes) {
    CommitArgs M = A;
    if (in_place) M.new_len = nullptr;
    if (f8) {
      if (A.D == 64) launch_commit_shape<true, 64>(M, st);
      else launch_commit_shape<true, 128>(M, st);
    } else {
      if (A.D == 64) launch_commit_shape<false, 64>(M, st);
      else launch_commit_shape<false, 128>(M, st);
    }
  }
  if (A.new_len && (in_place || !A.nodes)) hipLaunchKernelGGL(k_advance, dim3((A.B + 63) / 64), dim3(64), 0, st, A);
}

}  // namespace sv
