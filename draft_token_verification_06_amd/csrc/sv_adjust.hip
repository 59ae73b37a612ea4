// Logits adjustment (gfx950): penalties for repeated tokens, biases and
// grammar masks on the rows a verification call reads.
//
// Row r of a sequence follows the sequence's history and the row's path (the
// drafts before it, or the tree nodes down to it), so with n the occurrences
// of token t in history[prompt_len ..) and on the path, and seen(t) when t is
// anywhere in the history or on the path:
//   y = x(t);  seen: y = y > 0 ? y / repetition : y * repetition
//   n > 0:     y = y - frequency * n - presence
//   y += bias(t);  not allowed: y = -inf
// in float32, rounded once to the storage type.  Elements nothing applies to
// keep their bits.
//
// Bound: HBM (each row read once and written once).  A workgroup owns kChunk
// consecutive tokens of one sequence and every thread one 16-byte vector of
// them, over all rows: the history is counted once per chunk into LDS, each
// thread takes its vector's counts and biases into registers, and the row
// loop needs no barrier.  Path tokens are bit sets over the tree's nodes
// restricted to the chunk, nearly always empty, so a row costs its load, its
// mask byte and its store.
//
// Measured: B = 256, 9 rows of 128256 bf16, histories of 2048, biases: 226 us,
// 5.2 TB/s (a plain copy of 2 GiB: 4.9); 45 us more while the first rows waited
// for the counting.  Workgroups of 512 threads, 333 us: fewer of them cover the
// counting's barriers.  Grammar masks alone, in place on 32 windows: 24 us for
// 79 MB of mask and -inf.  Tree of 41 rows of 50257 fp16, 4 sequences: 17 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "sv_device.h"
#include "sv_launch.h"
#include "sv_plan.h"

namespace sv {

// Row starts are aligned to the element only (an odd vocabulary): vectors are
// moved with element alignment, which global memory instructions allow.
typedef unsigned int u32x4_e2_t __attribute__((ext_vector_type(4), aligned(2)));

// Storage type of a float value, as bits.
template <int DT> __device__ __forceinline__ uint32_t enc(float x);
template <> __device__ __forceinline__ uint32_t enc<DT_F32>(float x) { return __float_as_uint(x); }
template <> __device__ __forceinline__ uint32_t enc<DT_BF16>(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
template <> __device__ __forceinline__ uint32_t enc<DT_F16>(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

// kStream: with the nontemporal hint (rows that pass through once).
template <int DT, bool kStream> __device__ __forceinline__ uint4 load_elems(const char *p, int valid) {
  constexpr int kEPV = Elt<DT>::kEPV;
  if (valid >= kEPV) {
    const SV_GLOBAL u32x4_e2_t *g = as_global<u32x4_e2_t>(static_cast<const void *>(p));
    const u32x4_e2_t v = kStream ? __builtin_nontemporal_load(g) : *g;
    return make_uint4(v.x, v.y, v.z, v.w);
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < kEPV; ++k)
    if (k < valid) {
      if (DT == DT_F32) w[k] = Elt<DT>::raw(p, k);
      else w[k / 2] |= Elt<DT>::raw(p, k) << (16 * (k & 1));
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT, bool kStream> __device__ __forceinline__ void store_elems(char *p, uint4 v, int valid) {
  constexpr int kEPV = Elt<DT>::kEPV;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (valid >= kEPV) {
    SV_GLOBAL u32x4_e2_t *g = reinterpret_cast<SV_GLOBAL u32x4_e2_t *>(reinterpret_cast<uintptr_t>(p));
    const u32x4_e2_t x = {v.x, v.y, v.z, v.w};
    if (kStream) __builtin_nontemporal_store(x, g);
    else *g = x;
    return;
  }
#pragma unroll
  for (int k = 0; k < kEPV; ++k)
    if (k < valid) {
      if (DT == DT_F32) reinterpret_cast<uint32_t *>(p)[k] = w[k];
      else reinterpret_cast<uint16_t *>(p)[k] = static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1)));
    }
}

// The elements of v whose bit of m is set, those of w elsewhere.
template <int DT> __device__ __forceinline__ uint4 merge_elems(uint4 v, uint4 w, uint32_t m) {
  uint32_t a[4] = {v.x, v.y, v.z, v.w};
  const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (DT == DT_F32) {
      a[i] = (m >> i) & 1 ? a[i] : b[i];
    } else {
      const uint32_t keep = ((m >> (2 * i)) & 1 ? 0xFFFFu : 0u) | ((m >> (2 * i + 1)) & 1 ? 0xFFFF0000u : 0u);
      a[i] = (a[i] & keep) | (b[i] & ~keep);
    }
  }
  return make_uint4(a[0], a[1], a[2], a[3]);
}

constexpr int64_t kAdjustItems = 2048;  // workgroups wanted per launch (8 of 256 threads on each of 256 CUs)
constexpr uint32_t kSeenInPrompt = 0x80000000u;

// kMode: rows copied to another place, cached or streamed, or changed in place.
enum : int { ADJ_COPY = 0, ADJ_STREAM = 1, ADJ_IN_PLACE = 2 };

// tree: nothing for a window, or the TreeParents.
template <int DT, int kMode, class... Tree>
__global__ void __launch_bounds__(kAdjustThreads) k_adjust_logits(AdjustArgs A, Tree... tree) {
  constexpr bool kTree = sizeof...(Tree) > 0;
  using E = Elt<DT>;
  constexpr int kEPV = E::kEPV;
  constexpr bool kStream = kMode == ADJ_STREAM, kInPlace = kMode == ADJ_IN_PLACE;
  constexpr int kChunk = kAdjustThreads * kEPV;
  constexpr uint32_t kFull = (1u << kEPV) - 1;
  constexpr int kWords = kTreeMaxNodes / 64;
  __shared__ uint32_t s_count[kChunk];  // occurrences past the prompt; kSeenInPrompt
  __shared__ uint16_t s_bias[kChunk];   // 1 + index of the last bias entry that names the token
  __shared__ int32_t s_node[kTreeMaxNodes];
  __shared__ uint8_t s_parent[kTreeMaxNodes];
  __shared__ uint64_t s_in[kWords];               // nodes whose token lies in the chunk
  __shared__ uint64_t s_path[kTreeMaxNodes][kWords];  // those on each row's path

  const int tid = threadIdx.x;
  const int group = blockIdx.x % A.row_groups;
  const int item = blockIdx.x / A.row_groups;
  const int b = item / A.chunks;
  const int base = (item - b * A.chunks) * kChunk;
  const int live = A.row_count ? min(max(A.row_count[b], 0), A.R) : A.R;
  const int row0 = group * A.group_rows, rows = min(row0 + A.group_rows, live);
  if (row0 >= rows) return;  // the same for the whole workgroup
  const bool counted = A.repetition || A.presence || A.frequency;
  const bool history = counted && A.history;
  const bool biased = A.n_bias > 0;
  const bool paths = counted && A.tokens && A.R > 1;
  const int words = (A.R + 63) / 64;

  const int t0 = base + tid * kEPV;  // this thread's first token
  const int valid = min(kEPV, A.V - t0);
  const int64_t row_bytes = static_cast<int64_t>(A.V) * E::kBytes;
  const char *in = A.in + b * A.in_stride_bytes + static_cast<int64_t>(t0) * E::kBytes;
  char *out = A.out + b * A.out_stride_bytes + static_cast<int64_t>(t0) * E::kBytes;
  const uint8_t *allowed =
      A.allowed ? reinterpret_cast<const uint8_t *>(A.allowed + b * A.allowed_seq_stride) + t0 / 8 : nullptr;
  const int nibble = t0 & 7;  // float32 vectors: half a byte of the mask
  // kAhead rows at a time: their mask bytes, then their vectors, in flight
  // together (from a disallowed vector nothing is read).  Rows copied
  // elsewhere are all read, so the first ones set out before the counting.
  constexpr int kAhead = 4;
  struct Rows {
    uint32_t m[kAhead];
    uint4 x[kAhead];
  };
  auto fetch = [&](int r0, Rows &f, auto wanted) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int r = min(r0 + u, rows - 1);
      f.m[u] = kFull;
      if (allowed) f.m[u] = (allowed[r * A.allowed_row_stride * 4] >> nibble) & kFull;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int r = min(r0 + u, rows - 1);
      f.x[u] = make_uint4(0, 0, 0, 0);
      if (f.m[u] != 0 && wanted(r, f.m[u])) f.x[u] = load_elems<DT, kStream>(in + r * row_bytes, valid);
    }
  };
  const auto every = [](int, uint32_t) { return true; };
  Rows next;
  if (!kInPlace && valid > 0) fetch(row0, next, every);

  const float rho = A.repetition ? A.repetition[b] : 1.0f;
  const float pres = A.presence ? A.presence[b] : 0.0f;
  const float freq = A.frequency ? A.frequency[b] : 0.0f;

  if (history)
    for (int i = tid; i < kChunk; i += kAdjustThreads) s_count[i] = 0;
  if (biased)
    for (int i = tid; i < kChunk / 2; i += kAdjustThreads) reinterpret_cast<uint32_t *>(s_bias)[i] = 0;
  if (paths) {
    static_assert(kAdjustThreads >= kTreeMaxNodes, "one thread per node");
    if (tid < words * 64) {
      // row v's own node: the draft before row v, or the tree node's token
      int t = -1;
      if (tid >= 1 && tid < A.R) t = A.tokens[b * A.tokens_stride + (kTree ? tid : tid - 1)];
      const bool in = t >= base && t < A.V && t - base < kChunk;
      s_node[tid] = t;
      // the walks below read parents from LDS: a step through the argument
      // block would cost a trip to memory each
      s_parent[tid] = static_cast<uint8_t>(tid - 1);
      if constexpr (kTree) s_parent[tid] = (tree.parent[tid], ...);
      const uint64_t bits = __ballot(in);
      if ((tid & 63) == 0) s_in[tid >> 6] = bits;
    }
  }
  __syncthreads();
  if (history) {
    const int len = A.history_len ? min(max(A.history_len[b], 0), A.history_cap) : A.history_cap;
    const int prompt = A.prompt_len ? min(max(A.prompt_len[b], 0), len) : 0;
    const int32_t *h = A.history + b * A.history_stride;
    // kBatch loads in flight per thread: a long history costs few round trips
    constexpr int kBatch = 8;
    for (int i0 = tid; i0 < len; i0 += kBatch * kAdjustThreads) {
      int t[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) t[j] = i0 + j * kAdjustThreads < len ? h[i0 + j * kAdjustThreads] : -1;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (t[j] >= base && t[j] < A.V && t[j] - base < kChunk) {
          if (i0 + j * kAdjustThreads < prompt) atomicOr(&s_count[t[j] - base], kSeenInPrompt);
          else atomicAdd(&s_count[t[j] - base], 1u);
        }
    }
  }
  if (biased) {
    // the last entry that names a token counts: the largest index wins, in any order
    const int32_t *bt = A.bias_tokens + static_cast<int64_t>(b) * A.n_bias;
    for (int j = tid; j < A.n_bias; j += kAdjustThreads) {
      const int t = bt[j];
      if (t >= base && t < A.V && t - base < kChunk) {
        uint32_t *w = reinterpret_cast<uint32_t *>(s_bias) + ((t - base) >> 1);
        const int sh = 16 * ((t - base) & 1);
        uint32_t old = *w;
        while (((old >> sh) & 0xFFFFu) < static_cast<uint32_t>(j + 1)) {
          const uint32_t was = atomicCAS(w, old, (old & ~(0xFFFFu << sh)) | (static_cast<uint32_t>(j + 1) << sh));
          if (was == old) break;
          old = was;
        }
      }
    }
  }
  if (paths && tid < A.R) {
    uint64_t bits[kWords] = {};
    for (int v = tid; v > 0; v = s_parent[v]) {
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        if (w < words && w == (v >> 6)) bits[w] |= s_in[w] & (1ull << (v & 63));
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w)
      if (w < words) s_path[tid][w] = bits[w];
  }
  __syncthreads();

  if (valid <= 0) return;
  uint32_t count[kEPV];
  float bias[kEPV];
  // Elements that a count or a bias acts on.  The others keep their bits, which
  // a signalling NaN would not on its way through float32 (2% of the window
  // call of 1.1 GB).
  uint32_t named = 0;
#pragma unroll
  for (int k = 0; k < kEPV; ++k) {
    count[k] = history ? s_count[tid * kEPV + k] : 0u;
    bias[k] = 0.0f;
    named |= (count[k] != 0 ? 1u : 0u) << k;
  }
  if (biased) {
#pragma unroll
    for (int k = 0; k < kEPV; ++k) {
      const int j = s_bias[tid * kEPV + k];
      if (j > 0) {
        bias[k] = A.bias_values[static_cast<int64_t>(b) * A.n_bias + j - 1];
        named |= 1u << k;
      }
    }
  }
  auto near = [&](int r) {  // some token of the row's path lies in the chunk (the same for the workgroup)
    bool any = false;
    if (paths)
      for (int w = 0; w < words; ++w) any |= s_path[r][w] != 0;
    return any;
  };
  for (int r0 = row0; r0 < rows; r0 += kAhead) {
    Rows now;
    if (kInPlace) {
      fetch(r0, now, [&](int r, uint32_t m) { return named != 0 || m != kFull || near(r); });
    } else {
      now = next;
      if (r0 + kAhead < rows) fetch(r0 + kAhead, next, every);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int r = r0 + u;
      if (r >= rows) break;
      uint32_t on_path[kEPV] = {};
      uint32_t hit = named;
      if (near(r)) {
        for (int w = 0; w < words; ++w)
          for (uint64_t bits = s_path[r][w]; bits; bits &= bits - 1) {
            const int d = s_node[w * 64 + __builtin_ctzll(bits)] - t0;
#pragma unroll
            for (int k = 0; k < kEPV; ++k) on_path[k] += d == k;
            hit |= d >= 0 && d < kEPV ? 1u << d : 0u;
          }
      }
      if (kInPlace && hit == 0 && now.m[u] == kFull) continue;
      uint4 v = now.x[u];
      if (hit != 0 && now.m[u] != 0) {
        float y[kEPV];
        E::vec(v, y);
#pragma unroll
        for (int k = 0; k < kEPV; ++k) {
          const uint32_t n = (count[k] & ~kSeenInPrompt) + on_path[k];
          if (count[k] != 0 || n != 0) y[k] = y[k] > 0.0f ? y[k] / rho : y[k] * rho;
          if (n != 0) y[k] = y[k] - freq * static_cast<float>(n) - pres;
          if (bias[k] != 0.0f) y[k] += bias[k];
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = DT == DT_F32 ? enc<DT>(y[i % kEPV]) : enc<DT>(y[2 * i % kEPV]) | (enc<DT>(y[(2 * i + 1) % kEPV]) << 16);
        v = merge_elems<DT>(make_uint4(w[0], w[1], w[2], w[3]), v, hit);
      }
      constexpr uint32_t kInf = E::kNegInfPair;
      if (now.m[u] != kFull) v = merge_elems<DT>(v, make_uint4(kInf, kInf, kInf, kInf), now.m[u]);
      store_elems<DT, kStream>(out + r * row_bytes, v, valid);
    }
  }
}

int adjust_chunks(int dtype, int V) {
  const int chunk = kAdjustThreads * (dtype == DT_F32 ? 4 : 8);
  return (V + chunk - 1) / chunk;
}

namespace {

constexpr int64_t kAdjustStreamBytes = 256ll << 20;

template <int DT, int kMode>
void launch_shape(const AdjustArgs &A, const TreeParents *parents, dim3 grid, hipStream_t st) {
  if (parents)
    hipLaunchKernelGGL((k_adjust_logits<DT, kMode, TreeParents>), grid, dim3(kAdjustThreads), 0, st, A, *parents);
  else
    hipLaunchKernelGGL((k_adjust_logits<DT, kMode>), grid, dim3(kAdjustThreads), 0, st, A);
}

template <int kMode>
void launch_type(int dtype, const AdjustArgs &A, const TreeParents *parents, dim3 grid, hipStream_t st) {
  if (dtype == DT_F32)
    launch_shape<DT_F32, kMode>(A, parents, grid, st);
  else if (dtype == DT_BF16)
    launch_shape<DT_BF16, kMode>(A, parents, grid, st);
  else
    launch_shape<DT_F16, kMode>(A, parents, grid, st);
}

}  // namespace

void launch_adjust_logits(int dtype, AdjustArgs A, const TreeParents *parents, int B, hipStream_t st) {
  A.chunks = adjust_chunks(dtype, A.V);
  // Few sequences and many rows (a tree): rows go to several workgroups, each
  // of which counts the history again.  Four at least stay together, which is
  // what a thread keeps in flight.
  const int64_t items = static_cast<int64_t>(B) * A.chunks;
  const int64_t want = std::min<int64_t>((kAdjustItems + items - 1) / items, (A.R + 3) / 4);
  A.group_rows = static_cast<int32_t>((A.R + want - 1) / want);
  A.row_groups = (A.R + A.group_rows - 1) / A.group_rows;
  const dim3 grid(static_cast<unsigned>(items * A.row_groups));
  // Rows that do not fit the Infinity Cache between this call and the next
  // pass through it with the nontemporal hint; smaller ones are left there for
  // the verification that reads them.
  const int64_t bytes = 2 * static_cast<int64_t>(B) * A.R * A.V * (dtype == DT_F32 ? 4 : 2);
  if (A.in_place)
    launch_type<ADJ_IN_PLACE>(dtype, A, parents, grid, st);
  else if (bytes > kAdjustStreamBytes)
    launch_type<ADJ_STREAM>(dtype, A, parents, grid, st);
  else
    launch_type<ADJ_COPY>(dtype, A, parents, grid, st);
}

}  // namespace sv
