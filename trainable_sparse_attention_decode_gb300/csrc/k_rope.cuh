// Rotary positions: the arithmetic that the rotation (k_rope.cu), the 4-bit cache's append
// (k_quant4_cache.cu) and its attention share, so that a row comes out the same bits
// whichever of them turns it.
//
// Pair i of a row turns by the angle that its axis's position has in the table:
//     a' = a c - b s,   b' = b c + a s      (backward: s -> -s, the transpose)
// in fp32, every product and sum rounded on its own, then rounded to the row's type.
#pragma once

#include "nosa_internal.cuh"

#include <type_traits>

namespace nosa {

constexpr int kRopeMaxAxes = 4;

struct RopeArgs {
  const float2* table;   // [len][pairs] cosine and sine
  const int32_t* pos;    // [axes][batch x n]
  long long axis_stride; // batch x n
  int len, pairs;        // positions of the table; pairs of a row (0: no rotation)
  int interleaved;       // pairs (2i, 2i + 1) instead of (i, i + pairs)
  int one_axis;          // every pair's axis is 0
  uint32_t axes[kRopeMaxAxes];  // axis of pair i: bits 2 (i % 16) of word i / 16
  int* status;
};

#ifdef __CUDACC__

__device__ __forceinline__ uint32_t rope_axis(const RopeArgs& p, int i) {
  uint32_t w = p.axes[0];
#pragma unroll
  for (int k = 1; k < kRopeMaxAxes; ++k)
    if (i / 16 == k) w = p.axes[k];
  return (w >> (2 * (i % 16))) & 3u;
}

// EARLY: past L1, for kernels that read before their own griddep_wait (see launch_dependent).
template <bool EARLY, typename T> __device__ __forceinline__ T rope_load(const T* p) { return EARLY ? __ldcg(p) : *p; }

// Position of token row `at` on the axis of pair i; one that the table does not have is
// flagged and clamped.
template <bool EARLY = false>
__device__ __forceinline__ int rope_position(const RopeArgs& p, long long at, int i) {
  const int x = rope_load<EARLY>(p.pos + (long long)rope_axis(p, i) * p.axis_stride + at);
  if (x >= 0 && x < p.len) return x;
  if (p.status != nullptr) atomicOr(p.status, 2);  // NOSA_QUANT_INDEX
  return x < 0 ? 0 : p.len - 1;
}

// Cosine and sine of pair i of token row `at`.
__device__ __forceinline__ float2 rope_angle(const RopeArgs& p, long long at, int i) {
  return p.table[(long long)rope_position(p, at, i) * p.pairs + i];
}

// Element x (< 2 pairs) of a row: which pair it belongs to, whether it is the pair's
// first, and where the other one is.
struct RopePlace {
  int pair, other;
  bool first;
};
__device__ __forceinline__ RopePlace rope_place(const RopeArgs& p, int x) {
  if (p.interleaved) return {x >> 1, x ^ 1, (x & 1) == 0};
  const bool first = x < p.pairs;
  return {first ? x : x - p.pairs, first ? x + p.pairs : x - p.pairs, first};
}
__device__ __forceinline__ float rope_turn(float x, float other, bool first, float2 cs) {
  const float a = __fmul_rn(x, cs.x), b = __fmul_rn(other, cs.y);
  return first ? __fsub_rn(a, b) : __fadd_rn(a, b);
}

// The N elements x0, x0 + 1, ... of a row, f, turned in place and rounded to T (N a power of
// two from 2 to 8, x0 a multiple of it, all of them in one half where pairs are halves).
template <typename T, int N, bool EARLY>
__device__ __forceinline__ void rope_turn_vec(const RopeArgs& p, const T* row, long long at, int x0, float* f) {
  if (x0 >= 2 * p.pairs) return;
  float g[N];  // the other ones of the pairs
  int pair0;
  const bool first = x0 < p.pairs;
  if (p.interleaved) {
    pair0 = x0 / 2;
#pragma unroll
    for (int k = 0; k < N; ++k) g[k] = f[k ^ 1];
  } else {
    pair0 = first ? x0 : x0 - p.pairs;
    const T* src = row + (first ? x0 + p.pairs : x0 - p.pairs);
    using V = typename std::conditional<N * sizeof(T) == 16, uint4, uint2>::type;
    const V raw = rope_load<EARLY>(reinterpret_cast<const V*>(src));
    const T* o = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int k = 0; k < N; ++k) g[k] = to_f32(o[k]);
  }
  // one position for pairs of one axis, which are two to a 16-byte load; else each its own
  const int last = pair0 + (p.interleaved ? N / 2 : N) - 1;
  bool one = true;
  for (int i = pair0; i < last && !p.one_axis; ++i) one &= rope_axis(p, i) == rope_axis(p, last);
  float2 cs[N];
  const float2* at0 = p.table + (long long)rope_position<EARLY>(p, at, pair0) * p.pairs;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = pair0 + (p.interleaved ? k / 2 : k);
    cs[k] = rope_load<EARLY>((one ? at0 : p.table + (long long)rope_position<EARLY>(p, at, i) * p.pairs) + i);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) f[k] = to_f32(from_f32<T>(rope_turn(f[k], g[k], p.interleaved ? k % 2 == 0 : first, cs[k])));
}

#endif

struct RotateArgs {
  RopeArgs rope;
  const void* in[2];   // q, k: [batch][n][heads][d]
  void* out[2];
  long long in_b[2], in_t[2], in_h[2], out_b[2], out_t[2], out_h[2];  // elements between requests, tokens, heads
  int heads[2];
  int n, backward;
  long long rows;      // batch x n
};
cudaError_t launch_rotate(const Shape& s, const RotateArgs& a, cudaStream_t stream);

}  // namespace nosa
