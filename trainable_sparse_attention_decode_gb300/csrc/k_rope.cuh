// Rotary positions: the arithmetic that the rotation (k_rope.cu), the 4-bit cache's append
// (k_quant4_cache.cu) and its attention share, so that a row comes out the same bits
// whichever of them turns it.
//
// Pair i of a row turns by the angle that its axis's position has in the table:
//     a' = a c - b s,   b' = b c + a s      (backward: s -> -s, the transpose)
// in fp32, every product and sum rounded on its own, then rounded to the row's type.
#pragma once

#include "nosa_internal.cuh"

namespace nosa {

constexpr int kRopeMaxAxes = 4;

struct RopeArgs {
  const float2* table;   // [len][pairs] cosine and sine
  const int32_t* pos;    // [axes][batch x n]
  long long axis_stride; // batch x n
  int len, pairs;        // positions of the table; pairs of a row (0: no rotation)
  int interleaved;       // pairs (2i, 2i + 1) instead of (i, i + pairs)
  uint32_t axes[kRopeMaxAxes];  // axis of pair i: bits 2 (i % 16) of word i / 16
  int* status;
};

#ifdef __CUDACC__

// Position of token row `at` on the axis of pair i; one that the table does not have is
// flagged and clamped.
__device__ __forceinline__ int rope_position(const RopeArgs& p, long long at, int i) {
  uint32_t w = p.axes[0];
#pragma unroll
  for (int k = 1; k < kRopeMaxAxes; ++k)
    if (i / 16 == k) w = p.axes[k];
  const int x = p.pos[(long long)((w >> (2 * (i % 16))) & 3u) * p.axis_stride + at];
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
