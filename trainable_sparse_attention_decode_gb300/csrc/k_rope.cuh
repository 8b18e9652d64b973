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
  int wide;              // the table starts on a 32-byte boundary
  uint32_t axes[kRopeMaxAxes];  // axis of pair i: bits 2 (i % 16) of word i / 16
  int* status;
};

#ifdef __CUDACC__

__device__ __forceinline__ float rope_turn(float x, float other, bool first, float2 cs) {
  const float a = __fmul_rn(x, cs.x), b = __fmul_rn(other, cs.y);
  return first ? __fsub_rn(a, b) : __fadd_rn(a, b);
}

// Chunk i of d / 16: sixteen elements of a row, two vectors of eight. Where pairs are halves,
// a turned chunk has eight of each half; others are sixteen in a row.
struct RopeChunk {
  int lo, hi;  // where its vectors begin
  bool turned;
};
__device__ __forceinline__ RopeChunk rope_chunk(const RopeArgs& p, int i) {
  const bool turned = 8 * i < p.pairs;
  const bool split = turned && !p.interleaved;
  return {split ? 8 * i : 16 * i, split ? p.pairs + 8 * i : 16 * i + 8, turned};
}

// 32 bytes, a whole sector, at once.
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

// The axes of a chunk's pairs, two bits each.
__device__ __forceinline__ uint32_t rope_axes(const RopeArgs& p, int i) {
  uint32_t w = p.axes[0];
#pragma unroll
  for (int k = 1; k < kRopeMaxAxes; ++k)
    if (i / 2 == k) w = p.axes[k];
  return w >> (16 * (i & 1)) & 0xFFFFu;
}
// The position that `at` points to; one that the table does not have is flagged and clamped.
__device__ __forceinline__ int rope_position(const RopeArgs& p, const int32_t* at) {
  const int x = *at;
  if ((unsigned)x < (unsigned)p.len) return x;
  if (p.status != nullptr) atomicOr(p.status, 2);  // NOSA_QUANT_INDEX
  return x < 0 ? 0 : p.len - 1;
}
// Cosines and sines of pairs 8 i .. 8 i + 7 (axes w) of the token whose position on axis 0 is at
// `at`: two 32-byte loads where the pairs have one axis.
__device__ __forceinline__ void rope_angles(const RopeArgs& p, uint32_t w, const int32_t* at, int i, float2* cs) {
  if (w == (w & 3u) * 0x5555u) {
    const float4* src = reinterpret_cast<const float4*>(p.table + (long long)rope_position(p, at + (w & 3u) * p.axis_stride) * p.pairs + 8 * i);
    if (p.wide) {  // half the passes through L1: a warp's lanes are 64 bytes apart
#pragma unroll
      for (int k = 0; k < 2; ++k) load32(src + 2 * k, reinterpret_cast<uint32_t*>(cs + 4 * k));
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 x = src[k];
      cs[2 * k] = make_float2(x.x, x.y);
      cs[2 * k + 1] = make_float2(x.z, x.w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      cs[k] = p.table[(long long)rope_position(p, at + (w >> (2 * k) & 3u) * p.axis_stride) * p.pairs + 8 * i + k];
  }
}
// The sixteen elements of a turned chunk, unrounded.
__device__ __forceinline__ void rope_turn_chunk(bool interleaved, const float2* cs, float* x) {
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = x[2 * k], b = x[2 * k + 1];
      x[2 * k] = rope_turn(a, b, true, cs[k]);
      x[2 * k + 1] = rope_turn(b, a, false, cs[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = x[k], b = x[8 + k];
      x[k] = rope_turn(a, b, true, cs[k]);
      x[8 + k] = rope_turn(b, a, false, cs[k]);
    }
  }
}

// Eight elements in registers, as they are in memory.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
    f[4] = bf16_lo(r.z); f[5] = bf16_hi(r.z); f[6] = bf16_lo(r.w); f[7] = bf16_hi(r.w);
  }
  __device__ __forceinline__ void set(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

#endif

struct RotateArgs {
  RopeArgs rope;
  const void* in[2];   // q, k: [batch][n][heads][d]
  void* out[2];
  long long in_b[2], in_t[2], in_h[2], out_b[2], out_t[2], out_h[2];  // elements between requests, tokens, heads
  int heads[2];
  int n, backward;
  const int32_t* count;  // [batch] rows of a request that exist, or null
  long long rows;        // batch x n
};
cudaError_t launch_rotate(const Shape& s, const RotateArgs& a, cudaStream_t stream);

}  // namespace nosa
