// Write side of the 4-bit block cache: appending tokens, with the rotation of their keys on
// the way, and reading blocks back.
//
// Both read and write everything once. Reading back is bound by HBM (GB300: 4096 blocks of
// d = 128 in bf16, 174 MB, 28.7 us = 89 % of the measured copy rate; fp32, 307 MB, 46.7 us = 97 %).
// Appending is bound by its loads' latency and by its instructions together: the same blocks, 174 MB, 59 us
// = 43 % (without a rotation 56; fp32 86 us = 53 %). The loads by themselves take 38 (rotation: 7), the extremes
// 5, the codes and their way out 17; a block takes 16 warps 700 instructions each, at 2.5 a cycle. Tried: keys and
// values by one CTA 58 us (fp32 90), CTAs that stay and load the next block while they work on one
// 69 to 80, 4 or 6 CTAs an SM for 5 64 and 66. A token of 32 requests of 8 heads, every fourth of
// which completes a block: 6.0 us, latency.
#include "k_quant4.cuh"

#include <algorithm>

namespace nosa {
namespace {

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct UnitAppend4 {
  int n0, add;
};
// What the call does to unit u of request b: tokens before it, new ones (0 where the unit is left as it was).
template <bool EARLY>
__device__ __forceinline__ UnitAppend4 unit_append(const QAppendArgs& p, int b, int u, bool flag) {
  UnitAppend4 r;
  r.n0 = quant_len<EARLY>(p.lens, u, p.max_blocks, p.status, flag);
  r.add = quant_count<EARLY>(p.n_new, b, p.n, p.status, flag);
  if (r.n0 < 0) {
    r.n0 = r.add = 0;
  } else if (r.n0 > kQB * p.max_blocks - r.add) {
    if (flag) quant_flag(p.status, kQErrCapacity);
    r.add = 0;
  }
  return r;
}

// Chunk i (axes w) of a new token's key, turned and rounded, as two vectors: the key's row and
// where the token's positions are.
template <typename T>
__device__ __forceinline__ void new_key(const RopeArgs& p, const T* row, const int32_t* pos, uint32_t w, int i, const RopeChunk& ch, Vec8<T>* v) {
  v[0].load(row + ch.lo);
  v[1].load(row + ch.hi);
  if (!ch.turned) return;
  float2 cs[8];
  rope_angles(p, w, pos, i, cs);
  float x[16];
  v[0].get(x);
  v[1].get(x + 8);
  rope_turn_chunk(p.interleaved, cs, x);
  v[0].set(x);
  v[1].set(x + 8);
}

// Row t, dims x .. x + 7 of a tail unit: keys in 16-byte chunks, values in rows.
template <typename T, int D>
__device__ __forceinline__ void tail_load(const T* tail, bool key, int t, int x, Vec8<T>& v) {
  if (!key) {
    v.load(tail + kQB * D + t * D + x);
  } else if constexpr (sizeof(T) == 2) {
    v.load(tail + (x / 8 * kQB + t) * 8);
  } else {
    v.a = *reinterpret_cast<const float4*>(tail + (x / 4 * kQB + t) * 4);
    v.b = *reinterpret_cast<const float4*>(tail + ((x / 4 + 1) * kQB + t) * 4);
  }
}
template <typename T, int D>
__device__ __forceinline__ void tail_store(T* tail, bool key, int t, int x, const Vec8<T>& v) {
  if (!key) {
    v.store(tail + kQB * D + t * D + x);
  } else if constexpr (sizeof(T) == 2) {
    v.store(tail + (x / 8 * kQB + t) * 8);
  } else {
    *reinterpret_cast<float4*>(tail + (x / 4 * kQB + t) * 4) = v.a;
    *reinterpret_cast<float4*>(tail + ((x / 4 + 1) * kQB + t) * 4) = v.b;
  }
}

// Two numbers' nearest integers n in 0 .. 15 to (x - zero) * r, as kMagicBits + n: the last place
// of 1.5 2^23 is 1, so adding it rounds.
constexpr uint32_t kMagicBits = 0x4B400000u;
__device__ __forceinline__ uint2 code_bits(float2 x, float2 inv, float2 minus_zero, float2 r) {
  const float2 t = __ffma2_rn(__ffma2_rn(x, inv, minus_zero), r, make_float2(12582912.f, 12582912.f));
  return make_uint2(__float_as_uint(t.x), __float_as_uint(t.y));
}

// Extremes of a thread's elements, in a form that reductions by shuffles take: pairs of bf16
// numbers, or single fp32 numbers. NaN stays NaN.
template <typename T> struct Extreme;
template <> struct Extreme<__nv_bfloat16> {
  using V = uint32_t;
  static constexpr int PER = 2;  // elements of a value
  static __device__ __forceinline__ uint32_t none() { return 0xFF80FF80u; }
  static __device__ __forceinline__ __nv_bfloat162 b(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
  static __device__ __forceinline__ uint32_t u(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }
  static __device__ __forceinline__ uint32_t most(uint32_t x, uint32_t y) { return u(__hmax2_nan(b(x), b(y))); }
  static __device__ __forceinline__ uint32_t minus_least(uint32_t x, uint32_t y) { return u(__hmin2_nan(b(x), b(y))) ^ 0x80008000u; }
  static __device__ __forceinline__ uint32_t minus(uint32_t x) { return x ^ 0x80008000u; }
  static __device__ __forceinline__ void values(const Vec8<__nv_bfloat16>& v, uint32_t* x) { x[0] = v.r.x; x[1] = v.r.y; x[2] = v.r.z; x[3] = v.r.w; }
  static __device__ __forceinline__ float whole(uint32_t x) { return max_nan(bf16_lo(x), bf16_hi(x)); }
  // largest magnitude, as bits of an fp32 number; none() counts for nothing
  static __device__ __forceinline__ uint32_t size(uint32_t x) {
    const uint32_t lo = x << 16, hi = x & 0xFFFF0000u;
    return max(lo == 0xFF800000u ? 0u : lo & 0x7FFFFFFFu, hi == 0xFF800000u ? 0u : hi & 0x7FFFFFFFu);
  }
  template <int N> static __device__ __forceinline__ uint32_t sizes(const uint32_t* x) {
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < N; ++c) m = __vmaxu2(m, x[c] & 0x7FFF7FFFu);
    uint32_t top = max(m << 16, m & 0xFFFF0000u);
    if (top >= 0x7F800000u) {  // (seldom: something that is not finite, or none())
      top = 0;
#pragma unroll
      for (int c = 0; c < N; ++c) top = max(top, size(x[c]));
    }
    return top;
  }
};
template <> struct Extreme<float> {
  using V = float;
  static constexpr int PER = 1;
  static __device__ __forceinline__ float none() { return -INFINITY; }
  static __device__ __forceinline__ float most(float x, float y) { return max_nan(x, y); }
  static __device__ __forceinline__ float minus_least(float x, float y) { return max_nan(-x, -y); }
  static __device__ __forceinline__ float minus(float x) { return -x; }
  static __device__ __forceinline__ void values(const Vec8<float>& v, float* x) { v.get(x); }
  static __device__ __forceinline__ float whole(float x) { return x; }
  template <int N> static __device__ __forceinline__ uint32_t sizes(const float* x) {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < N; ++c) top = max(top, x[c] == -INFINITY ? 0u : __float_as_uint(x[c]) & 0x7FFFFFFFu);
    return top;
  }
};

// A block of a unit's tokens on its way into 4 bits, its keys and its values apart. CTAs of 2 D
// threads: thread (i, tp) has chunk i of D / 16 and a pair of tokens, of the keys the two of a word
// (4 (tp / 2) + tp % 2 and the second after it), of the values two of the four of a word (2 tp and
// 2 tp + 1). The block stays in registers, in the tokens' type, from its loads to its codes:
//   channels' extremes: over the thread's tokens, over the warp's by shuffles that halve the
//     values each lane has, over the warps through shared memory;
//   tokens' extremes: over four lanes;
//   codes: (x / scale - zero) / step + 1.5 2^23, whose last bits are the code; a word is the sum
//     of its codes' bits, shifted, less what the exponents add up to.
template <typename T, int D>
struct Quant4Block {
  using X = Extreme<T>;
  static constexpr int NT = 2 * D, WARPS = NT / 32, CH = D / 16, PITCH = 528;  // (bytes of 512, padded against bank conflicts)
  struct Shared {
    __align__(16) uint8_t code[CH * PITCH];
    __align__(16) uint8_t params[4 * D];             // steps and zeros as in the unit: 3 D bytes of the keys, 4 D of the values
    __align__(16) T part[WARPS][2 * D];              // channels: - least, largest
    __align__(16) float minus_zero[D], inv_step[D];  // channels
    __align__(16) uint32_t top[WARPS];               // largest magnitudes
  };
  const Q4AppendArgs& p;
  const T* tail;
  int Hkv, u, b, h, n0, tid, lane, warp, i, tp, first;
  uint32_t live0, live1;  // tokens that are not masked
  float e0, e1;           // logits of tokens `lane` and lane + 32

  // Block j of the new blocks (0: the one that the tail began).
  __device__ __forceinline__ Quant4Block(const Q4AppendArgs& p_, int Hkv_, int b_, int h_, int n0_, const T* tail_, int j)
      : p(p_), tail(tail_), Hkv(Hkv_), u(b_ * Hkv_ + h_), b(b_), h(h_), n0(n0_), tid(threadIdx.x), lane(threadIdx.x & 31),
        warp(threadIdx.x >> 5), i(threadIdx.x % CH), tp(threadIdx.x / CH), first(j * kQB - n0_ % kQB), e0(0.f), e1(0.f) {}

  // (first: the block's first token among the new ones, or before them)
  __device__ __forceinline__ long long at0() const { return (long long)b * p.a.n + first; }
  __device__ __forceinline__ void load_logits() {
    const float* old_e = reinterpret_cast<const float*>(tail + 2 * kQB * D);
    if (first + lane < 0)
      e0 = old_e[lane];
    else if (p.a.e != nullptr)
      e0 = (p.a.e + at0() * Hkv + h)[lane * Hkv];
    if (first + lane + 32 < 0)
      e1 = old_e[lane + 32];
    else if (p.a.e != nullptr)
      e1 = (p.a.e + at0() * Hkv + h)[(lane + 32) * Hkv];
  }
  __device__ __forceinline__ void find_live() {
    live0 = __ballot_sync(0xffffffffu, e0 != -INFINITY);
    live1 = __ballot_sync(0xffffffffu, e1 != -INFINITY);
  }
  __device__ __forceinline__ uint32_t live_from(int t) const { return (t < 32 ? live0 : live1) >> (t % 32); }

  // fp16 bits of a group's zero and step
  template <bool KEY>
  static __device__ __forceinline__ uint2 zero_step(float lo, float hi, float inv) {
    const uint32_t z = __half_as_ushort(__float2half_rd(lo * inv + 0.f));  // (no -0)
    const uint32_t s = __half_as_ushort(__float2half_ru(__fmul_rn(__fsub_rn(hi * inv, half_bits(z)), 1.f / 15.f)));
    return make_uint2(z, KEY ? (s + 0xFFu) & 0xFF00u : s);
  }
  static __device__ __forceinline__ float inv_of(uint32_t step) { return step != 0 ? __frcp_rn(half_bits(step)) : 0.f; }

  // The block's largest magnitude from the threads': whether it is finite and not below 2^-100
  // (whole CTA).
  __device__ __forceinline__ bool whole_top(Shared& sh, uint32_t& top) const {
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) sh.top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; w += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(&sh.top[w]);
      top = max(max(top, max(x.x, x.y)), max(x.z, x.w));
    }
    return top >= 0x0D800000u && top < 0x7F800000u;
  }
  static __device__ __forceinline__ float inv_scale(uint32_t top) { return __uint_as_float((256u - (top >> 23)) << 23); }
  static __device__ __forceinline__ uint32_t scale_bits(uint32_t top) {
    return top >= 0x7F800000u ? 0x7FC00000u : top >= 0x0D800000u ? ((top >> 23) - 2) << 23 : 0u;
  }
  // The unit that the table names; null and flagged where it names none.
  __device__ __forceinline__ uint8_t* unit_of(int to) const {
    if (to >= 0 && (long long)to < p.a.n_units) return p.a.units + (long long)to * quant4_unit_bytes(D);
    if (tid == 0) quant_flag(p.a.status, kQErrIndex);
    return nullptr;
  }

  __device__ __forceinline__ void keys(Shared& sh, int to) {
    const RopeChunk ch = rope_chunk(p.rope, i);
    const uint32_t axes = rope_axes(p.rope, i);
    const int kt = 4 * (tp / 2) + tp % 2;
    const T* k0 = static_cast<const T*>(p.a.k) + b * p.a.ks.b + h * p.a.ks.h + first * p.a.ks.t;
    Vec8<T> k[2][2];
    load_logits();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = kt + 2 * r;
      if (first + t < 0) {
        tail_load<T, D>(tail, true, t, ch.lo, k[r][0]);
        tail_load<T, D>(tail, true, t, ch.hi, k[r][1]);
      } else {
        new_key<T>(p.rope, k0 + t * p.a.ks.t, p.rope.pos + at0() + t, axes, i, ch, k[r]);
      }
    }
    find_live();
    const uint32_t l = live_from(kt);
    const bool live[2] = {(l & 1u) != 0, (l & 4u) != 0};
    if (!(live[0] && live[1])) {  // a masked token counts as its neighbour
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (!live[r]) {
          k[r][0] = k[1 - r][0];
          k[r][1] = k[1 - r][1];
        }
    }
    // ---- extremes ----
    uint32_t top;
    {
      constexpr int N = 32 / X::PER;  // values: of - least and of largest, one or two of the chunk's dims each
      typename X::V red[N], x[N / 2], y[N / 2];
      X::values(k[0][0], x); X::values(k[0][1], x + N / 4);
      X::values(k[1][0], y); X::values(k[1][1], y + N / 4);
#pragma unroll
      for (int c = 0; c < N / 2; ++c) {
        red[c] = X::minus_least(x[c], y[c]);
        red[N / 2 + c] = X::most(x[c], y[c]);
      }
      if (!live[0] && !live[1]) {
#pragma unroll
        for (int c = 0; c < N; ++c) red[c] = X::none();
      }
      constexpr int STEPS = CH == 8 ? 2 : 3, LEFT = N >> STEPS;
      int at = 0;  // of the values
#pragma unroll
      for (int step = 0; step < STEPS; ++step) {  // lanes of the same chunk: each keeps half of the values
        const int n = N / 2 >> step, away = 16 >> step;
        const bool up = (lane & away) != 0;
        at += up ? n : 0;
#pragma unroll
        for (int c = 0; c < N / 2; ++c) {
          if (c >= n) continue;
          const typename X::V send = up ? red[c] : red[c + n], keep = up ? red[c + n] : red[c];
          red[c] = X::most(keep, __shfl_xor_sync(0xffffffffu, send, away));
        }
      }
      const int c0 = at % (N / 2) * X::PER, dim = c0 < 8 ? ch.lo + c0 : ch.hi + c0 - 8;
      T* out = sh.part[warp] + at / (N / 2) * D + dim;
      if constexpr (LEFT == 2) {
        *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(red);
      } else {
#pragma unroll
        for (int c = 0; c < LEFT; c += 4) reinterpret_cast<uint4*>(out)[c / 4] = *reinterpret_cast<const uint4*>(red + c);
      }
      top = X::template sizes<LEFT>(red);
    }
    const bool ok = whole_top(sh, top);
    const float inv = ok ? inv_scale(top) : 0.f;
    // ---- steps and zeros ----
    if (tid < D) {
      float lo = -INFINITY, hi = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        lo = fmaxf(lo, to_f32(sh.part[w][tid]));  // (where there is a NaN, ok is false)
        hi = fmaxf(hi, to_f32(sh.part[w][D + tid]));
      }
      const uint2 zs = ok ? zero_step<true>(-lo, hi, inv) : make_uint2(0, 0);
      sh.minus_zero[tid] = -half_bits(zs.x);
      sh.inv_step[tid] = inv_of(zs.y);
      sh.params[quant4_order(tid, D)] = zs.y >> 8;
      reinterpret_cast<unsigned short*>(sh.params + D)[quant4_order(tid, D)] = zs.x;
    }
    __syncthreads();
    // ---- codes ----
    const uint32_t mask = ok ? (live[0] ? 0x0F0F0F0Fu : 0u) | (live[1] ? 0xF0F0F0F0u : 0u) : 0u;
    const int g = tp % 8, w = tp / 8;
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // the chunk's two vectors
      const int dim = half ? ch.hi : ch.lo;
      float x[2][8];
      k[0][half].get(x[0]);
      k[1][half].get(x[1]);
      uint8_t* row = sh.code + dim / 16 * PITCH + 16 * (4 * g + dim % 16 / 4) + 4 * w;
#pragma unroll
      for (int c = 0; c < 8; c += 4) {
        const float4 z = *reinterpret_cast<const float4*>(sh.minus_zero + dim + c), s = *reinterpret_cast<const float4*>(sh.inv_step + dim + c);
        uint2 n[2][2];  // of token r, dims 2 y and 2 y + 1: nibbles r + 2 y and r + 2 y + 4
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          n[r][0] = code_bits(make_float2(x[r][c], x[r][c + 1]), inv2, make_float2(z.x, z.y), make_float2(s.x, s.y));
          n[r][1] = code_bits(make_float2(x[r][c + 2], x[r][c + 3]), inv2, make_float2(z.z, z.w), make_float2(s.z, s.w));
        }
        const uint32_t lo = (n[1][1].x << 12) + (n[0][1].x << 8) + (n[1][0].x << 4) + n[0][0].x;
        const uint32_t hi = (n[1][1].y << 12) + (n[0][1].y << 8) + (n[1][0].y << 4) + n[0][0].y;
        *reinterpret_cast<uint32_t*>(row + 4 * c) = ((hi << 16) + lo - kMagicBits * 0x11111111u) & mask;
      }
    }
    __syncthreads();
    uint8_t* unit = unit_of(to);
    if (unit == nullptr) return;
    reinterpret_cast<uint4*>(unit)[tid] = *reinterpret_cast<const uint4*>(sh.code + tid / 32 * PITCH + tid % 32 * 16);
    if (tid < 3 * D / 16) reinterpret_cast<uint4*>(unit + 64 * D)[tid] = reinterpret_cast<const uint4*>(sh.params)[tid];
    if (warp == WARPS - 1) {
      float* e = reinterpret_cast<float*>(unit + quant4_e_off(D));
      e[lane] = e0;
      e[lane + 32] = e1;
      if (lane < 7) reinterpret_cast<uint32_t*>(e)[kQB + (lane == 0 ? 0 : lane + 1)] = lane == 0 ? scale_bits(top) : 0u;
    }
  }

  __device__ __forceinline__ void values(Shared& sh, int to) {
    const int vt = 2 * tp;
    const T* v0 = static_cast<const T*>(p.a.v) + b * p.a.vs.b + h * p.a.vs.h + first * p.a.vs.t;
    Vec8<T> v[2][2];
    load_logits();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = vt + r;
      if (first + t < 0) {
        tail_load<T, D>(tail, false, t, 16 * i, v[r][0]);
        tail_load<T, D>(tail, false, t, 16 * i + 8, v[r][1]);
      } else {
        const T* row = v0 + t * p.a.vs.t + 16 * i;
        if (p.wide) {  // sixteen elements in a row
#pragma unroll
          for (int y = 0; y < (int)sizeof(T) / 2; ++y) load32(row + y * 32 / sizeof(T), reinterpret_cast<uint32_t*>(v[r]) + 8 * y);
        } else {
          v[r][0].load(row);
          v[r][1].load(row + 8);
        }
      }
    }
    find_live();
    const uint32_t l = live_from(vt);
    const bool live[2] = {(l & 1u) != 0, (l & 2u) != 0};
    if (!(live[0] && live[1])) {  // a masked token counts for nothing
      const float zero[8] = {};
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (!live[r]) {
          v[r][0].set(zero);
          v[r][1].set(zero);
        }
    }
    uint32_t top = 0;
    float lo1 = 0.f, hi1 = 0.f;  // of the lane's one of the two tokens: even lanes the first, odd ones the second
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      constexpr int N = 16 / X::PER;
      typename X::V x[N];
      X::values(v[r][0], x);
      X::values(v[r][1], x + N / 2);
      typename X::V lo = X::minus(x[0]), hi = x[0];
#pragma unroll
      for (int c = 1; c < N; ++c) {
        lo = X::most(lo, X::minus(x[c]));
        hi = X::most(hi, x[c]);
      }
#pragma unroll
      for (int o = 1; o < 4; o *= 2) {
        lo = X::most(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = X::most(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      const float a = X::whole(lo), g = X::whole(hi);
      top = max(top, max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(g) & 0x7FFFFFFFu));
      if ((i & 1) == r) {
        lo1 = -a;
        hi1 = g;
      }
    }
    const bool ok = whole_top(sh, top);
    const float inv = ok ? inv_scale(top) : 0.f;
    const uint2 zs = ok && live[i & 1] ? zero_step<false>(lo1, hi1, inv) : make_uint2(0, 0);
    if (i % 4 < 2) {
      const int at = i / 4 * kQB + quant4_order(vt, kQB) + i % 4;  // (vt is even: the second token is next to the first)
      reinterpret_cast<unsigned short*>(sh.params)[at] = zs.y;
      reinterpret_cast<unsigned short*>(sh.params + 2 * D)[at] = zs.x;
    }
    const float mz = -half_bits(zs.x), rs = inv_of(zs.y);
    const float mz1 = __shfl_xor_sync(0xffffffffu, mz, 1), rs1 = __shfl_xor_sync(0xffffffffu, rs, 1);
    const float z2[2] = {i & 1 ? mz1 : mz, i & 1 ? mz : mz1}, r2[2] = {i & 1 ? rs1 : rs, i & 1 ? rs : rs1};
    float x[2][16];
    v[0][0].get(x[0]); v[0][1].get(x[0] + 8);
    v[1][0].get(x[1]); v[1][1].get(x[1] + 8);
    const int hh = tp & 1, c = tp / 2 % 4, w = tp / 8;
    const uint32_t mask = ok ? 0xFFFFFFFFu : 0u;
    uint32_t word[8];
#pragma unroll
    for (int d = 0; d < 8; d += 2) {  // dims d, d + 1 and the eighth ones after them, of the two tokens
      uint2 n[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          n[r][e] = code_bits(make_float2(x[r][d + 8 * e], x[r][d + 8 * e + 1]), make_float2(inv, inv), make_float2(z2[r], z2[r]), make_float2(r2[r], r2[r]));
      word[d] = (((((n[1][1].x << 4) + n[1][0].x) << 16) + (n[0][1].x << 4) + n[0][0].x - kMagicBits * 0x00110011u) & mask) << (8 * hh);
      word[d + 1] = (((((n[1][1].y << 4) + n[1][0].y) << 16) + (n[0][1].y << 4) + n[0][0].y - kMagicBits * 0x00110011u) & mask) << (8 * hh);
    }
    uint8_t* row = sh.code + i * PITCH + 16 * c + 4 * w;
#pragma unroll
    for (int d = 0; d < 4; ++d) {  // the other two tokens of the words are CH lanes away; each thread puts four words down
      const uint32_t other = __shfl_xor_sync(0xffffffffu, hh ? word[d] : word[d + 4], CH);
      *reinterpret_cast<uint32_t*>(row + 64 * (d + 4 * hh)) = (hh ? word[d + 4] : word[d]) | other;
    }
    __syncthreads();
    uint8_t* unit = unit_of(to);
    if (unit == nullptr) return;
    reinterpret_cast<uint4*>(unit + 32 * D)[tid] = *reinterpret_cast<const uint4*>(sh.code + tid / 32 * PITCH + tid % 32 * 16);
    if (tid < 4 * D / 16) reinterpret_cast<uint4*>(unit + quant4_vstep_off(D))[tid] = reinterpret_cast<const uint4*>(sh.params)[tid];
    if (tid == NT - 1) reinterpret_cast<uint32_t*>(unit + quant4_e_off(D))[kQB + 1] = scale_bits(top);
  }
};

// Blocks that the call completes: grid (KV heads x keys and values, most blocks, requests), so that
// neighbouring CTAs read the heads of the same tokens.
template <typename T, int D>
__global__ void __launch_bounds__(2 * D, (sizeof(T) == 2 ? 5 : 3) * 128 / D) quant4_blocks_kernel(Q4AppendArgs p, long long payload) {
  __shared__ typename Quant4Block<T, D>::Shared sh;
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.x / 2, Hkv = gridDim.x / 2, j = blockIdx.y, b = blockIdx.z, u = b * Hkv + h;
  const UnitAppend4 ap = unit_append<false>(p.a, b, u, false);
  if (j >= (ap.n0 % kQB + ap.add) / kQB) return;
  const int to = p.a.tab[(long long)u * p.a.max_blocks + ap.n0 / kQB + j];
  Quant4Block<T, D> q(p, Hkv, b, h, ap.n0, reinterpret_cast<const T*>(p.a.tail + u * payload), j);
  if (blockIdx.x % 2 == 0)
    q.keys(sh, to);
  else
    q.values(sh, to);
}

// The unit's tail and length; with BLOCK also the one block that at most 64 new tokens can
// complete (single tokens: one launch).
template <typename T, int D, bool BLOCK>
__global__ void __launch_bounds__(2 * D) quant4_tail_kernel(Q4AppendArgs p, long long payload) {
  const int h = blockIdx.x, Hkv = gridDim.x, b = blockIdx.z, u = b * Hkv + h, tid = threadIdx.x;
  if (BLOCK) griddep_wait();  // (the call's first launch)
  griddep_launch_dependents();
  const UnitAppend4 ap = unit_append<!BLOCK>(p.a, b, u, tid == 0);
  T* tail = reinterpret_cast<T*>(p.a.tail + u * payload);
  const int old = ap.n0 % kQB, done = (old + ap.add) / kQB;
  if constexpr (BLOCK) {
    __shared__ typename Quant4Block<T, D>::Shared sh;
    if (done > 0) {
      const int to = p.a.tab[(long long)u * p.a.max_blocks + ap.n0 / kQB];
      Quant4Block<T, D> q(p, Hkv, b, h, ap.n0, tail, 0);
      q.keys(sh, to);
      __syncthreads();
      q.values(sh, to);
    }
  }
  if (!BLOCK) griddep_wait();  // the blocks' launch has read the old tail
  __syncthreads();             // ... and so has this one, and the length
  const int first = done > 0 ? 0 : old, left = old + ap.add - done * kQB;
  constexpr int CH = D / 16;
  for (int id = tid; id < (left - first) * CH * 2; id += 2 * D) {
    const int i = id % CH, r = first + id / (2 * CH), tok = done * kQB + r - old;
    Vec8<T> x[2];
    if (id / CH % 2 == 0) {
      const RopeChunk ch = rope_chunk(p.rope, i);
      new_key<T>(p.rope, static_cast<const T*>(p.a.k) + b * p.a.ks.b + (long long)tok * p.a.ks.t + h * p.a.ks.h,
                 p.rope.pos + (long long)b * p.a.n + tok, rope_axes(p.rope, i), i, ch, x);
      tail_store<T, D>(tail, true, r, ch.lo, x[0]);
      tail_store<T, D>(tail, true, r, ch.hi, x[1]);
    } else {
      const T* row = static_cast<const T*>(p.a.v) + b * p.a.vs.b + (long long)tok * p.a.vs.t + h * p.a.vs.h + 16 * i;
      x[0].load(row);
      x[1].load(row + 8);
      tail_store<T, D>(tail, false, r, 16 * i, x[0]);
      tail_store<T, D>(tail, false, r, 16 * i + 8, x[1]);
    }
  }
  float* te = reinterpret_cast<float*>(tail + 2 * kQB * D);
  for (int r = first + tid; r < left; r += 2 * D)
    te[r] = p.a.e != nullptr ? p.a.e[((long long)b * p.a.n + (long long)done * kQB + r - old) * Hkv + h] : 0.f;
  if (tid == 0) p.a.lens_out[u] = p.a.lens[u] + ap.add;
}

template <typename T, int D>
cudaError_t append_variant(const Shape& s, const Q4AppendArgs& a, cudaStream_t stream) {
  if (a.a.n <= kQB) return launch_dependent(quant4_tail_kernel<T, D, true>, dim3(s.Hkv, 1, s.batch), 2 * D, 0, stream, a, s.payload);
  const int most = (int)std::min<long long>((a.a.n + kQB - 1LL) / kQB, a.a.max_blocks);
  const cudaError_t e = launch_dependent(quant4_blocks_kernel<T, D>, dim3(2 * s.Hkv, most, s.batch), 2 * D, 0, stream, a, s.payload);
  if (e != cudaSuccess) return e;
  return launch_dependent(quant4_tail_kernel<T, D, false>, dim3(s.Hkv, 1, s.batch), 2 * D, 0, stream, a, s.payload);
}

// Code (bits `at` to `at` + 3 of a word) as fp32.
__device__ __forceinline__ float code_f32(uint32_t word, int at) {
  return __uint_as_float((word >> at & 15u) | 0x4B000000u) - 8388608.f;
}
// 32 bytes, a whole sector, at once.
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Blocks read back: a CTA of D threads per block. A thread takes two of the keys' 16-byte
// loads, 8 tokens of four dims, and of the values the words of four tokens and sixteen dims; lanes
// are ordered so that a warp's stores are whole rows. Masked tokens are zeros.
template <typename T, int D>
__global__ void __launch_bounds__(D) quant4_read_kernel(Q4ReadArgs p) {
  constexpr int CH = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  for (long long n = blockIdx.x; n < p.n; n += gridDim.x) {
    const long long at = p.ids != nullptr ? p.ids[n] : n;
    if (at < 0 || at >= p.n_units) {
      if (tid == 0) quant_flag(p.status, kQErrIndex);
      continue;
    }
    const uint8_t* unit = p.units + at * quant4_unit_bytes(D);
    const float* e = reinterpret_cast<const float*>(unit + quant4_e_off(D));
    const int vm = tid % CH, vc = tid / CH % 4, vw = tid / CH / 4;
    uint4 kq[2];
    uint32_t ksteps = 0, vq[8];
    uint2 kzeros = make_uint2(0, 0), vsteps = kzeros, vzeros = kzeros;
    const int km = tid % (D / 4) / 4, kc = tid % 4, kg = tid / (D / 4);
    if (p.k != nullptr) {
#pragma unroll
      for (int r = 0; r < 2; ++r) kq[r] = reinterpret_cast<const uint4*>(unit)[km * 32 + 4 * (kg + 4 * r) + kc];
      const int o = 4 * (kc * CH + km);
      ksteps = *reinterpret_cast<const uint32_t*>(unit + quant4_kstep_off(D) + o);
      kzeros = *reinterpret_cast<const uint2*>(unit + quant4_kzero_off(D) + 2 * o);
    }
    if (p.v != nullptr) {
#pragma unroll
      for (int x = 0; x < 8; ++x) vq[x] = reinterpret_cast<const uint32_t*>(unit + 32 * D)[4 * (vm * 32 + 4 * x + vc) + vw];
      const int o = vm / 4 * kQB + 4 * (4 * vc + vw);
      vsteps = *reinterpret_cast<const uint2*>(unit + quant4_vstep_off(D) + 2 * o);
      vzeros = *reinterpret_cast<const uint2*>(unit + quant4_vzero_off(D) + 2 * o);
    }
    const float e0 = e[lane], e1 = e[lane + 32], ks = e[kQB], vs = e[kQB + 1];
    const uint32_t live[2] = {__ballot_sync(0xffffffffu, e0 != -INFINITY), __ballot_sync(0xffffffffu, e1 != -INFINITY)};
    auto is_live = [&](int t) { return (live[t / 32] >> (t % 32) & 1u) != 0; };
    if (p.e != nullptr && tid < kQB) p.e[n * kQB + tid] = tid < 32 ? e0 : e1;
    if (p.k != nullptr) {
      float st[4], z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        st[i] = half_bits(ksteps >> (8 * i) << 8 & 0xFF00u);
        z[i] = half_bits((i < 2 ? kzeros.x : kzeros.y) >> (16 * (i % 2)) & 0xFFFFu);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int g = kg + 4 * r;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t word = w == 0 ? kq[r].x : w == 1 ? kq[r].y : w == 2 ? kq[r].z : kq[r].w;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int t = 16 * w + 4 * (g / 2) + g % 2 + 2 * half;
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = is_live(t) ? fmaf(st[i], code_f32(word, 4 * (half + 2 * (i / 2) + 4 * (i % 2))), z[i]) * ks : 0.f;
            T* to = static_cast<T*>(p.k) + (n * kQB + t) * D + 16 * km + 4 * kc;
            if constexpr (sizeof(T) == 4)
              *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
            else
              *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]));
          }
        }
      }
    }
    if (p.v != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * vw + 4 * vc + i;
        const float st = half_bits((i < 2 ? vsteps.x : vsteps.y) >> (16 * (i % 2)) & 0xFFFFu);
        const float z = half_bits((i < 2 ? vzeros.x : vzeros.y) >> (16 * (i % 2)) & 0xFFFFu);
        float f[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) f[x] = is_live(t) ? fmaf(st, code_f32(vq[x % 8], 4 * (x / 8 + 2 * (i / 2) + 4 * (i % 2))), z) * vs : 0.f;
        T* to = static_cast<T*>(p.v) + (n * kQB + t) * D + 16 * vm;
        if constexpr (sizeof(T) == 4) {
          store32(to, reinterpret_cast<const uint32_t*>(f));
          store32(to + 8, reinterpret_cast<const uint32_t*>(f + 8));
        } else {
          uint32_t w[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) w[x] = bf16x2(f[2 * x], f[2 * x + 1]);
          store32(to, w);
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t read_variant(const Q4ReadArgs& a, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  return launch_dependent(quant4_read_kernel<T, D>, dim3((unsigned)std::min<long long>(a.n, 1 << 20)), D, 0, stream, a);
}

}  // namespace

cudaError_t launch_quant4_append(const Shape& s, const Q4AppendArgs& a, cudaStream_t stream) {
  if (s.dtype == 0) return s.d == 64 ? append_variant<float, 64>(s, a, stream) : append_variant<float, 128>(s, a, stream);
  return s.d == 64 ? append_variant<__nv_bfloat16, 64>(s, a, stream) : append_variant<__nv_bfloat16, 128>(s, a, stream);
}

cudaError_t launch_quant4_read(const Shape& s, const Q4ReadArgs& a, cudaStream_t stream) {
  if (s.dtype == 0) return s.d == 64 ? read_variant<float, 64>(a, stream) : read_variant<float, 128>(a, stream);
  return s.d == 64 ? read_variant<__nv_bfloat16, 64>(a, stream) : read_variant<__nv_bfloat16, 128>(a, stream);
}

}  // namespace nosa
