// Write side of the 4-bit block cache: appending tokens, with the rotation of their keys on
// the way, and reading blocks back.
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
// What the call does to unit u: tokens before it, new ones (0 where the unit is left as it was).
template <bool EARLY>
__device__ __forceinline__ UnitAppend4 unit_append(const QAppendArgs& p, int Hkv, int u, bool flag) {
  UnitAppend4 r;
  r.n0 = quant_len<EARLY>(p.lens, u, p.max_blocks, p.status, flag);
  r.add = quant_count<EARLY>(p.n_new, u / Hkv, p.n, p.status, flag);
  if (r.n0 < 0) {
    r.n0 = r.add = 0;
  } else if (r.n0 > kQB * p.max_blocks - r.add) {
    if (flag) quant_flag(p.status, kQErrCapacity);
    r.add = 0;
  }
  return r;
}

// Chunk i of new token `tok`'s key of (request b, head h), turned and rounded, as two vectors.
template <typename T>
__device__ __forceinline__ void new_key(const Q4AppendArgs& p, int b, int h, int tok, int i, const RopeChunk& ch, Vec8<T>* v) {
  const T* row = static_cast<const T*>(p.a.k) + b * p.a.ks.b + (long long)tok * p.a.ks.t + h * p.a.ks.h;
  v[0].load(row + ch.lo);
  v[1].load(row + ch.hi);
  if (!ch.turned) return;
  float2 cs[8];
  rope_angles<false>(p.rope, (long long)b * p.a.n + tok, i, cs);
  float x[16];
  v[0].get(x);
  v[1].get(x + 8);
  rope_turn_chunk(p.rope.interleaved, cs, x);
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
  static __device__ __forceinline__ uint32_t size(float x) { return x == -INFINITY ? 0u : __float_as_uint(x) & 0x7FFFFFFFu; }
};

// A block of a unit's tokens on its way into 4 bits. CTAs of 2 D threads: thread (i, tp) has
// chunk i of D / 16 and a pair of tokens, of the keys the two of a word (4 (tp / 2) + tp % 2 and
// the second after it), of the values two of the four of a word (2 tp and 2 tp + 1). The block
// stays in registers, in the tokens' type, from its loads to its codes:
//   channels' extremes: over the thread's tokens, over the warp's by shuffles that halve the
//     values each lane has, over the warps through shared memory;
//   tokens' extremes: over four lanes;
//   codes: (x / scale - zero) / step + 1.5 2^23, whose last bits are the code; a word is the sum
//     of its codes' bits, shifted, less what the exponents add up to.
template <typename T, int D>
struct Quant4Block {
  using X = Extreme<T>;
  static constexpr int NT = 2 * D, WARPS = NT / 32, CH = D / 16, PITCH = 528;  // (bytes of 512, padded against bank conflicts)
  static constexpr int REST = quant4_unit_bytes(D) - 64 * D;
  struct Shared {
    __align__(16) uint8_t code[2 * CH * PITCH];
    __align__(16) uint8_t rest[REST];  // steps, zeros, logits, scales: as in the unit from byte 64 D on
    __align__(16) T part[WARPS][2 * D];                // channels: - least, largest
    __align__(16) float minus_zero[D], inv_step[D];    // channels
    __align__(16) uint32_t top[2][WARPS];              // largest magnitudes of keys and values
  };
  const Q4AppendArgs& p;
  const T* tail;
  int Hkv, u, b, h, n0, old, tid;

  __device__ __forceinline__ Quant4Block(const Q4AppendArgs& p_, int Hkv_, int u_, int n0_, const T* tail_)
      : p(p_), tail(tail_), Hkv(Hkv_), u(u_), b(u_ / Hkv_), h(u_ % Hkv_), n0(n0_), old(n0_ % kQB), tid(threadIdx.x) {}

  __device__ __forceinline__ float logit(int first, int t) const {
    if (first + t < 0) return reinterpret_cast<const float*>(tail + 2 * kQB * D)[t];
    return p.a.e != nullptr ? p.a.e[((long long)b * p.a.n + first + t) * Hkv + h] : 0.f;
  }
  // fp16 bits of a group's zero and step
  template <bool KEY>
  static __device__ __forceinline__ uint2 zero_step(float lo, float hi, float inv) {
    const uint32_t z = __half_as_ushort(__float2half_rd(lo * inv + 0.f));  // (no -0)
    const uint32_t s = __half_as_ushort(__float2half_ru(__fmul_rn(__fsub_rn(hi * inv, half_bits(z)), 1.f / 15.f)));
    return make_uint2(z, KEY ? (s + 0xFFu) & 0xFF00u : s);
  }
  static __device__ __forceinline__ float inv_of(uint32_t step) { return step != 0 ? __frcp_rn(half_bits(step)) : 0.f; }

  // Block j of the new blocks (0: the one that the tail began) into its unit (whole CTA).
  __device__ __forceinline__ void run(int j, Shared& sh) const {
    const int to = p.a.tab[(long long)u * p.a.max_blocks + n0 / kQB + j];
    const int first = j * kQB - old;  // the block's first token among the new ones, or before them
    const int i = tid % CH, tp = tid / CH, lane = tid & 31, warp = tid >> 5;
    const RopeChunk ch = rope_chunk(p.rope, i);
    const int kt = 4 * (tp / 2) + tp % 2, vt = 2 * tp;
    Vec8<T> k[2][2], v[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = vt + r;
      if (first + t >= 0) {
        const T* row = static_cast<const T*>(p.a.v) + b * p.a.vs.b + (long long)(first + t) * p.a.vs.t + h * p.a.vs.h + 16 * i;
        if (p.wide) {  // sixteen elements in a row
#pragma unroll
          for (int y = 0; y < (int)sizeof(T) / 2; ++y) load32(row + y * 32 / sizeof(T), reinterpret_cast<uint32_t*>(v[r]) + 8 * y);
        } else {
          v[r][0].load(row);
          v[r][1].load(row + 8);
        }
      } else {
        tail_load<T, D>(tail, false, t, 16 * i, v[r][0]);
        tail_load<T, D>(tail, false, t, 16 * i + 8, v[r][1]);
      }
    }
    const float e0 = logit(first, lane), e1 = logit(first, lane + 32);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = kt + 2 * r;
      if (first + t >= 0) {
        new_key<T>(p, b, h, first + t, i, ch, k[r]);
      } else {
        tail_load<T, D>(tail, true, t, ch.lo, k[r][0]);
        tail_load<T, D>(tail, true, t, ch.hi, k[r][1]);
      }
    }
    if (warp == 0) {
      reinterpret_cast<float*>(sh.rest + 7 * D)[lane] = e0;
      reinterpret_cast<float*>(sh.rest + 7 * D)[lane + 32] = e1;
      if (lane < 6) reinterpret_cast<uint32_t*>(sh.rest + 7 * D)[kQB + 2 + lane] = 0;
    }
    const uint32_t l0 = __ballot_sync(0xffffffffu, e0 != -INFINITY), l1 = __ballot_sync(0xffffffffu, e1 != -INFINITY);
    const uint32_t kl = (kt < 32 ? l0 : l1) >> (kt % 32), vl = (vt < 32 ? l0 : l1) >> (vt % 32);
    const bool klive[2] = {(kl & 1u) != 0, (kl & 4u) != 0}, vlive[2] = {(vl & 1u) != 0, (vl & 2u) != 0};
    // A masked token counts as its neighbour, or not at all.
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float zero[8] = {};
      if (!klive[r]) {
        k[r][0] = k[1 - r][0];
        k[r][1] = k[1 - r][1];
      }
      if (!vlive[r]) {
        v[r][0].set(zero);
        v[r][1].set(zero);
      }
    }
    // ---- extremes ----
    uint32_t topk = 0, topv = 0;
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
      if (!klive[0] && !klive[1]) {
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
#pragma unroll
      for (int c = 0; c < LEFT; ++c) topk = max(topk, X::size(red[c]));
    }
    float vlo = 0.f, vhi = 0.f;  // of the lane's one of the two tokens: even lanes the first, odd ones the second
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
      const float l = X::whole(lo), g = X::whole(hi);
      topv = max(topv, max(__float_as_uint(l) & 0x7FFFFFFFu, __float_as_uint(g) & 0x7FFFFFFFu));
      if ((i & 1) == r) {
        vlo = -l;
        vhi = g;
      }
    }
    topk = __reduce_max_sync(0xffffffffu, topk);
    topv = __reduce_max_sync(0xffffffffu, topv);
    if (lane == 0) {
      sh.top[0][warp] = topk;
      sh.top[1][warp] = topv;
    }
    __syncthreads();
    // ---- scales, steps, zeros ----
#pragma unroll
    for (int w = 0; w < WARPS; w += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(&sh.top[0][w]), y = *reinterpret_cast<const uint4*>(&sh.top[1][w]);
      topk = max(max(topk, max(x.x, x.y)), max(x.z, x.w));
      topv = max(max(topv, max(y.x, y.y)), max(y.z, y.w));
    }
    const bool ok[2] = {topk >= 0x0D800000u && topk < 0x7F800000u, topv >= 0x0D800000u && topv < 0x7F800000u};  // finite, not below 2^-100
    const float kinv = ok[0] ? __uint_as_float((256u - (topk >> 23)) << 23) : 0.f;
    const float vinv = ok[1] ? __uint_as_float((256u - (topv >> 23)) << 23) : 0.f;
    if (tid < 2) {
      const uint32_t top = tid ? topv : topk;
      reinterpret_cast<uint32_t*>(sh.rest + 7 * D)[kQB + tid] = top >= 0x7F800000u ? 0x7FC00000u : top >= 0x0D800000u ? ((top >> 23) - 2) << 23 : 0u;
    }
    if (tid < D) {
      float lo = -INFINITY, hi = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        lo = fmaxf(lo, to_f32(sh.part[w][tid]));  // (where there is a NaN, ok is false)
        hi = fmaxf(hi, to_f32(sh.part[w][D + tid]));
      }
      const uint2 zs = ok[0] ? zero_step<true>(-lo, hi, kinv) : make_uint2(0, 0);
      sh.minus_zero[tid] = -half_bits(zs.x);
      sh.inv_step[tid] = inv_of(zs.y);
      sh.rest[quant4_order(tid, D)] = zs.y >> 8;
      reinterpret_cast<unsigned short*>(sh.rest + D)[quant4_order(tid, D)] = zs.x;
    }
    // ---- codes of the values ----
    {
      const uint2 zs = ok[1] && vlive[i & 1] ? zero_step<false>(vlo, vhi, vinv) : make_uint2(0, 0);
      if (i % 4 < 2) {
        const int at = i / 4 * kQB + quant4_order(vt, kQB) + i % 4;  // (vt is even: the second token is next to the first)
        reinterpret_cast<unsigned short*>(sh.rest + 3 * D)[at] = zs.y;
        reinterpret_cast<unsigned short*>(sh.rest + 5 * D)[at] = zs.x;
      }
      const float mz = -half_bits(zs.x), rs = inv_of(zs.y);
      const float mz1 = __shfl_xor_sync(0xffffffffu, mz, 1), rs1 = __shfl_xor_sync(0xffffffffu, rs, 1);
      const float z2[2] = {i & 1 ? mz1 : mz, i & 1 ? mz : mz1}, r2[2] = {i & 1 ? rs1 : rs, i & 1 ? rs : rs1};
      float x[2][16];
      v[0][0].get(x[0]); v[0][1].get(x[0] + 8);
      v[1][0].get(x[1]); v[1][1].get(x[1] + 8);
      const int hh = tp & 1, c = tp / 2 % 4, w = tp / 8;
      const uint32_t mask = ok[1] ? 0xFFFFFFFFu : 0u;
      uint32_t word[8];
#pragma unroll
      for (int d = 0; d < 8; d += 2) {  // dims d, d + 1 and the eighth ones after them, of the two tokens
        uint2 n[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            n[r][e] = code_bits(make_float2(x[r][d + 8 * e], x[r][d + 8 * e + 1]), make_float2(vinv, vinv), make_float2(z2[r], z2[r]), make_float2(r2[r], r2[r]));
        word[d] = (((((n[1][1].x << 4) + n[1][0].x) << 16) + (n[0][1].x << 4) + n[0][0].x - kMagicBits * 0x00110011u) & mask) << (8 * hh);
        word[d + 1] = (((((n[1][1].y << 4) + n[1][0].y) << 16) + (n[0][1].y << 4) + n[0][0].y - kMagicBits * 0x00110011u) & mask) << (8 * hh);
      }
      uint8_t* row = sh.code + (CH + i) * PITCH + 16 * c + 4 * w;
#pragma unroll
      for (int d = 0; d < 4; ++d) {  // the other two tokens of the words are CH lanes away; each thread puts four words down
        const uint32_t other = __shfl_xor_sync(0xffffffffu, hh ? word[d] : word[d + 4], CH);
        *reinterpret_cast<uint32_t*>(row + 64 * (d + 4 * hh)) = (hh ? word[d + 4] : word[d]) | other;
      }
    }
    __syncthreads();
    // ---- codes of the keys ----
    {
      const uint32_t mask = ok[0] ? (klive[0] ? 0x0F0F0F0Fu : 0u) | (klive[1] ? 0xF0F0F0F0u : 0u) : 0u;
      const int g = tp % 8, w = tp / 8;
      const float2 inv = make_float2(kinv, kinv);
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
            n[r][0] = code_bits(make_float2(x[r][c], x[r][c + 1]), inv, make_float2(z.x, z.y), make_float2(s.x, s.y));
            n[r][1] = code_bits(make_float2(x[r][c + 2], x[r][c + 3]), inv, make_float2(z.z, z.w), make_float2(s.z, s.w));
          }
          const uint32_t lo = (n[1][1].x << 12) + (n[0][1].x << 8) + (n[1][0].x << 4) + n[0][0].x;
          const uint32_t hi = (n[1][1].y << 12) + (n[0][1].y << 8) + (n[1][0].y << 4) + n[0][0].y;
          *reinterpret_cast<uint32_t*>(row + 4 * c) = ((hi << 16) + lo - kMagicBits * 0x11111111u) & mask;
        }
      }
    }
    __syncthreads();
    if (to < 0 || (long long)to >= p.a.n_units) {
      if (tid == 0) quant_flag(p.a.status, kQErrIndex);
      return;
    }
    uint8_t* unit = p.a.units + (long long)to * quant4_unit_bytes(D);
#pragma unroll
    for (int o = tid; o < 4 * D; o += NT)
      reinterpret_cast<uint4*>(unit)[o] = *reinterpret_cast<const uint4*>(sh.code + o / 32 * PITCH + o % 32 * 16);
    if (tid < REST / 16) reinterpret_cast<uint4*>(unit + 64 * D)[tid] = reinterpret_cast<const uint4*>(sh.rest)[tid];
    static_assert(REST / 16 <= NT, "one store of a thread");
  }
};

// Blocks that the call completes: grid (units, most blocks), so that neighbouring CTAs read the
// heads of the same tokens.
template <typename T, int D>
__global__ void __launch_bounds__(2 * D, (sizeof(T) == 2 ? 4 : 2) * 128 / D) quant4_blocks_kernel(Q4AppendArgs p, int Hkv, long long payload) {
  __shared__ typename Quant4Block<T, D>::Shared sh;
  griddep_wait();
  griddep_launch_dependents();
  const int u = blockIdx.x, j = blockIdx.y;
  const UnitAppend4 ap = unit_append<false>(p.a, Hkv, u, false);
  if (j >= (ap.n0 % kQB + ap.add) / kQB) return;
  Quant4Block<T, D>(p, Hkv, u, ap.n0, reinterpret_cast<const T*>(p.a.tail + u * payload)).run(j, sh);
}

// The unit's tail and length; with BLOCK also the one block that at most 64 new tokens can
// complete (single tokens: one launch).
template <typename T, int D, bool BLOCK>
__global__ void __launch_bounds__(2 * D) quant4_tail_kernel(Q4AppendArgs p, int Hkv, long long payload) {
  const int u = blockIdx.x, b = u / Hkv, h = u % Hkv, tid = threadIdx.x;
  if (BLOCK) griddep_wait();  // (the call's first launch)
  griddep_launch_dependents();
  const UnitAppend4 ap = unit_append<!BLOCK>(p.a, Hkv, u, tid == 0);
  T* tail = reinterpret_cast<T*>(p.a.tail + u * payload);
  const int old = ap.n0 % kQB, done = (old + ap.add) / kQB;
  if constexpr (BLOCK) {
    __shared__ typename Quant4Block<T, D>::Shared sh;
    if (done > 0) Quant4Block<T, D>(p, Hkv, u, ap.n0, tail).run(0, sh);
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
      new_key<T>(p, b, h, tok, i, ch, x);
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
  if (a.a.n <= kQB) return launch_dependent(quant4_tail_kernel<T, D, true>, dim3(s.U), 2 * D, 0, stream, a, s.Hkv, s.payload);
  const int most = (int)std::min<long long>((a.a.n + kQB - 1LL) / kQB, a.a.max_blocks);
  const cudaError_t e = launch_dependent(quant4_blocks_kernel<T, D>, dim3(s.U, most), 2 * D, 0, stream, a, s.Hkv, s.payload);
  if (e != cudaSuccess) return e;
  return launch_dependent(quant4_tail_kernel<T, D, false>, dim3(s.U), 2 * D, 0, stream, a, s.Hkv, s.payload);
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
