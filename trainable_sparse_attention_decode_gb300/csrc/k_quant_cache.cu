// Write side of the 8-bit block cache: appending tokens and evicting blocks.
//
// Appending reads the new tokens once and writes them once, in 8 bits: HBM bounds a
// prompt (GB300: 4 x 8192 tokens of 8 heads of 128 in bf16, 203 MB, 35.4 us = 85 % of the
// measured copy rate; what is left is the lengths' read ahead of the block's and the
// CTAs' barriers), latency a token (32 requests of 8 heads, every fourth completing a
// block: 4.8 us) and an eviction (256 units: one of 129 blocks 4.7 us, 1024 blocks down
// to 64 7.2 us).
#include "k_quant.cuh"

#include <algorithm>

namespace nosa {
namespace {

constexpr int kAppendThreads = 256;

// Eight consecutive elements as fp32.
template <typename T> struct Row8;
template <> struct Row8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const void* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  // largest magnitude as the bit pattern of an fp32 number
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t m = __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu), __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu));
    return max(m & 0xFFFF0000u, m << 16);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
    f[4] = bf16_lo(r.z); f[5] = bf16_hi(r.z); f[6] = bf16_lo(r.w); f[7] = bf16_hi(r.w);
  }
};
template <> struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ uint32_t amax() const {
    float f[8];
    get(f);
    uint32_t m = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) m = max(m, __float_as_uint(f[x]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

// Four fp32 values as four e4m3 codes (round to nearest even), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// A unit on its way through shared memory: runs of 512 bytes (32 lanes x 16) padded to
// 544, so that the words that a warp's patches write together, which lie 512 bytes
// apart in the unit, fall into different banks.
template <int D>
struct UnitImage {
  static constexpr int RUNS = 2 * kQB * D / 512, PITCH = 544;
  __align__(16) uint8_t code[RUNS * PITCH];
  __align__(16) float rest[kQB + 8];  // logits, scales, zeros
  uint32_t amax[2];
  static_assert(quant_unit_bytes(D) - quant_e_off(D) == (kQB + 8) * 4, "what follows the codes");
  __device__ __forceinline__ uint8_t* at(int off) { return code + off / 512 * PITCH + off % 512; }
};

// Quantises blocks of a unit's tokens: x -> e4m3(x * (448 / max |x|)), the maximum
// over the block's tokens whose logit is not -inf; the others become zeros. A thread
// owns patches of 4 tokens x 8 dims, the smallest piece whose key and value words are
// whole, so a block stays in registers between the maximum and the conversion and the
// input is read once; the image is put together in shared memory and leaves in 16-byte
// stores. (One wave of CTAs that load the next block while they store one was slower than
// a CTA per block: 50 us against 43 for 4 x 8192 tokens of 8 heads of 128 in bf16.)
template <typename T, int D>
struct BlockQuant {
  static constexpr int ELT = (int)sizeof(T), CE = 16 / ELT, NT = kAppendThreads;
  static constexpr int NP = 16 * (D / 8);  // patches of K (and of V)
  static constexpr int PPT = 2 * NP / NT;  // patches per thread: 2 (d = 128) or 1
  static_assert(PPT * NT == 2 * NP, "patches must divide over the threads");
  const QAppendArgs& p;
  const uint8_t* tail;
  int Hkv, u, b, h, n0, old, tid;
  Row8<T> row[PPT][4];
  float ev;
  int idx;

  __device__ __forceinline__ BlockQuant(const QAppendArgs& p_, int Hkv_, int u_, int n0_, const uint8_t* tail_)
      : p(p_), tail(tail_), Hkv(Hkv_), u(u_), b(u_ / Hkv_), h(u_ % Hkv_), n0(n0_), old(n0_ % kQB), tid(threadIdx.x) {}

  // Patch i of this thread: keys (isv 0) or values, 16-byte column pair c8, tokens 4 tg ...
  __device__ __forceinline__ void patch(int i, int& isv, int& c8, int& tg) const {
    const int id = tid + i * NT;
    isv = id / NP;
    c8 = id % NP % (D / 8);
    tg = id % NP / (D / 8);
  }

  // Starts the loads of block j of the new blocks (0: the one that the tail began).
  __device__ __forceinline__ void load(int j) {
    idx = p.tab[(long long)u * p.max_blocks + n0 / kQB + j];
    const int first = j * kQB - old;  // the block's first token among the new ones, or before them
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      int isv, c8, tg;
      patch(i, isv, c8, tg);
      const QStrides& st = isv ? p.vs : p.ks;
      const T* src = reinterpret_cast<const T*>(isv ? p.v : p.k) + b * st.b + h * st.h + (first + 4 * tg) * st.t + c8 * 8;
#pragma unroll
      for (int r = 0; r < 4; ++r, src += st.t) {
        const int t = 4 * tg + r;
        if (first >= 0 || first + t >= 0) {
          row[i][r].load(src);
        } else if (isv) {  // from the tail: values in rows, keys in 16-byte chunks
          row[i][r].load(tail + ((size_t)kQB * D + (size_t)t * D + c8 * 8) * ELT);
        } else if constexpr (CE == 8) {
          row[i][r].load(tail + ((size_t)c8 * kQB + t) * 16);
        } else {
          Row8<float>& f = row[i][r];
          f.a = *reinterpret_cast<const float4*>(tail + ((size_t)(2 * c8) * kQB + t) * 16);
          f.b = *reinterpret_cast<const float4*>(tail + ((size_t)(2 * c8 + 1) * kQB + t) * 16);
        }
      }
    }
    ev = 0.f;
    if (tid < kQB) {
      if (first + tid < 0)
        ev = reinterpret_cast<const float*>(tail + 2 * (size_t)kQB * D * ELT)[tid];
      else if (p.e != nullptr)
        ev = p.e[((long long)b * p.n + first + tid) * Hkv + h];
    }
  }

  // The loaded block into shared memory (whole CTA).
  __device__ __forceinline__ void encode(UnitImage<D>& img) {
    if (tid < kQB) img.rest[tid] = ev;
    if (tid < 2) img.amax[tid] = 0;
    __syncthreads();
    // Maximum of the magnitudes' bit patterns: a NaN or an infinity comes out on top.
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      int isv, c8, tg;
      patch(i, isv, c8, tg);
      const float4 e = reinterpret_cast<const float4*>(img.rest)[tg];
      if (e.x == -INFINITY) row[i][0].zero();
      if (e.y == -INFINITY) row[i][1].zero();
      if (e.z == -INFINITY) row[i][2].zero();
      if (e.w == -INFINITY) row[i][3].zero();
      uint32_t mx = max(max(row[i][0].amax(), row[i][1].amax()), max(row[i][2].amax(), row[i][3].amax()));
      mx = __reduce_max_sync(0xffffffffu, mx);
      if ((tid & 31) == 0) atomicMax(img.amax + isv, mx);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      int isv, c8, tg;
      patch(i, isv, c8, tg);
      const uint32_t bits = img.amax[isv];
      const float amax = __uint_as_float(bits);
      const float inv = amax >= 0x1p-100f ? 448.f / amax : 0.f;
      if (bits >= 0x7F800000u) {
#pragma unroll
        for (int r = 0; r < 4; ++r) row[i][r].zero();
      }
      float2 f[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        row[i][r].get(reinterpret_cast<float*>(f[r]));
#pragma unroll
        for (int x = 0; x < 4; ++x) f[r][x] = __fmul2_rn(f[r][x], make_float2(inv, inv));
      }
      if (isv) {  // one word: the patch's four tokens of one dim
        uint8_t* to = img.at(quant_v_off(4 * tg, c8 * 8, D));  // dims of a column pair are 64 bytes apart
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          *reinterpret_cast<uint32_t*>(to + 128 * x) = e4m3x4(f[0][x].x, f[1][x].x, f[2][x].x, f[3][x].x);
          *reinterpret_cast<uint32_t*>(to + 128 * x + 64) = e4m3x4(f[0][x].y, f[1][x].y, f[2][x].y, f[3][x].y);
        }
      } else {  // two words: four dims of tokens r and r + 2
        uint8_t* to = img.at(quant_k_off(4 * tg, c8 * 8, D));  // next token 64 bytes on, next four dims 16
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int x = 0; x < 4; x += 2)
            *reinterpret_cast<uint2*>(to + 64 * r + 8 * x) =
                make_uint2(e4m3x4(f[r][x].x, f[r][x].y, f[r][x + 1].x, f[r][x + 1].y),
                           e4m3x4(f[r + 2][x].x, f[r + 2][x].y, f[r + 2][x + 1].x, f[r + 2][x + 1].y));
      }
    }
    if (tid < 8) {
      const uint32_t bits = tid < 2 ? img.amax[tid] : 0u;
      const float amax = __uint_as_float(bits);
      img.rest[kQB + tid] = bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : amax >= 0x1p-100f ? amax / 448.f : 0.f;
    }
    __syncthreads();
  }

  // The image to unit `to` of the cache.
  __device__ __forceinline__ void store(UnitImage<D>& img, int to) const {
    if (to < 0 || (long long)to >= p.n_units) {
      if (tid == 0) quant_flag(p.status, kQErrIndex);
      return;
    }
    uint8_t* dst = p.units + (long long)to * quant_unit_bytes(D);
#pragma unroll
    for (int o = tid * 16; o < quant_e_off(D); o += NT * 16)
      *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(img.at(o));
    if (tid < (kQB + 8) / 4)
      reinterpret_cast<uint4*>(dst + quant_e_off(D))[tid] = reinterpret_cast<const uint4*>(img.rest)[tid];
  }
};

// What the call does to unit u: tokens before it, new ones (0 where the unit is left as it was).
struct UnitAppend {
  int n0, add;
};
template <bool EARLY>
__device__ __forceinline__ UnitAppend unit_append(const QAppendArgs& p, int Hkv, int u, bool flag) {
  UnitAppend r;
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

// Blocks that the call completes: grid (units, most blocks), so that neighbouring
// CTAs read the heads of the same tokens.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 2 || D == 64 ? 4 : 2)
quant_blocks_kernel(QAppendArgs p, int Hkv, long long payload) {
  __shared__ UnitImage<D> img;
  griddep_wait();
  griddep_launch_dependents();
  const int u = blockIdx.x, j = blockIdx.y;
  const UnitAppend a = unit_append<false>(p, Hkv, u, false);
  if (j >= (a.n0 % kQB + a.add) / kQB) return;
  BlockQuant<T, D> q(p, Hkv, u, a.n0, p.tail + u * payload);
  q.load(j);
  q.encode(img);
  q.store(img, q.idx);
}

// The unit's tail and length; with BLOCK also the one block that at most 64 new
// tokens can complete (single tokens: one launch).
template <typename T, int D, bool BLOCK>
__global__ void __launch_bounds__(kAppendThreads) quant_tail_kernel(QAppendArgs p, int Hkv, long long payload) {
  constexpr int ELT = (int)sizeof(T), CE = 16 / ELT, NCH = D / CE;
  const int u = blockIdx.x, b = u / Hkv, h = u % Hkv, tid = threadIdx.x;
  if (BLOCK) griddep_wait();  // (the call's first launch)
  griddep_launch_dependents();
  const UnitAppend a = unit_append<!BLOCK>(p, Hkv, u, tid == 0);
  uint8_t* tail = p.tail + u * payload;
  const int old = a.n0 % kQB, done = (old + a.add) / kQB;
  if constexpr (BLOCK) {
    __shared__ UnitImage<D> img;
    if (done > 0) {
      BlockQuant<T, D> q(p, Hkv, u, a.n0, tail);
      q.load(0);
      q.encode(img);
      q.store(img, q.idx);
    }
  }
  if (!BLOCK) griddep_wait();  // the blocks' launch has read the old tail
  __syncthreads();             // ... and so has this one, and the length
  const int first = done > 0 ? 0 : old, left = old + a.add - done * kQB;
  for (int i = tid; i < (left - first) * NCH; i += kAppendThreads) {
    const int r = first + i / NCH, c = i % NCH;
    const long long tok = (long long)done * kQB + r - old;
    const T* ksrc = reinterpret_cast<const T*>(p.k) + b * p.ks.b + tok * p.ks.t + h * p.ks.h + c * CE;
    const T* vsrc = reinterpret_cast<const T*>(p.v) + b * p.vs.b + tok * p.vs.t + h * p.vs.h + c * CE;
    *reinterpret_cast<uint4*>(tail + ((size_t)c * kQB + r) * 16) = *reinterpret_cast<const uint4*>(ksrc);
    *reinterpret_cast<uint4*>(tail + (size_t)kQB * D * ELT + (size_t)r * D * ELT + c * 16) =
        *reinterpret_cast<const uint4*>(vsrc);
  }
  float* te = reinterpret_cast<float*>(tail + 2 * (size_t)kQB * D * ELT);
  for (int r = first + tid; r < left; r += kAppendThreads)
    te[r] = p.e != nullptr ? p.e[((long long)b * p.n + (long long)done * kQB + r - old) * Hkv + h] : 0.f;
  if (tid == 0) p.lens_out[u] = p.lens[u] + a.add;
}

template <typename T, int D>
cudaError_t append_variant(const Shape& s, const QAppendArgs& a, cudaStream_t stream) {
  if (a.n <= kQB) {
    return launch_dependent(quant_tail_kernel<T, D, true>, dim3(s.U), kAppendThreads, 0, stream, a, s.Hkv, s.payload);
  } else {
    const int most = (int)std::min<long long>((a.n + kQB - 1LL) / kQB, a.max_blocks);
    const cudaError_t e =
        launch_dependent(quant_blocks_kernel<T, D>, dim3(s.U, most), kAppendThreads, 0, stream, a, s.Hkv, s.payload);
    if (e != cudaSuccess) return e;
    return launch_dependent(quant_tail_kernel<T, D, false>, dim3(s.U), kAppendThreads, 0, stream, a, s.Hkv, s.payload);
  }
}

// ---------------------------------------------------------------------------
// Eviction. One CTA per unit: the table row and the weights' bit patterns go to
// shared memory once, a radix selection (8 bits at a time over the order-preserving
// keys) finds the largest weight that still leaves, and a stable partition writes
// the row back: kept blocks in order, then the evicted ones, which are the next
// destinations of appended blocks. The row is read and written once (16 bytes an
// entry); with rows of hundreds of entries latency is all there is, so a pass costs
// one barrier: each has a histogram of its own, and every warp adds it up for itself.
// ---------------------------------------------------------------------------
constexpr int kEvictThreads = 256;
constexpr int kEvictAhead = 4;  // entries per thread fetched before the length is known

// Order-preserving key of a weight; NaN ranks above every number.
__device__ __forceinline__ uint32_t weight_key(uint32_t bits) {
  const float f = __uint_as_float(bits);
  return isnan(f) ? 0xFFFFFFFFu : ordered_key(f);
}

// Inclusive prefix sum over a warp's lanes.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Exclusive prefix sum over the block's threads, *total its sum. warp_s is not used twice.
__device__ __forceinline__ int block_scan(int v, int* warp_s, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int inc = warp_scan(v, lane);
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kEvictThreads / 32; ++w) {
    const int x = warp_s[w];
    if (w < warp) base += x;
    sum += x;
  }
  *total = sum;
  return base + inc - v;
}

__global__ void __launch_bounds__(kEvictThreads) quant_evict_kernel(QEvictArgs p) {
  extern __shared__ uint32_t evict_smem[];
  __shared__ int hist[4][256];
  __shared__ int eq_s[kEvictThreads / 32], kept_s[kEvictThreads / 32];
  const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const long long row = (long long)u * p.max_blocks;
#pragma unroll
  for (int k = 0; k < 4; ++k) hist[k][tid] = 0;
  griddep_wait();
  griddep_launch_dependents();
  // the first entries of the row are fetched together with its length
  uint32_t w0[kEvictAhead];
  int32_t t0[kEvictAhead];
#pragma unroll
  for (int k = 0; k < kEvictAhead; ++k) {
    const int i = tid + k * kEvictThreads;
    w0[k] = i < p.max_blocks ? __float_as_uint(p.mass[row + i]) : 0u;
    t0[k] = i < p.max_blocks ? p.tab[row + i] : 0;
  }
  const int n0 = quant_len(p.lens, u, p.max_blocks, p.status, tid == 0);
  const int full = n0 < 0 ? 0 : n0 / kQB, over = max(0, full - p.budget);
  if (over == 0) {  // nothing to evict: the row as it is
    for (int i = tid; i < p.max_blocks; i += kEvictThreads) {
      if (p.tab_out != p.tab) p.tab_out[row + i] = p.tab[row + i];
      if (p.mass_out != p.mass) p.mass_out[row + i] = p.mass[row + i];
      if (p.order != nullptr) p.order[row + i] = i;
    }
    if (tid == 0 && p.lens_out != p.lens) p.lens_out[u] = p.lens[u];
    return;
  }
  uint32_t* w = evict_smem;                                     // [full] weights (bit patterns)
  int32_t* tb = reinterpret_cast<int32_t*>(evict_smem + full);  // [full] table entries
  const int old = full - p.n_recent;                            // >= over: n_recent <= budget
#pragma unroll
  for (int k = 0; k < kEvictAhead; ++k) {
    const int i = tid + k * kEvictThreads;
    if (i < full) {
      w[i] = w0[k];
      tb[i] = t0[k];
    }
  }
  for (int i = tid + kEvictAhead * kEvictThreads; i < full; i += kEvictThreads) {
    w[i] = __float_as_uint(p.mass[row + i]);
    tb[i] = p.tab[row + i];
  }
  const float tail_mass = full < p.max_blocks ? p.mass[row + full] : 0.f;
  __syncthreads();
  uint32_t cut = 0;  // the over-th smallest key, a digit at a time
  int rank = over;   // ... among the keys that share the digits so far
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int shift = 24 - 8 * k;
    const uint32_t mask = k == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = tid; i < old; i += kEvictThreads) {
      const uint32_t key = weight_key(w[i]);
      if ((key & mask) == cut) atomicAdd(&hist[k][(key >> shift) & 255], 1);
    }
    __syncthreads();
    int c[8], sum = 0;  // the lane's eight bins
#pragma unroll
    for (int x = 0; x < 8; ++x) sum += c[x] = hist[k][8 * lane + x];
    int before = warp_scan(sum, lane) - sum;
    const int at = __ffs(__ballot_sync(0xffffffffu, before < rank && rank <= before + sum)) - 1;
    int bin = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) {  // (on lane `at`: the bin that reaches the rank)
      if (bin == x && before + c[x] < rank) {
        before += c[x];
        ++bin;
      }
    }
    cut |= (uint32_t)(8 * at + __shfl_sync(0xffffffffu, bin, at)) << shift;
    rank -= __shfl_sync(0xffffffffu, before, at);
  }
  // Blocks below the cut leave; of those at the cut, the `rank` ones of the highest indices.
  const int per = (old + kEvictThreads - 1) / kEvictThreads, i0 = min(old, tid * per), i1 = min(old, i0 + per);
  int eq = 0, above = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = weight_key(w[i]);
    eq += key == cut;
    above += key > cut;
  }
  int eq_total, kept_total;
  int eq_at = block_scan(eq, eq_s, &eq_total);
  const int eq_keep = eq_total - rank;
  int at = block_scan(above + max(0, min(eq, eq_keep - eq_at)), kept_s, &kept_total);
  int gone = full - over + (i0 - at);
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = weight_key(w[i]);
    const bool keep = key > cut || (key == cut && eq_at++ < eq_keep);
    const int to = keep ? at++ : gone++;
    p.tab_out[row + to] = tb[i];
    if (keep) p.mass_out[row + to] = __uint_as_float(w[i]);
    if (p.order != nullptr) p.order[row + to] = i;
  }
  for (int i = old + tid; i < full; i += kEvictThreads) {  // the newest blocks move up
    p.tab_out[row + i - over] = tb[i];
    p.mass_out[row + i - over] = __uint_as_float(w[i]);
    if (p.order != nullptr) p.order[row + i - over] = i;
  }
  // behind the kept blocks: the tail's weight, then zeros
  for (int i = full - over + tid; i <= full && i < p.max_blocks; i += kEvictThreads)
    p.mass_out[row + i] = i == full - over ? tail_mass : 0.f;
  for (int i = full + tid; i < p.max_blocks; i += kEvictThreads) {
    if (p.tab_out != p.tab) p.tab_out[row + i] = p.tab[row + i];
    if (p.mass_out != p.mass && i > full) p.mass_out[row + i] = p.mass[row + i];
    if (p.order != nullptr) p.order[row + i] = i;
  }
  if (tid == 0) p.lens_out[u] = n0 - kQB * over;
}

}  // namespace

cudaError_t launch_quant_append(const Shape& s, const QAppendArgs& a, cudaStream_t stream) {
  if (s.dtype == 0)
    return s.d == 64 ? append_variant<float, 64>(s, a, stream) : append_variant<float, 128>(s, a, stream);
  return s.d == 64 ? append_variant<__nv_bfloat16, 64>(s, a, stream) : append_variant<__nv_bfloat16, 128>(s, a, stream);
}

cudaError_t launch_quant_evict(const Shape& s, const QEvictArgs& a, cudaStream_t stream) {
  const size_t smem = (size_t)a.max_blocks * 8;
  static std::atomic<int> lim[64];
  if (smem > 40000) {  // (4.2 KB more are static)
    const cudaError_t e = raise_smem_limit((const void*)quant_evict_kernel, smem, lim);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(quant_evict_kernel, dim3(s.U), kEvictThreads, smem, stream, a);
}

}  // namespace nosa
