// Attention over the 8-bit block cache.
//
// Row (t, g) of unit u sees tokens [0, len - T_b + t]: its logits are
//     l_j = q . k_j / sqrt(d) + e_j   (e_j = -inf masks token j),
// out = sum_j softmax(l)_j v_j, lse = log sum_j exp(l_j), and the weights' sum over
// the rows and the tokens of a block goes to the block's accumulated weight.
//
// The cache is read once, so HBM bounds a call with few rows. Three launches:
//   stream  : the full blocks of all units, one after another, are one list of items
//             that one wave of CTAs (one per SM) shares equally: units differ in
//             length, so the shares are cut from the lengths on the device. A producer
//             warp keeps a ring of whole units in flight with bulk copies; the consumer
//             warps take the units in turn, each with a running maximum, sum and
//             output of its own. A warp that has a whole block to itself pays its
//             reductions and the output's rescaling once per 64 tokens and has four
//             independent chains of products. Where the CTA leaves a unit the warps
//             leave their parts to a helper warp, which joins them and has the next
//             unit's queries ready, and go on.
//   combine : a CTA per unit and 8 rows attends to the tail in fp32 while the stream
//             still runs, then joins the unit's parts.
//   weights : with accumulated weights, what the stream noted for each block is added
//             up relative to the rows' final sums: by the join where one CTA has all
//             rows of a unit (up to 8) and the table is short, else by a launch of its own.
//
// The products take the tensor cores' 16 x 8 x 16 shape with the codes as the large
// operand (tokens x dims, dims x tokens) and the rows as the small one: up to 8 rows
// (the query heads of a KV head) waste nothing, and the weights of a slice reach the
// second product with two 8 x 8 transposes. An e4m3 code is exact in fp16. Queries are
// brought to a largest magnitude in [2^14, 2^15) by a power of two per row, the top of
// fp16's range, so that an outlier takes no bits from the others: a bf16 element is exact
// down to 2^-31 of the row's largest, an fp32 one the sum of two fp16 terms (22 bits), and
// what is lost otherwise is at most 2^-39 of the largest. Weights are held in
// fp32 for the sums and rounded to fp16 (fp32 output: two terms) for the second
// product, scaled by 2^14 so that weights down to 2^-28 of the largest keep their 11
// bits. Each block's product starts from zero and enters the fp32 output with the
// block's value scale, so neither scale ever multiplies an operand.
//
// Measured on GB300 (bytes that the call cannot do without / time, of the measured copy
// rate of 6793 GB/s):
//   256 units x 65536 tokens, d = 128, 4 rows, weights   4.37 GB   668 us   96 %
//   128 units x 1 .. 32768 tokens, 3 rows, weights        0.58 GB   100 us   85 %
//   8 units x 131071 tokens, 4 rows                       0.27 GB    50 us   81 %
//   64 units x 16384 tokens, d = 64, 2 rows               0.14 GB    30 us   69 %
//   1 unit x 2031 tokens, d = 64, fp32                    0.3 MB    8.1 us
// The stream itself runs at the copy rate; what is left is fixed: 3.75 us until the
// first unit has landed (lengths, table, unit: three dependent reads), about 4 us between
// the first and the last CTA to end, 1.5 us for the last join inside a CTA, 3 us for the
// join launch after it and 2.5 us for the weights'. With 32 rows (8 drafted tokens of
// 4 heads, 32 units of 8200 tokens: 41 us; 128 rows over 16 units of 16384 tokens: 98 us)
// the products' instructions bound it: about 1300 of a warp and block at 1.7 a cycle, six
// consumer warps being all that the outputs' registers leave room for.
#pragma once

#include "k_quant.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

namespace nosa {

constexpr int kQaMinItems = 2;    // blocks of a CTA's share, at least
constexpr int kQcThreads = 256;   // combine
constexpr int kQcScan = 4;        // lengths of a thread, where the combine adds them up
constexpr float kQLog2e = 1.4426950408889634f;

struct QStreamParams {
  const uint8_t* units;
  long long n_units;
  const int32_t* tab;
  int max_blocks;
  const int32_t* lens;
  const void* q;
  QStrides qs;
  int T;
  const int32_t* q_len;
  int U, Hkv, Hq, G, tiles;
  const uint8_t* tail;
  long long payload;
  void* out;
  float* lse;
  float* mass;
  float decay;
  int* status;
  int ctas;  // CTAs of the stream
  bool give_up;  // every wait gives up at once (a test's)
  // workspace
  long long* total;   // items of the call
  long long* base;    // [units] full blocks of the units before, where there are many units
  float2* part_ml;    // [ctas + units x tiles][rows] maximum and sum of a part (or qa_missing)
  float* part_acc;    // ... [rows][d] its output (not normalised)
  float2* rowstat;    // [units x tiles][rows] final maximum and 1 / sum (-1: parts are missing)
  float* tail_w;      // [units x tiles][rows] weight of the tail
  float2* blk;        // [units x tiles][max_blocks][rows] maximum and sum of a block, or null (no weights asked for)
};

// 1 / sqrt(d)
template <int D> constexpr float kQScale = D == 64 ? 0.125f : 0.08838834764831845f;

#ifdef __CUDACC__

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }
// exp(x - m) for the base-2 exponential; x = -inf gives 0 for every finite m.
__device__ __forceinline__ float exp_from(float x, float m) { return exp2f((x - m) * kQLog2e); }

__device__ __forceinline__ float ex2(float x) {  // results below 2^-126 are 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 f32x2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether a phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A part that is missing, because a wait gave up: whatever it is joined with, the sum of the
// row is -infinity, which no other sum is.
__device__ __forceinline__ float2 qa_missing() { return make_float2(3.402823466e38f, -INFINITY); }

// CTAs that share `total` items, and the CTA that holds item x.
__device__ __forceinline__ int qa_active(long long total, int ctas) {
  const long long want = (total + kQaMinItems - 1) / kQaMinItems;
  return (int)(want < ctas ? want : ctas);
}
__device__ __forceinline__ int qa_cta_of(long long x, long long total, int active) {
  return (int)(((x + 1) * active - 1) / total);
}

// What row r of a tile is: its query (request, token, head), and the tokens it sees.
struct QRow {
  int t, g, sees;  // sees = 0 for a row that does not exist
};
__device__ __forceinline__ QRow qa_row(int r, int G, int n, int qn) {
  QRow w;
  w.t = r / G;
  w.g = r % G;
  w.sees = w.t < qn ? max(0, n - qn + w.t + 1) : 0;
  return w;
}

// Shape of a stream CTA. A warp has 8 NT rows; RG warps share a unit, each with its own
// rows, and IS units are worked on at once. Item i of the CTA goes to the warps of slot
// i % IS and to stage i % STAGES, and STAGES is a multiple of IS: a stage always has the
// same readers. Copies may land out of order, and a barrier's parity tells a phase only
// from its neighbours, so a warp may wait for a stage's next fill only after it has seen
// the fill before.
template <int D, int NT, int RG, bool F32>
struct QGeom {
  static constexpr int ROWS = 8 * NT * RG, KS = D / 16, UB = quant_unit_bytes(D);
  // Eight warps in all leave each one 255 registers, which 16 rows of output need; more
  // leave 168. Slots and ring for 8 rows, d = 128, measured at 256 units x 65536 tokens, us:
  // 4 slots and 8 stages 677, 3 and 9 671, 5 and 10 694, 3 and 6 721, 6 and 6 745, 2 and 8
  // 907 (two warps cannot keep up); the first leaves shared memory for the join's CTAs to
  // wait on the same SMs. d = 64 (64 units x 16384), 8 and 16 33.6, 4 and 16 33.9, 8 and 8 41.
  static constexpr int IS = NT == 2 ? 6 / RG : RG > 1 ? 8 / RG : D == 128 ? 4 : 8;
  static constexpr int W = IS * RG;             // consumer warps; a producer and a helper come on top
  static constexpr int THREADS = 32 * (W + 2);
  // What the compiler is told of the threads: 480 hold it to 136 registers, so that the join fits
  // beside the stream (kQcPerSm). fp32 takes the 144 that it may.
  static constexpr int BOUND = D == 64 && ROWS == 8 && !F32 ? 480 : THREADS;
  static constexpr int STAGES = D == 64 ? (NT == 1 ? 16 : 12) : NT == 1 ? 8 : 9;
  static constexpr int SL = 4;                  // slices of a block that a warp takes at once
  static constexpr int NQ = 2, ND = NT * RG == 1 ? 2 : 1;  // buffers for queries and for the warps' parts
  static constexpr int RP = D + 4;              // padded row of a part
  static constexpr int Q_BYTES = NT * RG * KS * 32 * (F32 ? 16 : 8);
  static constexpr int RED_BYTES = W * 8 * NT * RP * 4, ML_BYTES = W * 8 * NT * 8;
  static constexpr int Q_OFF = STAGES * UB;
  static constexpr int RED_OFF = Q_OFF + NQ * Q_BYTES;
  static constexpr int ML_OFF = RED_OFF + ND * RED_BYTES;
  static constexpr int ROW_OFF = ML_OFF + ND * ML_BYTES;
  static constexpr int NULL_OFF = ROW_OFF + NQ * ROWS * 8;
  static constexpr int BAR_OFF = NULL_OFF + (STAGES * 4 + 7) / 8 * 8;
  static constexpr int SMEM = BAR_OFF + (2 * STAGES + NQ + 2 * ND) * 8;
  static_assert(STAGES % IS == 0 && STAGES <= 32, "a stage has one slot and one producer lane");
  static_assert(UB % 16 == 0 && Q_OFF % 16 == 0 && RED_OFF % 16 == 0 && BAR_OFF % 8 == 0, "alignment");
  static_assert(SMEM <= 227 * 1024 - 256, "shared memory");
};

// A CTA's share as segments: consecutive blocks of one (unit, tile).
struct QWalk {
  const QStreamParams& p;
  int u, tile, j0, cnt, left, lane, have, len, tokens;
  // from the unit that holds the first item, `at` items into it, `left` items to go
  __device__ __forceinline__ QWalk(const QStreamParams& p_, int u_, long long at, int left_, int lane_)
      : p(p_), u(u_), cnt(0), left(left_), lane(lane_), have(-1), len(0), tokens(0) {
    tokens = fetch();
    const int nb = tokens / kQB;
    tile = (int)(at / nb);
    j0 = (int)(at % nb);
    cnt = min(nb - j0, left);
  }
  __device__ __forceinline__ int fetch() {  // tokens of unit u; 32 lengths at a time (whole warp)
    if (have < 0 || u >= have + 32) {
      have = u;
      len = u + lane < p.U ? max(0, quant_len(p.lens, u + lane, p.max_blocks, nullptr, false)) : 0;
    }
    return __shfl_sync(0xffffffffu, len, u - have);
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next() {
    left -= cnt;
    if (left <= 0) return;
    j0 = 0;
    if (++tile == p.tiles) {
      tile = 0;
      do {
        ++u;
        tokens = fetch();
      } while (tokens < kQB);
    }
    cnt = min(tokens / kQB, left);
  }
  __device__ __forceinline__ long long vu() const { return (long long)u * p.tiles + tile; }
};

// Queries of GROUPS x 8 rows (whole warp) as B operands, and the rows' factors; all
// loads come first, so that they cost one round trip.
template <int D, int GROUPS, bool F32>
__device__ __forceinline__ void qa_queries(const QStreamParams& p, int u, int row0, int n, int qn, uint8_t* q_s, float* rs_s,
                                           int* vis_s, int lane) {
  constexpr int KS = D / 16;
  using Raw = typename std::conditional<F32, uint4, uint2>::type;  // four elements
  const int g = lane >> 2, c = lane & 3, b = u / p.Hkv, h = u % p.Hkv;
  Raw raw[GROUPS][KS];
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    const QRow w = qa_row(row0 + 8 * i + g, p.G, n, qn);
    const long long src = b * p.qs.b + w.t * p.qs.t + (h * p.G + w.g) * p.qs.h + 4 * c;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      raw[i][k] = Raw{};
      // (not the read-only path: the kernel may be resident while its predecessor writes q)
      if (w.t < qn) raw[i][k] = *reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(p.q) + (src + 16 * k) * (F32 ? 4 : 2));
    }
  }
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    float f[KS][4];
    float mx = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const Raw x = raw[i][k];
      if constexpr (F32) {
        f[k][0] = __uint_as_float(x.x); f[k][1] = __uint_as_float(x.y);
        f[k][2] = __uint_as_float(x.z); f[k][3] = __uint_as_float(x.w);
      } else {
        f[k][0] = bf16_lo(x.x); f[k][1] = bf16_hi(x.x); f[k][2] = bf16_lo(x.y); f[k][3] = bf16_hi(x.y);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) mx = fmaxf(mx, fabsf(f[k][y]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // 2^(ex - 127) <= mx < 2^(ex - 126), kept where both powers below are normal numbers
    const uint32_t ex = min(max(__float_as_uint(mx) >> 23, 15u), 254u);
    const float down = __uint_as_float((268 - ex) << 23), up = __uint_as_float((ex - 14) << 23);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const float x0 = f[k][0] * down, x1 = f[k][1] * down, x2 = f[k][2] * down, x3 = f[k][3] * down;
      const uint32_t h0 = f16x2(x0, x1), h1 = f16x2(x2, x3);
      if constexpr (F32) {
        const float2 y0 = f32x2(h0), y1 = f32x2(h1);
        reinterpret_cast<uint4*>(q_s)[(i * KS + k) * 32 + lane] =
            make_uint4(h0, h1, f16x2(x0 - y0.x, x1 - y0.y), f16x2(x2 - y1.x, x3 - y1.y));
      } else {
        reinterpret_cast<uint2*>(q_s)[(i * KS + k) * 32 + lane] = make_uint2(h0, h1);
      }
    }
    if (c == 0) {
      rs_s[8 * i + g] = up;
      vis_s[8 * i + g] = qa_row(row0 + 8 * i + g, p.G, n, qn).sees;
    }
  }
}

// A warp's part of a segment once more, token by token in fp32, where it came out as NaN: the
// products take a masked token's value times a weight of 0, which is not 0 where the code is
// no number (0x7F, 0xFF). Here only the tokens that a row sees are looked at, and what stays
// NaN is the row's due. Blocks j0, j0 + IS, ... before j1 of unit u, rows first .. first + WR
// of the request, their parts red [WR][RP] and ml [WR] (whole warp; about 3.5 us a row and block).
// The products pay nothing for this. Clearing the codes of masked tokens on the way, with a
// mask per word, was measured: 256 units x 65536 tokens 674 us (668 without), 32 rows 41.3
// (40.0), 128 rows 101 (97.5), fp32 32 rows 74.0 (69.3).
template <int D, int WR, int RP, int IS, bool F32>
__device__ __noinline__ void qa_part_again(const QStreamParams& p, int u, int j0, int j1, int first, float* red, const float2* ml) {
  using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
  constexpr int DL = D / 32;  // dims of a lane
  const int b = u / p.Hkv, h = u % p.Hkv, lane = threadIdx.x & 31;
  const int n = max(0, quant_len(p.lens, u, p.max_blocks, nullptr, false)), qn = quant_count(p.q_len, b, p.T, nullptr, false);
  auto block = [&](int j) -> const uint8_t* {  // null: the table names no unit
    const int idx = p.tab[(long long)u * p.max_blocks + j];
    return idx < 0 || (long long)idx >= p.n_units ? nullptr : p.units + (long long)idx * quant_unit_bytes(D);
  };
#pragma unroll 1
  for (int r = 0; r < WR; ++r) {
    const QRow w = qa_row(first + r, p.G, n, qn);
    const float mu = finite_max(ml[r].x);
    if (w.sees == 0 || isnan(mu)) continue;
    bool due = false;  // a scale is NaN, and the row sees a token of its block
#pragma unroll 1
    for (int j = j0 + lane * IS; j < j1; j += 32 * IS) {
      const uint8_t* unit = block(j);
      if (unit == nullptr) continue;
      const float* es = reinterpret_cast<const float*>(unit + quant_e_off(D));
      if (!isnan(es[kQB + 1])) continue;
#pragma unroll 1
      for (int t = 0; t < kQB; ++t) due |= es[t] != -INFINITY && j * kQB + t < w.sees;
    }
    if (__any_sync(0xffffffffu, due)) continue;
    const T* q = static_cast<const T*>(p.q) + b * p.qs.b + w.t * p.qs.t + (h * p.G + w.g) * p.qs.h;
    float acc[DL] = {};
#pragma unroll 1
    for (int j = j0; j < j1; j += IS) {
      const uint8_t* unit = block(j);
      if (unit == nullptr) continue;
      const float* es = reinterpret_cast<const float*>(unit + quant_e_off(D));
      float wt[2];  // the lane's tokens lane and lane + 32; -1: masked or not seen
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int t = lane + 32 * y;
        float l = 0.f;
#pragma unroll 8
        for (int x = 0; x < D; x += 4) {
          const uint32_t k = *reinterpret_cast<const uint32_t*>(unit + quant_k_off(t, x, D));
          const float2 k0 = f32x2(e4m3x2_f16x2(k)), k1 = f32x2(e4m3x2_f16x2(k >> 16));
          l += to_f32(q[x]) * k0.x + to_f32(q[x + 1]) * k0.y + to_f32(q[x + 2]) * k1.x + to_f32(q[x + 3]) * k1.y;
        }
        wt[y] = es[t] == -INFINITY || j * kQB + t >= w.sees ? -1.f : exp_from(l * kQScale<D> * es[kQB] + es[t], mu);
      }
      float sum[DL] = {};
      bool any = false;
#pragma unroll 4
      for (int t = 0; t < kQB; t += 4) {  // a word has four tokens of a dim
        float v[DL][4];
#pragma unroll
        for (int x = 0; x < DL; ++x) {
          const uint32_t k = *reinterpret_cast<const uint32_t*>(unit + quant_v_off(t, lane * DL + x, D));
          const float2 v0 = f32x2(e4m3x2_f16x2(k)), v1 = f32x2(e4m3x2_f16x2(k >> 16));
          v[x][0] = v0.x; v[x][1] = v0.y; v[x][2] = v1.x; v[x][3] = v1.y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = __shfl_sync(0xffffffffu, t < 32 ? wt[0] : wt[1], (t + i) & 31);
          if (y < 0.f) continue;  // (the same for the warp)
          any = true;
#pragma unroll
          for (int x = 0; x < DL; ++x) sum[x] += y * v[x][i];
        }
      }
      if (!any) continue;
#pragma unroll
      for (int x = 0; x < DL; ++x) acc[x] += sum[x] * es[kQB + 1];
    }
#pragma unroll
    for (int x = 0; x < DL; ++x) {
      float& y = red[r * RP + lane * DL + x];
      if (isnan(y)) y = acc[x];
    }
  }
}

// First items of a thread's units, where the join does not add them up itself (out of line: 32 rows
// over 32 units of 8200 tokens 40.7 us, with the loop in the kernel 41.1).
static __device__ __noinline__ void qa_places(const QStreamParams& p, int a0, int a1, long long at) {
  for (int u = a0; u < a1; ++u) {
    p.base[u] = at;
    at += max(0, quant_len(p.lens, u, p.max_blocks, nullptr, false)) / kQB;
  }
}

template <int D, int NT, int RG, bool F32>
__global__ void __launch_bounds__(QGeom<D, NT, RG, F32>::BOUND, 1) quant_stream_kernel(QStreamParams p) {
  using Gm = QGeom<D, NT, RG, F32>;
  constexpr int KS = Gm::KS, ROWS = Gm::ROWS, STAGES = Gm::STAGES, UB = Gm::UB, SL = Gm::SL, W = Gm::W, IS = Gm::IS;
  constexpr int NQ = Gm::NQ, ND = Gm::ND, WR = 8 * NT, kThreads = Gm::THREADS;
  extern __shared__ __align__(128) uint8_t smem[];
  int* null_s = reinterpret_cast<int*>(smem + Gm::NULL_OFF);  // [STAGES] the table names no unit
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Gm::BAR_OFF);
  uint64_t* empty = full + STAGES;
  uint64_t* q_full = empty + STAGES;    // [NQ] queries of a segment are there
  uint64_t* dump_full = q_full + NQ;    // [ND] the warps' parts of a segment are there
  uint64_t* dump_free = dump_full + ND;
  // per buffer: queries, factors of the rows' logits, tokens they see, parts
  auto q_of = [&](int k) { return smem + Gm::Q_OFF + (k % NQ) * Gm::Q_BYTES; };
  auto rs_of = [&](int k) { return reinterpret_cast<float*>(smem + Gm::ROW_OFF) + (k % NQ) * 2 * ROWS; };
  auto vis_of = [&](int k) { return reinterpret_cast<int*>(rs_of(k) + ROWS); };
  auto red_of = [&](int k) { return reinterpret_cast<float*>(smem + Gm::RED_OFF + (k % ND) * Gm::RED_BYTES); };  // [W][WR][RP]
  auto ml_of = [&](int k) { return reinterpret_cast<float2*>(smem + Gm::ML_OFF + (k % ND) * Gm::ML_BYTES); };    // [W][WR]
  __shared__ long long s_scan[kThreads / 32];
  __shared__ long long s_before;
  __shared__ int s_unit;
  __shared__ volatile int s_bad;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], RG);
    }
    for (int s = 0; s < NQ; ++s) mbar_init(&q_full[s], 1);
    for (int s = 0; s < ND; ++s) {
      mbar_init(&dump_full[s], W);
      mbar_init(&dump_free[s], 1);
    }
    fence_mbar_init();
    s_bad = p.give_up;
  }
  griddep_wait();
  griddep_launch_dependents();
  // ---- the share: prefix sums of the units' full blocks ----
  const int per = (p.U + kThreads - 1) / kThreads;
  const int a0 = min(p.U, tid * per), a1 = min(p.U, a0 + per);
  long long mine = 0;
  for (int u = a0; u < a1; ++u) mine += max(0, quant_len(p.lens, u, p.max_blocks, p.status, cta == 0)) / kQB;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  long long total = 0, before = inc - mine;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  if (p.U > kQcScan * kQcThreads && tid % p.ctas == cta) qa_places(p, a0, a1, before);  // (a thread's by one of the CTAs)
  total *= p.tiles;
  before *= p.tiles;
  if (cta == 0 && tid == 0) *p.total = total;
  const int active = qa_active(total, p.ctas);
  if (cta >= active) return;  // (the whole CTA)
  const long long g0 = (long long)cta * total / active, g1 = (long long)(cta + 1) * total / active;
  if (before <= g0 && g0 < before + mine * p.tiles) {  // exactly one thread: the unit that holds item g0
    int u = a0;
    for (;; ++u) {
      const long long n = (long long)max(0, quant_len(p.lens, u, p.max_blocks, nullptr, false)) / kQB * p.tiles;
      if (g0 < before + n) break;
      before += n;
    }
    s_unit = u;
    s_before = before;
  }
  __syncthreads();
  const int items = (int)(g1 - g0);
  bool ok = true;  // no wait has given up
  // Waits (whole warp) for a phase, with a limit, unless another warp has given up.
  auto wait = [&](uint64_t* bar, int phase) {
    return __all_sync(0xffffffffu, s_bad == 0 && mbar_wait_bounded(bar, (uint32_t)(phase & 1)));
  };
  auto give_up = [&]() {  // (one lane)
    s_bad = 1;
    quant_flag(p.status, kQErrWait);
  };

  // Whether the consumers join their last segment's rows with the helper. Measured on
  // GB300, us (helper alone): d = 64, 1 unit x 2031 tokens in fp32 8.3 (9.0), 64 units x 16384
  // 29.9 (30.6), 32 rows 36 (37.5); d = 128, 32 rows over 32 units of 8200 42.2 (40.0): there
  // the join's registers disturb the main loop.
  constexpr bool kShareJoin = D == 64;
  // Rows first, first + step, ... of segment k: the warps' parts become the CTA's, in slot `to`.
  auto join_rows = [&](int k, long long to, int first, int step) {
    const float* red = red_of(k);
    const float2* ml = ml_of(k);
#pragma unroll 4
    for (int r = first; r < ROWS; r += step) {
      const int w0 = r / WR * IS, rr = r % WR;  // the warps of this row, and their row
      float M = ml[w0 * WR + rr].x;
#pragma unroll
      for (int w = 1; w < IS; ++w) M = max_nan(M, ml[(w0 + w) * WR + rr].x);
      const float mu = finite_max(M);
      float wt[IS], L = 0.f;
#pragma unroll
      for (int w = 0; w < IS; ++w) {
        const float2 y = ml[(w0 + w) * WR + rr];
        wt[w] = exp_from(y.x, mu);
        L += wt[w] * y.y;
      }
      if (lane < D / 4) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < IS; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(red + ((w0 + w) * WR + rr) * Gm::RP + 4 * lane);
          acc.x += wt[w] * y.x; acc.y += wt[w] * y.y; acc.z += wt[w] * y.z; acc.w += wt[w] * y.w;
        }
        reinterpret_cast<float4*>(p.part_acc + (to * ROWS + r) * D)[lane] = acc;
      }
      if (lane == 0) p.part_ml[to * ROWS + r] = make_float2(M, L);
    }
  };

  if (warp == W) {
    // ---- producer: lane s owns stage s and brings it items s, s + STAGES, ... ----
    int it = lane, u = s_unit, tile = 0, j = 0, nb = 0, idx = -1;
    long long pos = g0 - s_before + it;  // from the start of unit u
    auto seek = [&]() {                  // (u, tile, j) of the item, and its table entry
      if (it >= items) return;
      for (;;) {
        nb = max(0, quant_len(p.lens, u, p.max_blocks, nullptr, false)) / kQB;
        if (pos < (long long)nb * p.tiles) break;
        pos -= (long long)nb * p.tiles;
        ++u;
      }
      tile = (int)pos / nb;
      j = (int)pos - tile * nb;
      idx = p.tab[(long long)u * p.max_blocks + j];
    };
    if (lane >= STAGES) it = items;
    seek();
    int fills = 0;
    uint64_t since = global_ns();
    for (int spin = 0; __any_sync(0xffffffffu, it < items); ++spin) {
      bool moved = false;
      if (it < items && (fills == 0 || mbar_test(&empty[lane], (uint32_t)((fills - 1) & 1)))) {
        const bool bad = idx < 0 || (long long)idx >= p.n_units;
        null_s[lane] = bad;
        if (bad) {
          quant_flag(p.status, kQErrIndex);
          mbar_arrive(&full[lane]);
        } else {
          mbar_arrive_expect_tx(&full[lane], UB);
          bulk_g2s(smem + lane * UB, p.units + (long long)idx * UB, UB, &full[lane]);
        }
        ++fills;
        it += STAGES;
        pos += STAGES;
        seek();
        moved = true;
      }
      if (!__any_sync(0xffffffffu, moved)) __nanosleep(40);  // (leaves the issue slots to the others)
      if (__any_sync(0xffffffffu, moved)) {
        spin = 0;
        since = global_ns();
      } else if ((spin & 63) == 63 && (s_bad != 0 || global_ns() - since > 2000000000ull)) {
        ok = false;
      }
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
    }
    if (!ok && lane == 0) give_up();
    __syncthreads();
    if (s_bad != 0 && fills > 0) mbar_wait_bounded(&full[lane], (uint32_t)((fills - 1) & 1));  // drain
    return;
  }

  if (warp == W + 1) {
    // ---- helper: prepares the queries of coming segments, joins the warps' parts ----
    QWalk ahead(p, s_unit, g0 - s_before, items, lane);
    long long slot[NQ];
    int prepared = 0;
    auto prepare = [&]() {
      const int b = ahead.u / p.Hkv, qn = quant_count(p.q_len, b, p.T, p.status, lane == 0);
      constexpr int GR = F32 ? 1 : ROWS / 8;  // row groups at once: 32 rows of bf16 take 64 registers
#pragma unroll 1
      for (int r = 0; r < ROWS; r += 8 * GR)
        qa_queries<D, GR, F32>(p, ahead.u, ahead.tile * ROWS + r, ahead.tokens, qn, q_of(prepared) + r * KS * 4 * (F32 ? 16 : 8),
                               rs_of(prepared) + r, vis_of(prepared) + r, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[prepared % NQ]);
#pragma unroll
      for (int x = 0; x < NQ; ++x)
        if (x == prepared % NQ) slot[x] = cta + ahead.vu();
      ++prepared;
      ahead.next();
    };
    for (int x = 0; x < NQ && ahead.more(); ++x) prepare();
    for (int k = 0; k < prepared && ok; ++k) {
      if (!(ok = wait(&dump_full[k % ND], k / ND))) break;
      long long to = slot[0];
#pragma unroll
      for (int x = 1; x < NQ; ++x)
        if (x == k % NQ) to = slot[x];
      // (the last segment's consumers have nothing else to do and take most of its rows)
      const bool last = kShareJoin && k == prepared - 1 && !ahead.more();
      join_rows(k, to, last ? W : 0, last ? W + 1 : 1);
      __syncwarp();
      if (lane == 0) mbar_arrive(&dump_free[k % ND]);
      if (ahead.more()) prepare();  // (every warp has left segment k, whose queries were in this buffer)
    }
    if (!ok && lane == 0) give_up();
    __syncthreads();
    if (s_bad != 0) {  // none of the CTA's parts counts
      for (QWalk all(p, s_unit, g0 - s_before, items, lane); all.more(); all.next())
        if (lane < ROWS) p.part_ml[(cta + all.vu()) * ROWS + lane] = qa_missing();
    }
    return;
  }

  // ---- consumers ----
  const int g = lane >> 2, c = lane & 3;
  const int tok = 4 * (g >> 1) + (g & 1);  // this lane's tokens of a slice: tok and tok + 2
  const int is = warp % IS, rg = warp / IS;
  QWalk seg(p, s_unit, g0 - s_before, items, lane);
  int it0 = 0;  // first item of the segment
  for (int k = 0; seg.more(); ++k, it0 += seg.cnt, seg.next()) {
    if (!(ok = wait(&q_full[k % NQ], k / NQ))) break;
    const long long vu = seg.vu();
    const uint8_t* q_s = q_of(k) + rg * NT * KS * 32 * (F32 ? 16 : 8);
    const float* rs_s = rs_of(k) + rg * WR;
    const int* vis_s = vis_of(k) + rg * WR;
    float o[NT][KS][4], m_run[NT][2], l_run[NT][2], fac[1][2];
    int vis[1][2];  // (of more than 8 rows these two stay in shared memory)
    uint32_t qr[NT == 1 && !F32 ? KS : 1][2];
    int least = 0x7fffffff;  // tokens that all of this lane's rows see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (NT == 1) {
          fac[0][x] = rs_s[2 * c + x];
          vis[0][x] = vis_s[2 * c + x];
        }
        least = min(least, vis_s[nt * 8 + 2 * c + x]);
        m_run[nt][x] = -INFINITY;
        l_run[nt][x] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
    }
    if constexpr (NT == 1 && !F32) {
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const uint2 y = reinterpret_cast<const uint2*>(q_s)[x * 32 + lane];
        qr[x][0] = y.x;
        qr[x][1] = y.y;
      }
    }

    for (int it = it0 + (is + IS - it0 % IS) % IS; it < it0 + seg.cnt; it += IS) {
      const int s = it % STAGES, j = seg.j0 + it - it0;
      if (!(ok = wait(&full[s], it / STAGES))) break;
      const bool null_unit = null_s[s] != 0;
      const uint8_t* unit = smem + s * UB;
      const float* es = reinterpret_cast<const float*>(unit + quant_e_off(D));
      const float ks = es[kQB], vs = es[kQB + 1] * 0x1p-14f;
      const bool edge = j * kQB + kQB > least;
      float blk_l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) blk_l[nt][0] = blk_l[nt][1] = 0.f;
#pragma unroll
      for (int s0 = 0; s0 < 4; s0 += SL) {
        if (null_unit) break;
        const uint4* kw = reinterpret_cast<const uint4*>(unit) + s0 * 2 * D + lane;
        // ---- logits ----
        float sc[NT][SL][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int w = 0; w < SL; ++w) sc[nt][w][0] = sc[nt][w][1] = sc[nt][w][2] = sc[nt][w][3] = 0.f;
#pragma unroll
        for (int jj = 0; jj < KS / 2; ++jj) {
          uint4 v[SL];
#pragma unroll
          for (int w = 0; w < SL; ++w) v[w] = kw[w * 2 * D + jj * 32];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int kk = 2 * jj + y;
            uint32_t qb[NT][F32 ? 4 : 2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (F32) {
                const uint4 x = reinterpret_cast<const uint4*>(q_s)[(nt * KS + kk) * 32 + lane];
                qb[nt][0] = x.x; qb[nt][1] = x.y; qb[nt][2] = x.z; qb[nt][3] = x.w;
              } else if constexpr (NT == 1) {
                qb[nt][0] = qr[kk][0];
                qb[nt][1] = qr[kk][1];
              } else {
                const uint2 x = reinterpret_cast<const uint2*>(q_s)[(nt * KS + kk) * 32 + lane];
                qb[nt][0] = x.x;
                qb[nt][1] = x.y;
              }
            }
#pragma unroll
            for (int w = 0; w < SL; ++w) {
              const uint32_t w0 = y ? v[w].z : v[w].x, w1 = y ? v[w].w : v[w].y;
              const uint32_t a[4] = {e4m3x2_f16x2(w0), e4m3x2_f16x2(w1), e4m3x2_f16x2(w0 >> 16), e4m3x2_f16x2(w1 >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if constexpr (F32) mma16816(sc[nt][w], a, qb[nt][2], qb[nt][3]);
                mma16816(sc[nt][w], a, qb[nt][0], qb[nt][1]);
              }
            }
          }
        }
        // ---- softmax over the 16 SL tokens ----
        // (Warp-wide branches around the masks or the rescaling, and packed pairs, were all
        // slower: they keep the next products' loads from moving up. 256 units x 65536
        // tokens, us: as it is 669, masks behind a branch 675, packed 723.)
        float ev[SL][2];
#pragma unroll
        for (int w = 0; w < SL; ++w) {
          ev[w][0] = es[16 * (s0 + w) + tok];
          ev[w][1] = es[16 * (s0 + w) + tok + 2];
        }
        const int pos = j * kQB + 16 * s0 + tok;
        float corr[NT][2], vsc[NT][2];
        uint32_t pb[NT][SL][2], pl[F32 ? NT : 1][SL][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float f = (NT == 1 ? fac[0][x] : rs_s[nt * 8 + 2 * c + x]) * ks * kQScale<D>;  // (the power of two first)
            const int sees = NT == 1 ? vis[0][x] : vis_s[nt * 8 + 2 * c + x];
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < SL; ++w)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float& l = sc[nt][w][2 * y + x];
                l = l * f + ev[w][y];
                if (ev[w][y] == -INFINITY || (edge && pos + 16 * w + 2 * y >= sees)) l = -INFINITY;
                mx = max_nan(mx, l);
              }
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = max_nan(m_run[nt][x], mx), mu = finite_max(mn);
            corr[nt][x] = exp_from(m_run[nt][x], mu);
            vsc[nt][x] = mx == -INFINITY ? 0.f : vs;  // (nothing visible: whatever the scale)
            m_run[nt][x] = mn;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < SL; ++w)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float& l = sc[nt][w][2 * y + x];
                // times 2^14: for bf16 in the exponent, which costs 2^-21.5 of a weight
                if constexpr (F32) {
                  l = ex2((l - mu) * kQLog2e) * 16384.f;
                } else {
                  l = ex2(fmaf(l - mu, kQLog2e, 14.f));
                }
                sum += l;
              }
            l_run[nt][x] = l_run[nt][x] * corr[nt][x] + sum;
            blk_l[nt][x] = blk_l[nt][x] * corr[nt][x] + sum;
          }
#pragma unroll
          for (int w = 0; w < SL; ++w)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float x0 = sc[nt][w][2 * y], x1 = sc[nt][w][2 * y + 1];
              const uint32_t hh = f16x2(x0, x1);
              pb[nt][w][y] = transpose8x8(hh);
              if constexpr (F32) {
                const float2 r = f32x2(hh);
                pl[nt][w][y] = transpose8x8(f16x2(x0 - r.x, x1 - r.y));
              }
            }
        }
        // ---- o = o * corr + scale * (V^T P) ----
        const uint4* vw = kw + D;  // 16 D bytes on
#pragma unroll
        for (int jj = 0; jj < KS / 2; ++jj) {
          uint4 v[SL];
#pragma unroll
          for (int w = 0; w < SL; ++w) v[w] = vw[w * 2 * D + jj * 32];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float t[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) t[nt][0] = t[nt][1] = t[nt][2] = t[nt][3] = 0.f;
#pragma unroll
            for (int w = 0; w < SL; ++w) {
              const uint32_t w0 = y ? v[w].z : v[w].x, w1 = y ? v[w].w : v[w].y;
              const uint32_t a[4] = {e4m3x2_f16x2(w0), e4m3x2_f16x2(w1), e4m3x2_f16x2(w0 >> 16), e4m3x2_f16x2(w1 >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if constexpr (F32) mma16816(t[nt], a, pl[nt][w][0], pl[nt][w][1]);
                mma16816(t[nt], a, pb[nt][w][0], pb[nt][w][1]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                float& oo = o[nt][2 * jj + y][x];
                oo = oo * corr[nt][x & 1] + t[nt][x] * vsc[nt][x & 1];
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (p.blk != nullptr) {  // the block's sums, for the accumulated weights
        float2* note = p.blk + (vu * p.max_blocks + j) * ROWS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float t[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            t[x] = blk_l[nt][x];
            t[x] += __shfl_xor_sync(0xffffffffu, t[x], 4);
            t[x] += __shfl_xor_sync(0xffffffffu, t[x], 8);
            t[x] += __shfl_xor_sync(0xffffffffu, t[x], 16);
            t[x] *= 0x1p-14f;
          }
          const int r = rg * WR + nt * 8 + 2 * c;
          if (g == 0 && seg.tile * ROWS + r < p.T * p.G)
            *reinterpret_cast<float4*>(note + r) = make_float4(m_run[nt][0], t[0], m_run[nt][1], t[1]);
        }
      }
    }
    // ---- the warp's part of the segment goes to the helper ----
    if (ok && k >= ND) ok = wait(&dump_free[k % ND], k / ND - 1);
    if (!ok) break;
    float* red = red_of(k) + warp * WR * Gm::RP;
    float2* ml = ml_of(k) + warp * WR;
    float nan = 0.f;  // NaN where an output is
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float l = l_run[nt][x];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        l *= 0x1p-14f;
        if (g == 0) ml[nt * 8 + 2 * c + x] = make_float2(m_run[nt][x], l);
      }
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          red[(nt * 8 + 2 * c + (x & 1)) * Gm::RP + mt * 16 + g + 8 * (x >> 1)] = o[nt][mt][x];
          nan += o[nt][mt][x] * 0.f;
        }
    }
    __syncwarp();
    if (__any_sync(0xffffffffu, isnan(nan)))
      qa_part_again<D, WR, Gm::RP, IS, F32>(p, seg.u, seg.j0 + (is + IS - it0 % IS) % IS, seg.j0 + seg.cnt, seg.tile * ROWS + rg * WR, red, ml);
    __syncwarp();
    if (lane == 0) mbar_arrive(&dump_full[k % ND]);
    if (kShareJoin && seg.left == seg.cnt) {  // the last segment (its buffer's earlier fills have been joined)
      if (!(ok = wait(&dump_full[k % ND], k / ND))) break;
      join_rows(k, cta + vu, warp, W + 1);
    }
  }
  if (!ok && lane == 0) give_up();
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Tail attention and the join. Grid (units x tiles, row groups of 8, z): a CTA writes
// d / z dims of 8 rows. Before the stream has finished: the tail in fp32, its keys and
// values in registers. After: every thread merges its share
// of the unit's parts for four dims of a row, the shares join in shared memory.
// ---------------------------------------------------------------------------
constexpr int kQcRows = 8;
// The CTA has to fit beside a stream CTA, or it starts when that has ended and the tail
// is waited for. A stream CTA of d = 64 has ten warps, three of them on two of the SM's
// four schedulers, which leaves 48 registers a thread here (40 where the stream's are
// fp32): the values are then loaded after the keys are done with. Measured on GB300, us
// (64 registers): 32 units x 1000 tokens 10.0 (14.3), 128 x 3000 17.3 (21.8), fp32 8 x 3000
// 9.2 (15.0). (At 40 registers 20 bytes spill, outside the loops.) At d = 128 there is room for
// 80 beside a bf16 stream, and the values come along with the keys.
template <typename T, int D> constexpr int kQcPerSm = D == 64 ? (sizeof(T) == 4 ? 6 : 5) : 3;

template <typename T, int D>
__global__ void __launch_bounds__(kQcThreads, kQcPerSm<T, D>) quant_combine_kernel(QStreamParams p, int rows, bool weights) {
  constexpr int ELT = (int)sizeof(T), CE = 16 / ELT, NCH = D / CE;
  constexpr int KC = NCH / 4;                        // 16-byte key chunks of a thread: token tid % 64
  constexpr int TG = kQcThreads / NCH, TPT = kQB / TG;  // value tokens: TPT of one 16-byte column
  constexpr int CPW = 32 / TG;                       // columns of a warp; its lanes: token group x column
  constexpr bool kLate = D == 64;                    // values after the keys (fewer registers)
  __shared__ __align__(16) float q_s[kQcRows * D];
  __shared__ __align__(16) float o_s[kQcRows * D];   // the tail's output
  __shared__ float pd_s[4][kQcRows][kQB];            // partial logits
  __shared__ float w_s[kQcRows][kQB];                // weights, -1: masked
  __shared__ float4 ja_s[kQcThreads];
  __shared__ float2 jm_s[kQcThreads];
  __shared__ float m_s[kQcRows], l_s[kQcRows], tw_s[kQcRows];
  __shared__ float2 st_s[kQcRows];
  __shared__ int2 scan_s[kQcThreads / 32];
  griddep_launch_dependents();
  const int vu = blockIdx.x, u = vu / p.tiles, tile = vu % p.tiles, b = u / p.Hkv, h = u % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool flag = tid == 0 && blockIdx.y == 0 && blockIdx.z == 0;
  const int n = max(0, quant_len<true>(p.lens, u, p.max_blocks, p.status, flag));
  const int qn = quant_count<true>(p.q_len, b, p.T, p.status, flag);
  const int nb = n / kQB, nt = n % kQB;
  const int rt = blockIdx.y * kQcRows, r0 = tile * rows + rt;        // first row, in the tile and in the request
  const int live = min(kQcRows, max(0, qn * p.G - r0));              // rows that exist
  if (nt > 0 && live > 0) {
    const uint8_t* tail = p.tail + (long long)u * p.payload;
    const int t = tid % kQB, cg = tid / kQB;
    const int col = warp * CPW + lane % CPW, t0 = lane / CPW * TPT;
    uint4 kr[KC];
#pragma unroll
    for (int i = 0; i < KC; ++i)
      kr[i] = t < nt ? __ldcg(reinterpret_cast<const uint4*>(tail + ((size_t)(cg * KC + i) * kQB + t) * 16)) : make_uint4(0, 0, 0, 0);
    uint4 vr[TPT];
    auto load_values = [&]() {
#pragma unroll
      for (int i = 0; i < TPT; ++i)
        vr[i] = t0 + i < nt ? __ldcg(reinterpret_cast<const uint4*>(tail + (size_t)kQB * D * ELT + (size_t)(t0 + i) * D * ELT + col * 16))
                            : make_uint4(0, 0, 0, 0);
    };
    if (!kLate) load_values();
    const float* es = reinterpret_cast<const float*>(tail + 2 * (size_t)kQB * D * ELT);
    const float e0 = lane < nt ? __ldcg(es + lane) : -INFINITY, e1 = lane + 32 < nt ? __ldcg(es + lane + 32) : -INFINITY;
    for (int i = tid; i < live * NCH; i += kQcThreads) {
      const int r = i / NCH, x = i % NCH;
      const QRow w = qa_row(r0 + r, p.G, n, qn);
      const T* src = reinterpret_cast<const T*>(p.q) + b * p.qs.b + w.t * p.qs.t + (h * p.G + w.g) * p.qs.h + x * CE;
      const uint4 y = __ldcg(reinterpret_cast<const uint4*>(src));
      const T* e = reinterpret_cast<const T*>(&y);
#pragma unroll
      for (int k = 0; k < CE; ++k) q_s[r * D + x * CE + k] = to_f32(e[k]) * kQScale<D>;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kQcRows; ++r) {
      if (r < live) {
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          const T* kv = reinterpret_cast<const T*>(&kr[i]);
          const float* qv = q_s + r * D + (cg * KC + i) * CE;
#pragma unroll
          for (int x = 0; x < CE; ++x) dot += qv[x] * to_f32(kv[x]);
        }
        pd_s[cg][r][t] = dot;
      }
    }
    __syncthreads();
    if (warp < live) {  // a warp has a row
      const int sees = qa_row(r0 + warp, p.G, n, qn).sees - nb * kQB;
      float x0 = e0, x1 = e1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x0 += pd_s[k][warp][lane];
        x1 += pd_s[k][warp][32 + lane];
      }
      if (e0 == -INFINITY || lane >= sees) x0 = -INFINITY;
      if (e1 == -INFINITY || lane + 32 >= sees) x1 = -INFINITY;
      float m = max_nan(x0, x1);
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
      const float mu = finite_max(m), y0 = exp_from(x0, mu), y1 = exp_from(x1, mu);
      float l = y0 + y1;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
      w_s[warp][lane] = x0 == -INFINITY ? -1.f : y0;
      w_s[warp][32 + lane] = x1 == -INFINITY ? -1.f : y1;
      if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
      }
    }
    __syncthreads();
    if (kLate) load_values();
#pragma unroll 1
    for (int r = 0; r < live; ++r) {
      float acc[CE];
#pragma unroll
      for (int x = 0; x < CE; ++x) acc[x] = 0.f;
#pragma unroll
      for (int i = 0; i < TPT; ++i) {
        const float w = w_s[r][t0 + i];
        const T* vv = reinterpret_cast<const T*>(&vr[i]);
        if (!(w < 0.f)) {  // a masked token's value is not looked at
#pragma unroll
          for (int x = 0; x < CE; ++x) acc[x] += w * to_f32(vv[x]);
        }
      }
#pragma unroll
      for (int s = CPW; s < 32; s <<= 1)
#pragma unroll
        for (int x = 0; x < CE; ++x) acc[x] += __shfl_xor_sync(0xffffffffu, acc[x], s);
      if (lane < CPW) {
#pragma unroll
        for (int x = 0; x < CE; ++x) o_s[r * D + col * CE + x] = acc[x];
      }
    }
    __syncthreads();
  }
  // Items of the call and the first one of this unit and tile: added up here, while the
  // stream runs, where a thread has few lengths to read; else left by the stream.
  long long total = 0, first = 0;
  const bool few = p.U <= kQcScan * kQcThreads;
  if (few) {
    int all = 0, ahead = 0;
#pragma unroll
    for (int k = 0; k < kQcScan; ++k) {
      const int i = tid + k * kQcThreads;
      const int c = i < p.U ? max(0, quant_len<true>(p.lens, i, p.max_blocks, nullptr, false)) / kQB : 0;
      all += c;
      if (i < u) ahead += c;
    }
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, s);
      ahead += __shfl_xor_sync(0xffffffffu, ahead, s);
    }
    if (lane == 0) scan_s[warp] = make_int2(all, ahead);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQcThreads / 32; ++w) {
      total += scan_s[w].x;
      first += scan_s[w].y;
    }
    total *= p.tiles;
    first = first * p.tiles + (long long)tile * nb;
  }
  griddep_wait();  // the stream's parts
  // parts of this unit and tile: CTAs [c0, c0 + parts) of the stream, slot c + vu each
  int c0 = 0, parts = 0;
  if (nb > 0) {
    if (!few) {
      total = __ldcg(p.total);
      first = __ldcg(p.base + u) * p.tiles + (long long)tile * nb;
    }
    const int active = qa_active(total, p.ctas);
    c0 = qa_cta_of(first, total, active);
    parts = qa_cta_of(first + nb - 1, total, active) - c0 + 1;
  }
  const long long slot0 = (long long)c0 + vu;
  const int dims = D / gridDim.z, d0 = blockIdx.z * dims, cols = dims / 4, vec = live * cols;  // vec <= the threads
  int groups = 1;
  while (groups * 2 * vec <= kQcThreads && groups < parts) groups *= 2;
  const int at = vec > 0 ? tid % vec : 0, grp = vec > 0 ? tid / vec : 0;
  const bool on = vec > 0 && grp < groups;
  const int r = at / cols, x = at % cols;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto merge = [&](float2 ml, float4 y) {
    const float mn = max_nan(m, ml.x), mu = finite_max(mn);
    const float a = exp_from(m, mu), c = exp_from(ml.x, mu);
    acc.x = acc.x * a + y.x * c; acc.y = acc.y * a + y.y * c; acc.z = acc.z * a + y.z * c; acc.w = acc.w * a + y.w * c;
    l = l * a + ml.y * c;
    m = mn;
  };
  if (on) {
    const float* src = p.part_acc + (slot0 * rows + rt + r) * D + d0 + 4 * x;
    const float2* ml = p.part_ml + slot0 * rows + rt + r;
    for (int i0 = grp; i0 < parts; i0 += 4 * groups) {
      float2 mm[4];
      float4 yy[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * groups;
        mm[k] = i < parts ? __ldcg(ml + (long long)i * rows) : make_float2(-INFINITY, 0.f);
        yy[k] = i < parts ? __ldcg(reinterpret_cast<const float4*>(src + (long long)i * rows * D)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) merge(mm[k], yy[k]);
    }
  }
  if (groups > 1) {
    if (on && grp > 0) {
      ja_s[grp * vec + at] = acc;
      jm_s[grp * vec + at] = make_float2(m, l);
    }
    __syncthreads();
    if (on && grp == 0)
      for (int k = 1; k < groups; ++k) merge(jm_s[k * vec + at], ja_s[k * vec + at]);
  }
  if (on && grp == 0) {
    if (nt > 0) merge(make_float2(m_s[r], l_s[r]), *reinterpret_cast<const float4*>(o_s + r * D + d0 + 4 * x));
    const bool missing = l == -INFINITY;
    const float mu = finite_max(m), inv = missing ? __uint_as_float(0x7FC00000u) : l == 0.f ? 0.f : 1.f / l;
    const QRow w = qa_row(r0 + r, p.G, n, qn);
    const long long row = ((long long)b * p.T + w.t) * p.Hq + h * p.G + w.g;
    T* dst = reinterpret_cast<T*>(p.out) + row * D + d0 + 4 * x;
    if constexpr (ELT == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
      const __nv_bfloat162 y0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), y1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    }
    if (x == 0) {
      if (p.lse != nullptr && blockIdx.z == 0) p.lse[row] = l == 0.f ? -INFINITY : mu + logf(l);
      if (p.blk != nullptr) {
        const float tw = nt > 0 ? l_s[r] * exp_from(m_s[r], mu) * inv : 0.f;
        if (weights) {
          st_s[r] = make_float2(mu, missing ? -1.f : inv);
          tw_s[r] = tw;
        } else if (blockIdx.z == 0) {
          p.rowstat[(long long)vu * rows + rt + r] = make_float2(mu, missing ? -1.f : inv);
          p.tail_w[(long long)vu * rows + rt + r] = tw;
        }
      }
    }
  }
  if (p.blk != nullptr && !weights && blockIdx.z == 0 && tid >= live && tid < kQcRows) {  // rows that do not exist weigh nothing
    p.rowstat[(long long)vu * rows + rt + tid] = make_float2(0.f, 0.f);
    p.tail_w[(long long)vu * rows + rt + tid] = 0.f;
  }
  if (weights) {
    // All of the unit's rows are here: the accumulated weights too (unless parts are
    // missing). Eight lanes have a block's rows; CTA z of the unit takes every gridDim.z-th
    // run of 32 blocks.
    __syncthreads();
    const int row = tid % kQcRows, step = kQcThreads / kQcRows * gridDim.z;
    const float2 st = row < live ? st_s[row] : make_float2(0.f, 0.f);
    const float tw = row < live ? tw_s[row] : 0.f;
    if (__any_sync(0xffffffffu, st.y == -1.f)) return;  // (a warp has all rows)
    float* mass = p.mass + (long long)u * p.max_blocks;
    const float2* note = p.blk + (long long)u * p.max_blocks * kQcRows + row;
    for (int j0 = blockIdx.z * (kQcThreads / kQcRows) + tid / kQcRows; j0 - tid / kQcRows < p.max_blocks; j0 += 8 * step) {
      float2 ml[8];
      float old[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + k * step;
        ml[k] = j < nb && row < live ? __ldcg(note + (long long)j * kQcRows) : make_float2(-INFINITY, 0.f);
        old[k] = row == 0 && j < p.max_blocks && p.decay != 0.f ? mass[j] * p.decay : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + k * step;
        float w = j < nb ? ml[k].y * exp_from(ml[k].x, st.x) * st.y : j == nb ? tw : 0.f;
        w += __shfl_xor_sync(0xffffffffu, w, 1);
        w += __shfl_xor_sync(0xffffffffu, w, 2);
        w += __shfl_xor_sync(0xffffffffu, w, 4);
        if (row == 0 && j < p.max_blocks) mass[j] = old[k] + w;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Accumulated weights: mass = decay * mass + sum over the tiles and rows of
// (block sum) * exp(block maximum - row maximum) / row sum, the lanes in a fixed
// order. Entries without tokens only decay. A warp takes 32 / rows blocks at once,
// four times.
// ---------------------------------------------------------------------------
template <int ROWS>
__host__ __device__ constexpr int weights_per_cta() {
  return kQcThreads / 32 * (32 / ROWS) * 4;
}

template <int ROWS>
__global__ void __launch_bounds__(kQcThreads) quant_weights_kernel(QStreamParams p) {
  constexpr int PW = 32 / ROWS;  // blocks at once
  const int u = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane % ROWS;
  const int n = max(0, quant_len<true>(p.lens, u, p.max_blocks, nullptr, false)), nb = n / kQB, nt = n % kQB;
  const int first = blockIdx.y * weights_per_cta<ROWS>() + warp * PW * 4 + lane / ROWS;
  float* mass = p.mass + (long long)u * p.max_blocks;
  float old[4], w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = first + i * PW;
    old[i] = r == 0 && j < p.max_blocks && p.decay != 0.f ? __ldcg(mass + j) * p.decay : 0.f;
    w[i] = 0.f;
  }
  griddep_wait();
  griddep_launch_dependents();
  bool missing = false;
  for (int tile = 0; tile < p.tiles; ++tile) {
    const long long vu = (long long)u * p.tiles + tile;
    const bool on = tile * ROWS + r < p.T * p.G;
    const float2 st = on ? __ldcg(p.rowstat + vu * ROWS + r) : make_float2(0.f, 0.f);
    missing |= st.y == -1.f;
    float2 ml[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = first + i * PW;
      ml[i] = on && j < nb ? __ldcg(p.blk + (vu * p.max_blocks + j) * ROWS + r) : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = first + i * PW;
      if (on && j < nb) w[i] += ml[i].y * exp_from(ml[i].x, st.x) * st.y;
      if (j == nb && nt > 0) w[i] += __ldcg(p.tail_w + vu * ROWS + r);
    }
  }
  if (__any_sync(0xffffffffu, missing)) return;  // the unit's weights stay as they are
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = first + i * PW;
#pragma unroll
    for (int s = 1; s < ROWS; s <<= 1) w[i] += __shfl_xor_sync(0xffffffffu, w[i], s);
    if (r == 0 && j < p.max_blocks) mass[j] = old[i] + w[i];
  }
}

#endif  // __CUDACC__

// Launches one variant; defined per type in k_quant_attn_{bf16,f32}.cu.
struct QPlan {
  int rows, tiles, ctas;
};
QPlan quant_attn_plan(const Shape& s, int T);
cudaError_t launch_quant_stream_bf16(const Shape& s, const QPlan& pl, const QStreamParams& p, cudaStream_t stream);
cudaError_t launch_quant_stream_f32(const Shape& s, const QPlan& pl, const QStreamParams& p, cudaStream_t stream);

#ifdef __CUDACC__
template <int D, int NT, int RG, bool F32>
cudaError_t stream_variant(const QPlan& pl, const QStreamParams& p, cudaStream_t stream) {
  using Gm = QGeom<D, NT, RG, F32>;
  static std::atomic<int> lim[64];
  const cudaError_t e = raise_smem_limit((const void*)quant_stream_kernel<D, NT, RG, F32>, Gm::SMEM, lim);
  if (e != cudaSuccess) return e;
  return launch_dependent(quant_stream_kernel<D, NT, RG, F32>, dim3(pl.ctas), Gm::THREADS, Gm::SMEM, stream, p);
}

template <typename T, int D>
cudaError_t stream_launches(const Shape& s, const QPlan& pl, const QStreamParams& p, cudaStream_t stream) {
  constexpr bool F32 = sizeof(T) == 4;
  // 16 and 32 rows as row groups of 8, which convert the codes once each but leave
  // registers enough for eight consumer warps; 32 rows of bf16 as two groups of 16 on
  // six. Measured when they were chosen, at 4 requests x 8 KV heads x 16384 tokens of
  // d = 128, us: 16 rows 39 (one group of 16: 44), fp32 47 (59); 32 rows 62 (two groups
  // of 16: 60), fp32 78 (89). With the next unit's queries ready ahead: 36, 41, 53, 69.
  cudaError_t e;
  if (pl.rows == 8)
    e = stream_variant<D, 1, 1, F32>(pl, p, stream);
  else if (pl.rows == 16)
    e = stream_variant<D, 1, 2, F32>(pl, p, stream);
  else if constexpr (F32)
    e = stream_variant<D, 1, 4, F32>(pl, p, stream);
  else
    e = stream_variant<D, 2, 2, F32>(pl, p, stream);
  if (e != cudaSuccess) return e;
  // few units have many parts each: more CTAs share the join
  const int vu = s.U * pl.tiles, y = pl.rows / kQcRows, z = vu * y <= 16 ? 4 : vu * y <= 32 ? 2 : 1;
  // Where one CTA has all rows of a unit, the join does the accumulated weights too, if
  // they are few; long tables want the warps of a launch of their own. Measured at 128
  // units of d = 128 in bf16, us (joined / own launch): 32 blocks 22.1 / 23.1, 128 54.2 /
  // 54.3, 256 96.7 / 95.5, 512 105.4 / 100.0 (ragged); four CTAs a unit at 16 units: 375
  // blocks 27.1 / 27.6.
  const bool joined = p.mass != nullptr && pl.rows == kQcRows && p.max_blocks <= 128 * z;
  e = launch_dependent(quant_combine_kernel<T, D>, dim3(vu, y, z), kQcThreads, 0, stream, p, pl.rows, joined);
  if (e != cudaSuccess || p.mass == nullptr || joined) return e;
  auto weights = [&](auto kernel, int per) {
    return launch_dependent(kernel, dim3(s.U, (p.max_blocks + per - 1) / per), kQcThreads, 0, stream, p);
  };
  return pl.rows == 8    ? weights(quant_weights_kernel<8>, weights_per_cta<8>())
         : pl.rows == 16 ? weights(quant_weights_kernel<16>, weights_per_cta<16>())
                         : weights(quant_weights_kernel<32>, weights_per_cta<32>());
}
#endif

}  // namespace nosa
