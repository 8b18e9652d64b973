// Attention over the 8-bit block cache.
//
// Row (t, g) of unit u sees tokens [0, len - T_b + t]: its logits are
//     l_j = q . k_j / sqrt(d) + e_j   (e_j = -inf masks token j),
// out = sum_j softmax(l)_j v_j, lse = log sum_j exp(l_j), and the weights' sum over
// the rows and the tokens of a block goes to the block's accumulated weight.
//
// The cache is read once, so HBM bounds a call with few rows. Three launches:
//   stream  : the full blocks of all units, one after another, are one list of items
//             that one wave of CTAs shares equally (units differ in length, so the
//             shares are cut from the lengths on the device). A producer warp keeps a
//             ring of whole units in flight with bulk copies; four warps each own one
//             16-token slice of every unit with a running maximum, sum and output of
//             their own, and join when the CTA leaves a unit.
//   combine : one CTA per unit (and row tile) attends to the tail in fp32 while the
//             stream still runs, then joins the unit's parts.
//   weights : with accumulated weights, a warp per block adds up what the stream
//             noted for the block, relative to the rows' final sums.
//
// The products take the tensor cores' 16 x 8 x 16 shape with the codes as the large
// operand (tokens x dims, dims x tokens) and the rows as the small one: up to 8 rows
// (the query heads of a KV head) waste nothing, and the weights of a slice reach the
// second product with two 8 x 8 transposes. An e4m3 code is exact in fp16. Queries are
// brought to a largest magnitude in [1, 2) by a power of two per row, so that fp16
// holds a bf16 query exactly (what is lost lies 2^-25 below the row's largest
// element); an fp32 query is the sum of two fp16 terms (22 bits). Weights are held in
// fp32 for the sums and rounded to fp16 (fp32 output: two terms) for the second
// product, scaled by 2^14 so that weights down to 2^-28 of the largest keep their 11
// bits. Each slice's product starts from zero and enters the fp32 output with the
// block's value scale, so neither scale ever multiplies an operand.
#pragma once

#include "k_quant.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <map>
#include <mutex>

namespace nosa {

constexpr int kQaThreads = 160;   // four consumer warps and a producer warp
constexpr int kQaMinItems = 2;    // blocks of a CTA's share, at least
constexpr int kQcThreads = 256;   // combine
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
  // workspace
  long long* total;   // items of the call
  long long* base;    // [units x tiles] first item of each
  float2* part_ml;    // [ctas + units x tiles][rows] maximum and sum of a part
  float* part_acc;    // ... [rows][d] its output (not normalised)
  float2* rowstat;    // [units x tiles][rows] final maximum and 1 / sum
  float* tail_w;      // [units x tiles] weight of the tail
  float2* blk;        // [units x tiles][max_blocks][4][rows] maximum and sum of a slice, or null
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

template <int D, int NT, bool F32>
struct QGeom {
  static constexpr int ROWS = 8 * NT, KS = D / 16, UB = quant_unit_bytes(D);
  // ring depth: three CTAs per SM for 8 rows, two for more (their outputs need the registers)
  static constexpr int PER_SM = NT == 1 ? 3 : 2;
  static constexpr int STAGES = NT == 1 ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
  static constexpr int RP = D + 4;  // padded row of the joining buffer
  static constexpr int Q_OFF = STAGES * UB;
  static constexpr int RED_OFF = Q_OFF + NT * KS * 32 * (F32 ? 16 : 8);
  static constexpr int ML_OFF = RED_OFF + 4 * 8 * RP * 4;
  static constexpr int ROW_OFF = ML_OFF + 4 * 8 * 8;
  static constexpr int DESC_OFF = ROW_OFF + ROWS * 8;
  static constexpr int BAR_OFF = DESC_OFF + STAGES * 16;
  static constexpr int SMEM = BAR_OFF + (2 * STAGES + 1) * 8;
  static_assert(UB % 16 == 0 && Q_OFF % 16 == 0 && RED_OFF % 16 == 0 && DESC_OFF % 16 == 0, "alignment");
};

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kQaThreads, QGeom<D, NT, F32>::PER_SM) quant_stream_kernel(QStreamParams p) {
  using Gm = QGeom<D, NT, F32>;
  constexpr int KS = Gm::KS, ROWS = Gm::ROWS, STAGES = Gm::STAGES, UB = Gm::UB;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* q_s = smem + Gm::Q_OFF;
  float* red = reinterpret_cast<float*>(smem + Gm::RED_OFF);
  float2* red_ml = reinterpret_cast<float2*>(smem + Gm::ML_OFF);  // [4][8]
  float* rs_s = reinterpret_cast<float*>(smem + Gm::ROW_OFF);     // [ROWS] factor of a row's logits
  int* vis_s = reinterpret_cast<int*>(rs_s + ROWS);               // [ROWS] tokens it sees
  int4* desc = reinterpret_cast<int4*>(smem + Gm::DESC_OFF);      // unit, tile, block, flags
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Gm::BAR_OFF);
  uint64_t* empty = full + STAGES;
  uint64_t* join = empty + STAGES;
  __shared__ long long s_scan[8];
  __shared__ long long s_before;
  __shared__ int s_unit;
  __shared__ volatile int s_bad;
  enum { kFirst = 1, kLast = 2, kNull = 4 };

  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    mbar_init(join, 4);
    fence_mbar_init();
    s_bad = 0;
  }
  // ---- the share: prefix sums of the units' full blocks ----
  const int per = (p.U + kQaThreads - 1) / kQaThreads;
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
  for (int w = 0; w < kQaThreads / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
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

  if (warp == 4) {
    // ---- producer ----
    int u = s_unit, it = 0, issued = 0;
    long long ub = s_before;  // first item of unit u
    bool go = true;
    while (it < items && go) {
      const int nb = max(0, quant_len(p.lens, u, p.max_blocks, nullptr, false)) / kQB;
      const int32_t* row = p.tab + (long long)u * p.max_blocks;
      int at = (int)(g0 + it - ub);  // item inside the unit
      for (int tile = nb > 0 ? at / nb : p.tiles; tile < p.tiles && it < items && go; ++tile) {
        const int j0 = at - tile * nb, j1 = (int)min((long long)nb, (long long)j0 + (items - it));
        if (j0 == 0 && lane == 0) p.base[(long long)u * p.tiles + tile] = ub + (long long)tile * nb;
        int next = j0 + lane < j1 ? row[j0 + lane] : -1;
        for (int jb = j0; jb < j1 && go; jb += 32) {
          const int cur = next;
          next = jb + 32 + lane < j1 ? row[jb + 32 + lane] : -1;
          const int cnt = min(32, j1 - jb);
          for (int i = 0; i < cnt; ++i, ++it) {
            const int idx = __shfl_sync(0xffffffffu, cur, i);
            const int s = it % STAGES, j = jb + i;
            if (lane == 0) {
              if (it >= STAGES && !mbar_wait_bounded(&empty[s], (uint32_t)((it / STAGES - 1) & 1))) {
                s_bad = 1;
                quant_flag(p.status, kQErrWait);
              }
              if (s_bad == 0) {
                const bool bad = idx < 0 || (long long)idx >= p.n_units;
                desc[s] = make_int4(u, tile, j, (j == j0 ? kFirst : 0) | (j == j1 - 1 ? kLast : 0) | (bad ? kNull : 0));
                if (bad) {
                  quant_flag(p.status, kQErrIndex);
                  mbar_arrive(&full[s]);
                } else {
                  mbar_arrive_expect_tx(&full[s], UB);
                  bulk_g2s(smem + s * UB, p.units + (long long)idx * UB, UB, &full[s]);
                }
                issued = it + 1;
              }
            }
            go = __shfl_sync(0xffffffffu, s_bad == 0 ? 1 : 0, 0) != 0;
            if (!go) break;
          }
        }
        at += j1 - j0;
      }
      ub += (long long)nb * p.tiles;
      ++u;
    }
    __syncthreads();
    if (s_bad != 0 && lane == 0) {  // drain: the last copy issued into each stage
      for (int s = 0; s < STAGES; ++s) {
        int last = -1;
        for (int i = s; i < issued; i += STAGES) last = i;
        if (last >= 0) mbar_wait_bounded(&full[s], (uint32_t)((last / STAGES) & 1));
      }
    }
    return;
  }

  // ---- consumers ----
  const int g = lane >> 2, c = lane & 3;
  const int tok = 16 * warp + 4 * (g >> 1) + (g & 1);  // this lane's tokens: tok and tok + 2
  uint32_t joins = 0;
  // All four warps, with a limit: false where one of them gave up.
  auto sync4 = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(join);
    const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(join, joins & 1));
    ++joins;
    if (!ok && lane == 0) {
      s_bad = 1;
      quant_flag(p.status, kQErrWait);
    }
    return ok;
  };
  float o[NT][KS][4], m_run[NT][2], l_run[NT][2], fac[NT][2];
  int vis[NT][2];
  uint32_t qr[NT == 1 && !F32 ? KS : 1][2];
  int least = 0;  // tokens that every row of the tile sees
  for (int it = 0; it < items; ++it) {
    if (__any_sync(0xffffffffu, s_bad != 0)) break;
    const int s = it % STAGES;
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (uint32_t)((it / STAGES) & 1)))) {
      if (lane == 0) {
        s_bad = 1;
        quant_flag(p.status, kQErrWait);
      }
      break;
    }
    const int4 de = desc[s];
    const int u = de.x, tile = de.y, j = de.z;
    const long long vu = (long long)u * p.tiles + tile;
    if (de.w & kFirst) {
      // queries of the tile: warp w prepares row group w, w + 4, ...
      const int b = u / p.Hkv, h = u % p.Hkv;
      const int n = quant_len(p.lens, u, p.max_blocks, nullptr, false);
      const int qn = quant_count(p.q_len, b, p.T, p.status, true);
      for (int nt = warp; nt < NT; nt += 4) {
        const QRow w = qa_row(tile * ROWS + nt * 8 + g, p.G, n, qn);
        float f[KS][4];
        float mx = 0.f;
        const long long at = b * p.qs.b + w.t * p.qs.t + (h * p.G + w.g) * p.qs.h + 4 * c;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          f[k][0] = f[k][1] = f[k][2] = f[k][3] = 0.f;
          if (w.t < qn) {
            if constexpr (F32) {
              const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + at + 16 * k);
              f[k][0] = x.x; f[k][1] = x.y; f[k][2] = x.z; f[k][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(p.q) + at + 16 * k);
              f[k][0] = bf16_lo(x.x); f[k][1] = bf16_hi(x.x); f[k][2] = bf16_lo(x.y); f[k][3] = bf16_hi(x.y);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(f[k][i]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^ex <= mx < 2^(ex + 1), kept where both 2^ex and 2^-ex are normal numbers
        const int ex = min(max((int)(__float_as_uint(mx) >> 23), 1), 253) - 127;
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23), up = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const float x0 = f[k][0] * down, x1 = f[k][1] * down, x2 = f[k][2] * down, x3 = f[k][3] * down;
          const uint32_t h0 = f16x2(x0, x1), h1 = f16x2(x2, x3);
          if constexpr (F32) {
            const float2 y0 = f32x2(h0), y1 = f32x2(h1);
            reinterpret_cast<uint4*>(q_s)[(nt * KS + k) * 32 + lane] =
                make_uint4(h0, h1, f16x2(x0 - y0.x, x1 - y0.y), f16x2(x2 - y1.x, x3 - y1.y));
          } else {
            reinterpret_cast<uint2*>(q_s)[(nt * KS + k) * 32 + lane] = make_uint2(h0, h1);
          }
        }
        if (c == 0) {
          rs_s[nt * 8 + g] = up * kQScale<D>;
          vis_s[nt * 8 + g] = w.sees;
        }
      }
      if (!sync4()) break;
      least = 0x7fffffff;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          fac[nt][x] = rs_s[nt * 8 + 2 * c + x];
          vis[nt][x] = vis_s[nt * 8 + 2 * c + x];
          least = min(least, vis[nt][x]);
          m_run[nt][x] = -INFINITY;
          l_run[nt][x] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
      }
      if constexpr (NT == 1 && !F32) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint2 x = reinterpret_cast<const uint2*>(q_s)[k * 32 + lane];
          qr[k][0] = x.x;
          qr[k][1] = x.y;
        }
      }
    }

    float2* note = p.blk == nullptr ? nullptr : p.blk + ((vu * p.max_blocks + j) * 4 + warp) * ROWS;
    if (de.w & kNull) {
      if (note != nullptr && lane < ROWS) note[lane] = make_float2(-INFINITY, 0.f);
    } else {
      const uint8_t* unit = smem + s * UB;
      const uint4* kw = reinterpret_cast<const uint4*>(unit + warp * 32 * D) + lane;
      // ---- logits ----
      float sc[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[nt][0][x] = sc[nt][1][x] = 0.f;
#pragma unroll
      for (int jj = 0; jj < KS / 2; ++jj) {
        const uint4 w = kw[jj * 32];
        const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int k = 2 * jj + y;
          const uint32_t a[4] = {e4m3x2_f16x2(wd[2 * y]), e4m3x2_f16x2(wd[2 * y + 1]), e4m3x2_f16x2(wd[2 * y] >> 16),
                                 e4m3x2_f16x2(wd[2 * y + 1] >> 16)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (NT == 1 && !F32) {
              mma16816(sc[nt][y], a, qr[k][0], qr[k][1]);
            } else if constexpr (F32) {
              const uint4 x = reinterpret_cast<const uint4*>(q_s)[(nt * KS + k) * 32 + lane];
              mma16816(sc[nt][0], a, x.x, x.y);
              mma16816(sc[nt][1], a, x.z, x.w);
            } else {
              const uint2 x = reinterpret_cast<const uint2*>(q_s)[(nt * KS + k) * 32 + lane];
              mma16816(sc[nt][y], a, x.x, x.y);
            }
          }
        }
      }
      // ---- softmax over the warp's 16 tokens ----
      const float* es = reinterpret_cast<const float*>(unit + quant_e_off(D));
      const float e0 = es[tok], e1 = es[tok + 2];
      const float ks = es[kQB], vs = es[kQB + 1] * 0x1p-14f;
      const bool off0 = e0 == -INFINITY, off1 = e1 == -INFINITY;
      const int pos = j * kQB + tok;
      const bool edge = j * kQB + kQB > least;
      float corr[NT][2], vsc[NT][2];
      uint32_t pb[NT][2], pl[F32 ? NT : 1][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[2][2];  // [column][token]
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float f = fac[nt][x] * ks;
          float l0 = (sc[nt][0][x] + sc[nt][1][x]) * f + e0, l1 = (sc[nt][0][2 + x] + sc[nt][1][2 + x]) * f + e1;
          if (off0 || (edge && pos >= vis[nt][x])) l0 = -INFINITY;
          if (off1 || (edge && pos + 2 >= vis[nt][x])) l1 = -INFINITY;
          float mx = max_nan(l0, l1);
          mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = max_nan(m_run[nt][x], mx), mu = finite_max(mn);
          corr[nt][x] = exp_from(m_run[nt][x], mu);
          vsc[nt][x] = mx == -INFINITY ? 0.f : vs;  // (nothing visible: whatever the block holds)
          pr[x][0] = exp_from(l0, mu);
          pr[x][1] = exp_from(l1, mu);
          const float sum = pr[x][0] + pr[x][1];
          l_run[nt][x] = l_run[nt][x] * corr[nt][x] + sum;
          m_run[nt][x] = mn;
          if (note != nullptr) {
            float t = sum;
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            if (g == 0) note[nt * 8 + 2 * c + x] = make_float2(mn, t);
          }
        }
        const float q00 = pr[0][0] * 16384.f, q10 = pr[1][0] * 16384.f, q01 = pr[0][1] * 16384.f, q11 = pr[1][1] * 16384.f;
        const uint32_t h0 = f16x2(q00, q10), h1 = f16x2(q01, q11);
        pb[nt][0] = transpose8x8(h0);
        pb[nt][1] = transpose8x8(h1);
        if constexpr (F32) {
          const float2 y0 = f32x2(h0), y1 = f32x2(h1);
          pl[nt][0] = transpose8x8(f16x2(q00 - y0.x, q10 - y0.y));
          pl[nt][1] = transpose8x8(f16x2(q01 - y1.x, q11 - y1.y));
        }
      }
      // ---- o = o * corr + scale * (V^T P) ----
      const uint4* vw = kw + D;  // 16 D bytes on
#pragma unroll
      for (int jj = 0; jj < KS / 2; ++jj) {
        const uint4 w = vw[jj * 32];
        const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t a[4] = {e4m3x2_f16x2(wd[2 * y]), e4m3x2_f16x2(wd[2 * y + 1]), e4m3x2_f16x2(wd[2 * y] >> 16),
                                 e4m3x2_f16x2(wd[2 * y + 1] >> 16)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(t, a, pb[nt][0], pb[nt][1]);
            if constexpr (F32) mma16816(t, a, pl[nt][0], pl[nt][1]);
            float* oo = o[nt][2 * jj + y];
#pragma unroll
            for (int x = 0; x < 4; ++x) oo[x] = oo[x] * corr[nt][x & 1] + t[x] * vsc[nt][x & 1];
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);

    if (de.w & kLast) {
      // ---- the four warps' parts become the CTA's part of the unit ----
      const long long slot = cta + vu;
      bool ok = true;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt > 0 && !(ok = ok && sync4())) break;  // the buffer is free
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float l = l_run[nt][x];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          if (g == 0) red_ml[warp * 8 + 2 * c + x] = make_float2(m_run[nt][x], l);
        }
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            red[(warp * 8 + 2 * c + (x & 1)) * Gm::RP + mt * 16 + g + 8 * (x >> 1)] = o[nt][mt][x];
        if (!(ok = ok && sync4())) break;
        for (int i = tid; i < 8 * D / 4; i += 128) {
          const int r = i / (D / 4), x = i % (D / 4);
          float M = red_ml[r].x;
#pragma unroll
          for (int w = 1; w < 4; ++w) M = max_nan(M, red_ml[w * 8 + r].x);
          const float mu = finite_max(M);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float L = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 ml = red_ml[w * 8 + r];
            const float wt = exp_from(ml.x, mu);
            const float4 y = *reinterpret_cast<const float4*>(red + (w * 8 + r) * Gm::RP + 4 * x);
            acc.x += wt * y.x; acc.y += wt * y.y; acc.z += wt * y.z; acc.w += wt * y.w;
            L += wt * ml.y;
          }
          const long long at = slot * ROWS + nt * 8 + r;
          reinterpret_cast<float4*>(p.part_acc + at * D)[x] = acc;
          if (x == 0) p.part_ml[at] = make_float2(M, L);
        }
      }
      if (!ok) break;
      if (!sync4()) break;  // the buffers are free for the next unit
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Tail attention and the join. Grid (units x tiles, z): CTA y of z owns d / z dims.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kQcThreads) quant_combine_kernel(QStreamParams p, int rows) {
  constexpr int ELT = (int)sizeof(T), CE = 16 / ELT, NCH = D / CE, MAXR = 32;
  extern __shared__ __align__(16) uint8_t csmem[];
  float* q_s = reinterpret_cast<float*>(csmem);      // [rows][D]
  float* p_s = q_s + rows * D;                       // [rows][64] logits, then weights (-1: masked)
  float* o_s = p_s + rows * kQB;                     // [rows][dims] the tail's output, then the join's parts
  __shared__ float m_s[MAXR], l_s[MAXR], inv_s[MAXR];
  __shared__ int sees_s[MAXR];
  griddep_launch_dependents();
  const int vu = blockIdx.x, u = vu / p.tiles, tile = vu % p.tiles, b = u / p.Hkv, h = u % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = max(0, quant_len(p.lens, u, p.max_blocks, p.status, tid == 0));
  const int qn = quant_count(p.q_len, b, p.T, p.status, tid == 0);
  const int nb = n / kQB, nt = n % kQB;
  const int r0 = tile * rows, live = min(rows, max(0, qn * p.G - r0));  // rows of the tile that exist
  const int dims = D / gridDim.y, d0 = blockIdx.y * dims;
  const uint8_t* tail = p.tail + (long long)u * p.payload;
  if (tid < live) sees_s[tid] = qa_row(r0 + tid, p.G, n, qn).sees;
  if (nt > 0) {
    const float scale = kQScale<D>;
    for (int i = tid; i < live * (D / CE); i += kQcThreads) {
      const int r = i / (D / CE), x = i % (D / CE);
      const QRow w = qa_row(r0 + r, p.G, n, qn);
      const T* src = reinterpret_cast<const T*>(p.q) + b * p.qs.b + w.t * p.qs.t + (h * p.G + w.g) * p.qs.h + x * CE;
      const uint4 y = *reinterpret_cast<const uint4*>(src);
      const T* e = reinterpret_cast<const T*>(&y);
#pragma unroll
      for (int k = 0; k < CE; ++k) q_s[r * D + x * CE + k] = to_f32(e[k]) * scale;
    }
    __syncthreads();
    // logits: a thread has one token and every fourth row
    const int t = tid % kQB, rg = tid / kQB;
    const float e = t < nt ? reinterpret_cast<const float*>(tail + 2 * (size_t)kQB * D * ELT)[t] : -INFINITY;
    float dot[MAXR / 4];
#pragma unroll
    for (int k = 0; k < MAXR / 4; ++k) dot[k] = 0.f;
    if (t < nt) {
#pragma unroll 4
      for (int ch = 0; ch < NCH; ++ch) {
        const uint4 y = *reinterpret_cast<const uint4*>(tail + ((size_t)ch * kQB + t) * 16);
        const T* kv = reinterpret_cast<const T*>(&y);
#pragma unroll
        for (int k = 0; k < MAXR / 4; ++k) {
          const int r = rg + 4 * k;
          if (r < live) {
#pragma unroll
            for (int x = 0; x < CE; ++x) dot[k] += q_s[r * D + ch * CE + x] * to_f32(kv[x]);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < MAXR / 4; ++k) {
      const int r = rg + 4 * k;
      if (r < live) p_s[r * kQB + t] = (e == -INFINITY || nb * kQB + t >= sees_s[r]) ? -INFINITY : dot[k] + e;
    }
    __syncthreads();
    for (int r = warp; r < live; r += kQcThreads / 32) {
      const float x0 = p_s[r * kQB + lane], x1 = p_s[r * kQB + 32 + lane];
      float m = max_nan(x0, x1);
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
      const float mu = finite_max(m), y0 = exp_from(x0, mu), y1 = exp_from(x1, mu);
      float l = y0 + y1;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
      p_s[r * kQB + lane] = x0 == -INFINITY ? -1.f : y0;
      p_s[r * kQB + 32 + lane] = x1 == -INFINITY ? -1.f : y1;
      if (lane == 0) {
        m_s[r] = m;
        l_s[r] = l;
      }
    }
    __syncthreads();
    const T* vt = reinterpret_cast<const T*>(tail + (size_t)kQB * D * ELT) + d0;
    for (int i = tid; i < live * dims; i += kQcThreads) {
      const int r = i / dims, x = i % dims;
      float acc = 0.f;
#pragma unroll 8
      for (int t2 = 0; t2 < nt; ++t2) {
        const float w = p_s[r * kQB + t2];
        if (w >= 0.f || w != w) acc += w * to_f32(vt[t2 * D + x]);  // a masked token's value is not looked at
      }
      o_s[i] = acc;
    }
  } else {
    if (tid < live) {
      m_s[tid] = -INFINITY;
      l_s[tid] = 0.f;
    }
    for (int i = tid; i < live * dims; i += kQcThreads) o_s[i] = 0.f;
  }
  __syncthreads();
  griddep_wait();  // the stream's parts
  // parts of this unit and tile: CTAs [c0, c1] of the stream, slot c + vu each
  int c0 = 0, parts = 0;
  if (nb > 0) {
    const long long total = *p.total, first = p.base[vu];
    const int active = qa_active(total, p.ctas);
    c0 = qa_cta_of(first, total, active);
    parts = qa_cta_of(first + nb - 1, total, active) - c0 + 1;
  }
  const long long slot0 = (long long)c0 + vu;
  float tw = 0.f;
  for (int r = warp; r < live; r += kQcThreads / 32) {
    float m = m_s[r];
    for (int i = lane; i < parts; i += 32) m = max_nan(m, p.part_ml[(slot0 + i) * rows + r].x);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
    const float mu = finite_max(m);
    float l = 0.f;
    for (int i = lane; i < parts; i += 32) {
      const float2 ml = p.part_ml[(slot0 + i) * rows + r];
      l += ml.y * exp_from(ml.x, mu);
    }
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    const float lt = l_s[r] * exp_from(m_s[r], mu);
    l += lt;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __syncwarp();
    if (lane == 0) {
      const float tail_scale = exp_from(m_s[r], mu) * inv;
      m_s[r] = mu;
      inv_s[r] = inv;
      l_s[r] = tail_scale;
      if (blockIdx.y == 0) {
        const QRow w = qa_row(r0 + r, p.G, n, qn);
        if (p.lse != nullptr)
          p.lse[((long long)b * p.T + w.t) * p.Hq + h * p.G + w.g] = l == 0.f ? -INFINITY : mu + logf(l);
        if (p.blk != nullptr) p.rowstat[(long long)vu * rows + r] = make_float2(mu, inv);
      }
      tw += lt * inv;
    }
  }
  __syncthreads();
  if (p.blk != nullptr && blockIdx.y == 0) {
    // the tail's weight over the rows, in a fixed order; rows that do not exist weigh nothing
    __shared__ float tw_s[kQcThreads / 32];
    if (lane == 0) tw_s[warp] = tw;
    for (int r = live + tid; r < rows; r += kQcThreads) p.rowstat[(long long)vu * rows + r] = make_float2(0.f, 0.f);
    __syncthreads();
    if (tid == 0) {
      float s = 0.f;
      for (int w = 0; w < kQcThreads / 32; ++w) s += tw_s[w];
      p.tail_w[vu] = s;
    }
  }
  // outputs: groups of threads take every gth part, joined through shared memory
  const int vec = live * dims / 4;  // float4 outputs
  int groups = 1;
  while (groups * 2 * vec <= kQcThreads && groups * 2 <= parts) groups *= 2;
  float4* part_s = reinterpret_cast<float4*>(o_s + rows * dims);  // [groups][vec] where groups > 1
  for (int base = 0; base < vec; base += kQcThreads) {
    const int slot_i = groups > 1 ? tid % vec : base + tid, grp = groups > 1 ? tid / vec : 0;
    const bool on = slot_i < vec && grp < groups;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    int r = 0, x = 0;
    if (on) {
      r = slot_i / (dims / 4);
      x = slot_i % (dims / 4);
      const float mu = m_s[r], inv = inv_s[r];
      const float* src = p.part_acc + (slot0 * rows + r) * D + d0 + 4 * x;
      const float2* ml = p.part_ml + slot0 * rows + r;
#pragma unroll 4
      for (int i = grp; i < parts; i += groups) {
        const float w = exp_from(ml[(long long)i * rows].x, mu) * inv;
        const float4 y = *reinterpret_cast<const float4*>(src + (long long)i * rows * D);
        acc.x += w * y.x; acc.y += w * y.y; acc.z += w * y.z; acc.w += w * y.w;
      }
    }
    if (groups > 1) {
      if (on && grp > 0) part_s[grp * vec + slot_i] = acc;
      __syncthreads();
      if (on && grp == 0)
        for (int k = 1; k < groups; ++k) {
          const float4 y = part_s[k * vec + slot_i];
          acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
        }
    }
    if (on && grp == 0) {
      const float ts = l_s[r];
      const float4 y = *reinterpret_cast<const float4*>(o_s + r * dims + 4 * x);
      if (nt > 0) {
        acc.x += ts * y.x; acc.y += ts * y.y; acc.z += ts * y.z; acc.w += ts * y.w;
      }
      const QRow w = qa_row(r0 + r, p.G, n, qn);
      T* dst = reinterpret_cast<T*>(p.out) + (((long long)b * p.T + w.t) * p.Hq + h * p.G + w.g) * D + d0 + 4 * x;
      dst[0] = from_f32<T>(acc.x);
      dst[1] = from_f32<T>(acc.y);
      dst[2] = from_f32<T>(acc.z);
      dst[3] = from_f32<T>(acc.w);
    }
  }
}

// ---------------------------------------------------------------------------
// Accumulated weights: a warp per block. mass = decay * mass + sum over the tiles,
// slices and rows of (slice sum) * exp(slice maximum - row maximum) / row sum, the
// lanes in a fixed order. Entries without tokens only decay.
// ---------------------------------------------------------------------------
template <int ROWS>
__global__ void __launch_bounds__(kQcThreads) quant_weights_kernel(QStreamParams p) {
  const int u = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = max(0, quant_len(p.lens, u, p.max_blocks, nullptr, false)), nb = n / kQB, nt = n % kQB;
  griddep_wait();
  for (int j = blockIdx.y * (kQcThreads / 32) + warp; j < p.max_blocks; j += gridDim.y * (kQcThreads / 32)) {
    float w = 0.f;
    if (j < nb) {
      for (int tile = 0; tile < p.tiles; ++tile) {
        const long long vu = (long long)u * p.tiles + tile;
        const float2* note = p.blk + (vu * p.max_blocks + j) * 4 * ROWS;
#pragma unroll
        for (int i = 0; i < ROWS / 8; ++i) {
          const int x = lane + 32 * i;
          const float2 ml = note[x], st = p.rowstat[vu * ROWS + x % ROWS];
          w += ml.y * exp_from(ml.x, st.x) * st.y;
        }
      }
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) w += __shfl_xor_sync(0xffffffffu, w, s);
    } else if (j == nb && nt > 0) {
      for (int tile = 0; tile < p.tiles; ++tile) w += p.tail_w[(long long)u * p.tiles + tile];
    }
    if (lane == 0) {
      float* m = p.mass + (long long)u * p.max_blocks + j;
      *m = (p.decay == 0.f ? 0.f : *m * p.decay) + w;
    }
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
// Launches `kernel` so that it may begin while the one before it in the stream runs
// (it waits with griddepcontrol.wait before it reads that kernel's results).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int NT, bool F32>
cudaError_t stream_variant(const QPlan& pl, const QStreamParams& p, cudaStream_t stream) {
  constexpr int smem = QGeom<D, NT, F32>::SMEM;
  static std::atomic<int> lim[64];
  const cudaError_t e = raise_smem_limit((const void*)quant_stream_kernel<D, NT, F32>, smem, lim);
  if (e != cudaSuccess) return e;
  quant_stream_kernel<D, NT, F32><<<pl.ctas, kQaThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t stream_launches(const Shape& s, const QPlan& pl, const QStreamParams& p, cudaStream_t stream) {
  constexpr bool F32 = sizeof(T) == 4;
  cudaError_t e = pl.rows == 8    ? stream_variant<D, 1, F32>(pl, p, stream)
                  : pl.rows == 16 ? stream_variant<D, 2, F32>(pl, p, stream)
                                  : stream_variant<D, 4, F32>(pl, p, stream);
  if (e != cudaSuccess) return e;
  const int vu = s.U * pl.tiles;
  const int z = vu * 4 <= 304 ? 4 : vu * 2 <= 304 ? 2 : 1;
  const size_t smem = (size_t)pl.rows * (D + kQB + D / z) * 4 + kQcThreads * 16;
  e = launch_dependent(quant_combine_kernel<T, D>, dim3(vu, z), kQcThreads, smem, stream, p, pl.rows);
  if (e != cudaSuccess || p.mass == nullptr) return e;
  const int y = std::min(p.max_blocks, std::max(1, (p.max_blocks + 31) / 32));
  const dim3 grid(s.U, y);
  return pl.rows == 8    ? launch_dependent(quant_weights_kernel<8>, grid, kQcThreads, 0, stream, p)
         : pl.rows == 16 ? launch_dependent(quant_weights_kernel<16>, grid, kQcThreads, 0, stream, p)
                         : launch_dependent(quant_weights_kernel<32>, grid, kQcThreads, 0, stream, p);
}
#endif

}  // namespace nosa
