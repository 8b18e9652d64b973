// Attention over the 4-bit block cache: a CTA per row of a unit goes through the unit's
// tokens block by block with a running maximum and sum; the accumulated weights are added
// up from the blocks' sums by a second launch.
#include "k_quant4.cuh"

namespace nosa {
namespace {

constexpr int kThreads = 256;

struct Q4AttnParams {
  QAttnArgs a;
  RopeArgs rope;
  int Hq, Hkv, G, rows;
  long long payload;
  float2* rowstat;  // [units][rows] final maximum and 1 / sum
  float* tail_w;    // [units][rows] weight of the tail
  float2* blk;      // [units][rows][max_blocks] maximum and sum of a block, or null
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) quant4_rows_kernel(Q4AttnParams p) {
  constexpr int CE = 16 / (int)sizeof(T), PER = D / 4;  // dims of a thread: four threads have a token
  __shared__ float q_s[D], l_s[kQB], w_s[kQB], o_s[kThreads];
  const int u = blockIdx.x, row = blockIdx.y, b = u / p.Hkv, h = u % p.Hkv, tid = threadIdx.x;
  const int n = max(0, quant_len(p.a.lens, u, p.a.max_blocks, p.a.status, row == 0 && tid == 0));
  const int qn = quant_count(p.a.q_len, b, p.a.T, p.a.status, row == 0 && tid == 0);
  const int t = row / p.G, g = row % p.G, sees = t < qn ? max(0, n - qn + t + 1) : 0;
  if (t >= qn) {
    if (tid == 0 && p.blk != nullptr) p.rowstat[(long long)u * p.rows + row] = make_float2(0.f, 0.f);
    if (tid == 0 && p.blk != nullptr) p.tail_w[(long long)u * p.rows + row] = 0.f;
    return;
  }
  const T* q = static_cast<const T*>(p.a.q) + b * p.a.qs.b + t * p.a.qs.t + (h * p.G + g) * p.a.qs.h;
  if (tid < D) {
    T y = q[tid];
    if (tid < 2 * p.rope.pairs) {
      const RopePlace w = rope_place(p.rope, tid);
      y = from_f32<T>(rope_turn(to_f32(y), to_f32(q[w.other]), w.first, rope_angle(p.rope, (long long)b * p.a.T + t, w.pair)));
    }
    q_s[tid] = to_f32(y);
  }
  __syncthreads();
  const float scale = D == 64 ? 0.125f : 0.08838834764831845f;
  const int nb = n / kQB, nt = n % kQB;
  float m = -INFINITY, l = 0.f, acc = 0.f, tail_l = 0.f, tail_m = -INFINITY;
  for (int j = 0; j < nb + (nt > 0); ++j) {
    const bool is_tail = j == nb;
    const uint8_t* unit = is_tail ? p.a.tail + u * p.payload : nullptr;
    if (!is_tail) {
      const int idx = p.a.tab[(long long)u * p.a.max_blocks + j];
      if (idx < 0 || (long long)idx >= p.a.n_units) {
        if (tid == 0 && row == 0) quant_flag(p.a.status, kQErrIndex);
        if (tid == 0 && p.blk != nullptr) p.blk[((long long)u * p.rows + row) * p.a.max_blocks + j] = make_float2(-INFINITY, 0.f);
        continue;
      }
      unit = p.a.units + (long long)idx * quant4_unit_bytes(D);
    }
    const float* es = reinterpret_cast<const float*>(unit + (is_tail ? 2 * kQB * D * (int)sizeof(T) : quant4_e_off(D)));
    const int tk = tid / 4, x0 = tid % 4 * PER;
    float dot = 0.f;
    for (int x = x0; x < x0 + PER; ++x) {
      float k;
      if (is_tail) {
        k = to_f32(reinterpret_cast<const T*>(unit)[((size_t)(x / CE) * kQB + tk) * CE + x % CE]);
      } else {
        const int bit = quant4_k_bit(tk, x), o = quant4_order(x, D);
        k = fmaf(half_bits(unit[quant4_kstep_off(D) + o] << 8), (float)(unit[bit / 8] >> (bit % 8) & 15),
                 half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_kzero_off(D))[o]));
      }
      dot += q_s[x] * k;
    }
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
    const bool live = es[tk] != -INFINITY && j * kQB + tk < sees && (!is_tail || tk < nt);
    if (tid % 4 == 0) l_s[tk] = live ? dot * scale * (is_tail ? 1.f : es[kQB]) + es[tk] : -INFINITY;
    __syncthreads();
    float mx = -INFINITY;
    bool nan = false;
    for (int i = 0; i < kQB; ++i) {
      mx = fmaxf(mx, l_s[i]);
      nan |= isnan(l_s[i]);
    }
    if (nan) mx = __uint_as_float(0x7FC00000u);
    const float mn = nan || isnan(m) ? __uint_as_float(0x7FC00000u) : fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
    if (tid < kQB) w_s[tid] = l_s[tid] == -INFINITY ? -1.f : expf(l_s[tid] - mu);
    __syncthreads();
    float sum = 0.f;
    for (int i = 0; i < kQB; ++i) sum += w_s[i] == -1.f ? 0.f : w_s[i];
    const float corr = m == -INFINITY ? 0.f : expf(m - mu);
    l = l * corr + sum;
    acc *= corr;
    if (is_tail) {
      tail_l = sum;
      tail_m = mn;
    } else if (tid == 0 && p.blk != nullptr) {
      p.blk[((long long)u * p.rows + row) * p.a.max_blocks + j] = make_float2(mn, sum);
    }
    // a thread has one dim of every (256 / d)-th token
    const int x = tid % D;
    for (int i = tid / D; i < kQB; i += kThreads / D) {
      if (w_s[i] == -1.f) continue;
      float v;
      if (is_tail) {
        v = to_f32(reinterpret_cast<const T*>(unit)[(size_t)kQB * D + (size_t)i * D + x]);
      } else {
        const int bit = quant4_v_bit(i, x), o = x / 64 * kQB + quant4_order(i, kQB);
        v = fmaf(half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_vstep_off(D))[o]), (float)(unit[32 * D + bit / 8] >> (bit % 8) & 15),
                 half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_vzero_off(D))[o])) *
            es[kQB + 1];
      }
      acc += w_s[i] * v;
    }
    m = mn;
    __syncthreads();
  }
  o_s[tid] = acc;
  __syncthreads();
  const long long at = ((long long)b * p.a.T + t) * p.Hq + h * p.G + g;
  const float mu = m == -INFINITY ? 0.f : m, inv = l == 0.f ? 0.f : 1.f / l;
  if (tid < D) {
    float o = 0.f;
    for (int i = tid; i < kThreads; i += D) o += o_s[i];
    static_cast<T*>(p.a.out)[at * D + tid] = from_f32<T>(o * inv);
  }
  if (tid == 0) {
    if (p.a.lse != nullptr) p.a.lse[at] = l == 0.f ? -INFINITY : mu + logf(l);
    if (p.blk != nullptr) {
      p.rowstat[(long long)u * p.rows + row] = make_float2(mu, inv);
      p.tail_w[(long long)u * p.rows + row] = nt > 0 && l != 0.f && tail_m != -INFINITY ? tail_l * expf(tail_m - mu) * inv : 0.f;
    }
  }
}

__global__ void __launch_bounds__(kThreads) quant4_mass_kernel(Q4AttnParams p) {
  const int u = blockIdx.x, j = blockIdx.y * kThreads + threadIdx.x;
  if (j >= p.a.max_blocks) return;
  const int n = max(0, quant_len(p.a.lens, u, p.a.max_blocks, nullptr, false));
  float w = 0.f;
  for (int r = 0; r < p.rows; ++r) {
    const float2 st = p.rowstat[(long long)u * p.rows + r];
    if (j == n / kQB) w += p.tail_w[(long long)u * p.rows + r];
    if (j >= n / kQB || st.y == 0.f) continue;
    const float2 y = p.blk[((long long)u * p.rows + r) * p.a.max_blocks + j];
    if (y.x != -INFINITY) w += y.y * expf(y.x - st.x) * st.y;
  }
  float* mass = p.a.mass + (long long)u * p.a.max_blocks + j;
  *mass = (p.a.decay != 0.f ? *mass * p.a.decay : 0.f) + w;
}

template <typename T, int D>
cudaError_t attention_variant(const Shape& s, const Q4AttnParams& p, cudaStream_t stream) {
  quant4_rows_kernel<T, D><<<dim3(s.U, p.rows), kThreads, 0, stream>>>(p);
  if (p.a.mass != nullptr) quant4_mass_kernel<<<dim3(s.U, (p.a.max_blocks + kThreads - 1) / kThreads), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t quant4_attn_workspace(const Shape& s, int max_blocks, int T, bool mass) {
  const size_t rows = (size_t)s.U * T * s.G;
  return 256 + (mass ? rows * (12 + 8 * (size_t)max_blocks) + 256 : 0);
}

cudaError_t launch_quant4_attention(const Shape& s, const QAttnArgs& a, const RopeArgs& rope, cudaStream_t stream) {
  Q4AttnParams p{};
  p.a = a;
  p.rope = rope;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.G = s.G;
  p.rows = a.T * s.G;
  p.payload = s.payload;
  if (a.mass != nullptr) {
    const size_t rows = (size_t)s.U * p.rows;
    p.rowstat = reinterpret_cast<float2*>(a.ws);
    p.blk = p.rowstat + rows;
    p.tail_w = reinterpret_cast<float*>(p.blk + rows * a.max_blocks);
  }
  if (s.dtype == 0) return s.d == 64 ? attention_variant<float, 64>(s, p, stream) : attention_variant<float, 128>(s, p, stream);
  return s.d == 64 ? attention_variant<__nv_bfloat16, 64>(s, p, stream) : attention_variant<__nv_bfloat16, 128>(s, p, stream);
}

}  // namespace nosa
