// Attention over the 8-bit block cache.
//
// Row (t, g) of unit u sees tokens [0, len - T_b + t]: its logits are
//     l_j = q . k_j / sqrt(d) + e_j   (e_j = -inf masks token j),
// out = sum_j softmax(l)_j v_j, lse = log sum_j exp(l_j), and the weights' sum over
// the rows and the tokens of a block goes to the block's accumulated weight.
#include "k_quant.cuh"

#include <cuda_fp8.h>

#include <algorithm>

namespace nosa {
namespace {

constexpr int kRows = 8;
constexpr int kThreads = 128;

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// One CTA per unit walks its row tiles and blocks with fp32 arithmetic.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) quant_attn_kernel(QAttnArgs p, int Hq, int Hkv, int G, long long payload) {
  __shared__ float q_s[kRows][D];
  __shared__ float p_s[kRows][kQB];
  __shared__ float m_s[kRows], l_s[kRows], c_s[kRows], d_s[kRows];
  const int u = blockIdx.x, b = u / Hkv, h = u % Hkv, tid = threadIdx.x;
  const int n = max(0, quant_len(p.lens, u, p.max_blocks, p.status, tid == 0));
  const int qn = quant_count(p.q_len, b, p.T, p.status, tid == 0);
  const int nb = n / kQB, nt = n % kQB, R = qn * G;
  const uint8_t* tail = p.tail + u * payload;
  const float scale = (float)(1.0 / sqrt((double)D));
  for (int r0 = 0; r0 < p.T * G; r0 += kRows) {
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kThreads) {
      const int r = r0 + i / D;
      q_s[i / D][i % D] = r < R ? to_f32(reinterpret_cast<const T*>(p.q)[b * p.qs.b + (r / G) * p.qs.t + (h * G + r % G) * p.qs.h + i % D]) : 0.f;
    }
    if (tid < kRows) { m_s[tid] = -INFINITY; l_s[tid] = 0.f; }
    float acc[kRows];
    for (int r = 0; r < kRows; ++r) acc[r] = 0.f;
    for (int pass = 0; pass < (p.mass ? 2 : 1); ++pass) {
      for (int j = 0; j <= nb; ++j) {
        const bool is_tail = j == nb;
        const int cnt = is_tail ? nt : kQB;
        const int idx = is_tail ? 0 : p.tab[(long long)u * p.max_blocks + j];
        const bool bad = idx < 0 || (!is_tail && idx >= p.n_units);
        if (bad && pass == 0 && tid == 0) quant_flag(p.status, kQErrIndex);
        if (cnt == 0) continue;
        const uint8_t* un = p.units + (long long)(bad ? 0 : idx) * quant_unit_bytes(D);
        __syncthreads();
        {
          const int t = tid % kQB;
          for (int r = tid / kQB; r < kRows; r += kThreads / kQB) {
            const int gr = r0 + r, last = n - qn + gr / G;  // newest visible token
            float lg = -INFINITY;
            if (!bad && gr < R && t < cnt && j * kQB + t <= last) {
              const float e = is_tail ? reinterpret_cast<const float*>(tail + 2 * (size_t)kQB * D * sizeof(T))[t]
                                      : reinterpret_cast<const float*>(un + quant_e_off(D))[t];
              if (e != -INFINITY) {
                float dot = 0.f;
                for (int x = 0; x < D; ++x)
                  dot += q_s[r][x] * (is_tail ? to_f32(*reinterpret_cast<const T*>(tail + k_off(t, x, kQB, sizeof(T))))
                                              : e4m3_f32(un[quant_k_off(t, x, D)]));
                if (!is_tail) dot *= reinterpret_cast<const float*>(un + quant_scale_off(D))[0];
                lg = dot * scale + e;
              }
            }
            p_s[r][t] = lg;
          }
        }
        __syncthreads();
        if (tid < kRows) {
          if (pass == 0) {
            float m = m_s[tid];
            for (int t = 0; t < kQB; ++t) { const float x = p_s[tid][t]; m = (x > m || isnan(x)) ? x : m; }
            c_s[tid] = m_s[tid] == -INFINITY ? 0.f : expf(m_s[tid] - m);
            m_s[tid] = m;
          }
          float sum = 0.f;
          for (int t = 0; t < kQB; ++t) {
            const float x = p_s[tid][t];
            const float e = x == -INFINITY ? 0.f : expf(x - m_s[tid]);
            p_s[tid][t] = x == -INFINITY ? -1.f : e;
            sum += e;
          }
          if (pass == 0) l_s[tid] = l_s[tid] * c_s[tid] + sum;
          d_s[tid] = l_s[tid] != 0.f ? sum / l_s[tid] : 0.f;
        }
        __syncthreads();
        if (pass == 1) {
          if (tid == 0 && j < p.max_blocks) {
            float w = 0.f;
            for (int r = 0; r < kRows; ++r) w += d_s[r];
            float* m = p.mass + (long long)u * p.max_blocks + j;
            *m = (r0 > 0 ? *m : p.decay == 0.f ? 0.f : *m * p.decay) + w;
          }
          continue;
        }
        for (int x = tid; x < D; x += kThreads) {
          const float vs = is_tail || bad ? 1.f : reinterpret_cast<const float*>(un + quant_scale_off(D))[1];
          for (int r = 0; r < kRows; ++r) {
            float o = 0.f;
            for (int t = 0; t < kQB; ++t) {
              const float w = p_s[r][t];
              if (w < 0.f) continue;  // masked: whatever its value holds
              o += w * (is_tail ? to_f32(*reinterpret_cast<const T*>(tail + v_off(t, x, kQB, D, sizeof(T))))
                                : vs * e4m3_f32(un[quant_v_off(t, x, D)]));
            }
            acc[r] = acc[r] * c_s[r] + o;
          }
        }
      }
      if (pass == 0) {
        __syncthreads();
        for (int r = 0; r < kRows; ++r) {
          const int gr = r0 + r;
          if (gr >= R) continue;
          const long long o = ((long long)b * p.T + gr / G) * Hq + h * G + gr % G;
          if (tid < D) reinterpret_cast<T*>(p.out)[o * D + tid] = from_f32<T>(l_s[r] != 0.f ? acc[r] / l_s[r] : 0.f);
          if (tid == 0 && p.lse != nullptr) p.lse[o] = l_s[r] != 0.f ? m_s[r] + logf(l_s[r]) : -INFINITY;
        }
      }
    }
  }
  if (p.mass != nullptr)  // entries without tokens only decay
    for (int j = nb + (nt > 0) + tid; j < p.max_blocks; j += kThreads) {
      float* m = p.mass + (long long)u * p.max_blocks + j;
      *m = p.decay == 0.f ? 0.f : *m * p.decay;
    }
}

template <typename T, int D>
cudaError_t attn_variant(const Shape& s, const QAttnArgs& a, cudaStream_t stream) {
  quant_attn_kernel<T, D><<<s.U, kThreads, 0, stream>>>(a, s.Hq, s.Hkv, s.G, s.payload);
  return cudaGetLastError();
}

}  // namespace

size_t quant_attn_workspace(const Shape&, int, int, bool) { return 16; }

cudaError_t launch_quant_attention(const Shape& s, const QAttnArgs& a, cudaStream_t stream) {
  if (s.dtype == 0) return s.d == 64 ? attn_variant<float, 64>(s, a, stream) : attn_variant<float, 128>(s, a, stream);
  return s.d == 64 ? attn_variant<__nv_bfloat16, 64>(s, a, stream) : attn_variant<__nv_bfloat16, 128>(s, a, stream);
}

}  // namespace nosa
