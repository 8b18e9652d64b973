// Write side of the 4-bit block cache: appending tokens, with the rotation of their keys on
// the way, and reading blocks back.
#include "k_quant4.cuh"

#include <algorithm>

namespace nosa {
namespace {

constexpr int kThreads = 256;

struct UnitAppend4 {
  int n0, add;
};
// What the call does to unit u: tokens before it, new ones (0 where the unit is left as it was).
__device__ __forceinline__ UnitAppend4 unit_append(const QAppendArgs& p, int Hkv, int u, bool flag) {
  UnitAppend4 r;
  r.n0 = quant_len(p.lens, u, p.max_blocks, p.status, flag);
  r.add = quant_count(p.n_new, u / Hkv, p.n, p.status, flag);
  if (r.n0 < 0) {
    r.n0 = r.add = 0;
  } else if (r.n0 > kQB * p.max_blocks - r.add) {
    if (flag) quant_flag(p.status, kQErrCapacity);
    r.add = 0;
  }
  return r;
}

// Element x of new token `tok` of (request b, head h), as the cache takes it: keys turned
// and rounded to their type.
template <typename T>
__device__ __forceinline__ T new_element(const Q4AppendArgs& p, bool key, int b, int h, int tok, int x) {
  const QStrides& st = key ? p.a.ks : p.a.vs;
  const T* row = static_cast<const T*>(key ? p.a.k : p.a.v) + b * st.b + (long long)tok * st.t + h * st.h;
  if (!key || x >= 2 * p.rope.pairs) return row[x];
  const RopePlace w = rope_place(p.rope, x);
  return from_f32<T>(rope_turn(to_f32(row[x]), to_f32(row[w.other]), w.first, rope_angle(p.rope, (long long)b * p.a.n + tok, w.pair)));
}

// Element x of row t of a tail unit.
template <typename T, int D>
__device__ __forceinline__ size_t tail_at(bool key, int t, int x) {
  constexpr int CE = 16 / (int)sizeof(T);
  return key ? ((size_t)(x / CE) * kQB + t) * CE + x % CE : (size_t)kQB * D + (size_t)t * D + x;
}

// Blocks that the call completes: grid (units, most blocks).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) quant4_blocks_kernel(Q4AppendArgs p, int Hkv, long long payload) {
  __shared__ T x_s[kQB][D];
  __shared__ float e_s[kQB], zero_s[D > 128 ? D : 128], step_s[128];
  __shared__ unsigned amax_s;
  const int u = blockIdx.x, j = blockIdx.y, b = u / Hkv, h = u % Hkv, tid = threadIdx.x;
  const UnitAppend4 ap = unit_append(p.a, Hkv, u, false);
  const int old = ap.n0 % kQB;
  if (j >= (old + ap.add) / kQB) return;
  const int to = p.a.tab[(long long)u * p.a.max_blocks + ap.n0 / kQB + j];
  if (to < 0 || (long long)to >= p.a.n_units) {
    if (tid == 0) quant_flag(p.a.status, kQErrIndex);
    return;
  }
  uint8_t* unit = p.a.units + (long long)to * quant4_unit_bytes(D);
  const T* tail = reinterpret_cast<const T*>(p.a.tail + u * payload);
  const int first = j * kQB - old;  // the block's first token among the new ones, or before them
  if (tid < kQB) {
    float e = 0.f;
    if (first + tid < 0)
      e = reinterpret_cast<const float*>(tail + 2 * kQB * D)[tid];
    else if (p.a.e != nullptr)
      e = p.a.e[((long long)b * p.a.n + first + tid) * Hkv + h];
    e_s[tid] = e;
    reinterpret_cast<float*>(unit + quant4_e_off(D))[tid] = e;
  }
  for (int part = 0; part < 2; ++part) {
    const bool key = part == 0;
    const int groups = key ? D : kQB * D / 64;  // channels, or runs of 64 dims of a token
    if (tid == 0) amax_s = 0;
    __syncthreads();
    unsigned mx = 0;
    for (int i = tid; i < kQB * D; i += kThreads) {
      const int t = i / D, x = i % D;
      const T y = first + t < 0 ? tail[tail_at<T, D>(key, t, x)] : new_element<T>(p, key, b, h, first + t, x);
      x_s[t][x] = y;
      if (e_s[t] != -INFINITY) mx = max(mx, __float_as_uint(to_f32(y)) & 0x7FFFFFFFu);
    }
    atomicMax(&amax_s, mx);
    __syncthreads();
    const unsigned top = amax_s;
    const bool bad = top >= 0x7F800000u, none = top < 0x0D800000u;  // not finite; below 2^-100
    const float inv = none || bad ? 0.f : __uint_as_float((256u - (top >> 23)) << 23);
    if (tid == 0)
      reinterpret_cast<float*>(unit + quant4_e_off(D))[kQB + part] =
          bad ? __uint_as_float(0x7FC00000u) : none ? 0.f : __uint_as_float(((top >> 23) - 2) << 23);
    if (tid < groups) {
      float lo = INFINITY, hi = -INFINITY;
      for (int i = 0; i < 64; ++i) {
        const int t = key ? i : tid % kQB, x = key ? tid : tid / kQB * 64 + i;
        if (e_s[t] == -INFINITY) continue;
        const float y = to_f32(x_s[t][x]) * inv;
        lo = fminf(lo, y);
        hi = fmaxf(hi, y);
      }
      unsigned short z = 0, s = 0;
      if (!bad && !none && lo <= hi) {
        z = __half_as_ushort(__float2half_rd(lo));
        s = __half_as_ushort(__float2half_ru(__fmul_rn(__fsub_rn(hi, half_bits(z)), 1.f / 15.f)));
        if (key) s = (s + 0xFF) & 0xFF00;
      }
      zero_s[tid] = half_bits(z);
      step_s[tid] = half_bits(s);
      if (key) {
        unit[quant4_kstep_off(D) + quant4_order(tid, D)] = s >> 8;
        reinterpret_cast<unsigned short*>(unit + quant4_kzero_off(D))[quant4_order(tid, D)] = z;
      } else {
        const int at = tid / kQB * kQB + quant4_order(tid % kQB, kQB);
        reinterpret_cast<unsigned short*>(unit + quant4_vstep_off(D))[at] = s;
        reinterpret_cast<unsigned short*>(unit + quant4_vzero_off(D))[at] = z;
      }
    }
    __syncthreads();
    // a thread has words of eight codes: it looks for the codes that belong there
    for (int i = tid; i < 8 * D; i += kThreads) {
      const int m = i / 128, lane = i / 4 % 32, w = i % 4, g = lane / 4, c = lane % 4;
      uint32_t word = 0;
      for (int k = 0; k < 8; ++k) {
        const int half = k % 2, i4 = k / 4 + k / 2 % 2 * 2;
        const int t = 16 * w + (key ? 4 * (g / 2) + g % 2 + 2 * half : 4 * c + i4);
        const int x = 16 * m + (key ? 4 * c + i4 : g + 8 * half);
        const int grp = key ? x : x / 64 * kQB + t;
        const float s = step_s[grp];
        if (e_s[t] == -INFINITY || !(s > 0.f)) continue;
        const float y = __fsub_rn(to_f32(x_s[t][x]) * inv, zero_s[grp]);
        word |= (uint32_t)(int)(fmaf(y, __frcp_rn(s), 12582912.f) - 12582912.f) << (4 * k);
      }
      reinterpret_cast<uint32_t*>(unit + part * 32 * D)[i] = word;
    }
    __syncthreads();
  }
  if (tid < 6) reinterpret_cast<uint32_t*>(unit + quant4_e_off(D))[kQB + 2 + tid] = 0;
}

// The units' tails and lengths.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) quant4_tail_kernel(Q4AppendArgs p, int Hkv, long long payload) {
  const int u = blockIdx.x, b = u / Hkv, h = u % Hkv, tid = threadIdx.x;
  const UnitAppend4 ap = unit_append(p.a, Hkv, u, tid == 0);
  __syncthreads();  // every thread has the length
  const int old = ap.n0 % kQB, done = (old + ap.add) / kQB;
  const int first = done > 0 ? 0 : old, left = old + ap.add - done * kQB;
  T* tail = reinterpret_cast<T*>(p.a.tail + u * payload);
  for (int i = tid; i < (left - first) * D; i += kThreads) {
    const int r = first + i / D, x = i % D, tok = done * kQB + r - old;
    tail[tail_at<T, D>(true, r, x)] = new_element<T>(p, true, b, h, tok, x);
    tail[tail_at<T, D>(false, r, x)] = new_element<T>(p, false, b, h, tok, x);
  }
  float* te = reinterpret_cast<float*>(tail + 2 * kQB * D);
  for (int r = first + tid; r < left; r += kThreads)
    te[r] = p.a.e != nullptr ? p.a.e[((long long)b * p.a.n + (long long)done * kQB + r - old) * Hkv + h] : 0.f;
  if (tid == 0) p.a.lens_out[u] = p.a.lens[u] + ap.add;
}

template <typename T, int D>
cudaError_t append_variant(const Shape& s, const Q4AppendArgs& a, cudaStream_t stream) {
  const int most = (int)std::min<long long>((a.a.n + kQB - 1LL) / kQB, a.a.max_blocks);
  if (most > 0) quant4_blocks_kernel<T, D><<<dim3(s.U, most), kThreads, 0, stream>>>(a, s.Hkv, s.payload);
  quant4_tail_kernel<T, D><<<s.U, kThreads, 0, stream>>>(a, s.Hkv, s.payload);
  return cudaGetLastError();
}

// Blocks read back: a CTA per block. Masked tokens are zeros.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) quant4_read_kernel(Q4ReadArgs p) {
  for (long long n = blockIdx.x; n < p.n; n += gridDim.x) {
    const long long at = p.ids != nullptr ? p.ids[n] : n;
    if (at < 0 || at >= p.n_units) {
      if (threadIdx.x == 0) quant_flag(p.status, kQErrIndex);
      continue;
    }
    const uint8_t* unit = p.units + at * quant4_unit_bytes(D);
    const float* e = reinterpret_cast<const float*>(unit + quant4_e_off(D));
    for (int i = threadIdx.x; i < kQB * D; i += kThreads) {
      const int t = i / D, x = i % D, kb = quant4_k_bit(t, x), vb = quant4_v_bit(t, x);
      const int ko = quant4_order(x, D), vo = x / 64 * kQB + quant4_order(t, kQB);
      const int kc = unit[kb / 8] >> (kb % 8) & 15, vc = unit[32 * D + vb / 8] >> (vb % 8) & 15;
      const float ks = half_bits(unit[quant4_kstep_off(D) + ko] << 8), kz = half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_kzero_off(D))[ko]);
      const float vs = half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_vstep_off(D))[vo]);
      const float vz = half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_vzero_off(D))[vo]);
      const bool live = e[t] != -INFINITY;
      if (p.k != nullptr) static_cast<T*>(p.k)[n * kQB * D + i] = from_f32<T>(live ? fmaf(ks, (float)kc, kz) * e[kQB] : 0.f);
      if (p.v != nullptr) static_cast<T*>(p.v)[n * kQB * D + i] = from_f32<T>(live ? fmaf(vs, (float)vc, vz) * e[kQB + 1] : 0.f);
    }
    if (p.e != nullptr && threadIdx.x < kQB) p.e[n * kQB + threadIdx.x] = e[threadIdx.x];
  }
}

template <typename T, int D>
cudaError_t read_variant(const Q4ReadArgs& a, cudaStream_t stream) {
  if (a.n > 0) quant4_read_kernel<T, D><<<(int)std::min<long long>(a.n, 1 << 20), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
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
