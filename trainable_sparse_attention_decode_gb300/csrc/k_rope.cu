// Rotation of query and key rows by their positions.
//
// Every row is read and written once, so HBM bounds a prompt; the table's rows are shared by
// a token's heads. A thread has one chunk (eight pairs) of up to HPT heads of a token, whose
// angles it loads once; its loads of all heads are in flight together.
#include "k_quant.cuh"
#include "k_rope.cuh"

namespace nosa {
namespace {

constexpr int kRotateThreads = 256;

template <typename T, int HPT>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(RotateArgs p, int chunks, int groups, int tokens, int same) {
  griddep_wait();
  griddep_launch_dependents();
  const int heads = p.heads[0] + p.heads[1], per = groups * chunks;  // threads of a token
  for (int id = threadIdx.x; id < tokens * per; id += kRotateThreads) {
    const long long at = (long long)blockIdx.x * tokens + id / per;
    if (at >= p.rows) break;
    const int g = id % per / chunks, i = id % chunks;
    const long long b = at < 0x7FFFFFFF ? (unsigned)at / (unsigned)p.n : at / p.n, t = at - b * p.n;
    if (p.count != nullptr && t >= p.count[b]) continue;
    const RopeChunk ch = rope_chunk(p.rope, i);
    Vec8<T> v[HPT][2];
    const T* src[HPT];
    long long to[HPT];
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
      const int hh = g + k * groups, w = hh >= p.heads[0], h = hh - (w ? p.heads[0] : 0);
      src[k] = nullptr;
      to[k] = 0;
      if (hh < heads && (ch.turned || !(same >> w & 1))) {
        src[k] = static_cast<const T*>(p.in[w]) + b * p.in_b[w] + t * p.in_t[w] + h * p.in_h[w];
        to[k] = b * p.out_b[w] + t * p.out_t[w] + h * p.out_h[w];
        v[k][0].load(src[k] + ch.lo);
        v[k][1].load(src[k] + ch.hi);
      }
    }
    float2 cs[8];
    if (ch.turned) {
      rope_angles<false>(p.rope, at, i, cs);
      if (p.backward) {
#pragma unroll
        for (int k = 0; k < 8; ++k) cs[k].y = -cs[k].y;
      }
    }
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
      if (src[k] == nullptr) continue;
      const int w = g + k * groups >= p.heads[0];
      if (ch.turned) {
        float x[16];
        v[k][0].get(x);
        v[k][1].get(x + 8);
        rope_turn_chunk(p.rope.interleaved, cs, x);
        v[k][0].set(x);
        v[k][1].set(x + 8);
      }
      T* dst = static_cast<T*>(p.out[w]) + to[k];
      v[k][0].store(dst + ch.lo);
      v[k][1].store(dst + ch.hi);
    }
  }
}

template <typename T, int HPT>
cudaError_t rotate_variant(const Shape& s, const RotateArgs& a, cudaStream_t stream) {
  const int heads = a.heads[0] + a.heads[1], chunks = s.d / 16, groups = (heads + HPT - 1) / HPT, per = groups * chunks;
  const int tokens = per >= kRotateThreads ? 1 : kRotateThreads / per;
  int same = 0;  // in place: rows behind the turned dims stay
  for (int i = 0; i < 2; ++i) same |= (a.in[i] == a.out[i]) << i;
  const long long grid = (a.rows + tokens - 1) / tokens;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_dependent(rotate_kernel<T, HPT>, dim3((unsigned)grid), kRotateThreads, 0, stream, a, chunks, groups, tokens, same);
}

}  // namespace

cudaError_t launch_rotate(const Shape& s, const RotateArgs& a, cudaStream_t stream) {
  const int heads = a.heads[0] + a.heads[1];
  if (a.rows * heads == 0) return cudaSuccess;
  // few rows: a thread for each head, all of them at once
  const bool few = a.rows * heads * (s.d / 16) <= 152LL * 2048;
  if (s.dtype == 0) return few ? rotate_variant<float, 1>(s, a, stream) : rotate_variant<float, 2>(s, a, stream);
  return few ? rotate_variant<__nv_bfloat16, 1>(s, a, stream) : rotate_variant<__nv_bfloat16, 4>(s, a, stream);
}

}  // namespace nosa
