// Rotation of query and key rows by their positions.
//
// Every row is read and written once, so HBM bounds a prompt; the table's rows are shared by
// a token's heads. A thread has one chunk (eight pairs) of up to HPT heads of a token, whose
// angles it loads once; its loads of all heads are in flight together. Small CTAs come and go
// one by one, which keeps reads and writes mixed: 4 x 8192 tokens of 40 heads of 128 in bf16
// (671 MB), us by threads of a CTA: 256 144, 128 111, 64 110, 32 101 = 99 % of the measured copy
// rate (fp32: 213, 216, 197, 198); 1500 tokens, where launching counts: 64 5.8, 32 7.2. Heads of a
// thread, at 256 threads: 1 161, 2 135, 4 144, 5 129. A token of 32 requests: 2.3 us, latency.
#include "k_quant.cuh"
#include "k_rope.cuh"

#include <algorithm>

namespace nosa {
namespace {

constexpr int kRotateFew = 512, kRotateMany = 64;  // threads of a CTA, at most

template <typename T, int HPT>
__global__ void __launch_bounds__(HPT == 1 ? kRotateFew : kRotateMany, HPT == 1 ? 1 : 10) rotate_kernel(RotateArgs p, int chunks, int groups, int tokens, int same) {
  griddep_wait();
  griddep_launch_dependents();
  const int heads = p.heads[0] + p.heads[1], per = groups * chunks;  // threads of a token
  for (int id = threadIdx.x; id < tokens * per; id += blockDim.x) {
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
      rope_angles(p.rope, rope_axes(p.rope, i), p.rope.pos + at, i, cs);
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
cudaError_t rotate_variant(const Shape& s, const RotateArgs& a, int full, cudaStream_t stream) {
  const int heads = a.heads[0] + a.heads[1], chunks = s.d / 16, groups = (heads + HPT - 1) / HPT, per = groups * chunks;
  const int tokens = std::max(1, full / per);
  const int threads = std::min(HPT == 1 ? kRotateFew : full, (tokens * per + 31) / 32 * 32);
  int same = 0;  // in place: rows behind the turned dims stay
  for (int i = 0; i < 2; ++i) same |= (a.in[i] == a.out[i]) << i;
  const long long grid = (a.rows + tokens - 1) / tokens;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_dependent(rotate_kernel<T, HPT>, dim3((unsigned)grid), threads, 0, stream, a, chunks, groups, tokens, same);
}

}  // namespace

cudaError_t launch_rotate(const Shape& s, const RotateArgs& a, cudaStream_t stream) {
  const int heads = a.heads[0] + a.heads[1];
  if (a.rows * heads == 0) return cudaSuccess;
  // Few chunks: a thread for each head. Chunks, us by threads for each head (several heads a thread), 40 heads
  // of 128: 10 000 2.0 (2.8), 50 000 2.5 (2.8), 77 000 3.0 (2.9), 100 000 3.2 (3.2), 150 000 4.7 (4.2), 400 000 8.8
  // (6.2); 8 heads of 128 and 24 of 64 cross there too.
  const long long work = a.rows * heads * (s.d / 16);
  const bool few = work <= 152 * 512;
  const int full = few ? 256 : work <= 4 << 20 ? kRotateMany : kRotateMany / 2;
  if (s.dtype == 0) return few ? rotate_variant<float, 1>(s, a, full, stream) : rotate_variant<float, 2>(s, a, full, stream);
  if (few) return rotate_variant<__nv_bfloat16, 1>(s, a, full, stream);
  // Four heads a thread, or five where that saves the warps a round: one of 32 threads takes 32 / per tokens, or a
  // token in several rounds. us (four heads, five) for 270 MB, of d = 128 5 heads 55 46, 8 47 48, 9 60 48, 16 47 47, 20
  // 62 45, 24 55 57, 25 50 59, 32 46 47, 36 63 44, 40 58 44, 48 51 55, 64 44 48 and, against the rule, 60 46 49; of d = 64
  // 9 52 48, 32 46 51, 36 67 47, 40 61 44, 64 45 51 and, against it, 24 54 48, 25 53 47.
  const auto rounds = [&](int heads_each) {  // of 32 tokens
    const int per = (heads + heads_each - 1) / heads_each * (s.d / 16);
    return per <= 32 ? 32 / (32 / per) : (per + 31) / 32 * 32;
  };
  return rounds(5) < rounds(4) ? rotate_variant<__nv_bfloat16, 5>(s, a, full, stream) : rotate_variant<__nv_bfloat16, 4>(s, a, full, stream);
}

}  // namespace nosa
