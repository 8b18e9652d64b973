// Rotation of query and key rows by their positions.
#include "k_rope.cuh"

namespace nosa {
namespace {

constexpr int kRotateThreads = 256;

// A thread has a pair of a row, or two elements behind the rotated ones.
template <typename T>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(RotateArgs p, int d) {
  const int heads = p.heads[0] + p.heads[1];
  const long long total = p.rows * heads * (d / 2);
  for (long long i = blockIdx.x * (long long)kRotateThreads + threadIdx.x; i < total; i += (long long)gridDim.x * kRotateThreads) {
    const int x = (int)(i % (d / 2));
    const long long row = i / (d / 2);
    const int hh = (int)(row % heads), w = hh >= p.heads[0], h = hh - w * p.heads[0];
    const long long at = row / heads, b = at / p.n, t = at % p.n;
    const T* src = static_cast<const T*>(p.in[w]) + b * p.in_b[w] + t * p.in_t[w] + h * p.in_h[w];
    T* dst = static_cast<T*>(p.out[w]) + b * p.out_b[w] + t * p.out_t[w] + h * p.out_h[w];
    if (x >= p.rope.pairs) {
      dst[2 * x] = src[2 * x];
      dst[2 * x + 1] = src[2 * x + 1];
      continue;
    }
    const int x0 = p.rope.interleaved ? 2 * x : x, x1 = p.rope.interleaved ? 2 * x + 1 : x + p.rope.pairs;
    float2 cs = rope_angle(p.rope, at, x);
    if (p.backward) cs.y = -cs.y;
    const float a = to_f32(src[x0]), c = to_f32(src[x1]);
    dst[x0] = from_f32<T>(rope_turn(a, c, true, cs));
    dst[x1] = from_f32<T>(rope_turn(c, a, false, cs));
  }
}

}  // namespace

cudaError_t launch_rotate(const Shape& s, const RotateArgs& a, cudaStream_t stream) {
  const long long total = a.rows * (a.heads[0] + a.heads[1]) * (s.d / 2);
  if (total == 0) return cudaSuccess;
  const long long want = (total + kRotateThreads - 1) / kRotateThreads;
  const int grid = (int)(want < 152 * 16 ? want : 152 * 16);
  if (s.dtype == 0)
    rotate_kernel<float><<<grid, kRotateThreads, 0, stream>>>(a, s.d);
  else
    rotate_kernel<__nv_bfloat16><<<grid, kRotateThreads, 0, stream>>>(a, s.d);
  return cudaGetLastError();
}

}  // namespace nosa
