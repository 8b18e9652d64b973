// 4-bit block cache: unit layout and kernel parameters shared by k_quant4_cache.cu (append,
// reading back), the attention and the entry points in nosa_quant4.cu.
//
// A unit holds 64 tokens of one KV head as codes n in 0..15 that stand for
// (step * n + zero) * scale: keys with a step and a zero per channel (dim), because the
// channels of keys differ in size and offset, values with a step and a zero per token and
// run of 64 dims, and one scale, a power of two, for the keys and one for the values, which
// brings the block's largest magnitude to [4, 8) so that 16 bits hold steps and zeros.
// The steps of keys have three significant bits (the format of 5 exponent and 2 mantissa
// bits): their product with a bf16 query element (8 bits) is exact in fp16, so the attention
// scales the queries of a block once and its logits keep fp32's precision.
//
// The codes lie in the order in which the lanes of a warp need them as the A operand of a
// 16 x 16 matrix product (tokens x dims for the keys, dims x tokens for the values): one
// 32-bit word has a lane's four operand registers of two codes each, and the words of the
// block's four 16-token slices are one 16-byte load. A code under a mask is a subnormal fp16
// number (2^-24 n, or 2^-20 n four bits further up): no conversion. include/nosa.h states
// the offsets; the functions below are their only other statement.
#pragma once

#include "k_quant.cuh"
#include "k_rope.cuh"

#include <cuda_fp16.h>

namespace nosa {

__host__ __device__ constexpr int quant4_kstep_off(int d) { return 64 * d; }   // e5m2 bytes [d]
__host__ __device__ constexpr int quant4_kzero_off(int d) { return 65 * d; }   // fp16 [d]
__host__ __device__ constexpr int quant4_vstep_off(int d) { return 67 * d; }   // fp16 [d / 64][64]
__host__ __device__ constexpr int quant4_vzero_off(int d) { return 69 * d; }
__host__ __device__ constexpr int quant4_e_off(int d) { return 71 * d; }       // fp32 [64], then the two scales
__host__ __device__ constexpr int quant4_unit_bytes(int d) { return (71 * d + 4 * kQB + 8 + 31) / 32 * 32; }

// Code (token t, dim x) of the keys as 8 * (byte of its word) + 4 * (nibble of the word).
__host__ __device__ constexpr int quant4_k_bit(int t, int x) {
  const int tt = t % 16, g = 2 * (tt / 4) + tt % 2, half = tt % 4 / 2, i = x % 4;
  return 8 * (512 * (x / 16) + 16 * (4 * g + x % 16 / 4) + 4 * (t / 16)) + 4 * (half + 2 * (i / 2) + 4 * (i % 2));
}
// ... and of the values (from the start of the value codes, 32 d bytes on).
__host__ __device__ constexpr int quant4_v_bit(int t, int x) {
  const int i = t % 4;
  return 8 * (512 * (x / 16) + 16 * (4 * (x % 8) + t % 16 / 4) + 4 * (t / 16)) + 4 * (x % 16 / 8 + 2 * (i / 2) + 4 * (i % 2));
}
// Index of channel x among d steps (or zeros), of token t among a run's 64: what a lane
// needs of them is consecutive.
__host__ __device__ constexpr int quant4_order(int x, int n) { return 4 * (x % 16 / 4 * (n / 16) + x / 16) + x % 4; }

struct Q4AppendArgs {
  QAppendArgs a;
  RopeArgs rope;
  int wide;  // v's rows start on 32-byte boundaries
};
struct Q4ReadArgs {
  const uint8_t* units;
  long long n_units;
  const int32_t* ids;  // [n] or null: 0, 1, ...
  long long n;
  void* k;             // [n][64][d] or null
  void* v;
  float* e;            // [n][64] or null
  int* status;
};
cudaError_t launch_quant4_append(const Shape& s, const Q4AppendArgs& a, cudaStream_t stream);
cudaError_t launch_quant4_read(const Shape& s, const Q4ReadArgs& a, cudaStream_t stream);
size_t quant4_attn_workspace(const Shape& s, int max_blocks, int T, bool mass);
cudaError_t launch_quant4_attention(const Shape& s, const QAttnArgs& a, const RopeArgs& rope, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ float half_bits(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }

// Keys (token t, dims x .. x + 3) and values (tokens t .. t + 3, dim x) of a unit, without
// the block's scale; x (t) a multiple of 4.
template <int D>
__device__ __forceinline__ void quant4_keys(const uint8_t* unit, int t, int x, float* f) {
  const int bit = quant4_k_bit(t, x), o = quant4_order(x, D);  // (nibbles 0, 4, 2, 6 from there)
  const uint32_t w = *reinterpret_cast<const uint32_t*>(unit + bit / 32 * 4) >> (bit % 32);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = fmaf(half_bits(unit[quant4_kstep_off(D) + o + i] << 8), (float)(w >> (16 * (i % 2) + 8 * (i / 2)) & 15),
                half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_kzero_off(D))[o + i]));
}
template <int D>
__device__ __forceinline__ void quant4_values(const uint8_t* unit, int t, int x, float* f) {
  const int bit = quant4_v_bit(t, x), o = x / 64 * kQB + quant4_order(t, kQB);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(unit + 32 * D + bit / 32 * 4) >> (bit % 32);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = fmaf(half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_vstep_off(D))[o + i]),
                (float)(w >> (16 * (i % 2) + 8 * (i / 2)) & 15),
                half_bits(reinterpret_cast<const unsigned short*>(unit + quant4_vzero_off(D))[o + i]));
}
#endif

}  // namespace nosa
