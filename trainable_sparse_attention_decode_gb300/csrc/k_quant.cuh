// 8-bit block cache: unit layout and kernel parameters shared by k_quant_cache.cu
// (append, eviction), k_quant_attn.cu (attention) and the entry points in
// nosa_quant.cu.
//
// A unit holds 64 tokens of one KV head: keys and values as e4m3 codes that stand
// for code * scale (one scale for the keys, one for the values), and the tokens'
// fp32 eviction logits. The codes are stored in the order in which the lanes of a
// warp need them as the A operand of a 16 x 16 matrix product (tokens x dims for
// the keys, dims x tokens for the values): each lane reads its part of a 16-token
// slice with 16-byte loads that are consecutive over the lanes, and one 4-byte
// word converts to two operand registers. Slices follow one another, so a warp
// that owns one slice reads one contiguous run (K then V). include/nosa.h states
// the offsets; the functions below are their only other statement.
#pragma once

#include "nosa_internal.cuh"

namespace nosa {

constexpr int kQB = 64;             // tokens of a block
constexpr int kQMaxBlocks = 16384;  // table entries per unit (eviction holds a row in shared memory)
constexpr int kQMaxQueries = 128;   // query tokens of one attention call

// Device status bits (nosa.h, NOSA_QUANT_*).
enum : int { kQErrWait = 1, kQErrIndex = 2, kQErrCapacity = 4 };

__host__ __device__ constexpr int quant_e_off(int d) { return 2 * kQB * d; }
__host__ __device__ constexpr int quant_scale_off(int d) { return 2 * kQB * d + 4 * kQB; }
__host__ __device__ constexpr int quant_unit_bytes(int d) { return (quant_scale_off(d) + 8 + 31) / 32 * 32; }

// Byte offset of the key code (token t, dim x) in a unit of head dimension d.
__host__ __device__ constexpr int quant_k_off(int t, int x, int d) {
  const int tt = t % 16, g = 2 * (tt / 4) + tt % 2, half = tt % 4 / 2;
  return t / 16 * 32 * d + (x / 32 * 32 + g * 4 + x % 16 / 4) * 16 + (x % 32 / 16 * 2 + half) * 4 + x % 4;
}
// ... and of the value code.
__host__ __device__ constexpr int quant_v_off(int t, int x, int d) {
  const int tt = t % 16;
  return t / 16 * 32 * d + 16 * d + (x / 32 * 32 + x % 8 * 4 + tt / 4) * 16 + (x % 32 / 8) * 4 + tt % 4;
}

struct QStrides {
  long long b, t, h;  // elements between requests, tokens, heads
};

struct QAppendArgs {
  const void* k;
  const void* v;
  const float* e;  // [batch][n][Hkv] or null (zeros)
  QStrides ks, vs;
  int n;                 // token positions per request
  const int32_t* n_new;  // [batch] valid ones, or null (all n)
  uint8_t* units;
  long long n_units;
  const int32_t* tab;  // [U][max_blocks]
  int max_blocks;
  uint8_t* tail;
  const int32_t* lens;  // [U]
  int32_t* lens_out;    // [U], may be lens
  int* status;          // or null
};

struct QEvictArgs {
  int max_blocks, budget, n_recent;
  const int32_t* tab;
  const float* mass;
  const int32_t* lens;
  int32_t* tab_out;
  float* mass_out;
  int32_t* lens_out;
  int32_t* order;  // or null
  int* status;
};

struct QAttnArgs {
  const uint8_t* units;
  long long n_units;
  const int32_t* tab;
  int max_blocks;
  const uint8_t* tail;
  const int32_t* lens;
  const void* q;
  QStrides qs;
  int T;                 // query positions per request
  const int32_t* q_len;  // [batch] valid ones, or null (all T)
  void* out;             // [batch][T][Hq][d]
  float* lse;            // [batch][T][Hq] or null
  float* mass;           // [U][max_blocks] or null
  float decay;
  uint8_t* ws;
  bool give_up;  // a test's: every wait gives up at once
  bool turned;   // q was written by the launch before (see quant_stream_kernel)
  int* status;
};

int quant_sm_count();  // of the current device
cudaError_t launch_quant_append(const Shape& s, const QAppendArgs& a, cudaStream_t stream);
cudaError_t launch_quant_evict(const Shape& s, const QEvictArgs& a, cudaStream_t stream);
size_t quant_attn_workspace(const Shape& s, int max_blocks, int T, bool mass);
cudaError_t launch_quant_attention(const Shape& s, const QAttnArgs& a, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ void quant_flag(int* status, int bit) {
  if (status != nullptr) atomicOr(status, bit);
}
// Tokens of unit u: lens[u], or -1 (flagged by `flag`) where it is not a length of this cache.
// EARLY: read before the kernel's own griddep_wait (see launch_dependent).
template <bool EARLY = false>
__device__ __forceinline__ int quant_len(const int32_t* lens, int u, int max_blocks, int* status, bool flag) {
  const int n = EARLY ? __ldcg(lens + u) : lens[u];
  if (n >= 0 && n <= kQB * max_blocks) return n;
  if (flag) quant_flag(status, kQErrIndex);
  return -1;
}
// Valid new tokens of request b out of n.
template <bool EARLY = false>
__device__ __forceinline__ int quant_count(const int32_t* count, int b, int n, int* status, bool flag) {
  if (count == nullptr) return n;
  const int c = EARLY ? __ldcg(count + b) : count[b];
  if (c >= 0 && c <= n) return c;
  if (flag) quant_flag(status, kQErrIndex);
  return c < 0 ? 0 : n;
}

// Launches `kernel` so that it may become resident while the one before it in the
// stream still runs. Every kernel of the cache is launched so, and each of its CTAs
// calls griddep_wait before it ends: where a kernel has ended, all before it have.
// The first kernel of a call waits before it reads anything and only then lets its
// successor start (griddep_launch_dependents), so that a successor inside the call may
// read, before its own wait, what was there before the call: a wait returns when all that
// came before has been performed in the device's memory, that is, in L2, and no CTA of the
// successor starts before every CTA of the first kernel has come past its wait. Only a
// copy that an earlier kernel left in the SM's L1 could be older, so such reads go past L1
// (__ldcg). Nothing that the call itself writes is read early, but for a weight by the one
// thread that then writes it.
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
#endif

}  // namespace nosa
