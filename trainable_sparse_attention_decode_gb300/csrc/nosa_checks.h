// Argument checks that the entry points of the block caches and of the rotation share.
#pragma once

#include "nosa.h"
#include "k_quant.cuh"

#include <cstdlib>
#include <cstring>
#include <string>

namespace nosa {

void set_thread_error(const std::string& msg);  // defined with the other entry points

inline nosa_status refuse(nosa_status st, const std::string& why) {
  set_thread_error(why);
  return st;
}
inline nosa_status invalid(const std::string& why) { return refuse(NOSA_ERR_INVALID_ARG, why); }

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline nosa_status check_config(const nosa_config* cfg) {
  char why[256];
  const nosa_status vs = nosa_config_validate(cfg, why, sizeof(why));
  return vs == NOSA_OK ? NOSA_OK : refuse(vs, why);
}

// The checks that every call on a cache makes first: the configuration and the table's width.
inline nosa_status check_cache(const nosa_config* cfg, int32_t max_blocks) {
  const nosa_status vs = check_config(cfg);
  if (vs != NOSA_OK) return vs;
  if (max_blocks < 1) return invalid("max_blocks must be >= 1");
  if (max_blocks > kQMaxBlocks)
    return refuse(NOSA_ERR_UNSUPPORTED, "max_blocks must be <= " + std::to_string(kQMaxBlocks));
  return NOSA_OK;
}

inline Shape quant_shape(const nosa_config& c) {
  Shape s{};
  s.batch = c.batch;
  s.Hq = c.n_q_heads;
  s.Hkv = c.n_kv_heads;
  s.U = c.batch * c.n_kv_heads;
  s.G = c.n_q_heads / c.n_kv_heads;
  s.d = c.head_dim;
  s.B = c.block;
  s.dtype = c.dtype;
  s.elt = c.dtype == NOSA_F32 ? 4 : 2;
  s.payload = (long long)nosa_payload_bytes(&c);
  return s;
}

// Strides (elements) of [batch][n][heads][d]: given, or those of a contiguous array.
// Every row must start on a 16-byte boundary.
inline nosa_status take_strides(const char* name, const int64_t* st, int n, int heads, const Shape& s, QStrides& out) {
  out = QStrides{(long long)n * heads * s.d, (long long)heads * s.d, s.d};
  if (st == nullptr) return NOSA_OK;
  out = QStrides{st[0], st[1], st[2]};
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] % (16 / s.elt) != 0)
      return invalid(std::string(name) + ": strides must be >= 0 and multiples of 16 bytes");
  return NOSA_OK;
}

// What an append and an attention call are given, checked.
inline nosa_status take_append(const Shape& s, int32_t max_blocks, int32_t n_tokens, const void* k, const int64_t* k_strides,
                               const void* v, const int64_t* v_strides, const float* e, const int32_t* n_new, void* units,
                               int64_t n_units, const int32_t* block_tab, void* tail, const int32_t* lens, int32_t* lens_out,
                               int32_t* status, QAppendArgs& a) {
  if (n_tokens < 0) return invalid("n_tokens must be >= 0");
  if (n_units < 0 || (n_units > 0 && !units) || !block_tab || !tail || !lens || !lens_out ||
      (n_tokens > 0 && (!k || !v)))
    return invalid("NULL or negative argument");
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(units, 16) || !aligned_to(tail, 16) ||
      !aligned_to(e, 4) || !aligned_to(n_new, 4) || !aligned_to(block_tab, 4) || !aligned_to(lens, 4) ||
      !aligned_to(lens_out, 4) || !aligned_to(status, 4))
    return invalid("misaligned pointer (k, v, units, tail 16 bytes)");
  nosa_status st;
  if ((st = take_strides("k", k_strides, n_tokens, s.Hkv, s, a.ks)) != NOSA_OK) return st;
  if ((st = take_strides("v", v_strides, n_tokens, s.Hkv, s, a.vs)) != NOSA_OK) return st;
  a.k = k;
  a.v = v;
  a.e = e;
  a.n = n_tokens;
  a.n_new = n_new;
  a.units = static_cast<uint8_t*>(units);
  a.n_units = n_units;
  a.tab = block_tab;
  a.max_blocks = max_blocks;
  a.tail = static_cast<uint8_t*>(tail);
  a.lens = lens;
  a.lens_out = lens_out;
  a.status = status;
  return NOSA_OK;
}

// NOSA_INJECT_FAIL=wait: the attention's waits give up at once (a test hook, read at every
// call; no GPU fault is involved).
inline bool inject_wait() {
  const char* g = std::getenv("NOSA_INJECT_FAIL");
  return g != nullptr && std::strcmp(g, "wait") == 0;
}

inline nosa_status take_attention(const Shape& s, int32_t max_blocks, int32_t n_queries, const void* units, int64_t n_units,
                                  const int32_t* block_tab, const void* tail, const int32_t* lens, const void* q,
                                  const int64_t* q_strides, const int32_t* q_len, void* out, float* lse, float* mass,
                                  float decay, void* workspace, int32_t* status, QAttnArgs& a) {
  if (n_queries < 1) return invalid("n_queries must be >= 1");
  if (n_queries > kQMaxQueries)
    return refuse(NOSA_ERR_UNSUPPORTED, "n_queries must be <= " + std::to_string(kQMaxQueries));
  if (n_units < 0 || (n_units > 0 && !units) || !block_tab || !tail || !lens || !q || !out || !workspace)
    return invalid("NULL or negative argument");
  if (q == out) return invalid("out must not be q");
  if (mass && !(decay >= 0.f && decay <= 1.f)) return invalid("decay must be in [0, 1]");
  if (!aligned_to(units, 16) || !aligned_to(tail, 16) || !aligned_to(q, 16) || !aligned_to(out, 16) ||
      !aligned_to(workspace, 256) || !aligned_to(block_tab, 4) || !aligned_to(lens, 4) || !aligned_to(q_len, 4) ||
      !aligned_to(lse, 4) || !aligned_to(mass, 4) || !aligned_to(status, 4))
    return invalid("misaligned pointer (units, tail, q, out 16 bytes; workspace 256 bytes)");
  const nosa_status st = take_strides("q", q_strides, n_queries, s.Hq, s, a.qs);
  if (st != NOSA_OK) return st;
  a.max_blocks = max_blocks;
  a.units = static_cast<const uint8_t*>(units);
  a.n_units = n_units;
  a.tab = block_tab;
  a.tail = static_cast<const uint8_t*>(tail);
  a.lens = lens;
  a.q = q;
  a.T = n_queries;
  a.q_len = q_len;
  a.out = out;
  a.lse = lse;
  a.mass = mass;
  a.decay = decay;
  a.ws = static_cast<uint8_t*>(workspace);
  a.give_up = inject_wait();
  a.status = status;
  return NOSA_OK;
}

inline nosa_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return NOSA_OK;
  cudaGetLastError();  // (reported here)
  return refuse(NOSA_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
}

}  // namespace nosa
