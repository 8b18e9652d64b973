// Entry points of the 8-bit block cache: argument checks and launches. The
// kernels live in k_quant_cache.cu and k_quant_attn.cu.
#include "nosa_checks.h"

using namespace nosa;

extern "C" {

size_t nosa_quant_unit_bytes(const nosa_config* cfg) {
  return nosa_config_validate(cfg, nullptr, 0) == NOSA_OK ? quant_unit_bytes(cfg->head_dim) : 0;
}

nosa_status nosa_quant_append(const nosa_config* cfg, int32_t max_blocks, int32_t n_tokens, const void* k,
                              const int64_t* k_strides, const void* v, const int64_t* v_strides, const float* e,
                              const int32_t* n_new, void* units, int64_t n_units, const int32_t* block_tab, void* tail,
                              const int32_t* lens, int32_t* lens_out, int32_t* status, void* stream) {
  nosa_status st = check_cache(cfg, max_blocks);
  if (st != NOSA_OK) return st;
  const Shape s = quant_shape(*cfg);
  QAppendArgs a{};
  if ((st = take_append(s, max_blocks, n_tokens, k, k_strides, v, v_strides, e, n_new, units, n_units, block_tab, tail, lens,
                        lens_out, status, a)) != NOSA_OK)
    return st;
  DeviceGuard guard(cfg->device);
  return launched(launch_quant_append(s, a, static_cast<cudaStream_t>(stream)), "quantising append");
}

size_t nosa_quant_attention_workspace_bytes(const nosa_config* cfg, int32_t max_blocks, int32_t n_queries,
                                            int32_t with_mass) {
  if (check_cache(cfg, max_blocks) != NOSA_OK || n_queries < 1 || n_queries > kQMaxQueries) return 0;
  DeviceGuard guard(cfg->device);
  return quant_attn_workspace(quant_shape(*cfg), max_blocks, n_queries, with_mass != 0);
}

nosa_status nosa_quant_attention(const nosa_config* cfg, int32_t max_blocks, int32_t n_queries, const void* units,
                                 int64_t n_units, const int32_t* block_tab, const void* tail, const int32_t* lens,
                                 const void* q, const int64_t* q_strides, const int32_t* q_len, void* out, float* lse,
                                 float* mass, float decay, void* workspace, size_t workspace_bytes, int32_t* status,
                                 void* stream) {
  nosa_status st = check_cache(cfg, max_blocks);
  if (st != NOSA_OK) return st;
  const Shape s = quant_shape(*cfg);
  QAttnArgs a{};
  if ((st = take_attention(s, max_blocks, n_queries, units, n_units, block_tab, tail, lens, q, q_strides, q_len, out, lse, mass,
                           decay, workspace, status, a)) != NOSA_OK)
    return st;
  DeviceGuard guard(cfg->device);
  if (workspace_bytes < quant_attn_workspace(s, max_blocks, n_queries, mass != nullptr))
    return invalid("workspace too small (see nosa_quant_attention_workspace_bytes)");
  return launched(launch_quant_attention(s, a, static_cast<cudaStream_t>(stream)), "8-bit cache attention");
}

nosa_status nosa_quant_evict(const nosa_config* cfg, int32_t max_blocks, int32_t budget, int32_t n_recent,
                             const int32_t* block_tab, const float* mass, const int32_t* lens, int32_t* tab_out,
                             float* mass_out, int32_t* lens_out, int32_t* order, int32_t* status, void* stream) {
  const nosa_status st = check_cache(cfg, max_blocks);
  if (st != NOSA_OK) return st;
  if (budget < 1 || n_recent < 0 || n_recent > budget) return invalid("need budget >= 1 and 0 <= n_recent <= budget");
  if (!block_tab || !mass || !lens || !tab_out || !mass_out || !lens_out) return invalid("NULL argument");
  if (!aligned_to(block_tab, 4) || !aligned_to(mass, 4) || !aligned_to(lens, 4) || !aligned_to(tab_out, 4) ||
      !aligned_to(mass_out, 4) || !aligned_to(lens_out, 4) || !aligned_to(order, 4) || !aligned_to(status, 4))
    return invalid("misaligned pointer");
  QEvictArgs a{};
  a.max_blocks = max_blocks;
  a.budget = budget;
  a.n_recent = n_recent;
  a.tab = block_tab;
  a.mass = mass;
  a.lens = lens;
  a.tab_out = tab_out;
  a.mass_out = mass_out;
  a.lens_out = lens_out;
  a.order = order;
  a.status = status;
  DeviceGuard guard(cfg->device);
  return launched(launch_quant_evict(quant_shape(*cfg), a, static_cast<cudaStream_t>(stream)), "eviction");
}

}  // extern "C"
