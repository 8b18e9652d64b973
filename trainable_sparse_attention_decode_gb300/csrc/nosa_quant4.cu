// Entry points of the rotation and of the 4-bit block cache: argument checks and launches.
// The kernels live in k_rope.cu, k_quant4_cache.cu and k_quant_attn.cuh.
#include "nosa_checks.h"
#include "k_quant4.cuh"

using namespace nosa;

namespace {

// The rotation that a call was given (NULL: none) as kernels take it.
nosa_status take_rope(const nosa_config& cfg, const nosa_rope* rope, const int32_t* positions, int n, int32_t* status, RopeArgs& out) {
  out = RopeArgs{};
  if (rope == nullptr) return NOSA_OK;
  if (!rope->table || (n > 0 && !positions)) return invalid("the rotation needs a table and positions");
  if (!aligned_to(rope->table, 16) || !aligned_to(positions, 4)) return invalid("misaligned pointer (table 16 bytes, positions 4)");
  if (rope->rot_dim < 16 || rope->rot_dim % 16 != 0 || rope->rot_dim > cfg.head_dim)
    return invalid("rot_dim must be a multiple of 16 in [16, head_dim]");
  if (rope->table_len < 1) return invalid("table_len must be >= 1");
  if (rope->n_axes < 1 || rope->n_axes > kRopeMaxAxes) return invalid("n_axes must be in [1, 4]");
  out.pairs = rope->rot_dim / 2;
  if (rope->axes != nullptr)
    for (int i = 0; i < out.pairs; ++i) {
      if (rope->axes[i] < 0 || rope->axes[i] >= rope->n_axes) return invalid("an axis is not in [0, n_axes)");
      out.axes[i / 16] |= (uint32_t)rope->axes[i] << (2 * (i % 16));
    }
  out.table = reinterpret_cast<const float2*>(rope->table);
  out.pos = positions;
  out.axis_stride = (long long)cfg.batch * n;
  out.len = rope->table_len;
  out.interleaved = rope->interleaved != 0;
  out.wide = aligned_to(rope->table, 32);
  out.status = status;
  return NOSA_OK;
}

}  // namespace

extern "C" {

nosa_status nosa_rotate(const nosa_config* cfg, const nosa_rope* rope, const int32_t* positions, int32_t n_tokens,
                        const void* q, const int64_t* q_strides, void* q_out, const int64_t* q_out_strides,
                        const void* k, const int64_t* k_strides, void* k_out, const int64_t* k_out_strides,
                        int32_t backward, int32_t* status, void* stream) {
  nosa_status st = check_config(cfg);
  if (st != NOSA_OK) return st;
  if (n_tokens < 0) return invalid("n_tokens must be >= 0");
  if (!rope) return invalid("rope is NULL");
  if (!q != !q_out || !k != !k_out) return invalid("q and q_out, k and k_out come together");
  if (!aligned_to(q, 16) || !aligned_to(q_out, 16) || !aligned_to(k, 16) || !aligned_to(k_out, 16) || !aligned_to(status, 4))
    return invalid("misaligned pointer (q, k and their outputs 16 bytes)");
  const Shape s = quant_shape(*cfg);
  RotateArgs a{};
  if ((st = take_rope(*cfg, rope, positions, n_tokens, status, a.rope)) != NOSA_OK) return st;
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int64_t* strides[2][2] = {{q_strides, q_out_strides}, {k_strides, k_out_strides}};
  for (int i = 0; i < 2; ++i) {
    if (in[i] == nullptr) continue;
    const int heads = i ? s.Hkv : s.Hq;
    QStrides x, y;
    if ((st = take_strides(i ? "k" : "q", strides[i][0], n_tokens, heads, s, x)) != NOSA_OK) return st;
    if ((st = take_strides(i ? "k_out" : "q_out", strides[i][1], n_tokens, heads, s, y)) != NOSA_OK) return st;
    if (in[i] == out[i] && (x.b != y.b || x.t != y.t || x.h != y.h)) return invalid("in place, the strides must be the same");
    const int64_t st[3] = {y.b, y.t, y.h}, size[3] = {cfg->batch, n_tokens, heads};
    for (int k = 0; k < 3; ++k)
      if (st[k] == 0 && size[k] > 1) return invalid("an output's stride is 0");
    a.in[i] = in[i];
    a.out[i] = out[i];
    a.heads[i] = heads;
    a.in_b[i] = x.b; a.in_t[i] = x.t; a.in_h[i] = x.h;
    a.out_b[i] = y.b; a.out_t[i] = y.t; a.out_h[i] = y.h;
  }
  a.n = n_tokens;
  a.rows = (long long)cfg->batch * n_tokens;
  a.backward = backward != 0;
  DeviceGuard guard(cfg->device);
  return launched(launch_rotate(s, a, static_cast<cudaStream_t>(stream)), "rotation");
}

size_t nosa_quant4_unit_bytes(const nosa_config* cfg) {
  return nosa_config_validate(cfg, nullptr, 0) == NOSA_OK ? quant4_unit_bytes(cfg->head_dim) : 0;
}

nosa_status nosa_quant4_append(const nosa_config* cfg, int32_t max_blocks, int32_t n_tokens, const void* k,
                               const int64_t* k_strides, const void* v, const int64_t* v_strides, const float* e,
                               const int32_t* n_new, const nosa_rope* rope, const int32_t* positions, void* units,
                               int64_t n_units, const int32_t* block_tab, void* tail, const int32_t* lens,
                               int32_t* lens_out, int32_t* status, void* stream) {
  nosa_status st = check_cache(cfg, max_blocks);
  if (st != NOSA_OK) return st;
  const Shape s = quant_shape(*cfg);
  Q4AppendArgs a{};
  if ((st = take_append(s, max_blocks, n_tokens, k, k_strides, v, v_strides, e, n_new, units, n_units, block_tab, tail, lens,
                        lens_out, status, a.a)) != NOSA_OK)
    return st;
  if ((st = take_rope(*cfg, rope, positions, n_tokens, status, a.rope)) != NOSA_OK) return st;
  const int sector = 32 / s.elt;
  a.wide = aligned_to(v, 32) && a.a.vs.b % sector == 0 && a.a.vs.t % sector == 0 && a.a.vs.h % sector == 0;
  DeviceGuard guard(cfg->device);
  return launched(launch_quant4_append(s, a, static_cast<cudaStream_t>(stream)), "4-bit cache append");
}

nosa_status nosa_quant4_read(const nosa_config* cfg, const void* units, int64_t n_units, const int32_t* ids, int64_t n,
                             void* k_out, void* v_out, float* e_out, int32_t* status, void* stream) {
  const nosa_status st = check_config(cfg);
  if (st != NOSA_OK) return st;
  if (n < 0 || n_units < 0 || (n_units > 0 && !units)) return invalid("NULL or negative argument");
  if (!ids && n > n_units) return invalid("n is more than the units");
  if (!aligned_to(units, 16) || !aligned_to(k_out, 32) || !aligned_to(v_out, 32) || !aligned_to(ids, 4) || !aligned_to(e_out, 4) ||
      !aligned_to(status, 4))
    return invalid("misaligned pointer (units 16 bytes; k_out, v_out 32)");
  Q4ReadArgs a{};
  a.units = static_cast<const uint8_t*>(units);
  a.n_units = n_units;
  a.ids = ids;
  a.n = n;
  a.k = k_out;
  a.v = v_out;
  a.e = e_out;
  a.status = status;
  DeviceGuard guard(cfg->device);
  return launched(launch_quant4_read(quant_shape(*cfg), a, static_cast<cudaStream_t>(stream)), "4-bit cache read");
}

size_t nosa_quant4_attention_workspace_bytes(const nosa_config* cfg, int32_t max_blocks, int32_t n_queries, int32_t with_mass) {
  if (check_cache(cfg, max_blocks) != NOSA_OK || n_queries < 1 || n_queries > kQMaxQueries) return 0;
  DeviceGuard guard(cfg->device);
  return quant4_attn_workspace(quant_shape(*cfg), max_blocks, n_queries, with_mass != 0);
}

nosa_status nosa_quant4_attention(const nosa_config* cfg, int32_t max_blocks, int32_t n_queries, const void* units,
                                  int64_t n_units, const int32_t* block_tab, const void* tail, const int32_t* lens,
                                  const void* q, const int64_t* q_strides, const int32_t* q_len, const nosa_rope* rope,
                                  const int32_t* positions, void* out, float* lse, float* mass, float decay, void* workspace,
                                  size_t workspace_bytes, int32_t* status, void* stream) {
  nosa_status st = check_cache(cfg, max_blocks);
  if (st != NOSA_OK) return st;
  const Shape s = quant_shape(*cfg);
  QAttnArgs a{};
  if ((st = take_attention(s, max_blocks, n_queries, units, n_units, block_tab, tail, lens, q, q_strides, q_len, out, lse, mass,
                           decay, workspace, status, a)) != NOSA_OK)
    return st;
  RopeArgs r;
  if ((st = take_rope(*cfg, rope, positions, n_queries, status, r)) != NOSA_OK) return st;
  DeviceGuard guard(cfg->device);
  if (workspace_bytes < quant4_attn_workspace(s, max_blocks, n_queries, mass != nullptr))
    return invalid("workspace too small (see nosa_quant4_attention_workspace_bytes)");
  return launched(launch_quant4_attention(s, a, r, static_cast<cudaStream_t>(stream)), "4-bit cache attention");
}

}  // extern "C"
