// Plan, workspace and dispatch of the attention over the 8-bit and 4-bit block caches.
#include "k_quant_attn.cuh"

namespace nosa {

int quant_sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && (n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

struct Layout {
  size_t base, part_ml, part_acc, rowstat, tail_w, blk, total;
};
Layout layout(const Shape& s, const QPlan& pl, int max_blocks, bool mass) {
  const size_t vu = (size_t)s.U * pl.tiles, slots = vu + pl.ctas;
  Layout w;
  size_t at = 256;  // the item count
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  w.base = take((size_t)s.U * 8);
  w.part_ml = take(slots * pl.rows * 8);
  w.part_acc = take(slots * pl.rows * s.d * 4);
  w.rowstat = take(vu * pl.rows * 8);
  w.tail_w = take(vu * pl.rows * 4);
  w.blk = take(mass ? vu * max_blocks * pl.rows * 8 : 0);
  w.total = at;
  return w;
}

}  // namespace

// Rows of a tile: 8, 16 or 32, the least that holds the call's rows: the rows of a
// tile share one pass over the cache, and every row costs its products.
QPlan quant_attn_plan(const Shape& s, int T) {
  QPlan pl;
  const int rows = T * s.G;
  pl.rows = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  pl.tiles = (rows + pl.rows - 1) / pl.rows;
  pl.ctas = quant_sm_count();
  return pl;
}

size_t quant_attn_workspace(const Shape& s, int max_blocks, int T, bool mass) {
  return layout(s, quant_attn_plan(s, T), max_blocks, mass).total;
}

static QStreamParams stream_params(const Shape& s, const QPlan& pl, const QAttnArgs& a) {
  const Layout w = layout(s, pl, a.max_blocks, a.mass != nullptr);
  QStreamParams p{};
  p.units = a.units;
  p.n_units = a.n_units;
  p.tab = a.tab;
  p.max_blocks = a.max_blocks;
  p.lens = a.lens;
  p.q = a.q;
  p.qs = a.qs;
  p.T = a.T;
  p.q_len = a.q_len;
  p.U = s.U;
  p.Hkv = s.Hkv;
  p.Hq = s.Hq;
  p.G = s.G;
  p.tiles = pl.tiles;
  p.tail = a.tail;
  p.payload = s.payload;
  p.out = a.out;
  p.lse = a.lse;
  p.mass = a.mass;
  p.decay = a.decay;
  p.status = a.status;
  p.ctas = pl.ctas;
  p.give_up = a.give_up;
  p.total = reinterpret_cast<long long*>(a.ws);
  p.base = reinterpret_cast<long long*>(a.ws + w.base);
  p.part_ml = reinterpret_cast<float2*>(a.ws + w.part_ml);
  p.part_acc = reinterpret_cast<float*>(a.ws + w.part_acc);
  p.rowstat = reinterpret_cast<float2*>(a.ws + w.rowstat);
  p.tail_w = reinterpret_cast<float*>(a.ws + w.tail_w);
  p.blk = a.mass != nullptr ? reinterpret_cast<float2*>(a.ws + w.blk) : nullptr;
  return p;
}

cudaError_t launch_quant_attention(const Shape& s, const QAttnArgs& a, cudaStream_t stream) {
  const QPlan pl = quant_attn_plan(s, a.T);
  const QStreamParams p = stream_params(s, pl, a);
  return s.dtype == 0 ? launch_quant_stream_f32(s, pl, p, stream) : launch_quant_stream_bf16(s, pl, p, stream);
}

cudaError_t launch_quant4_attention(const Shape& s, const QAttnArgs& a, const RopeArgs& rope, cudaStream_t stream) {
  const QPlan pl = quant_attn_plan(s, a.T);
  QStreamParams p = stream_params(s, pl, a);
  p.rope = rope;
  return s.dtype == 0 ? launch_quant4_stream_f32(s, pl, p, stream) : launch_quant4_stream_bf16(s, pl, p, stream);
}

}  // namespace nosa
