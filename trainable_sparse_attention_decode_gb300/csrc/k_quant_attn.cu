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
  p.turned = a.turned;
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

// The queries are turned first, into the workspace: in the stream's helper warp and in the join the
// rotation cost 9 to 16 us a call (8 units x 131071 tokens; 32 rows), by their registers most of it.
cudaError_t launch_quant4_attention(const Shape& s, const QAttnArgs& args, const RopeArgs& rope, cudaStream_t stream) {
  const QPlan pl = quant_attn_plan(s, args.T);
  QAttnArgs a = args;
  if (rope.pairs > 0) {
    RotateArgs r{};
    r.rope = rope;
    r.in[0] = a.q;
    r.in_b[0] = a.qs.b;
    r.in_t[0] = a.qs.t;
    r.in_h[0] = a.qs.h;
    a.qs = QStrides{(long long)a.T * s.Hq * s.d, (long long)s.Hq * s.d, s.d};
    a.q = r.out[0] = a.ws + quant_attn_workspace(s, a.max_blocks, a.T, a.mass != nullptr);
    a.turned = true;
    r.out_b[0] = a.qs.b;
    r.out_t[0] = a.qs.t;
    r.out_h[0] = a.qs.h;
    r.heads[0] = s.Hq;
    r.n = a.T;
    r.count = a.q_len;
    r.rows = (long long)s.batch * a.T;
    const cudaError_t e = launch_rotate(s, r, stream);
    if (e != cudaSuccess) return e;
  }
  const QStreamParams p = stream_params(s, pl, a);
  return s.dtype == 0 ? launch_quant4_stream_f32(s, pl, p, stream) : launch_quant4_stream_bf16(s, pl, p, stream);
}

size_t quant4_attn_workspace(const Shape& s, int max_blocks, int T, bool mass) {
  return quant_attn_workspace(s, max_blocks, T, mass) + (size_t)s.batch * T * s.Hq * s.d * s.elt;
}

}  // namespace nosa
