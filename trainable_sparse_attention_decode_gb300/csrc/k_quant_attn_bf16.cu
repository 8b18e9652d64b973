// bf16 instantiations of the attention over the 8-bit block cache (see k_quant_attn.cuh).
#include "k_quant_attn.cuh"

namespace nosa {
cudaError_t launch_quant_stream_bf16(const Shape& s, const QPlan& pl, const QStreamParams& p, cudaStream_t stream) {
  return s.d == 64 ? stream_launches<__nv_bfloat16, 64>(s, pl, p, stream) : stream_launches<__nv_bfloat16, 128>(s, pl, p, stream);
}
}  // namespace nosa
