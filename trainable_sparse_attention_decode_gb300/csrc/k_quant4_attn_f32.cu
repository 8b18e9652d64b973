// fp32 instantiations of the attention over the 4-bit block cache (see k_quant_attn.cuh).
#include "k_quant_attn.cuh"

namespace nosa {
cudaError_t launch_quant4_stream_f32(const Shape& s, const QPlan& pl, const QStreamParams& p, cudaStream_t stream) {
  return s.d == 64 ? stream_launches<float, 64, 4>(s, pl, p, stream) : stream_launches<float, 128, 4>(s, pl, p, stream);
}
}  // namespace nosa
