// kvq_rect_d64.cu -- attention to shared prefixes and encoder keys, head_dim 64.
#include "kvq_rect.cuh"

namespace kvq {
int launch_rect_d64(const AttnParams& p, const RectParams& rp, int dtype, void* stream) {
  return launch_rect_d<64>(p, rp, dtype, static_cast<cudaStream_t>(stream));
}
}  // namespace kvq
