// kvq_rect_d256.cu -- attention to shared prefixes and encoder keys, head_dim 256.
#include "kvq_rect.cuh"

namespace kvq {
int launch_rect_d256(const AttnParams& p, const RectParams& rp, int dtype, void* stream) {
  return launch_rect_d<256>(p, rp, dtype, static_cast<cudaStream_t>(stream));
}
}  // namespace kvq
