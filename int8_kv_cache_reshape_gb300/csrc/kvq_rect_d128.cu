// kvq_rect_d128.cu -- attention to shared prefixes and encoder keys, head_dim 128.
#include "kvq_rect.cuh"

namespace kvq {
int launch_rect_d128(const AttnParams& p, const RectParams& rp, int dtype, void* stream) {
  return launch_rect_d<128>(p, rp, dtype, static_cast<cudaStream_t>(stream));
}
}  // namespace kvq
