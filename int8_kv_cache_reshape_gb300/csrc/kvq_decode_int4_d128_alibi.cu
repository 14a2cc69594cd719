// kvq_decode_int4_d128_alibi.cu -- the 4-bit decode kernels and fused step for
// head_dim 128 with ALiBi (one translation unit per head_dim and ALiBi setting keeps
// the build parallel).
#include "kvq_decode_int4.cuh"

namespace kvq {
int launch_int4_decode_d128_alibi(const AttnParams& p, const PrefillMaps& maps, int ntiles, void* stream) {
  return launch_int4_decode_d<128, true>(p, maps, ntiles, static_cast<cudaStream_t>(stream));
}
int launch_int4_step_d128_alibi(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, int64_t* warps,
                            void* stream) {
  return launch_int4_step_d<128, true>(p, sp, maps, warps, static_cast<cudaStream_t>(stream));
}
}  // namespace kvq
