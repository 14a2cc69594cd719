// kvq_decode_int4_d128.cu -- the 4-bit decode kernels and fused step for
// head_dim 128 (one translation unit per head_dim and ALiBi setting keeps
// the build parallel).
#include "kvq_decode_int4.cuh"

namespace kvq {
int launch_int4_decode_d128_alibi(const AttnParams& p, const PrefillMaps& maps, int ntiles, void* stream);
int launch_int4_step_d128_alibi(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, int64_t* warps,
                            void* stream);
int launch_int4_decode_d128(const AttnParams& p, const PrefillMaps& maps, bool alibi, int ntiles, void* stream) {
  return alibi ? launch_int4_decode_d128_alibi(p, maps, ntiles, stream)
               : launch_int4_decode_d<128, false>(p, maps, ntiles, static_cast<cudaStream_t>(stream));
}
int launch_int4_step_d128(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, bool alibi, int64_t* warps,
                            void* stream) {
  return alibi ? launch_int4_step_d128_alibi(p, sp, maps, warps, stream)
               : launch_int4_step_d<128, false>(p, sp, maps, warps, static_cast<cudaStream_t>(stream));
}
}  // namespace kvq
