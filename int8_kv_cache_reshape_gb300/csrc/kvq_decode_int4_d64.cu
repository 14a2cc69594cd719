// kvq_decode_int4_d64.cu -- the 4-bit decode kernels and fused step for
// head_dim 64 (one translation unit per head_dim and ALiBi setting keeps
// the build parallel).
#include "kvq_decode_int4.cuh"

namespace kvq {
int launch_int4_decode_d64_alibi(const AttnParams& p, const PrefillMaps& maps, int ntiles, void* stream);
int launch_int4_step_d64_alibi(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, int64_t* warps,
                            void* stream);
int launch_int4_decode_d64(const AttnParams& p, const PrefillMaps& maps, bool alibi, int ntiles, void* stream) {
  return alibi ? launch_int4_decode_d64_alibi(p, maps, ntiles, stream)
               : launch_int4_decode_d<64, false>(p, maps, ntiles, static_cast<cudaStream_t>(stream));
}
int launch_int4_step_d64(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, bool alibi, int64_t* warps,
                            void* stream) {
  return alibi ? launch_int4_step_d64_alibi(p, sp, maps, warps, stream)
               : launch_int4_step_d<64, false>(p, sp, maps, warps, static_cast<cudaStream_t>(stream));
}
}  // namespace kvq
