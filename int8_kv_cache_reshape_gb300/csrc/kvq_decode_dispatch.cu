// kvq_decode_dispatch.cu -- head_dim (and ALiBi) dispatch of the split-KV
// decode, the tensor-core prefill and the rectangular attention kernels (one
// translation unit per head_dim and ALiBi setting holds the instances).
#include "kvq_internal.h"
#include "kvq_merge.cuh"

namespace kvq {

// The merge runs right after the decode kernel on the stream, launched as its
// programmatic dependent (the decode kernel lets it be scheduled at once; it
// waits for the decode grid before reading): no launch gap between the two.
int launch_merge(const AttnParams& p, int dtype, int head_dim, int64_t num_merges, void* stream) {
  if (num_merges <= 0) return KVQ_OK;
  void (*kern)(AttnParams);
  switch (head_dim) {
    case 64: kern = is_int4(dtype) ? merge_splits_kernel<64, true> : merge_splits_kernel<64, false>; break;
    case 128: kern = is_int4(dtype) ? merge_splits_kernel<128, true> : merge_splits_kernel<128, false>; break;
    case 256: kern = is_int4(dtype) ? merge_splits_kernel<256, true> : merge_splits_kernel<256, false>; break;
    default: return KVQ_E_UNSUPPORTED;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_merges);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  return KVQ_OK;
}

namespace {
template <int D, int PARTS, int BATCH>
int rect_merge(const AttnParams& p, const RectParams& rp, const RectMergePlan& m, void* stream) {
  // (eight warps, fewer where an item's rows need fewer)
  const unsigned rows = (unsigned)(m.most_rows < 8 / PARTS ? m.most_rows : 8 / PARTS);
  // (few items: a CTA for each of an item's turns)
  const int turns = (m.most_rows + (int)rows - 1) / (int)rows;
  const int ctas = m.items * turns <= (int64_t)m.sms * 8 ? turns : 1;
  return launch_dependent(merge_rect_kernel<D, PARTS, BATCH>, (unsigned)(m.items * ctas), 32u * PARTS * rows, stream, p,
                          rp, ctas);
}
template <int D>
int rect_merge_d(const AttnParams& p, const RectParams& rp, const RectMergePlan& m, void* stream) {
  // Warps a row: as many as have partials to read, while all rows' warps are on
  // the device at once.  (Calls of 8-bit rows behind 8,192 keys, 4 / 2 / 1 warps a row: head_dim
  // 128, 512 rows 24.1 / 24.6 / 25.7 us, 1,216 rows 36.7 / 33.9 / 34.4, 2,048 rows 47.8 / 44.6 /
  // 43.0; head_dim 256, 256 rows 23.5 / 24.8 / 26.7, 1,536 rows 64.7 / 61.8 / 59.2.)
  const int64_t room = (int64_t)m.sms * 8 * rect_merge_ctas(D) / (m.rows > 0 ? m.rows : 1);
  if (m.most_splits > 16 && room >= 4) return rect_merge<D, 4, 8>(p, rp, m, stream);
  if (m.most_splits > 8 && room >= 2) return rect_merge<D, 2, 8>(p, rp, m, stream);
  return rect_merge<D, 1, 8>(p, rp, m, stream);
}
}  // namespace

int launch_rect_merge(const AttnParams& p, const RectParams& rp, int head_dim, const RectMergePlan& m, void* stream) {
  if (m.items <= 0) return KVQ_OK;
  switch (head_dim) {
    case 64: return rect_merge_d<64>(p, rp, m, stream);
    case 128: return rect_merge_d<128>(p, rp, m, stream);
    case 256: return rect_merge_d<256>(p, rp, m, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}

int launch_merge_step(const AttnParams& p, const StepParams& sp, int dtype, int head_dim,
                      int64_t warps, void* stream) {
  if (sp.num_tiles <= 0) return KVQ_OK;
  void (*kern)(AttnParams, StepParams, int64_t);
  switch (head_dim) {
    case 64: kern = is_int4(dtype) ? merge_step_kernel<64, true> : merge_step_kernel<64, false>; break;
    case 128: kern = is_int4(dtype) ? merge_step_kernel<128, true> : merge_step_kernel<128, false>; break;
    case 256: kern = is_int4(dtype) ? merge_step_kernel<256, true> : merge_step_kernel<256, false>; break;
    default: return KVQ_E_UNSUPPORTED;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sp.num_tiles);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p, sp, warps) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  return KVQ_OK;
}

#define KVQ_DECLARE(D)                                                                       \
  int launch_rect_d##D(const AttnParams&, const RectParams&, int, void*);                    \
  int launch_decode_d##D(const AttnParams&, int, int, void*);                               \
  int launch_decode_d##D##_alibi(const AttnParams&, int, int, void*);                       \
  int launch_step_d##D(const AttnParams&, const StepParams&, int, int64_t*, void*);         \
  int launch_step_d##D##_alibi(const AttnParams&, const StepParams&, int, int64_t*, void*); \
  int launch_int4_decode_d##D(const AttnParams&, const PrefillMaps&, bool, int, void*);     \
  int launch_int4_step_d##D(const AttnParams&, const StepParams&, const PrefillMaps&, bool, \
                            int64_t*, void*);                                               \
  int launch_prefill_d##D(const AttnParams&, const PrefillMaps&, int, int64_t, void*);      \
  int launch_prefill_d##D##_alibi(const AttnParams&, const PrefillMaps&, int, int64_t, void*);
KVQ_DECLARE(64)
KVQ_DECLARE(128)
KVQ_DECLARE(256)
#undef KVQ_DECLARE

int launch_decode(const AttnParams& p, const PrefillMaps& maps, int dtype, int head_dim, int ntiles,
                  void* stream) {
  if (p.num_chunks <= 0) return KVQ_OK;
  const bool al = uses_alibi(p);
  if (is_int4(dtype)) {
    switch (head_dim) {
      case 64: return launch_int4_decode_d64(p, maps, al, ntiles, stream);
      case 128: return launch_int4_decode_d128(p, maps, al, ntiles, stream);
      case 256: return launch_int4_decode_d256(p, maps, al, ntiles, stream);
      default: return KVQ_E_UNSUPPORTED;
    }
  }
  switch (head_dim) {
    case 64: return al ? launch_decode_d64_alibi(p, dtype, ntiles, stream)
                       : launch_decode_d64(p, dtype, ntiles, stream);
    case 128: return al ? launch_decode_d128_alibi(p, dtype, ntiles, stream)
                        : launch_decode_d128(p, dtype, ntiles, stream);
    case 256: return al ? launch_decode_d256_alibi(p, dtype, ntiles, stream)
                        : launch_decode_d256(p, dtype, ntiles, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}

namespace {
int step_dispatch(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, int dtype,
                  int head_dim, bool al, int64_t* warps, void* stream) {
  if (is_int4(dtype)) {
    switch (head_dim) {
      case 64: return launch_int4_step_d64(p, sp, maps, al, warps, stream);
      case 128: return launch_int4_step_d128(p, sp, maps, al, warps, stream);
      case 256: return launch_int4_step_d256(p, sp, maps, al, warps, stream);
      default: return KVQ_E_UNSUPPORTED;
    }
  }
  switch (head_dim) {
    case 64: return al ? launch_step_d64_alibi(p, sp, dtype, warps, stream)
                       : launch_step_d64(p, sp, dtype, warps, stream);
    case 128: return al ? launch_step_d128_alibi(p, sp, dtype, warps, stream)
                        : launch_step_d128(p, sp, dtype, warps, stream);
    case 256: return al ? launch_step_d256_alibi(p, sp, dtype, warps, stream)
                        : launch_step_d256(p, sp, dtype, warps, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}
}  // namespace

int step_warps(int dtype, int heads_kv, int head_dim, bool alibi, int max_rows, int64_t* warps) {
  AttnParams p{};
  p.heads_kv = heads_kv;
  StepParams sp{};
  sp.max_rows = max_rows;
  *warps = 0;
  return step_dispatch(p, sp, PrefillMaps{}, dtype, head_dim, alibi, warps, nullptr);
}

int launch_decode_step(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, int dtype,
                       int head_dim, int64_t warps, void* stream) {
  return step_dispatch(p, sp, maps, dtype, head_dim, uses_alibi(p), &warps, stream);
}

int launch_rect(const AttnParams& p, const RectParams& rp, int dtype, int head_dim, void* stream) {
  if (rp.num_units <= 0) return KVQ_OK;
  switch (head_dim) {
    case 64: return launch_rect_d64(p, rp, dtype, stream);
    case 128: return launch_rect_d128(p, rp, dtype, stream);
    case 256: return launch_rect_d256(p, rp, dtype, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}

int launch_prefill(const AttnParams& p, const PrefillMaps& maps, int dtype, int head_dim,
                   int64_t ctas, void* stream) {
  if (ctas <= 0) return KVQ_OK;
  const bool al = uses_alibi(p);
  switch (head_dim) {
    case 64: return al ? launch_prefill_d64_alibi(p, maps, dtype, ctas, stream)
                       : launch_prefill_d64(p, maps, dtype, ctas, stream);
    case 128: return al ? launch_prefill_d128_alibi(p, maps, dtype, ctas, stream)
                        : launch_prefill_d128(p, maps, dtype, ctas, stream);
    case 256: return al ? launch_prefill_d256_alibi(p, maps, dtype, ctas, stream)
                        : launch_prefill_d256(p, maps, dtype, ctas, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}

}  // namespace kvq
