// kvq_gather.cu -- gather_cache: rows of the paged caches read back, through a
// slot mapping, as the values they stand for.  No counterpart on the pages
// (the inverse of their reshape kernel).
//
// value = code * scale in fp32: the code (4-bit rows: the code times its
// group's multiplier) converts exactly, so an fp32 output carries one
// rounding, and a bf16 output is that fp32 value rounded once more.
//
// HBM bound, almost all of it the output.  A thread takes 8 values of K and of
// V: one code word of a 4-bit row, 8 bytes of an 8-bit one; its fp32 values go
// out in one 32-byte store each where the outputs' alignment allows (else two
// of 16), so a warp's stores cover whole lines.  With 4 values a thread the
// kernel was bound by its instructions (166 for 8 values, 36.1 us for 20,011
// tokens x 8 heads of 128 as fp32); now 29.2 us, 190 MB at 6.5 TB/s.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;

// 8 consecutive values, dims 8 part .. 8 part + 7, of a row.
template <int DT, int D>
__device__ __forceinline__ void load_values(const uint8_t* row, int part, float tensor_scale, float (&v)[8]) {
  if constexpr (DT == KVQ_AUTO) {
    const uint4 w = dev::ldg_stream_coherent(row + 16 * part);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = dev::bf16_lo(x[i]);
      v[2 * i + 1] = dev::bf16_hi(x[i]);
    }
  } else if constexpr (is_int4(DT)) {
    const uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(row + 4 * part));
    const uint4 tail = __ldcg(reinterpret_cast<const uint4*>(row + D / 2));  // s, m_0..3, m_4..7
    const int g = part / (D / 64);
    const float s = __uint_as_float(tail.x);
    const float m = (float)(((g < 4 ? tail.y : tail.z) >> (8 * (g & 3))) & 0xFFu);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // a nibble below the pattern of 2^23 is 2^23 + code + 8
      const uint32_t u = ((w >> (4 * (i / 2) + 16 * (i & 1))) & 15u) | 0x4B000000u;
      v[i] = s * ((__uint_as_float(u) - 8388616.0f) * m);
    }
  } else {
    const float s = is_per_token_head(DT) ? __ldcg(reinterpret_cast<const float*>(row + D)) : tensor_scale;
    const uint2 w = __ldcg(reinterpret_cast<const uint2*>(row + 8 * part));
    uint32_t h[4];
    dev::word_to_f16x2x2<DT>(w.x, h[0], h[1]);
    dev::word_to_f16x2x2<DT>(w.y, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      v[2 * i] = f.x * s;
      v[2 * i + 1] = f.y * s;
    }
  }
}

// How the outputs are stored: bf16; fp32 by 32 bytes; fp32 by 16.
enum { kOutBf16 = 0, kOutFp32 = 1, kOutFp32Half = 2 };
template <int OUT>
__device__ __forceinline__ void store_values(void* out, int64_t at, const float (&v)[8]) {
  if constexpr (OUT == kOutBf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
        make_uint4(dev::pack_bf16x2(v[0], v[1]), dev::pack_bf16x2(v[2], v[3]), dev::pack_bf16x2(v[4], v[5]),
                   dev::pack_bf16x2(v[6], v[7]));
  } else {
    float* o = static_cast<float*>(out) + at;
    if constexpr (OUT == kOutFp32) {
      asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                   :: "l"(o), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]),
                   "f"(v[7]) : "memory");
    } else {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

// D / 8 threads per row, grid-stride over rows.
template <int DT, int D, int OUT>
__global__ void __launch_bounds__(kThreads)
gather_cache_kernel(const GatherArgs a) {
  constexpr int kTpr = D / 8, kRowsPerStep = kThreads / kTpr;
  constexpr int64_t kRow = row_bytes(DT, D);
  const int part = threadIdx.x % kTpr;
  // (a programmatic dependent of whatever ran before on the stream: what that
  // wrote is read by coherent loads)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t step = (int64_t)gridDim.x * kRowsPerStep;
  // (token, head) of this thread's row, advanced by the step's: one division
  const int64_t r = (int64_t)blockIdx.x * kRowsPerStep + threadIdx.x / kTpr;
  int64_t t = r / a.heads_kv;
  int h = (int)(r - t * a.heads_kv);
  const int64_t dt = step / a.heads_kv;
  const int dh = (int)(step - dt * a.heads_kv);
  while (t < a.num_tokens) {
    const int64_t slot = __ldcg(a.slot_mapping + t);
    float k[8], v[8];
    if (slot >= 0 && slot < a.num_slots) {
      const int64_t off = (slot * a.heads_kv + h) * kRow;
      load_values<DT, D>(a.key_cache + off, part, a.k_scale, k);
      load_values<DT, D>(a.value_cache + off, part, a.v_scale, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) k[i] = v[i] = 0.0f;
    }
    store_values<OUT>(a.key_out, t * a.key_stride + (int64_t)h * D + 8 * part, k);
    store_values<OUT>(a.value_out, t * a.value_stride + (int64_t)h * D + 8 * part, v);
    t += dt;
    h += dh;
    if (h >= a.heads_kv) {
      h -= a.heads_kv;
      ++t;
    }
  }
}

template <int DT, int D, int OUT>
int launch(const GatherArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  constexpr int kRowsPerStep = kThreads / (D / 8);
  int64_t blocks = (a.num_tokens * a.heads_kv + kRowsPerStep - 1) / kRowsPerStep;
  // (6 of 256 threads are resident per SM; 8: 31.0 us for the rows above, 16: 29.2,
  // 64: 30.1)
  const int64_t cap = (int64_t)sms * 16;
  if (blocks > cap) blocks = cap;
  return launch_dependent(gather_cache_kernel<DT, D, OUT>, (unsigned)blocks, kThreads, stream, a);
}

template <int DT, int D>
int launch_n(const GatherArgs& a, bool fp32, cudaStream_t stream) {
  if (!fp32) return launch<DT, D, kOutBf16>(a, stream);
  // (token strides are multiples of 8 elements)
  const bool wide = ((reinterpret_cast<uintptr_t>(a.key_out) | reinterpret_cast<uintptr_t>(a.value_out)) & 31) == 0;
  return wide ? launch<DT, D, kOutFp32>(a, stream) : launch<DT, D, kOutFp32Half>(a, stream);
}

template <int DT>
int launch_d(const GatherArgs& a, int head_dim, bool fp32, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_n<DT, 64>(a, fp32, stream);
    case 128: return launch_n<DT, 128>(a, fp32, stream);
    case 256: return launch_n<DT, 256>(a, fp32, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}

}  // namespace

int launch_gather_cache(const GatherArgs& a, int dtype, int head_dim, bool fp32, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case KVQ_AUTO: return launch_d<KVQ_AUTO>(a, head_dim, fp32, s);
    case KVQ_FP8_E4M3: return launch_d<KVQ_FP8_E4M3>(a, head_dim, fp32, s);
    case KVQ_FP8_E5M2: return launch_d<KVQ_FP8_E5M2>(a, head_dim, fp32, s);
    case KVQ_INT8_PER_TOKEN_HEAD: return launch_d<KVQ_INT8_PER_TOKEN_HEAD>(a, head_dim, fp32, s);
    case KVQ_FP8_PER_TOKEN_HEAD: return launch_d<KVQ_FP8_PER_TOKEN_HEAD>(a, head_dim, fp32, s);
    case KVQ_FP8_E5M2_PER_TOKEN_HEAD: return launch_d<KVQ_FP8_E5M2_PER_TOKEN_HEAD>(a, head_dim, fp32, s);
    case KVQ_INT4_PER_TOKEN_HEAD: return launch_d<KVQ_INT4_PER_TOKEN_HEAD>(a, head_dim, fp32, s);
    default: return KVQ_E_UNSUPPORTED;
  }
}

}  // namespace kvq
