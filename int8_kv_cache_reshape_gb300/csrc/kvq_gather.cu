// kvq_gather.cu -- gather_cache: rows of the paged caches read back, through a
// slot mapping, as the values they stand for.  No counterpart on the pages
// (the inverse of their reshape kernel).
//
// value = code * scale in fp32: the code (4-bit rows: the code times its
// group's multiplier) converts exactly, so an fp32 output carries one
// rounding, and a bf16 output is that fp32 value rounded once more.
//
// HBM bound, almost all of it the output: a thread stores 16 bytes of K and
// of V (4 fp32 or 8 bf16 values), so a warp's stores cover whole lines, and
// loads the 2 to 16 bytes of codes behind them and the row's tail (the same
// few sectors for all of a row's threads).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;

// N consecutive values from dim d0 (a multiple of N) of a row.
template <int DT, int D, int N>
__device__ __forceinline__ void load_values(const uint8_t* row, int d0, float tensor_scale, float (&v)[N]) {
  if constexpr (DT == KVQ_AUTO) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint2 w = dev::ldg_stream8(row + 2 * (d0 + i));
      v[i] = dev::bf16_lo(w.x);
      v[i + 1] = dev::bf16_hi(w.x);
      v[i + 2] = dev::bf16_lo(w.y);
      v[i + 3] = dev::bf16_hi(w.y);
    }
  } else if constexpr (is_int4(DT)) {
    // 8 dims a word; N = 4: the two nibbles 2k and 2k + 1 of each half
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(row + (d0 / 8) * 4));
    const float s = __ldg(reinterpret_cast<const float*>(row + D / 2));
    const int m = __ldg(row + D / 2 + 4 + d0 / (D / 8));
    const int k0 = N == 4 ? (d0 & 4) / 2 : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (int)((w >> (4 * (k0 + i / 2) + 16 * (i & 1))) & 15u) - 8;
      v[i] = s * (float)(m * c);
    }
  } else {
    const float s = is_per_token_head(DT) ? __ldg(reinterpret_cast<const float*>(row + D)) : tensor_scale;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      uint32_t lo, hi;
      dev::word_to_f16x2x2<DT>(__ldg(reinterpret_cast<const uint32_t*>(row + d0 + i)), lo, hi);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      v[i] = a.x * s;
      v[i + 1] = a.y * s;
      v[i + 2] = b.x * s;
      v[i + 3] = b.y * s;
    }
  }
}

template <int N>
__device__ __forceinline__ uint4 pack_out(const float (&v)[N]) {
  if constexpr (N == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    return make_uint4(dev::pack_bf16x2(v[0], v[1]), dev::pack_bf16x2(v[2], v[3]), dev::pack_bf16x2(v[4], v[5]),
                      dev::pack_bf16x2(v[6], v[7]));
}

// N: values per 16 output bytes (4: fp32, 8: bf16); D / N threads per row,
// grid-stride over rows.
template <int DT, int D, int N>
__global__ void __launch_bounds__(kThreads)
gather_cache_kernel(const uint8_t* __restrict__ key_cache, const uint8_t* __restrict__ value_cache,
                    int64_t num_slots, int heads_kv, const int64_t* __restrict__ slot_mapping,
                    int64_t num_tokens, uint4* __restrict__ key_out, uint4* __restrict__ value_out,
                    int64_t key_stride, int64_t value_stride, float k_scale, float v_scale) {
  constexpr int kTpr = D / N, kRowsPerStep = kThreads / kTpr;
  constexpr int64_t kRow = row_bytes(DT, D);
  const int part = threadIdx.x % kTpr;
  const int64_t rows = num_tokens * heads_kv, step = (int64_t)gridDim.x * kRowsPerStep;
  for (int64_t r = (int64_t)blockIdx.x * kRowsPerStep + threadIdx.x / kTpr; r < rows; r += step) {
    // (a 64-bit division costs more than the rest of the row)
    const int64_t t = rows <= 0x7FFFFFFF ? (int64_t)((uint32_t)r / (uint32_t)heads_kv) : r / heads_kv;
    const int h = (int)(r - t * heads_kv);
    const int64_t slot = slot_mapping[t];
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (slot >= 0 && slot < num_slots) {
      const int64_t off = (slot * heads_kv + h) * kRow;
      float a[N], b[N];
      load_values<DT, D, N>(key_cache + off, part * N, k_scale, a);
      load_values<DT, D, N>(value_cache + off, part * N, v_scale, b);
      k = pack_out<N>(a);
      v = pack_out<N>(b);
    }
    key_out[(t * key_stride + (int64_t)h * D) / N + part] = k;
    value_out[(t * value_stride + (int64_t)h * D) / N + part] = v;
  }
}

template <int DT, int D, int N>
int launch(const GatherArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  constexpr int kRowsPerStep = kThreads / (D / N);
  int64_t blocks = (a.num_tokens * a.heads_kv + kRowsPerStep - 1) / kRowsPerStep;
  const int64_t cap = (int64_t)sms * 8;  // 8 resident 256-thread blocks per SM
  if (blocks > cap) blocks = cap;
  gather_cache_kernel<DT, D, N><<<(unsigned)blocks, kThreads, 0, stream>>>(
      a.key_cache, a.value_cache, a.num_slots, a.heads_kv, a.slot_mapping, a.num_tokens,
      static_cast<uint4*>(a.key_out), static_cast<uint4*>(a.value_out), a.key_stride, a.value_stride,
      a.k_scale, a.v_scale);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_E_CUDA;
}

template <int DT, int D>
int launch_n(const GatherArgs& a, bool fp32, cudaStream_t stream) {
  return fp32 ? launch<DT, D, 4>(a, stream) : launch<DT, D, 8>(a, stream);
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
