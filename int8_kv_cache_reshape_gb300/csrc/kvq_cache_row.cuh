// kvq_cache_row.cuh -- the cache writer's per-row quantisation, shared by
// the reshape_and_cache kernel and the fused decode step.
//
// vllm PR 39445 page, Breakdown item 1 (the reshape kernel writing the fp8
// cache with scalar e4m3 quantisation) and vllm PR 38378 page, Breakdown
// item 3 (_reshape_cache_per_token_head: per-(token, head) absmax scale
// computed on the fly and stored inline).  A (token, kv_head) row is handled
// by D/8 threads, each with one 16-byte load of K and of V.
#pragma once

#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace row {

template <int DT>
__device__ __forceinline__ void quantise8(const uint4 x, float s, uint32_t& lo, uint32_t& hi) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = __fdiv_rn(dev::bf16_lo(w[i]), s);
    float b = __fdiv_rn(dev::bf16_hi(w[i]), s);
    if constexpr (DT == KVQ_INT8_PER_TOKEN_HEAD) {
      code[i] = dev::enc_int8(a) | (dev::enc_int8(b) << 8);
    } else if constexpr (DT == KVQ_FP8_E5M2) {
      code[i] = dev::enc_e5m2x2(a, b);
    } else {
      code[i] = dev::enc_e4m3x2(a, b);
    }
  }
  lo = code[0] | (code[1] << 16);
  hi = code[2] | (code[3] << 16);
}

__device__ __forceinline__ float absmax8(const uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = fmaxf(m, fabsf(dev::bf16_lo(w[i])));
    m = fmaxf(m, fabsf(dev::bf16_hi(w[i])));
  }
  return m;
}

// 4-bit codes.  The format's quotients are correctly rounded; a division costs
// some ten instructions and only decides which integer is nearest, so the
// codes come from products with reciprocals a little too large and a little
// too small: rint is monotonic, and where both give the same integer, so does
// the rounded quotient between them.  Where they differ (a quotient whose
// distance from halfway is about 2^-20 of itself or less: up to 2^-17, at 6.5)
// the division decides.
//
// Reference form: an element's code + 8 under its group's step s * m_g.
__device__ __forceinline__ uint32_t enc_int4(float x, float step) {
  const int v = __float2int_rn(__fdiv_rn(x, step));
  return (uint32_t)(max(-7, min(7, v)) + 8);
}
// Eight consecutive elements' code word: element e in nibble e / 2, the odd
// ones four nibbles up.
static __device__ __noinline__ uint32_t quantise8_int4_exact(const uint4 x, float step) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    code |= enc_int4(dev::bf16_lo(w[i]), step) << (4 * i) | enc_int4(dev::bf16_hi(w[i]), step) << (4 * i + 16);
  return code;
}
// (|x| <= gmax of every element; step > 0)
__device__ __forceinline__ uint32_t quantise8_int4(const uint4 x, float gmax, float step) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const float inv = dev::rcp_approx(step);
  const float hi = inv * (1.0f + 0x1p-20f), lo = inv * (1.0f - 0x1p-20f);
  // x * inv + 1.5 2^23 + 8 holds rint(x * inv) + 8 in its lowest bits, on top
  // of the pattern of 1.5 2^23: the sum of the patterns times 16^j, less the
  // constant's, is the code word (modulo 2^32)
  const float magic = 12582912.0f + 8.0f;
  uint32_t code = 0, differ = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = dev::bf16_lo(w[i]), b = dev::bf16_hi(w[i]);
    const uint32_t a0 = __float_as_uint(fmaf(a, lo, magic)), a1 = __float_as_uint(fmaf(a, hi, magic));
    const uint32_t b0 = __float_as_uint(fmaf(b, lo, magic)), b1 = __float_as_uint(fmaf(b, hi, magic));
    differ |= (a0 ^ a1) | (b0 ^ b1);
    code += a0 * (1u << (4 * i)) + b0 * (1u << (4 * i + 16));
  }
  code -= 0x4B400000u * 0x11111111u;
  // (steps so small that the reciprocal or the clamp matters: a quotient above
  // 7.25, or none, also goes the exact way)
  return differ == 0 && gmax * hi < 7.25f ? code : quantise8_int4_exact(x, step);
}
// A group's multiplier min(127, ceil((gmax / s) / 7)), the same way.
__device__ __forceinline__ uint32_t int4_multiplier(float gmax, float rowmax, float s) {
  const float u = gmax * dev::rcp_approx(s) * (1.0f / kInt4MaxCode);
  const float near = rintf(u), d = u - near;
  // (s = rowmax / 889 is far above the subnormals: the largest group is at
  // 889 / 7 = 127 but for rounding, clamped from above)
  const bool normal = rowmax > 0x1p-100f;
  if (normal && gmax == rowmax) return (uint32_t)kInt4MaxMul;
  if (normal && fabsf(d) > 0x1p-12f) return (uint32_t)(int)fminf(kInt4MaxMul, d > 0.0f ? near + 1.0f : near);
  return (uint32_t)(int)fminf(kInt4MaxMul, ceilf(__fdiv_rn(__fdiv_rn(gmax, s), kInt4MaxCode)));
}
// Magnitudes of 8 bf16 values: the packed maximum.
__device__ __forceinline__ uint32_t absmax8_packed(const uint4 x) {
  return dev::max_u16x2(dev::max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                        dev::max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
}
__device__ __forceinline__ float max_of_packed(uint32_t m) {
  return __uint_as_float(max(m << 16, m & 0xFFFF0000u));
}

// Writes one row's share (8 elements) of codes, and for per-token-head the
// scale tail.  TPR threads (a power of two, aligned in the warp) own a row.
template <int DT, int TPR>
__device__ __forceinline__ void write_part(const uint4 x, float tensor_scale, uint8_t* row,
                                           int part, bool active) {
  constexpr int kRowCodes = 8 * TPR;  // head_dim
  if constexpr (DT == KVQ_AUTO) {
    if (active) *reinterpret_cast<uint4*>(row + part * 16) = x;
  } else if constexpr (DT == KVQ_FP8_E4M3 || DT == KVQ_FP8_E5M2) {
    uint32_t lo, hi;
    quantise8<DT>(x, tensor_scale, lo, hi);
    if (active) *reinterpret_cast<uint2*>(row + part * 8) = make_uint2(lo, hi);
  } else {
    float m = absmax8(x);
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float s = __fdiv_rn(m, per_token_head_qmax(DT));
    uint32_t lo = 0, hi = 0;
    if (s != 0.0f) quantise8<code_format(DT)>(x, s, lo, hi);
    if (active) {
      *reinterpret_cast<uint2*>(row + part * 8) = make_uint2(lo, hi);
      if (part == 0)
        *reinterpret_cast<uint4*>(row + kRowCodes) = make_uint4(__float_as_uint(s), 0u, 0u, 0u);
    }
  }
}

// The (token, kv_head) rows of K and V, D/8 threads per row, the rows of a
// step of `threads` threads (a multiple of 32) side by side, over
// [first_step, steps) strided by `stride` steps.  Rows past the end still
// take part in the shuffles (per-token-head) with a clamped, in-bounds read;
// they write nothing.
template <int DT, int D>
__device__ __forceinline__ void write_rows(const uint16_t* __restrict__ key,
                                           const uint16_t* __restrict__ value, int64_t num_tokens,
                                           int64_t key_stride, int64_t value_stride, int heads_kv,
                                           uint8_t* __restrict__ key_cache,
                                           uint8_t* __restrict__ value_cache, int64_t num_slots,
                                           const int64_t* __restrict__ slot_mapping,
                                           float k_scale, float v_scale, int threads, int tid,
                                           int64_t first_step, int64_t stride) {
  constexpr int TPR = D / 8;
  constexpr int kRow = row_bytes(DT, D);
  const int rows_per_step = threads / TPR;
  const int part = tid % TPR;
  const int64_t total_rows = num_tokens * heads_kv;
  for (int64_t r0 = first_step * rows_per_step; r0 < total_rows; r0 += stride * rows_per_step) {
    const int64_t r = r0 + tid / TPR;
    const bool in_range = r < total_rows;
    const int64_t rr = in_range ? r : total_rows - 1;
    // (a 64-bit division costs more than the rest of the addressing)
    const int64_t t = total_rows <= 0x7FFFFFFF ? (int64_t)((uint32_t)rr / (uint32_t)heads_kv) : rr / heads_kv;
    const int h = (int)(rr - t * heads_kv);
    const int64_t slot = slot_mapping[t];
    const bool active = in_range && slot >= 0 && slot < num_slots;
    const uint4 kx = dev::ldg_stream(key + t * key_stride + (int64_t)h * D + part * 8);
    const uint4 vx = dev::ldg_stream(value + t * value_stride + (int64_t)h * D + part * 8);
    const int64_t dst = (active ? (slot * heads_kv + h) : 0) * (int64_t)kRow;
    write_part<DT, TPR>(kx, k_scale, key_cache + dst, part, active);
    write_part<DT, TPR>(vx, v_scale, value_cache + dst, part, active);
  }
}

// 4-bit rows, 16 elements a thread (8: 36.7 us for 20,011 tokens x 8 heads of
// 128; 16: 25.1, 108 MB at 4.3 TB/s, bound by its instructions).
// Writes one 4-bit row's share of 16 elements (x0, x1: the first 8, the rest):
// TPR = D / 16 threads (aligned in the warp) own a row.  A group is D / 8
// dims: half a share, a share or two.
template <int D>
__device__ __forceinline__ void write_part_int4(const uint4 x0, const uint4 x1, uint8_t* row, int part,
                                                bool active) {
  constexpr int TPR = D / 16;
  const uint32_t m0 = absmax8_packed(x0), m1 = absmax8_packed(x1);
  uint32_t mp = dev::max_u16x2(m0, m1);
  if constexpr (D == 256) mp = dev::max_u16x2(mp, __shfl_xor_sync(0xffffffffu, mp, 1));
  const float g0 = max_of_packed(D == 64 ? m0 : mp), g1 = D == 64 ? max_of_packed(m1) : g0;
#pragma unroll
  for (int off = D == 256 ? 2 : 1; off < TPR; off <<= 1)
    mp = dev::max_u16x2(mp, __shfl_xor_sync(0xffffffffu, mp, off));
  const float m = max_of_packed(mp);
  const float s = __fdiv_rn(m, kInt4Levels);
  uint32_t mul0 = 0, mul1 = 0;
  uint2 code = make_uint2(0x88888888u, 0x88888888u);
  if (s > 0.0f) {
    mul0 = int4_multiplier(g0, m, s);
    mul1 = D == 64 ? int4_multiplier(g1, m, s) : mul0;
    const float step0 = __fmul_rn(s, (float)mul0), step1 = __fmul_rn(s, (float)mul1);
    if (step0 > 0.0f) code.x = quantise8_int4(x0, g0, step0);
    if (step1 > 0.0f) code.y = quantise8_int4(x1, g1, step1);
  }
  // the four multipliers of each half of the row in one word: {s, m_0..3} and
  // {m_4..7, 0} go out as two 8-byte stores of the halves' first threads
  uint32_t word;
  if constexpr (D == 64) {
    word = (mul0 | mul1 << 8) << (16 * (part & 1));
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
  } else {
    constexpr int GT = D / 128;  // threads of a group
    word = mul0 << (8 * ((part / GT) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, GT);
    word |= __shfl_xor_sync(0xffffffffu, word, 2 * GT);
  }
  if (active) {
    *reinterpret_cast<uint2*>(row + part * 8) = code;
    if (part % (TPR / 2) == 0)
      *reinterpret_cast<uint2*>(row + D / 2 + (part == 0 ? 0 : 8)) =
          part == 0 ? make_uint2(__float_as_uint(s), word) : make_uint2(word, 0u);
  }
}

// write_rows for 4-bit rows, 16 elements of K and of V per thread: what is
// computed per group and row (scale, multiplier, reciprocals, shuffles) is
// most of the work with 8.  (Coherent loads: the kernel may be a programmatic
// dependent of the one that wrote its inputs.)
template <int D>
__device__ __forceinline__ void write_rows_int4(const uint16_t* __restrict__ key,
                                                const uint16_t* __restrict__ value, int64_t num_tokens,
                                                int64_t key_stride, int64_t value_stride, int heads_kv,
                                                uint8_t* __restrict__ key_cache,
                                                uint8_t* __restrict__ value_cache, int64_t num_slots,
                                                const int64_t* __restrict__ slot_mapping, int threads,
                                                int tid, int64_t first_step, int64_t stride) {
  constexpr int TPR = D / 16;
  constexpr int kRow = row_bytes(KVQ_INT4_PER_TOKEN_HEAD, D);
  const int rows_per_step = threads / TPR;
  const int part = tid % TPR;
  const int64_t total_rows = num_tokens * heads_kv;
  const int64_t step = stride * rows_per_step;
  // (token, head) of this thread's row, advanced by the step's: one division
  int64_t r = first_step * rows_per_step + tid / TPR;
  int64_t t = r / heads_kv;
  int h = (int)(r - t * heads_kv);
  const int64_t dt = step / heads_kv;
  const int dh = (int)(step - dt * heads_kv);
  for (int64_t r0 = first_step * rows_per_step; r0 < total_rows; r0 += step) {
    // (threads past the end take part in the shuffles with the last token's
    // rows and write nothing)
    const bool in_range = t < num_tokens;
    const int64_t tt = in_range ? t : num_tokens - 1;
    const int64_t slot = __ldcg(slot_mapping + tt);
    const uint16_t* ks = key + tt * key_stride + (int64_t)h * D + part * 16;
    const uint16_t* vs = value + tt * value_stride + (int64_t)h * D + part * 16;
    const uint4 k0 = dev::ldg_stream_coherent(ks), k1 = dev::ldg_stream_coherent(ks + 8);
    const uint4 v0 = dev::ldg_stream_coherent(vs), v1 = dev::ldg_stream_coherent(vs + 8);
    const bool active = in_range && slot >= 0 && slot < num_slots;
    const int64_t dst = (active ? (slot * heads_kv + h) : 0) * (int64_t)kRow;
    write_part_int4<D>(k0, k1, key_cache + dst, part, active);
    write_part_int4<D>(v0, v1, value_cache + dst, part, active);
    t += dt;
    h += dh;
    if (h >= heads_kv) {
      h -= heads_kv;
      ++t;
    }
  }
}

}  // namespace row
}  // namespace kvq
