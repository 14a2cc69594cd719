// kvq_rotary.cu -- rotary_and_cache: a step's queries and keys rotated by
// their positions, the keys and values stored in the paged caches.
//
// Row t of the cos / sin table's position p_t turns each pair (a, b) of the
// first R dims into (a c - b s, b c + a s); pair j is the dims (j, j + R/2),
// or (2j, 2j + 1) interleaved.  Products and sums are rounded to fp32 one by
// one (no fused multiply-add), so the rotated keys are a function of the
// inputs that any fp32 evaluation reproduces, and so are the stored bytes;
// keys are quantised from their fp32 values (a bf16 rounding in between, as a
// rotation kernel of its own would leave, would move codes), queries rounded
// once to bf16.
//
// HBM bound: per token 2 (Hq + 2 Hkv) D bytes in, 2 Hq D and 2 Hkv row bytes
// out, a table row.  A thread holds 16 consecutive dims of a row (D/16 threads
// a row): what quantising costs per row and group is shared by twice the
// elements of an 8-dim thread, and a row's codes leave as 16-byte stores.  The
// other half of a pair comes from a lane of the row by shuffles of packed
// bf16.  A unit of threads takes kQHeads query heads of a token, whose cos and
// sin stay in registers, or one kv head's K and V rows; the two kinds are mixed, since one
// is bound by memory and the other by its instructions.
// 20,011 tokens of 32 / 8 heads of 128: 80 us for 4-bit rows (446 MB, 5.6 TB/s: 0.82 of a
// measured copy; 93 us with the kinds one after the other, 86 us without the fetches into
// L2 a unit ahead), 82 us int8 and fp8, 81 us bf16; what is left above the copy's 66 to 74 us is
// latency and the codes' instructions.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_cache_row.cuh"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kQHeads = 4;  // query heads of a unit

__device__ __forceinline__ void unpack8(const uint4 x, float* f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = dev::bf16_lo(w[i]);
    f[2 * i + 1] = dev::bf16_hi(w[i]);
  }
}

// cos and sin of a thread's 16 dims, two dims a register pair.  With the other
// half of a pair beside each dim, a rotated dim is x c + y t: t is -s for the
// first of a pair and s for the second, so the sum rounds as the difference
// does, and a product serves two dims.
template <bool IL>
struct Angles {
  uint64_t c[2][4], t[2][4];
  bool turned[2];  // the 8-dim piece is rotated
  // piece q = 2 part + h; R8 = rotated dims / 16 (pieces of a half)
  __device__ __forceinline__ void load(const float* row, int part, int R8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int q = 2 * part + h;
      turned[h] = q < 2 * R8;
      if constexpr (IL) {
        const int j = turned[h] ? 4 * q : 0;
        const float4 a = *reinterpret_cast<const float4*>(row + j);
        const float4 b = *reinterpret_cast<const float4*>(row + 8 * R8 + j);
        c[h][0] = dev::pack2(a.x, a.x), c[h][1] = dev::pack2(a.y, a.y);
        c[h][2] = dev::pack2(a.z, a.z), c[h][3] = dev::pack2(a.w, a.w);
        t[h][0] = dev::pack2(-b.x, b.x), t[h][1] = dev::pack2(-b.y, b.y);
        t[h][2] = dev::pack2(-b.z, b.z), t[h][3] = dev::pack2(-b.w, b.w);
      } else {
        const int j = turned[h] ? 8 * (q < R8 ? q : q - R8) : 0;
        const ulonglong2* const c2 = reinterpret_cast<const ulonglong2*>(row + j);
        const ulonglong2* const s2 = reinterpret_cast<const ulonglong2*>(row + 8 * R8 + j);
        const uint64_t flip = q < R8 ? 0x8000000080000000ull : 0ull;
        const ulonglong2 a = c2[0], b = c2[1], d = s2[0], e = s2[1];
        c[h][0] = a.x, c[h][1] = a.y, c[h][2] = b.x, c[h][3] = b.y;
        t[h][0] = d.x ^ flip, t[h][1] = d.y ^ flip, t[h][2] = e.x ^ flip, t[h][3] = e.y ^ flip;
      }
    }
  }
};

// The thread's 16 dims x[0], x[1] (8 each), rotated.  Every lane of the warp
// calls it (shuffles).  Halves: piece q's other half is piece q -+ R8, the
// words of lane (q -+ R8) / 2's piece of parity (q -+ R8) % 2, the same for all lanes.
template <int TPR, bool IL>
__device__ __forceinline__ void rotate16(const uint4 (&x)[2], const Angles<IL>& a, int part, int R8, float* f) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {x[h].x, x[h].y, x[h].z, x[h].w};
    uint32_t o[4];
    if constexpr (IL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = dev::prmt(w[i], 0u, 0x1032u);  // the other of the pair
    } else {
      const int q = 2 * part + h;
      const int from = (q < R8 ? q + R8 : q < 2 * R8 ? q - R8 : q) >> 1;
      const uint4 mine = (R8 & 1) ? x[h ^ 1] : x[h];
      o[0] = __shfl_sync(0xffffffffu, mine.x, from, TPR);
      o[1] = __shfl_sync(0xffffffffu, mine.y, from, TPR);
      o[2] = __shfl_sync(0xffffffffu, mine.z, from, TPR);
      o[3] = __shfl_sync(0xffffffffu, mine.w, from, TPR);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t v = dev::pack2(dev::bf16_lo(w[i]), dev::bf16_hi(w[i]));
      const uint64_t y = dev::pack2(dev::bf16_lo(o[i]), dev::bf16_hi(o[i]));
      // (scalar sums: a packed sum of packed products comes back fused)
      const float2 p = dev::unpack2(dev::mul2(v, a.c[h][i])), r = dev::unpack2(dev::mul2(y, a.t[h][i]));
      f[8 * h + 2 * i] = a.turned[h] ? __fadd_rn(p.x, r.x) : dev::bf16_lo(w[i]);
      f[8 * h + 2 * i + 1] = a.turned[h] ? __fadd_rn(p.y, r.y) : dev::bf16_hi(w[i]);
    }
  }
}

// Eight codes of x / s.  The quotients are correctly rounded by definition, and
// coding is monotonic: where the products with a reciprocal a little too small
// and one a little too large give the same code, so does the quotient between
// them; elsewhere (and where s or its reciprocal is not normal) it is divided.
template <int F>
__device__ __forceinline__ uint32_t code2(float a, float b) {
  if constexpr (F == KVQ_INT8_PER_TOKEN_HEAD) return dev::enc_int8(a) | (dev::enc_int8(b) << 8);
  else if constexpr (F == KVQ_FP8_E5M2) return dev::enc_e5m2x2(a, b);
  else return dev::enc_e4m3x2(a, b);
}
template <int F>
static __device__ __noinline__ uint2 codes8_exact(const float4 u, const float4 v, float s) {
  return make_uint2(code2<F>(__fdiv_rn(u.x, s), __fdiv_rn(u.y, s)) | code2<F>(__fdiv_rn(u.z, s), __fdiv_rn(u.w, s)) << 16,
                    code2<F>(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s)) | code2<F>(__fdiv_rn(v.z, s), __fdiv_rn(v.w, s)) << 16);
}
template <int F>
__device__ __forceinline__ uint2 codes8(const float* f, float s) {
  const float inv = dev::rcp_approx(s);
  const float lo = inv * (1.0f - 0x1p-22f), hi = inv * (1.0f + 0x1p-22f);
  uint32_t c[4], differ = 0;
  if constexpr (F == KVQ_INT8_PER_TOKEN_HEAD) {
    // x lo + 1.5 2^23 holds rint(x lo) in its lowest byte (|x| <= 127 s up to rounding:
    // nothing to clamp)
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      b[i] = __float_as_uint(fmaf(f[i], lo, 12582912.0f));
      differ |= b[i] ^ __float_as_uint(fmaf(f[i], hi, 12582912.0f));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = dev::prmt(b[2 * i], b[2 * i + 1], 0x0040u) & 0xFFFFu;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = code2<F>(f[2 * i] * lo, f[2 * i + 1] * lo);
      differ |= c[i] ^ code2<F>(f[2 * i] * hi, f[2 * i + 1] * hi);
    }
  }
  if (differ != 0 || !(s > 0x1p-120f && s < 0x1p120f))
    return codes8_exact<F>(make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7]), s);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// 4-bit codes of 8 elements under their group's step (see kvq_cache_row.cuh).
static __device__ __noinline__ uint32_t int4_codes8_exact(const float4 u, const float4 v, float step) {
  return row::enc_int4(u.x, step) | row::enc_int4(u.y, step) << 16 | row::enc_int4(u.z, step) << 4 |
         row::enc_int4(u.w, step) << 20 | row::enc_int4(v.x, step) << 8 | row::enc_int4(v.y, step) << 24 |
         row::enc_int4(v.z, step) << 12 | row::enc_int4(v.w, step) << 28;
}
__device__ __forceinline__ uint32_t int4_codes8(const float* f, float gmax, float step) {
  const float inv = dev::rcp_approx(step);
  const float hi = inv * (1.0f + 0x1p-20f), lo = inv * (1.0f - 0x1p-20f);
  const float magic = 12582912.0f + 8.0f;
  uint32_t code = 0, differ = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a0 = __float_as_uint(fmaf(f[2 * i], lo, magic)), a1 = __float_as_uint(fmaf(f[2 * i], hi, magic));
    const uint32_t b0 = __float_as_uint(fmaf(f[2 * i + 1], lo, magic));
    const uint32_t b1 = __float_as_uint(fmaf(f[2 * i + 1], hi, magic));
    differ |= (a0 ^ a1) | (b0 ^ b1);
    code += a0 * (1u << (4 * i)) + b0 * (1u << (4 * i + 16));
  }
  code -= 0x4B400000u * 0x11111111u;
  if (differ == 0 && gmax * hi < 7.25f) return code;
  return int4_codes8_exact(make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7]), step);
}

__device__ __forceinline__ float absmax8(const float* f) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// A thread's 16 values of a row into the cache row (every lane of the warp
// calls it; only `active` ones store).
template <int DT, int D>
__device__ __forceinline__ void store_row(const float* f, float tensor_scale, uint8_t* to, int part, bool active) {
  constexpr int TPR = D / 16;
  if constexpr (DT == KVQ_AUTO) {
    if (active) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = dev::pack_bf16x2(f[2 * i], f[2 * i + 1]);
      reinterpret_cast<uint4*>(to)[2 * part] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(to)[2 * part + 1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  } else if constexpr (is_int4(DT)) {
    const float m0 = absmax8(f), m1 = absmax8(f + 8);
    float m = fmaxf(m0, m1);
    if constexpr (D == 256) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const float g0 = D == 64 ? m0 : m, g1 = D == 64 ? m1 : m;
#pragma unroll
    for (int off = D == 256 ? 2 : 1; off < TPR; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float s = __fdiv_rn(m, kInt4Levels);
    uint32_t mul0 = 0, mul1 = 0;
    uint2 code = make_uint2(0x88888888u, 0x88888888u);
    if (s > 0.0f) {
      mul0 = row::int4_multiplier(g0, m, s);
      mul1 = D == 64 ? row::int4_multiplier(g1, m, s) : mul0;
      const float step0 = __fmul_rn(s, (float)mul0), step1 = __fmul_rn(s, (float)mul1);
      if (step0 > 0.0f) code.x = int4_codes8(f, g0, step0);
      if (step1 > 0.0f) code.y = int4_codes8(f + 8, g1, step1);
    }
    uint32_t word;  // the four multipliers of each half of the row
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
      *reinterpret_cast<uint2*>(to + part * 8) = code;
      if (part % (TPR / 2) == 0)
        *reinterpret_cast<uint2*>(to + D / 2 + (part == 0 ? 0 : 8)) =
            part == 0 ? make_uint2(__float_as_uint(s), word) : make_uint2(word, 0u);
    }
  } else {
    float s = tensor_scale;
    if constexpr (is_per_token_head(DT)) {
      float m = fmaxf(absmax8(f), absmax8(f + 8));
#pragma unroll
      for (int off = TPR / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      s = __fdiv_rn(m, per_token_head_qmax(DT));
    }
    uint4 c = make_uint4(0, 0, 0, 0);
    if (s != 0.0f) {
      const uint2 u = codes8<code_format(DT)>(f, s), v = codes8<code_format(DT)>(f + 8, s);
      c = make_uint4(u.x, u.y, v.x, v.y);
    }
    if (active) {
      reinterpret_cast<uint4*>(to)[part] = c;
      if (is_per_token_head(DT) && part == 0)
        *reinterpret_cast<uint4*>(to + D) = make_uint4(__float_as_uint(s), 0u, 0u, 0u);
    }
  }
}

__device__ __forceinline__ void prefetch_l2(const void* at) { asm volatile("prefetch.global.L2 [%0];" :: "l"(at)); }

template <int DT, int D, bool IL>
__global__ void __launch_bounds__(kThreads, 2) rotary_and_cache_kernel(const RotaryArgs a, uint64_t share,
                                                                       bool from_memory) {
  constexpr int TPR = D / 16, kUnits = 32 / TPR;  // threads of a row, units of a warp
  constexpr int kRow = row_bytes(DT, D);
  // (a programmatic dependent of whatever ran before on the stream)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, part = lane % TPR;
  const int R8 = a.rotary_dim / 16;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t T = a.num_tokens;
  const int qblocks = (a.heads_q + kQHeads - 1) / kQHeads;
  // Warps' worth of K/V units spread evenly among those of query units: of the
  // first w, floor(w share / 2^32) are K/V units (share: their part of all,
  // rounded up, times 2^32).
  const int64_t kv_w = (T * a.heads_kv + kUnits - 1) / kUnits, q_w = (T * qblocks + kUnits - 1) / kUnits;
  // A unit's token, head (or block of heads), position and slot, one unit ahead: the
  // table row's address waits for the position.
  struct Unit {
    int64_t t, pos, slot;
    int b;
    bool is_kv, in_range;
  };
  auto unit_of = [&](int64_t w) {
    Unit x;
    const int64_t kv0 = (int64_t)(((uint64_t)w * share) >> 32);
    x.is_kv = (int64_t)(((uint64_t)(w + 1) * share) >> 32) > kv0;
    const uint32_t per = (uint32_t)(x.is_kv ? a.heads_kv : qblocks);
    const int64_t u = (x.is_kv ? kv0 : w - kv0) * kUnits + lane / TPR;
    const int64_t tu = u <= 0x7FFFFFFF ? (int64_t)((uint32_t)u / per) : u / per;
    // (threads past the end take part in the shuffles with the last token's
    // rows and store nothing)
    x.in_range = tu < T;
    x.t = x.in_range ? tu : T - 1;
    x.b = x.in_range ? (int)(u - tu * per) : 0;
    x.pos = __ldcg(a.positions + x.t);
    x.slot = x.is_kv ? __ldcg(a.slot_mapping + x.t) : 0;
    return x;
  };
  const int64_t all = kv_w + q_w;
  int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= all) return;
  Unit next = unit_of(w);
  for (; w < all; w += warps) {
    const Unit cur = next;
    if (w + warps < all) {
      next = unit_of(w + warps);
      if (from_memory) {
        if (next.is_kv) {
          const int64_t at = (int64_t)next.b * D + part * 16;
          prefetch_l2(a.key + next.t * a.key_stride + at);
          prefetch_l2(a.value + next.t * a.value_stride + at);
        } else {
          const int h0 = next.b * kQHeads, nh = min(kQHeads, a.heads_q - h0);
          const uint16_t* const qs = a.query + next.t * a.query_stride + (int64_t)h0 * D + part * 16;
#pragma unroll
          for (int i = 0; i < kQHeads; ++i)
            if (i < nh) prefetch_l2(qs + i * D);
        }
      }
    }
    const int64_t t = cur.t;
    const int b = cur.b;
    const bool in_range = cur.in_range, is_kv = cur.is_kv;
    const bool known = cur.pos >= 0 && cur.pos < a.max_position;
    const float* const angles = a.cos_sin + (known ? cur.pos : 0) * a.rotary_dim;
    Angles<IL> ang;
    if (is_kv) {
      const int64_t slot = cur.slot;
      const uint16_t* ks = a.key + t * a.key_stride + (int64_t)b * D + part * 16;
      const uint16_t* vs = a.value + t * a.value_stride + (int64_t)b * D + part * 16;
      const uint4 k[2] = {dev::ldg_stream_coherent(ks), dev::ldg_stream_coherent(ks + 8)};
      const uint4 v[2] = {dev::ldg_stream_coherent(vs), dev::ldg_stream_coherent(vs + 8)};
      ang.load(angles, part, R8);
      const bool active = in_range && known && slot >= 0 && slot < a.num_slots;
      const int64_t at = (active ? slot * a.heads_kv + b : 0) * (int64_t)kRow;
      float f[16];
      rotate16<TPR, IL>(k, ang, part, R8, f);
      store_row<DT, D>(f, a.k_scale, a.key_cache + at, part, active);
      unpack8(v[0], f);
      unpack8(v[1], f + 8);
      store_row<DT, D>(f, a.v_scale, a.value_cache + at, part, active);
    } else {
      const int h0 = b * kQHeads, nh = min(kQHeads, a.heads_q - h0);
      const uint16_t* qs = a.query + t * a.query_stride + (int64_t)h0 * D + part * 16;
      uint16_t* qo = a.query_out + t * a.query_out_stride + (int64_t)h0 * D + part * 16;
      uint4 x[kQHeads][2];
#pragma unroll
      for (int i = 0; i < kQHeads; ++i) {
        x[i][0] = i < nh ? dev::ldg_stream_coherent(qs + i * D) : make_uint4(0, 0, 0, 0);
        x[i][1] = i < nh ? dev::ldg_stream_coherent(qs + i * D + 8) : make_uint4(0, 0, 0, 0);
      }
      ang.load(angles, part, R8);
#pragma unroll
      for (int i = 0; i < kQHeads; ++i) {
        float f[16];
        rotate16<TPR, IL>(x[i], ang, part, R8, f);
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = known ? dev::pack_bf16x2(f[2 * e], f[2 * e + 1]) : 0u;
        if (in_range && i < nh) {
          *reinterpret_cast<uint4*>(qo + i * D) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(qo + i * D + 8) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
  }
}

template <int DT, int D>
int launch(const RotaryArgs& a, bool interleaved, void* stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return KVQ_E_CUDA;
  constexpr int kUnits = 32 / (D / 16);
  const int64_t kv_w = (a.num_tokens * a.heads_kv + kUnits - 1) / kUnits;
  const int64_t warps = kv_w + (a.num_tokens * ((a.heads_q + kQHeads - 1) / kQHeads) + kUnits - 1) / kUnits;
  // (2^31 warps read terabytes; the kernel's products stay within 64 bits)
  if (warps >= ((int64_t)1 << 31)) return KVQ_E_UNSUPPORTED;
  const uint64_t share = (((uint64_t)kv_w << 32) + (uint64_t)warps - 1) / (uint64_t)warps;
  const int64_t blocks = std::min<int64_t>((warps + kThreads / 32 - 1) / (kThreads / 32), (int64_t)sms * 2);
  // The next unit's rows are fetched into L2 a unit ahead where they are not there
  // already, as a projection's output is up to about half of it.  Without / with, int8 rows:
  // 32 / 8 heads of 128, 42 MB 16.6 / 16.7 us, 64 MB 24.6 / 24.1, 100 MB 39.7 / 37.1, 246 MB 91
  // / 83; 16 / 16 of 64, 42 MB 17.9 / 17.6, 64 MB 27.5 / 26.0; 16 / 2 of 256, 64 MB 23.7 / 24.5,
  // 100 MB 37.7 / 37.0: the sides meet between 42 and 90 MB.
  const int64_t in_bytes = 2 * a.num_tokens * ((int64_t)a.heads_q + 2 * a.heads_kv) * D;
  const bool from_memory = in_bytes > (64 << 20);
  return interleaved
             ? launch_dependent(rotary_and_cache_kernel<DT, D, true>, (unsigned)blocks, kThreads, stream, a, share, from_memory)
             : launch_dependent(rotary_and_cache_kernel<DT, D, false>, (unsigned)blocks, kThreads, stream, a, share, from_memory);
}

template <int DT>
int launch_d(const RotaryArgs& a, int head_dim, bool interleaved, void* stream) {
  switch (head_dim) {
    case 64: return launch<DT, 64>(a, interleaved, stream);
    case 128: return launch<DT, 128>(a, interleaved, stream);
    case 256: return launch<DT, 256>(a, interleaved, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}

}  // namespace

int launch_rotary_and_cache(const RotaryArgs& a, int dtype, int head_dim, bool interleaved, void* stream) {
  switch (dtype) {
    case KVQ_AUTO: return launch_d<KVQ_AUTO>(a, head_dim, interleaved, stream);
    case KVQ_FP8_E4M3: return launch_d<KVQ_FP8_E4M3>(a, head_dim, interleaved, stream);
    case KVQ_FP8_E5M2: return launch_d<KVQ_FP8_E5M2>(a, head_dim, interleaved, stream);
    case KVQ_INT8_PER_TOKEN_HEAD: return launch_d<KVQ_INT8_PER_TOKEN_HEAD>(a, head_dim, interleaved, stream);
    case KVQ_FP8_PER_TOKEN_HEAD: return launch_d<KVQ_FP8_PER_TOKEN_HEAD>(a, head_dim, interleaved, stream);
    case KVQ_FP8_E5M2_PER_TOKEN_HEAD: return launch_d<KVQ_FP8_E5M2_PER_TOKEN_HEAD>(a, head_dim, interleaved, stream);
    case KVQ_INT4_PER_TOKEN_HEAD: return launch_d<KVQ_INT4_PER_TOKEN_HEAD>(a, head_dim, interleaved, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}

}  // namespace kvq
