// kvq_decode_int4.cuh -- split-KV attention of small row tiles (decode) over
// the 4-bit paged cache, and the fused decode step of that cache.
//
// What it computes is the attention of kvq_decode.cuh (same masks, soft cap,
// ALiBi, sinks, partial rows and merge) for rows of D/2 code bytes and a
// 16-byte tail of scales: k_jd = s_j m_jg c_jd.  m c is an integer of at most
// 10 bits, so it enters the f16 MMAs exactly; s_j multiplies the fp32 scores
// (K) and joins the softmax weights (V).
//
// GB300 design.  A 4-bit chunk of 16 tokens is 2560 bytes a head at D = 128,
// so at the memory's rate a warp has some 450 issue slots for it, and a
// kernel that fetches its rows lane by lane (kvq_decode.cuh) spends more than
// that (560 instructions, with a quarter of them for loads, and 71 us for
// the 64-request decode batch).  Here:
//   * One warp per kv head, all heads of a group side by side in a CTA on the
//     same chunks (the plan's head lockstep).  A token's rows of all heads
//     lie next to each other, so 16 tokens of a block are one run of whole
//     128-byte lines: one bulk tensor copy each for K and V, with no address,
//     predicate or register in the consumers.  (Copies a token at a time
//     reached the copy engine's rate, not the memory's: a 640-byte copy
//     every 40-50 cycles of an SM, 375 us against 243 for 32 x 32768 keys.)
//   * No producer warp (a ninth costs as many registers as three more): the
//     warps of a group issue the copies in turn, chunk k by warp k mod Hg, a
//     chunk behind the ring's end, so that the wait for the slot's last
//     readers is over before it is asked for.  Records (slots, masks) are
//     prepared by the lanes, kInt4Turns turns at a time.
//   * The copies write the 128-byte swizzle, and MMA row g is token pi(g) =
//     {0,4,2,6,12,8,14,10}[g] of a half (row g + 8 the token after it).  The
//     order is chosen for 8 heads of 128 (5 lines a token): K's 16-byte reads
//     (eight lanes: two rows) and V's (rows pi(2c)) of heads 0, 2, 4, 5 and 7
//     then cover the 32 banks once, the others' take 1.5 to 2 times as many
//     wavefronts (by address arithmetic; 1, 2 and 4 heads: 1.4 to 2.9 times).
//     The token order of a softmax is free.
//   * A warp takes both halves of a chunk in one go (32 tokens): waits,
//     records, masks and votes once for two sets of MMAs.
//   * The lazy reference maximum and the value scales' power-of-two reference
//     move on one warp vote; the common chunk has no shuffle.
// Measured: 64 requests of 1,024 to 4,096 keys (32 q and 8 kv heads of 128) in
// 48 us with the merge, 179 MB at 3.7 TB/s (the first data comes 7 us after
// the launch, the merge takes 4); 32 requests of 32,768 keys (64 q heads) in
// 229 us, 5.9 TB/s, 88 % of a plain copy's rate.  The same 32 requests in other
// shapes (8 q heads a kv head): 16 kv heads 463 us (5.8 TB/s), 4 heads 124 (5.4), 2 heads
// 79 (4.2), 1 head 69 (2.4: three eighths of its stages are padding, 13 groups a
// CTA issue their own copies); 16 rows a tile 356 (3.8: 8 warps a CTA, twice the
// MMAs); ALiBi 274 (4.9); head_dim 64 155 (5.2), 256 446 (5.4).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "kvq_cache_row.cuh"
#include "kvq_decode.cuh"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_tcgen05.cuh"

namespace kvq {

template <int D>
struct Int4Row {
  static constexpr int kCodes = D / 2;
  static constexpr int kRow = row_bytes(KVQ_INT4_PER_TOKEN_HEAD, D);
  static constexpr int kKBytes = D / 8 >= 16 ? 16 : D / 8;  // bytes of a K piece
  static constexpr int kK16 = D / 8 / kKBytes;              // K pieces per lane per row
  static constexpr int kKWords = D / 32;                    // K code words per lane per row
  static constexpr int kVWords = D / 64;                    // V code words per lane per row
  static constexpr int kRun = 2 * kKBytes;                  // consecutive dims of a K piece
  static constexpr int kKsteps = D / 16, kMtiles = D / 16;
  // A lane's 8-dim K words: the first half belongs to its first group, the
  // rest to its second: groups 2c and 2c + 1 (D = 256: c and c + 4).
};

namespace i4 {

__device__ __forceinline__ int pi_of(int g) { return (int)((0xAE8C6240u >> (4 * g)) & 15u); }

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int group, int slot, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], "
      "[%5];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(slot), "r"(bar) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// Bounded wait of a whole warp: false on a timeout (about a second), here or
// in another warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (true) {
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort != 0u)) return false;
    if (__any_sync(0xffffffffu, clock64() - t0 > 2000000000LL)) {
      *abort = 1u;
      return false;
    }
  }
}

}  // namespace i4

// The fused step's plan: one tile per request (its kv heads share the chunk
// ranges), {first chunk, first key, end, rows}, and the prefix sum of their
// chunk counts.  A request with more rows than the launch was built for (or
// more queries than keys) is left out and flags the error word (if `flag`).
__device__ __forceinline__ void plan_step_int4(const AttnParams& p, const StepParams& sp, int32_t* prefix,
                                               int4* tiles, bool flag) {
  __shared__ int32_t warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  const int nt = sp.num_req;
  const int per = (nt + nthr - 1) / nthr;
  const int t0 = min(nt, tid * per), t1 = min(nt, t0 + per);
  int local = 0;
  for (int r = t0; r < t1; ++r) {
    const int Q = sp.in_query_start_loc[r + 1] - sp.in_query_start_loc[r];
    const int L = sp.in_seq_lens[r];
    int4 ti = make_int4(0, 0, 0, 0);
    if (Q <= 0 || L < Q || Q > sp.max_rows / p.group) {
      if (flag && Q != 0) atomicExch(p.error_flag, 2);  // (1 is a timeout)
    } else {
      const int lo = p.window > 0 ? max(0, L - Q - p.window + 1) : 0;
      ti = make_int4(lo / kInt4Chunk, lo, L, Q * p.group);
    }
    tiles[r] = ti;
    local += ti.z > 0 ? (ti.z - 1) / kInt4Chunk + 1 - ti.x : 0;
    prefix[r] = local;  // (within this thread's requests, for now)
  }
  int incl = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int run = incl - local;
  for (int w = 0; w < warp; ++w) run += warp_sums[w];
  int before = run;
  for (int r = t0; r < t1; ++r) {
    const int end = run + prefix[r];
    prefix[r] = before;
    before = end;
  }
  if (tid == nthr - 1) prefix[nt] = run + local;
  __syncthreads();
}

template <int D, int NT, bool AL, bool DEV>
__global__ void __launch_bounds__(32 * int4_max_warps(D, NT), 1)
int4_decode_kernel(const AttnParams p, const StepParams sp, const Int4Geom ge,
                   const __grid_constant__ PrefillMaps maps) {
  using Row = Int4Row<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t abort_word;
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);  // (uniform)
  const int g = lane >> 2;
  const int c = lane & 3;

  // The merge of the cut tiles (its own kernel, after this one) may be
  // scheduled now: it waits for this grid to complete.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int grp = warp / ge.hg, j = warp % ge.hg;  // the group, and the warp's head in it
  // ---- this warp's segment of the flat chunk sequence of its head -----------
  // (segment, head group): the SMs first, so that few segments have their
  // own copy queue and warp schedulers each
  const int glin = grp * gridDim.x + blockIdx.x;
  const int seg = glin / ge.hsplit, hgrp = glin % ge.hsplit;
  const int head = hgrp * ge.hg + j;
  const int gw = seg * p.heads_kv + head;
  int seg0 = 0, n = 0, first_piece = 0;
  if constexpr (!DEV) {
    if (seg < ge.segments) {
      const WarpSeg ws = p.warp_seg[gw];
      seg0 = ws.seg0;
      n = ws.n;
      first_piece = ws.piece;
    }
  }
  // (the swizzle goes by shared-memory addresses: stages on 1 KB)
  const uint32_t smem0 = (dev::smem_u32(smem) + 1023u) & ~1023u;
  const uint32_t sbase = smem0 + (uint32_t)(grp * ge.stages * ge.stage_bytes);
  const uint32_t meta0 = smem0 + (uint32_t)(ge.gpc * ge.stages * ge.stage_bytes);
  const uint32_t meta = meta0 + (uint32_t)(grp * ge.stages * 32);  // per stage: record (16), full, empty
  volatile uint32_t* const abort = &abort_word;
  if (threadIdx.x == 0) {
    abort_word = 0u;
    for (int i = 0; i < ge.gpc * ge.stages; ++i) {
      tc::mbar_init(meta0 + 32u * i + 16, 1);
      tc::mbar_init(meta0 + 32u * i + 24, ge.hg);
    }
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
    tc::mbar_fence_init();
  }

  // ---- the fused step's prologue -------------------------------------------
  if constexpr (DEV) {
    StageLane st;
    stage_issue(sp, st);
    row::write_rows_int4<D>(sp.key, sp.value, sp.num_tokens, sp.key_stride, sp.value_stride, p.heads_kv,
                            sp.key_cache, sp.value_cache, sp.num_slots, sp.slot_mapping, blockDim.x,
                            threadIdx.x, blockIdx.x, gridDim.x);
    stage_finish(sp, st);
    // (the bulk copies below read rows that other CTAs stored: both sides
    // order their proxies)
    asm volatile("fence.proxy.async.global;" ::: "memory");
  }
  // The fused step's plan: of up to kInt4PlanReq requests by every CTA for
  // itself, so that all that leads to the first copies lies before the
  // grid barrier (unless the inputs are still on their way from the host);
  // else by the first CTA, for all of them.  The merge reads the first CTA's.
  // A CTA with a plan of its own arrives at the barrier as soon as its rows
  // are written and waits there when the plan, the records and the first
  // piece are ready (arriving then took a step of 64 requests 3 us more).
  __shared__ int32_t prefix_s[DEV ? kInt4PlanReq + 1 : 1];
  __shared__ int4 tiles_s[DEV ? kInt4PlanReq : 1];
  const bool own_plan = DEV && sp.num_req <= kInt4PlanReq && sp.stage_bytes == 0;
  const volatile int32_t* prefix = own_plan ? prefix_s : sp.prefix;
  const volatile int4* tiles = own_plan ? tiles_s : sp.tiles;
  __shared__ uint32_t gen_s;  // the barrier's generation before it opens
  auto arrive_grid = [&]() {
    __syncthreads();  // (the CTA's rows are written)
    if (threadIdx.x == 0) {
      gen_s = *(volatile uint32_t*)(sp.barrier + 1);
      __threadfence();
      if (atomicAdd(sp.barrier, 1u) == gridDim.x - 1) {
        atomicExch(sp.barrier, 0u);
        __threadfence();
        atomicAdd(sp.barrier + 1, 1u);
      }
    }
  };
  auto join_grid = [&]() -> bool {
    int ok = 1;
    if (threadIdx.x == 0) {
      const long long t0 = clock64();
      while (*(volatile uint32_t*)(sp.barrier + 1) == gen_s) {
        if (clock64() - t0 > 2000000000LL) {  // about a second
          ok = 0;
          atomicExch(p.error_flag, 1);
          break;
        }
      }
      __threadfence();
    }
    ok = __syncthreads_and(ok);
    asm volatile("fence.proxy.async.global;" ::: "memory");
    return ok != 0;
  };
  if constexpr (DEV) {
    if (own_plan) {
      arrive_grid();
      plan_step_int4(p, sp, prefix_s, tiles_s, blockIdx.x == 0);
      if (blockIdx.x == 0)
        for (int r = threadIdx.x; r <= sp.num_req; r += blockDim.x) {
          sp.prefix[r] = prefix_s[r];
          if (r < sp.num_req) sp.tiles[r] = tiles_s[r];
        }
    } else {
      if (blockIdx.x == 0) plan_step_int4(p, sp, sp.prefix, sp.tiles, true);
      arrive_grid();
      if (!join_grid()) return;
    }
  }
  __syncthreads();

  if constexpr (DEV) {
    const int64_t T = prefix[sp.num_req];
    const int segs = int4_step_segments(T, ge.segments);
    if (seg < segs) {
      seg0 = (int)((int64_t)seg * T / segs);
      n = (int)((int64_t)(seg + 1) * T / segs) - seg0;
      // the last request whose first chunk is seg0 or an earlier one
      int hi = sp.num_req;
      while (hi - first_piece > 1) {
        const int mid = (first_piece + hi) >> 1;
        if (prefix[mid] <= seg0) first_piece = mid;
        else hi = mid;
      }
    }
  }
  if (n <= 0) {  // (the whole group: its heads share the chunk range)
    if (own_plan) (void)join_grid();
    return;
  }
  // Host plans are launched as programmatic dependents of whatever ran before
  // on the stream: only the plan has been read so far.  Where that is the
  // call's own prefill or rectangular attention, nothing here depends on it, and
  // all that it depends on was done when it started: the decode's CTAs take the
  // SMs that it leaves, and the first waits for its end before its own (so that what
  // follows the decode follows both; its first group always has chunks).
  if (!DEV && !p.beside_prefill) asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- copies ----------------------------------------------------------------
  // Chunk k of the segment is copied by warp k mod hg of the group.
  const int S = ge.stages, ahead = S - 1;
  const int tok_bytes = ge.hg * Row::kRow;  // a token's rows of the group
  const uint32_t v_off = 2u * ge.half_bytes;  // V's rows in a stage
  // Records of this warp's next kInt4Turns turns, one per lane: {first token, piece
  // relative to the segment's first, live tokens}, {first slot of each half of
  // the chunk (-1: none of its keys, or no block)}.
  // (Filled together; the three dependent loads cost a group of one warp its
  // lead every 16 chunks, wider groups nothing.)
  __shared__ uint4 recs_s[int4_max_warps(D, NT)][kInt4Turns][2];
  const uint32_t recs = dev::smem_u32(recs_s[warp]);
  int cur_piece = first_piece;
  auto fill_records = [&](int turn0) {
    const int pos = j + ge.hg * (turn0 + lane);
    int slot[2] = {-1, -1}, tok0 = 0, rel = 0;
    uint32_t live = 0;
    if (lane < kInt4Turns && pos < n) {
      const int flat = seg0 + pos;
      int chunk, req, lo, hi;
      if constexpr (DEV) {
        while (cur_piece + 1 < sp.num_req && prefix[cur_piece + 1] <= flat) ++cur_piece;
        chunk = tiles[cur_piece].x + (flat - prefix[cur_piece]);
        req = cur_piece;
        lo = tiles[cur_piece].y;
        hi = tiles[cur_piece].z;
      } else {
        // (a piece's descriptor and the next one's start are read together)
        while (true) {
          const int4* d = reinterpret_cast<const int4*>(p.pieces + cur_piece);
          const int4 a = __ldg(d), b = __ldg(d + 1), e = __ldg(d + 2);
          const int next = cur_piece + 1 < p.num_pieces ? __ldg(&p.pieces[cur_piece + 1].flat0) : 0x7FFFFFFF;
          if (flat < next) {
            chunk = e.y + (flat - e.x);
            req = a.x;
            lo = b.z;
            hi = b.w;
            break;
          }
          ++cur_piece;
        }
      }
      tok0 = chunk * kInt4Chunk;
      rel = cur_piece - first_piece;
      // (the fused step's table width is not known on the host: check it
      // here; the bounds-checked build checks the host plan's positions too)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tk = tok0 + 16 * u, lb = tk / p.block_size;
        const int l = min(max(lo - tk, 0), 16), h = min(max(hi - tk, 0), 16);
        if (h <= l) continue;  // no key of the piece (nor, perhaps, a block)
        const bool in_table = lb < p.block_table_stride;
        if constexpr (KVQ_CHECKED && !DEV)
          if (!in_table) atomicExch(p.error_flag, 2);
        int blk = -1;
        if (!(DEV || KVQ_CHECKED) || in_table) blk = p.block_table[(int64_t)req * p.block_table_stride + lb];
        if (blk >= 0 && (int64_t)blk < p.num_blocks) {
          slot[u] = blk * p.block_size + (tk - lb * p.block_size);
          live |= (((1u << h) - 1u) & ~((1u << l) - 1u)) << (16 * u);
        }
      }
    }
    if (lane < kInt4Turns) {
      i4::sts128(recs + 32u * lane, make_uint4((uint32_t)tok0, (uint32_t)rel, live, 0u));
      i4::sts128(recs + 32u * lane + 16, make_uint4((uint32_t)slot[0], (uint32_t)slot[1], 0u, 0u));
    }
    __syncwarp();
  };
  int turn = 0;  // this warp's next turn
  // This warp's next chunk into stage s, whose parity of use is u (first:
  // the stage has not been used before).
  auto issue = [&](int s, uint32_t u, bool first) -> bool {
    if (turn % kInt4Turns == 0 && !(own_plan && turn == 0)) fill_records(turn);
    const uint32_t full = meta + 32u * s + 16;
    if (!first && !i4::warp_wait(full + 8, u ^ 1u, abort)) return false;
    const uint4 rec = dev::lds128(recs + 32u * (turn % kInt4Turns));
    const uint2 sl = i4::lds64(recs + 32u * (turn % kInt4Turns) + 16);
    const int halves = ((int)sl.x >= 0) + ((int)sl.y >= 0);
    if (lane == 0) {
      i4::sts128(meta + 32u * s, rec);
      if (halves) i4::mbar_arrive_expect_tx(full, (uint32_t)(halves * 2 * kChunkTokens * tok_bytes));
      else i4::mbar_arrive(full);
    }
    __syncwarp();
    // lanes 0-3: K and V of the first half, K and V of the second
    const int slot = (int)(lane & 2 ? sl.y : sl.x);
    if (lane < 4 && slot >= 0) {
      const uint32_t dst = sbase + (uint32_t)(s * ge.stage_bytes) + (lane & 1 ? v_off : 0u) +
                           (lane & 2 ? (uint32_t)ge.half_bytes : 0u);
      const CUtensorMap* map = lane & 1 ? &maps.v : &maps.k;
      // (16 tokens are whole lines: their first line's number is exact)
      if (ge.hsplit == 1) i4::tma_2d(dst, map, (slot >> 4) * (tok_bytes >> 3), full);
      else i4::tma_4d(dst, map, hgrp, slot, full);
    }
    ++turn;
    return true;
  };
  // ---- per-piece state ---------------------------------------------------------
  const float log2e = 1.4426950408889634f;
  const float cap = p.soft_cap;
  const float base_scale = p.sm_scale * (cap > 0.0f ? 1.0f : log2e) * dev::kInt4Unit;
  const float cap_l2 = cap * log2e;
  const float inv_cap = cap > 0.0f ? 1.0f / cap : 0.0f;
  const int G = p.group;
  // r / G of a tile's row (r < kTileMaxRows; exact: r + 1/2 is half a row or more
  // from a multiple of G).  An integer division here, two for each score of a
  // piece's last chunk, took 6 us of a step of seven requests.
  const float inv_g = 1.0f / (float)G;
  auto div_g = [&](int r) -> int { return (int)(((float)r + 0.5f) * inv_g); };
  const int W = p.window;
  int cur = -1;                 // current piece, relative to the segment's first
  int all_lo = 0, all_hi = 0;   // tokens that all its rows see
  int len = 0, pos0 = 0, row0 = 0, row_end = 0;  // its keys, first query's position, rows
  float score_mul = 0.0f;
  uint32_t qf[NT][Row::kKsteps][2];
  float o[NT][Row::kMtiles][4];
  // a row's reference maximum less 6, in log2 units (the weights carry 2^6);
  // kUnset before its first visible key
  constexpr float kUnset = -1.0e30f;
  float m_off[NT][2], l_run[NT][2];
  // value scales enter as s 2^-ev, ev the exponent of the largest so far
  int ev = -1000;
  float sv_lim = 0.0f, to_ref = 0.0f;
  float al_slope[NT][2];
  int al_pos[NT][2];
  const int tok_g = i4::pi_of(g);  // MMA row g's token of a chunk; row g + 8's is the next

  // 2^e, e in [-126, 127] (-127: zero)
  auto exp2_int = [](int e) -> float { return __int_as_float((127 + e) << 23); };

  // A piece's descriptor (read again where it is needed: it does not stay in
  // registers) and its request's first query token.
  struct Piece {
    int req, row0, nrows, part, q0, pos0, len;
    bool bad;  // (bounds-checked build) its rows lie outside q / out
  };
  auto piece_at = [&](int rel) {
    Piece pc;
    if constexpr (DEV) {
      // The tile's part inside this segment; a cut tile's partial rows go to
      // one of the warp's two 16-row slots: 2 gw for the tile the segment
      // starts in, 2 gw + 1 for the one it ends in.
      const int r = first_piece + rel;
      const int f0 = prefix[r], f1 = prefix[r + 1];
      pc.req = r;
      pc.row0 = 0;
      pc.nrows = tiles[r].w;
      pc.len = tiles[r].z;
      pc.pos0 = pc.len - div_g(pc.nrows);
      pc.part = f0 < seg0 || f1 > seg0 + n ? (2 * gw + (f0 <= seg0 ? 0 : 1)) * kTileMaxRows : -1;
      pc.q0 = p.query_start_loc[r];
    } else {
      const int4* d = reinterpret_cast<const int4*>(p.pieces + first_piece + rel);
      const int4 a = __ldg(d), b = __ldg(d + 1), e = __ldg(d + 2);
      pc.req = a.x;
      pc.row0 = a.z;
      pc.nrows = a.w;
      pc.part = b.x;
      pc.len = b.w;  // (all keys its rows see; without causality all keys)
      pc.q0 = e.z;
      pc.pos0 = e.w;
    }
    pc.bad = false;
    if constexpr (KVQ_CHECKED && !DEV) {
      pc.bad = pc.q0 < 0 || pc.q0 + div_g(pc.row0 + pc.nrows - 1) >= p.total_q_tokens;
      if (pc.bad && lane == 0) atomicExch(p.error_flag, 2);
    }
    return pc;
  };
  // Start a piece: Q fragments (B operand of S^T = K Q^T) and masks.  Q enters
  // the MMA exactly: bf16 values scaled by a power of two only.  Lane c holds
  // dims 4 kRun i + kRun c + [0, kRun) of its rows.
  auto start_piece = [&](int rel) {
    const Piece pc = piece_at(rel);
    const int q0 = pc.q0;
    const int p_min = pc.pos0;
    const int p_max = pc.pos0 + div_g(pc.row0 + pc.nrows - 1);
    len = pc.len;
    pos0 = pc.pos0;
    row0 = pc.row0;
    row_end = pc.row0 + pc.nrows;
    all_lo = W > 0 ? p_max - W + 1 : 0;
    all_hi = p.causal ? p_min + 1 : len;
    float qv[NT][D / 4];
    float qmax = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int nr = 8 * t + g;
      const bool valid = nr < pc.nrows && !pc.bad;
      const int R = pc.row0 + (valid ? nr : 0);
      const int rq = div_g(R);
      const uint16_t* src =
          p.q + ((int64_t)(q0 + rq) * p.heads_q + head * G + R - rq * G) * D + Row::kRun * c;
#pragma unroll
      for (int i = 0; i < D / 4 / Row::kRun; ++i) {
#pragma unroll
        for (int h = 0; h < Row::kRun / 8; ++h) {
          const uint4 w = valid ? *reinterpret_cast<const uint4*>(src + 4 * Row::kRun * i + 8 * h)
                                : make_uint4(0, 0, 0, 0);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2) {
            const int e = Row::kRun * i + 8 * h + 2 * e2;
            qv[t][e] = dev::bf16_lo(ws[e2]);
            qv[t][e + 1] = dev::bf16_hi(ws[e2]);
            qmax = fmaxf(qmax, fmaxf(fabsf(qv[t][e]), fabsf(qv[t][e + 1])));
          }
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
    // Power-of-two shift that puts the largest |q| just under 2^15.
    int shift = 0;
    if (qmax > 0.0f && qmax < 3.0e38f) {
      int e;
      frexpf(qmax, &e);
      shift = max(-126, min(126, 15 - e));
    }
    const float q_mul = __int_as_float((127 + shift) << 23);
    const float q_unmul = __int_as_float((127 - shift) << 23);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int s = 0; s < Row::kKsteps; ++s) {
        qf[t][s][0] = dev::pack_f16x2(qv[t][4 * s] * q_mul, qv[t][4 * s + 1] * q_mul);
        qf[t][s][1] = dev::pack_f16x2(qv[t][4 * s + 2] * q_mul, qv[t][4 * s + 3] * q_mul);
      }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int nr = min(8 * t + 2 * c + e, pc.nrows - 1);
        if constexpr (AL) {
          const int rq = div_g(pc.row0 + nr);
          al_slope[t][e] = p.alibi_slopes[head * G + pc.row0 + nr - rq * G] * log2e;
          al_pos[t][e] = pos0 + rq;
        }
        m_off[t][e] = kUnset;
        l_run[t][e] = 0.0f;
      }
    score_mul = base_scale * q_unmul;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < Row::kMtiles; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
    ev = -1000;
    sv_lim = __uint_as_float(1u);  // (any positive scale moves it)
    to_ref = 0.0f;
  };

  // Finish a piece: its rows' outputs (or partials) straight from the MMA
  // fragments.
  auto finish_piece = [&](int rel) {
    const Piece pc = piece_at(rel);
    const int q0 = pc.q0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          l_run[t][e] += __shfl_xor_sync(0xffffffffu, l_run[t][e], off);
    const float unit = ev > -1000 ? exp2_int(ev) : 1.0f;
    // An attention sink joins the normaliser of a whole (uncut) tile here;
    // a cut tile's merge adds it once.
    if (p.sinks && pc.part < 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int nr = min(8 * t + 2 * c + e, pc.nrows - 1);
          const float sk = p.sinks[head * G + pc.row0 + nr - div_g(pc.row0 + nr) * G] * log2e;
          if (m_off[t][e] > kUnset && sk != -INFINITY)
            l_run[t][e] += exp2f(fminf(sk - m_off[t][e], 126.0f));
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int nr = 8 * t + 2 * c + e;
        if (nr >= pc.nrows) continue;
        const float l = l_run[t][e];
        // The value scales' power of two comes last: o / l is of the codes' size,
        // while 2^15 / l times the smallest scales' power would be subnormal (at l
        // = 2^30, a few ten thousand keys, it keeps 8 bits).
        const float sc = l > 0.0f ? dev::kInt4Unit / l : 0.0f;
        auto val = [&](int i, int h) -> float { return o[t][i][e + 2 * h] * sc * unit; };
        if (pc.part < 0) {
          if (pc.bad) continue;
          const int R = pc.row0 + nr, rq = div_g(R);
          uint16_t* dst = p.out + ((int64_t)(q0 + rq) * p.heads_q + head * G + R - rq * G) * D + g * (D / 8);
          // (the lane's group of D / 8 dims: m-tile i holds dims 2 i, 2 i + 1)
#pragma unroll
          for (int i = 0; i < Row::kMtiles; i += 4)
            *reinterpret_cast<uint4*>(dst + 2 * i) =
                make_uint4(dev::pack_bf16x2(val(i, 0), val(i, 1)), dev::pack_bf16x2(val(i + 1, 0), val(i + 1, 1)),
                           dev::pack_bf16x2(val(i + 2, 0), val(i + 2, 1)),
                           dev::pack_bf16x2(val(i + 3, 0), val(i + 3, 1)));
        } else {
          float* dst = p.part_o + (int64_t)(pc.part + nr) * D + g * (D / 8);
#pragma unroll
          for (int i = 0; i < Row::kMtiles; i += 2)
            *reinterpret_cast<float4*>(dst + 2 * i) =
                make_float4(val(i, 0), val(i, 1), val(i + 1, 0), val(i + 1, 1));
          if (g == 0)
            p.part_lse[pc.part + nr] = l > 0.0f ? m_off[t][e] + 6.0f + log2f(l) : -INFINITY;
        }
      }
  };

  // ---- stream the segment --------------------------------------------------------
  // Byte offsets, in a half, of what this lane reads: its K pieces of token
  // pi(g) and the next one (rows g and g + 8), those rows' tails, and its V
  // codes of tokens pi(2c), pi(2c + 1) and the ones after them.
  auto at = [&](int tok, int off) -> uint32_t {
    const uint32_t o = (uint32_t)(tok * tok_bytes + j * Row::kRow + off);
    return ge.swizzle ? o ^ ((o >> 3) & 0x70u) : o;
  };
  uint32_t k_at[2][Row::kK16], t_at[2], v_at[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    t_at[h] = at(tok_g + h, Row::kCodes);
#pragma unroll
    for (int q = 0; q < Row::kK16; ++q) k_at[h][q] = at(tok_g + h, Row::kKBytes * c + 64 * q);
#pragma unroll
    for (int r = 0; r < 2; ++r) v_at[2 * h + r] = v_off + at(i4::pi_of(2 * c + r) + h, Row::kVWords * 4 * g);
  }
  // multiplier bytes of this lane in a tail's two words: 2c and 2c + 1; at D
  // = 256 its K groups are c and c + 4
  const bool up = c >= 2;
  const uint32_t pair_sel = c & 1 ? 0x4342u : 0x4140u;          // (byte, 0x64) twice
  const uint32_t kpair_sel = (uint32_t)c | 0x40u | ((uint32_t)c << 8) | 0x4000u;

  // Iteration i reads chunk i and has chunk i + ahead copied (the first
  // `ahead` iterations only copy); the last one finishes the last piece.  The
  // first piece starts while the first copies are in flight; in the fused
  // step before the grid barrier (then in an iteration of its own).
  int st = 0, kst = 0, kw = 0;     // stage of chunk i; stage and warp of chunk i + ahead
  uint32_t par = 0, kpar = 0;
  if (DEV && own_plan) fill_records(0);
  for (int i = own_plan ? -ahead - 1 : -ahead;; ++i) {
    const bool before = i < -ahead;
    if (!before && i + ahead < n) {
      if (kw == j && !issue(kst, kpar, i < 1)) break;
      if (++kw == ge.hg) kw = 0;
      if (++kst == S) {
        kst = 0;
        kpar ^= 1u;
      }
    }
    if (!before && i < 0) continue;
    const uint32_t sb = sbase + (uint32_t)(st * ge.stage_bytes);
    const uint32_t mb = meta + 32u * st;
    uint4 rec = make_uint4(0u, 0u, 0u, 0u);
    if (i == n) rec.y = 0xFFFFFFFEu;
    else if (i > 0) {
      if (!i4::warp_wait(mb + 16, par, abort)) break;
      rec = dev::lds128(mb);
    }
    if ((int)rec.y != cur) {
      if (cur >= 0) finish_piece(cur);
      if (i == n) {
        if (!DEV && p.beside_prefill && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
      }
      cur = (int)rec.y;
      start_piece(cur);
    }
    if (before) {
      if (!join_grid()) return;
      continue;
    }
    if (i == 0) {
      if (!i4::warp_wait(mb + 16, par, abort)) break;
      rec = dev::lds128(mb);
    }
    const int tok0 = (int)rec.x;

    const uint32_t live = rec.z;
    const bool full = live == 0xFFFFFFFFu && tok0 >= all_lo && tok0 + kInt4Chunk <= all_hi;
    const uint32_t bias = 0x64646464u;  // f16 1024 + byte
    // S^T = K Q^T: the two halves of the chunk, 16 tokens x 8 rows per n-tile
    // each; and what the values' part needs of this stage.
    float s[2][NT][4], zm[2][2], sv[2][2];
    uint32_t vm[2][2], vc[2][4][Row::kVWords];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t ub = sb + (uint32_t)(u * ge.half_bytes);
      // tails: {s, m_0..3, m_4..7} of rows g and g + 8
      const uint4 tk[2] = {dev::lds128(ub + t_at[0]), dev::lds128(ub + t_at[1])};
      uint4 kc[2][Row::kK16];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < Row::kK16; ++q) {
          if constexpr (Row::kKBytes == 8) {
            const uint2 w = i4::lds64(ub + k_at[h][q]);
            kc[h][q] = make_uint4(w.x, w.y, 0, 0);
          } else {
            kc[h][q] = dev::lds128(ub + k_at[h][q]);
          }
        }
      dev::Int4Mul km[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        zm[u][h] = score_mul * __uint_as_float(tk[h].x);
        if constexpr (D == 256) {
          km[h][0] = dev::int4_mul(dev::prmt(tk[h].y, bias, kpair_sel));
          km[h][1] = dev::int4_mul(dev::prmt(tk[h].z, bias, kpair_sel));
        } else {
          const uint32_t pr = dev::prmt(up ? tk[h].z : tk[h].y, bias, pair_sel);
          km[h][0] = dev::int4_mul(dev::prmt(pr, pr, 0x1010u));
          km[h][1] = dev::int4_mul(dev::prmt(pr, pr, 0x3232u));
        }
      }
#pragma unroll
      for (int q = 0; q < Row::kK16; ++q) {
        const uint32_t w0[4] = {kc[0][q].x, kc[0][q].y, kc[0][q].z, kc[0][q].w};
        const uint32_t w1[4] = {kc[1][q].x, kc[1][q].y, kc[1][q].z, kc[1][q].w};
#pragma unroll
        for (int w = 0; w < Row::kKBytes / 4; ++w) {
          const int wi = q * (Row::kKBytes / 4) + w, half = wi >= Row::kKWords / 2 ? 1 : 0;
          uint32_t f[4], f8[4];
          dev::int4_to_f16x2x4(w0[w], km[0][half], f);
          dev::int4_to_f16x2x4(w1[w], km[1][half], f8);
          const uint32_t a0[4] = {f[0], f8[0], f[1], f8[1]}, a1[4] = {f[2], f8[2], f[3], f8[3]};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (wi == 0) dev::mma_f16_16816_zero(s[u][t], a0, qf[t][0][0], qf[t][0][1]);
            else dev::mma_f16_16816(s[u][t], a0, qf[t][2 * wi][0], qf[t][2 * wi][1]);
            dev::mma_f16_16816(s[u][t], a1, qf[t][2 * wi + 1][0], qf[t][2 * wi + 1][1]);
          }
        }
      }
      // values: codes of tokens pi(2c), pi(2c + 1) and the ones after them;
      // scales and multipliers of rows g and g + 8
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t a = ub + v_at[r];
        if constexpr (Row::kVWords == 1) {
          vc[u][r][0] = i4::lds32(a);
        } else if constexpr (Row::kVWords == 2) {
          const uint2 w = i4::lds64(a);
          vc[u][r][0] = w.x;
          vc[u][r][1] = w.y;
        } else {
          const uint4 w = dev::lds128(a);
          vc[u][r][0] = w.x;
          vc[u][r][1] = w.y;
          vc[u][r][2] = w.z;
          vc[u][r][3] = w.w;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 tv = dev::lds128(ub + v_off + t_at[h]);
        sv[u][h] = __uint_as_float(tv.x);
        vm[u][h] = dev::prmt(up ? tv.z : tv.y, bias, pair_sel);
      }
    }
    if (live != 0xFFFFFFFFu) {
      // Tokens outside the piece's keys (or in no block): whatever the stage
      // holds there takes no part.  (Their scores are replaced below.)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = (live >> (16 * u + tok_g + h)) & 1u;
          sv[u][h] = in ? sv[u][h] : 0.0f;
          vm[u][h] = in ? vm[u][h] : 0x64006400u;
        }
    }
    // every lane has read the stage
    __syncwarp();
    if (lane == 0) i4::mbar_arrive(mb + 24);

    // Weights P = 2^(z - m_off), z the score in log2 units.  A row's reference
    // moves only when a weight would pass 2^14 (f16's range), the value
    // scales' only when one is a binade larger: one vote for both.
    auto score = [&](int u, int t, int e) -> float {
      float v = s[u][t][e] * zm[u][e >> 1];
      if (cap > 0.0f) v = cap_l2 * dev::tanh_exp(v * inv_cap);
      const int at = 16 * u + tok_g + (e >> 1), tok = tok0 + at;
      if constexpr (AL)  // bias from the exact integer distance, after the cap
        v = fmaf(al_slope[t][e & 1], (float)(tok - al_pos[t][e & 1]), v);
      if (!full) {  // (rare: the edges of a request's keys) the column's own keys
        const int pn = pos0 + div_g(min(row0 + 8 * t + 2 * c + (e & 1), row_end - 1));
        const bool vis = ((live >> at) & 1u) && tok >= (W > 0 ? pn - W + 1 : 0) && tok < (p.causal ? pn + 1 : len);
        v = vis ? v : -INFINITY;
      }
      return v;
    };
    // (x: the weights' exponents, or, where a score takes more than a product,
    // the scores until the reference has been settled)
    const bool plain = !AL && full && !(cap > 0.0f);
    float x[2][NT][4], xmax = -INFINITY;
    if (plain) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[u][t][e] = fmaf(s[u][t][e], zm[u][e >> 1], -m_off[t][e & 1]);
            xmax = fmaxf(xmax, x[u][t][e]);
          }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[u][t][e] = score(u, t, e);
            xmax = fmaxf(xmax, x[u][t][e] - m_off[t][e & 1]);
          }
    }
    const float sv_max = fmaxf(fmaxf(sv[0][0], sv[0][1]), fmaxf(sv[1][0], sv[1][1]));
    if (__any_sync(0xffffffffu, xmax > 14.0f || sv_max >= sv_lim)) {
      float mx = sv_max;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      float alpha_v = 1.0f;
      if (mx > 0.0f) {
        // (a finite row's scale is below 2^119)
        const int e = max(-126, min(118, (int)((__float_as_uint(mx) >> 23) & 0xFFu) - 127));
        if (e > ev) {
          alpha_v = exp2_int(max(ev - e, -127));
          ev = e;
          to_ref = exp2_int(-e);
          sv_lim = exp2_int(e + 1);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float z[4];
#pragma unroll
          for (int i2 = 0; i2 < 4; ++i2) {
            const int u = i2 >> 1, k = e + 2 * (i2 & 1);
            z[i2] = plain ? s[u][t][k] * zm[u][k >> 1] : x[u][t][k];
          }
          float cm = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, off));
          // (only a row that passed its limit moves: to the chunk's maximum,
          // whose weight is 2^6)
          const float mn = cm > m_off[t][e] + 14.0f ? cm - 6.0f : m_off[t][e];
          alpha[e] = dev::fast_exp2(m_off[t][e] - mn);
          m_off[t][e] = mn;
          l_run[t][e] *= alpha[e];
#pragma unroll
          for (int i2 = 0; i2 < 4; ++i2) x[i2 >> 1][t][e + 2 * (i2 & 1)] = z[i2] - mn;
        }
#pragma unroll
        for (int i2 = 0; i2 < Row::kMtiles; ++i2) {
          o[t][i2][0] *= alpha[0] * alpha_v;
          o[t][i2][1] *= alpha[1] * alpha_v;
          o[t][i2][2] *= alpha[0] * alpha_v;
          o[t][i2][3] *= alpha[1] * alpha_v;
        }
      }
    } else if (!plain) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][t][e] -= m_off[t][e & 1];
    }

    // O^T += V^T P^T : head_dim x 8 rows per n-tile.  The low halves of word
    // w of a row hold the even dims of its 8, the high halves the odd ones:
    // nibble q of each pairs two tokens' codes of dim 8 w + 2 q (+ 1), the
    // two rows of m-tile 4 w + q.
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float f0 = sv[u][0] * to_ref, f1 = sv[u][1] * to_ref;
      uint32_t pb0[NT], pb1[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float p0 = dev::fast_exp2(x[u][t][0]), p1 = dev::fast_exp2(x[u][t][1]);
        const float p2 = dev::fast_exp2(x[u][t][2]), p3 = dev::fast_exp2(x[u][t][3]);
        l_run[t][0] += p0 + p2;
        l_run[t][1] += p1 + p3;
        // P^T (tokens x rows) -> B operand of O^T = V^T P^T via transposes.
        pb0[t] = dev::movmatrix_trans(dev::pack_f16x2(p0 * f0, p1 * f0));
        pb1[t] = dev::movmatrix_trans(dev::pack_f16x2(p2 * f1, p3 * f1));
      }
      // V's multipliers, transposed to the token pairs its codes form
      const dev::Int4Mul vf0 = dev::int4_mul(dev::movmatrix_trans(vm[u][0]));
      const dev::Int4Mul vf1 = dev::int4_mul(dev::movmatrix_trans(vm[u][1]));
#pragma unroll
      for (int w = 0; w < Row::kVWords; ++w) {
        uint32_t e01[4], o01[4], e23[4], o23[4];
        dev::int4_to_f16x2x4(dev::prmt(vc[u][0][w], vc[u][1][w], 0x5410u), vf0, e01);
        dev::int4_to_f16x2x4(dev::prmt(vc[u][0][w], vc[u][1][w], 0x7632u), vf0, o01);
        dev::int4_to_f16x2x4(dev::prmt(vc[u][2][w], vc[u][3][w], 0x5410u), vf1, e23);
        dev::int4_to_f16x2x4(dev::prmt(vc[u][2][w], vc[u][3][w], 0x7632u), vf1, o23);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t a[4] = {e01[q], o01[q], e23[q], o23[q]};
#pragma unroll
          for (int t = 0; t < NT; ++t) dev::mma_f16_16816(o[t][4 * w + q], a, pb0[t], pb1[t]);
        }
      }
    }

    if (++st == S) {
      st = 0;
      par ^= 1u;
    }
  }
  // A wait was given up: the error word, NaN rows for this and the segment's
  // remaining pieces, and a bounded wait for what may still be in flight
  // before the CTA's shared memory is released.
  if (lane == 0) atomicExch(p.error_flag, 1);
  for (int rel = max(cur, 0); first_piece + rel < (DEV ? sp.num_req : p.num_pieces); ++rel) {
    const int f0 = DEV ? prefix[first_piece + rel] : p.pieces[first_piece + rel].flat0;
    if (f0 >= seg0 + n) break;
    const Piece pc = piece_at(rel);
    for (int r = 0; r < pc.nrows && !pc.bad; ++r) {
      const int R = pc.row0 + r;
      for (int d = lane; d < D; d += 32) {
        if (pc.part >= 0) p.part_o[(int64_t)(pc.part + r) * D + d] = NAN;
        else p.out[((int64_t)(pc.q0 + R / G) * p.heads_q + head * G + R % G) * D + d] = 0x7FC0u;
      }
      if (pc.part >= 0 && lane == 0) p.part_lse[pc.part + r] = 0.0f;
    }
  }
  for (int s = 0; s < S; ++s)
    (void)tc::mbar_wait(meta + 32u * s + 16, s < kst ? kpar : kpar ^ 1u, 200000000LL);
  if (!DEV && p.beside_prefill && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The launches' shared memory limit, raised once per device.
inline bool int4_raise_smem(const void* kern, std::atomic<bool>* raised) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (dev < kMaxCachedDevices && raised[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kInt4MaxSmem) !=
      cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (dev < kMaxCachedDevices) raised[dev].store(true, std::memory_order_release);
  return true;
}

template <int D, int NT, bool AL>
int launch_int4_decode(const AttnParams& p, const PrefillMaps& maps, cudaStream_t stream) {
  Int4Geom ge = int4_geom(p.heads_kv, D, NT);
  ge.segments = p.num_warps / p.heads_kv;
  auto kern = int4_decode_kernel<D, NT, AL, false>;
  static std::atomic<bool> raised[kMaxCachedDevices];
  if (!int4_raise_smem(reinterpret_cast<const void*>(kern), raised)) return KVQ_E_CUDA;
  // A programmatic dependent of the kernel before it on the stream (it waits
  // for that one's completion after reading its plan).
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  const int groups = ge.segments * ge.hsplit, least = (groups + ge.gpc - 1) / ge.gpc;
  // (beside units a CTA an SM that they leave: one more would wait for a unit to end.
  // 64 requests, 16 of them behind 2,048 keys and all of some 1,000 of their own, 16 / 4 heads
  // of 256: 78 us with a CTA for every SM of the device, 55 so)
  if (p.decode_sms > 0 && p.decode_sms < sms) sms = p.decode_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(least > sms ? least : groups < sms ? groups : sms));
  cfg.blockDim = dim3((unsigned)(32 * ge.hg * ge.gpc));
  cfg.dynamicSmemBytes = ge.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  StepParams none{};
  if (cudaLaunchKernelEx(&cfg, kern, p, none, ge, maps) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  return KVQ_OK;
}

// The fused step: every CTA resident at once (a cooperative launch), as many
// as fit on the device; *warps counts segments times kv heads (0 asks for
// that number instead).
template <int D, int NT, bool AL>
int launch_int4_step(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, int64_t* warps,
                     cudaStream_t stream) {
  Int4Geom ge = int4_geom(p.heads_kv, D, NT);
  auto kern = int4_decode_kernel<D, NT, AL, true>;
  int dev = 0, sms = 0, per_sm = 0;
  const int threads = 32 * ge.hg * ge.gpc;
  // resident CTAs per SM of each geometry (a step asks twice, and the query
  // costs microseconds), by device and kv heads
  constexpr int kHeads = 64;
  static std::atomic<int> resident[kMaxCachedDevices][kHeads];
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  const bool kept = dev < kMaxCachedDevices && p.heads_kv < kHeads;
  if (kept) per_sm = resident[dev][p.heads_kv].load(std::memory_order_acquire);
  if (per_sm <= 0) {
    static std::atomic<bool> raised[kMaxCachedDevices];
    if (!int4_raise_smem(reinterpret_cast<const void*>(kern), raised) ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, ge.smem) != cudaSuccess ||
        per_sm <= 0) {
      cudaGetLastError();
      return KVQ_E_CUDA;
    }
    if (kept) resident[dev][p.heads_kv].store(per_sm, std::memory_order_release);
  }
  const int64_t ctas = (int64_t)sms * per_sm;
  ge.segments = (int)(ctas * ge.gpc / ge.hsplit);
  if (ge.segments == 0) return KVQ_E_UNSUPPORTED;  // more head groups than resident
  const int64_t want = (int64_t)ge.segments * p.heads_kv;
  if (*warps == 0) {
    *warps = want;
    return KVQ_OK;
  }
  if (*warps != want) return KVQ_E_INVALID_ARG;
  AttnParams pp = p;
  StepParams ss = sp;
  PrefillMaps mm = maps;
  void* args[] = {&pp, &ss, &ge, &mm};
  if (cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3((unsigned)ctas), dim3(threads),
                                  args, ge.smem, stream) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  return KVQ_OK;
}

template <int D, bool AL>
int launch_int4_decode_d(const AttnParams& p, const PrefillMaps& maps, int ntiles, cudaStream_t stream) {
  return ntiles == 1 ? launch_int4_decode<D, 1, AL>(p, maps, stream)
                     : launch_int4_decode<D, 2, AL>(p, maps, stream);
}
template <int D, bool AL>
int launch_int4_step_d(const AttnParams& p, const StepParams& sp, const PrefillMaps& maps, int64_t* warps,
                       cudaStream_t stream) {
  return sp.max_rows <= 8 ? launch_int4_step<D, 1, AL>(p, sp, maps, warps, stream)
                          : launch_int4_step<D, 2, AL>(p, sp, maps, warps, stream);
}

}  // namespace kvq
