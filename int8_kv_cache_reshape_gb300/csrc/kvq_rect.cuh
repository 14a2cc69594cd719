// kvq_rect.cuh -- attention of many rows to one run of cached keys, without
// a causal edge inside it: the keys of a prefix that requests share, or an
// encoder's keys (5th-generation tensor cores, accumulators in tensor memory).
//
// What it computes: a unit is up to 256 packed (query token, head) rows of
// one kv head -- 128 at head_dim 256 -- and a range of keys read through one
// block-table row.  For each row r: the reference m_r, l_r = sum_j 2^(z_rj -
// m_r + 6) and o_r = sum_j 2^(z_rj - m_r + 6) v_j / l_r over the range's keys
// that it sees (all, but for a sliding window), z in log2 units with the scale, the
// soft cap and the ALiBi bias.  Units that hold all keys of their rows write
// bf16 rows; others leave (o_r, m_r + log2 l_r) in fp32 for the merge.
//
// Why a kernel of its own beside the prefill (kvq_prefill.cuh): a prefix is
// converted to f16 once per 256 rows, so the converters stay below the MMAs'
// pace; two row tiles share each KV tile and the tensor core always has the
// other tile's product to run while one tile's softmax works; the keys
// of one row tile may be cut among many CTAs, which a causal prefill need not be.
//
// Layout (one CTA per SM, one unit per CTA; 16 warps):
//   warps 0, 1 issue the MMAs, a thread for each softmax group (head_dim 256: warp 0)
//   warp 2     resolves 16-key chunks through the block table into slots, up to
//              four KV tiles ahead
//   warp 3     the KV tiles' side data: per-key scales, chunk mask
//   converters two warps (head_dim 256: four) for K and as many for V, each thread 16
//              codes (4-bit: 32) of a key at a time, loaded into registers a KV tile
//              ahead, converted exactly to f16 and stored in the 128-byte swizzle into
//              two-stage rings; bf16 rows are copied as they are (cp.async, dead keys
//              zero)
//   softmax    two warpgroups (head_dim 256: one), thread = row = tensor-memory lane;
//              it holds the item's 64 scores of its row in registers
// Items: an item is S = Q K^T of a row tile against 64 keys and then O += P V; the
// softmax turns S into P in place.  A softmax group has its own items, k = 0, 1, ..,
// and two S buffers, so that S(k + 1) is there when it is done with S(k); S(k + 2)
// follows P V (k).  Each group's MMAs come from a thread of their own: the
// barriers and commits of an item take a thread some 700 cycles beside its MMAs,
// which is 640 cycles' work (4 x 1,024 tokens of 32 / 8 heads of 128 to 4,096 fp8 keys:
// 235 us with one thread for both, 215 us with two).
//   two row tiles (129 to 256 rows): each group has a row tile and all keys
//   one row tile (up to 128 rows): both have its rows and take the halves of each
//     KV tile, with an O of their own: two partials a row, or, where the unit holds
//     all keys, joined through shared memory
//   head_dim 256: O takes half of tensor memory; one row tile, one group
// (Items of 128 keys leave no room for a second S: with P in S's place the next S
// waits for the P V, 4,280 cycles a 128-key tile of two row tiles of which 2,048 are MMA
// work; with P beside one S of both groups the chain S, load, S is as long.  N = 64
// reads Q from shared memory twice as often: 2,560 cycles of its bandwidth a tile.)
// Numbers as in the prefill: Q enters as f16 scaled by a power of two per row
// (bf16 rows: as it is), scales multiply fp32 scores, value scales fold into P against
// a running power of two, the reference m is an integer that moves when a score
// exceeds it by 2^8, every sum is fp32.  P is f16 (11 bits; bf16 rows: two bf16
// numbers, 16 bits): the operand type of the MMA.
// Bound by the chain S, softmax, P of a row tile: a 128-key tile of two row tiles takes
// some 3,800 cycles where its MMAs take 2,560, the tensor pipe is busy 57 to 62 %
// of the time, the issue slots 52 to 54 %.  4 x 1,024 tokens of 32 / 8 heads of 128 to 4,096 fp8
// keys: 205 to 215 us, 1.06 PFLOP/s.  Short runs are bound by a unit's fixed time, about
// 6 to 8 us (Q, first keys and instructions, the rows' way out).
// Every wait is bounded (about a second); a unit that gave up leaves NaN rows and
// sets the schedule's error word.
#pragma once

#include "kvq_prefill.cuh"

namespace kvq {

template <int DT, int D>
struct RectGeom {
  static constexpr bool kAuto = DT == KVQ_AUTO, kInt4 = is_int4(DT), kPth = is_per_token_head(DT);
  static constexpr int kRT = rect_row_tiles(D);       // row tiles with an O of their own
  static constexpr int kM = 128, kN = prefill_keys(D);
  static constexpr int kThreads = 512;
  static constexpr int kConv = kRT == 2 ? 64 : 128;   // converter threads of K, and of V
  static constexpr int kSoftWg = kRT == 2 ? 2 : 3;    // first softmax warpgroup
  static constexpr int kStages = 2, kSide = 4, kSlotRing = 4;
  static constexpr int kQBytes = kM * D * 2;          // a row tile's Q
  static constexpr int kTileBytes = kN * D * 2;       // a KV tile's K or V
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kRT * kQBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffSk = kOffV + kStages * kTileBytes;   // kSide x kN f32
  static constexpr int kOffSv = kOffSk + kSide * kN * 4;        // kSide x kN f32
  static constexpr int kOffSMask = kOffSv + kSide * kN * 4;     // kSide u32 masks, kSide i32 exponents
  static constexpr int kOffSlots = kOffSMask + kSide * 8;       // kSlotRing x 16 i32
  static constexpr int kOffQScale = kOffSlots + kSlotRing * 64; // kM f32 (of one row tile)
  static constexpr int kOffBar = kOffQScale + kM * 4;
  static constexpr int kBytes = kOffBar + 320;
  static constexpr int kItem = 64;                    // keys of an item
  static constexpr int kItems = kN / kItem;           // items of a KV tile
  static constexpr int kColO = 0, kColS = kRT * D;    // O of each group; its two S (P in place)
  static constexpr int kTmemCols = 512;
  static constexpr int kBarSlots = 0, kBarSlotsFree = 4, kBarSide = 8, kBarKFull = 12, kBarVFull = 14, kBarKEmpty = 16,
                       kBarVEmpty = 18, kBarSFull = 20, kBarPFull = 24, kBarODone = 28, kBarQFull = 30, kBarDrain = 32,
                       kBarOFinal = 34, kNumBars = 36;
  static constexpr int kOffTmemSlot = kOffBar + 8 * kNumBars, kOffAbort = kOffTmemSlot + 4;
  static_assert(kColS + kRT * 2 * kItem <= kTmemCols, "tensor memory");
  static_assert(kQBytes % 1024 == 0 && kTileBytes % 1024 == 0 && kOffBar % 8 == 0 && kOffSk % 16 == 0, "alignment");
  static_assert(kOffAbort + 4 <= kBytes && (size_t)kBytes + 1024 == rect_smem_bytes(D), "shared memory");
};

// Registers a thread of each warpgroup, out of the launch's 512 x 128.
template <int D>
struct RectRegs {
  static constexpr int kIssue = D >= 256 ? 96 : 104, kConvert = 104, kSoftmax = D >= 256 ? 208 : 152;
  static_assert(kIssue + (D >= 256 ? 2 : 1) * kConvert + rect_row_tiles(D) * kSoftmax <= 4 * 128,
                "the groups' registers come out of the launch's");
};

// wait_or_abort with the second look and the rest out of the way (what the warps
// run between waits has to stay in the instruction caches).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  if (__builtin_expect(tc::mbar_try_wait(bar, parity), 1)) return true;
  const long long t0 = clock64();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (*abort != 0u || clock64() - t0 > 2000000000LL) {  // about a second
      *abort = 1u;
      return false;
    }
  }
  return true;
}

template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}

// GEN: with a soft cap or ALiBi (an instance of its own keeps the code of the others
// small).
template <int DT, int D, bool GEN>
__global__ void __launch_bounds__(512, 1) rect_attention_kernel(const AttnParams p, const RectParams rp) {
  using Geo = RectGeom<DT, D>;
  using Regs = RectRegs<D>;
  constexpr int kM = Geo::kM, kN = Geo::kN, kRT = Geo::kRT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
  const uint32_t bars = base + Geo::kOffBar;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(sm + Geo::kOffAbort);

  // (the plan, which no kernel writes, ahead of the wait below)
  const int4* const rec = reinterpret_cast<const int4*>(rp.units + blockIdx.x);
  const int4 u0 = __ldg(rec), u1 = __ldg(rec + 1);
  const int part_stride = __ldg(&rp.units[blockIdx.x].part_stride);
  const int kv_head = u0.x, row0 = u0.y, nrows = u0.z, kv_lo = u0.w;
  const int kv_hi = u1.x, tok0 = u1.y, req = u1.z, part0 = u1.w;
  const int G = p.group;
  const bool two = kRT == 2 && nrows > kM;  // two row tiles, else one
  // a softmax thread's row: tile t (one row tile: both groups take it), row m;
  // its token's row of q and out and position
  const int t = wg - Geo::kSoftWg, m = tid & 127, tile = two && t == 1 ? 1 : 0, R = tile * kM + m;
  const bool row_valid = t >= 0 && R < nrows;
  int2 token = make_int2(0, 0);
  int row_g = 0;
  if (row_valid) {
    const int packed = row0 + R, q = packed / G;
    row_g = packed - q * G;
    token = __ldg(reinterpret_cast<const int2*>(rp.tokens) + tok0 + q);
  }

  // (a barrier a thread: code that runs once is fetched line by line, some 250
  // cycles each)
  if (tid < Geo::kNumBars) {
    const int arrivals = tid >= Geo::kBarSlotsFree && tid < Geo::kBarSide  ? 2 * Geo::kConv / 32 + 1
                         : tid >= Geo::kBarKFull && tid < Geo::kBarKEmpty  ? Geo::kConv / 32
                         : tid >= Geo::kBarKEmpty && tid < Geo::kBarSFull  ? kRT
                         : (tid >= Geo::kBarPFull && tid < Geo::kBarODone) ||
                                   (tid >= Geo::kBarQFull && tid < Geo::kBarDrain)
                             ? 4
                             : 1;
    tc::mbar_init(bar(tid), (uint32_t)arrivals);
    if (tid == 0) *abort_flag = 0u;
    tc::mbar_fence_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(base + Geo::kOffTmemSlot, Geo::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + Geo::kOffTmemSlot);
  // A programmatic dependent of the kernel ahead: nothing that it wrote is
  // read before this wait, and what comes after this kernel may start only now.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int kv_first = kv_lo / kN * kN;
  const int T = (kv_hi - kv_first + kN - 1) / kN;  // KV tiles (one at least)
  constexpr int kChunks = kN / 16;
  constexpr uint32_t kAllChunks = (1u << kChunks) - 1u;

  auto wait = [&](int b, int phase) {  // (of a whole warp)
    return __all_sync(0xffffffffu, wait_bar(bar(b), (uint32_t)(phase & 1), abort_flag));
  };
  // the live keys of KV tile g, relative to its first
  auto live_lo = [&](int g) { return max(kv_lo - (kv_first + g * kN), 0); };
  auto live_hi = [&](int g) { return min(kv_hi - (kv_first + g * kN), kN); };

  if (wg == 0) {
    regs_down<Regs::kIssue>();
    if (warp < kRT) {
      // ---- MMA issuer of softmax group `warp` (see the items above): one thread,
      // so that a wait costs one barrier test and no vote --------------------
      if (elect_one()) {
        auto wait1 = [&](int b, int phase) { return wait_bar(bar(b), (uint32_t)(phase & 1), abort_flag); };
        constexpr uint32_t idesc_s = Geo::kAuto ? tc::idesc_bf16(kM, Geo::kItem) : tc::idesc_f16(kM, Geo::kItem);
        constexpr uint32_t idesc_o = (Geo::kAuto ? tc::idesc_bf16(kM, D) : tc::idesc_f16(kM, D)) | tc::kBMajorMN;
        // the group's items of a KV tile: all, or (one row tile) one of the halves
        const bool all = kRT == 1 || two;
        const int qt = two ? warp : 0, count = all ? Geo::kItems * T : T;
        const uint64_t dq = tc::desc_sw128(base + Geo::kOffQ + (uint32_t)(qt * Geo::kQBytes));
        const uint32_t s_at = tmem + (uint32_t)(Geo::kColS + warp * 2 * Geo::kItem);
        const uint32_t o_at = tmem + (uint32_t)(Geo::kColO + warp * D);
        const uint64_t dk0 = tc::desc_sw128(base + Geo::kOffK), dv0 = tc::desc_sw128_mn(base + Geo::kOffV, kN * 128, 1024);
        bool ok = wait1(Geo::kBarQFull + qt, 0);
        for (int k = -2; k < count && ok; ++k) {
          if (k >= 0) {
            // O += P V (k)
            const int g = all ? k / Geo::kItems : k, h = all ? k % Geo::kItems : warp, st = g & 1;
            if (!(ok = wait1(Geo::kBarPFull + 2 * warp + (k & 1), k >> 1))) break;
            if ((!all || h == 0) && !(ok = wait1(Geo::kBarVFull + st, g >> 1))) break;
            tc::fence_after_sync();
            const uint64_t dv = dv0 + (uint64_t)((st * Geo::kTileBytes + h * Geo::kItem * 128) >> 4);
            const uint32_t p_at = s_at + (uint32_t)((k & 1) * Geo::kItem);
#pragma unroll
            for (int kk = 0; kk < Geo::kItem / 16; ++kk) {
              const uint64_t dvk = dv + (uint64_t)(kk * (2048 >> 4));
              tc::mma_ts(o_at, p_at + (uint32_t)(kk * 8), dvk, idesc_o, (k > 0 || kk > 0) ? 1u : 0u);
              // (bf16 rows: P = hi + lo, both bf16, lo 32 columns on)
              if constexpr (Geo::kAuto) tc::mma_ts(o_at, p_at + (uint32_t)(32 + kk * 8), dvk, idesc_o, 1u);
            }
            if (!all || h == Geo::kItems - 1) tc::mma_commit(bar(Geo::kBarVEmpty + st));
            // (the S after next stands for the others)
            if (k >= count - 2) tc::mma_commit(bar((k == count - 1 ? Geo::kBarOFinal : Geo::kBarODone) + warp));
          }
          const int k2 = k + 2;
          if (k2 < count) {
            // S (k + 2)
            const int g = all ? k2 / Geo::kItems : k2, h = all ? k2 % Geo::kItems : warp, st = g & 1;
            if ((!all || h == 0) && !(ok = wait1(Geo::kBarKFull + st, g >> 1))) break;
            tc::fence_after_sync();
            const uint64_t dk = dk0 + (uint64_t)((st * Geo::kTileBytes + h * Geo::kItem * 128) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t qoff = (kk >> 2) * (kM * 128) + (kk & 3) * 32, koff = (kk >> 2) * (kN * 128) + (kk & 3) * 32;
              // (kind::f16: the instruction descriptor names the 16-bit type)
              tc::mma_bf16(s_at + (uint32_t)((k & 1) * Geo::kItem), dq + (uint64_t)(qoff >> 4), dk + (uint64_t)(koff >> 4),
                           idesc_s, kk > 0 ? 1u : 0u);
            }
            tc::mma_commit(bar(Geo::kBarSFull + 2 * warp + (k & 1)));
            if (!all || h == Geo::kItems - 1) tc::mma_commit(bar(Geo::kBarKEmpty + st));
          }
        }
        if (!ok) {
          // drain what was issued before the tensor memory is freed
          tc::mma_commit(bar(Geo::kBarDrain + warp));
          (void)tc::mbar_wait(bar(Geo::kBarDrain + warp), 0u, 200000000LL);
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---- slots of the KV tiles' 16-key chunks --------------------------
      // (entries are loaded a tile ahead; the block size is a multiple of 16;
      // q = hi32(j floor((2^32 - 1) / B)) is the quotient or one less)
      const int32_t* const btab = p.block_table + (int64_t)req * p.block_table_stride;
      const uint32_t bsz = (uint32_t)p.block_size, bdiv = 0xFFFFFFFFu / bsz;
      int32_t* const table = reinterpret_cast<int32_t*>(sm + Geo::kOffSlots);
      // lane c < kChunks looks after chunk c
      auto fetch = [&](int g, int& blk, int& off) {
        blk = -1;
        off = 0;
        const int j0 = kv_first + g * kN + 16 * lane;
        if (lane < kChunks && g < T && j0 + 16 > kv_lo && j0 < kv_hi) {
          uint32_t q = __umulhi((uint32_t)j0, bdiv), r = (uint32_t)j0 - q * bsz;
          if (r >= bsz) {
            ++q;
            r -= bsz;
          }
          blk = __ldcg(btab + q);
          off = (int)r;
        }
      };
      int blk, off;
      fetch(0, blk, off);
      for (int g = 0; g < T; ++g) {
        const int e = g & 3;
        if (g >= 4 && !__all_sync(0xffffffffu, wait_bar(bar(Geo::kBarSlotsFree + e), (uint32_t)(((g >> 2) - 1) & 1),
                                                             abort_flag)))
          break;
        const bool in = blk >= 0 && (int64_t)blk < p.num_blocks;
        const uint32_t mask = __ballot_sync(0xffffffffu, in);
        if (lane < kChunks) table[e * 16 + lane] = in ? blk * (int)bsz + off : 0;  // < num_blocks * block_size < 2^31
        if (lane == 15) table[e * 16 + 15] = (int32_t)mask;
        warp_arrive(bar(Geo::kBarSlots + e));
        fetch(g + 1, blk, off);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ---- side data for the softmax, in slot g mod 4 ----------------------
      // (its last reader, of KV tile g - 4, is done: P(g - 2) V(g - 2) is complete)
      const int32_t* const table = reinterpret_cast<const int32_t*>(sm + Geo::kOffSlots);
      float* const sk = reinterpret_cast<float*>(sm + Geo::kOffSk);
      float* const sv = reinterpret_cast<float*>(sm + Geo::kOffSv);
      uint32_t* const smask = reinterpret_cast<uint32_t*>(sm + Geo::kOffSMask);
      int32_t* const sev = reinterpret_cast<int32_t*>(sm + Geo::kOffSMask + Geo::kSide * 4);
      constexpr int kKeys = kN / 32;  // keys of a thread
      constexpr int64_t kRow = row_bytes(DT, D);
      const int64_t tail = kv_head * kRow + code_bytes(DT, D), tok_bytes = (int64_t)p.heads_kv * kRow;
      float ks[kKeys], vs[kKeys];
      uint32_t valid = 0;
      int ev = -1000;  // exponent of the value scales' reference
      auto load = [&](int g) -> bool {
        const int e = g & 3;
        if (!wait(Geo::kBarSlots + e, g >> 2)) return false;
        valid = (uint32_t)table[e * 16 + 15];
        if constexpr (Geo::kPth) {
          const int lo = live_lo(g), hi = live_hi(g);
#pragma unroll
          for (int x = 0; x < kKeys; ++x) {
            const int nn = lane + 32 * x;
            ks[x] = vs[x] = 0.0f;  // (of a dead key)
            if (((valid >> (nn >> 4)) & 1u) && nn >= lo && nn < hi) {
              const int64_t off = (int64_t)(table[e * 16 + (nn >> 4)] + (nn & 15)) * tok_bytes + tail;
              ks[x] = __ldcg(reinterpret_cast<const float*>(p.key_cache + off));
              vs[x] = __ldcg(reinterpret_cast<const float*>(p.value_cache + off));
            }
          }
        }
        warp_arrive(bar(Geo::kBarSlotsFree + e));
        return true;
      };
      bool ok = true;
      for (int g = 0; g < T; ++g) {
        if (!(ok = load(g))) break;
        const int sd = g & 3;
        float to_ref = 0.0f;
        if constexpr (Geo::kPth) {
          // value scales relative to the largest power of two so far, 2^ev
          float vmax = 0.0f;  // (a NaN or negative scale is ignored)
#pragma unroll
          for (int x = 0; x < kKeys; ++x) vmax = fmaxf(vmax, vs[x]);
          const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(vmax));
          // (2^e above the largest scale, by its exponent bits)
          if (mb != 0u) ev = max(ev, max(-125, min(126, (int)(mb >> 23) - 126)));
          // (no positive scale yet: values are zero)
          to_ref = ev > -1000 ? __int_as_float((127 - ev) << 23) : 0.0f;
        }
        if (g >= 2 && !wait(Geo::kBarVEmpty + (g & 1), (g >> 1) - 1)) break;
        if (lane == 0) smask[sd] = valid;
        if constexpr (Geo::kPth) {
#pragma unroll
          for (int x = 0; x < kKeys; ++x) {
            sk[sd * kN + lane + 32 * x] = ks[x];
            sv[sd * kN + lane + 32 * x] = vs[x] * to_ref;
          }
          if (lane == 0) sev[sd] = ev;
        }
        warp_arrive(bar(Geo::kBarSide + sd));
      }
      __syncwarp();
    }
  } else if (wg < Geo::kSoftWg) {
    // ---- converters: K, then V ---------------------------------------------
    regs_down<Regs::kConvert>();
    const bool for_v = tid - 128 >= Geo::kConv;
    const int ct = (tid - 128) % Geo::kConv;
    const uint8_t* const cache = for_v ? p.value_cache : p.key_cache;
    const uint32_t tiles = base + (for_v ? Geo::kOffV : Geo::kOffK);
    const int bar_empty = for_v ? Geo::kBarVEmpty : Geo::kBarKEmpty, bar_full = for_v ? Geo::kBarVFull : Geo::kBarKFull;
    const int32_t* const table = reinterpret_cast<const int32_t*>(sm + Geo::kOffSlots);
    constexpr int64_t kRow = row_bytes(DT, D);
    const int64_t tok_bytes = (int64_t)p.heads_kv * kRow;
    const uint8_t* const head_at = cache + kv_head * kRow;
    if constexpr (Geo::kAuto) {
      // 16-byte pieces of bf16 rows straight into the operand tile; a stage's
      // copies are in flight while the next stage's are issued
      constexpr int kPieces = D / 8, kStepN = Geo::kConv / kPieces, kCopies = kN / kStepN;
      const int pc = ct % kPieces, n0 = ct / kPieces;
      auto done = [&](int g) {
        tc::fence_async_smem();
        warp_arrive(bar(bar_full + (g & 1)));
      };
      bool ok = true;
      for (int g = 0; g < T; ++g) {
        const int e = g & 3, st = g & 1;
        if (!(ok = wait(Geo::kBarSlots + e, g >> 2))) break;
        if (g >= 2 && !(ok = wait(bar_empty + st, (g >> 1) - 1))) break;
        const uint32_t valid = (uint32_t)table[e * 16 + 15];
        const int lo = live_lo(g), hi = live_hi(g);
#pragma unroll 8
        for (int i = 0; i < kCopies; ++i) {
          const int nn = n0 + i * kStepN;
          const bool on = ((valid >> (nn >> 4)) & 1u) && nn >= lo && nn < hi;
          const int64_t slot = on ? table[e * 16 + (nn >> 4)] + (nn & 15) : 0;
          dev::cp_async_16(tiles + (uint32_t)(st * Geo::kTileBytes + (pc >> 3) * kN * 128 + nn * 128 +
                                              (((pc & 7) ^ (nn & 7)) << 4)),
                           head_at + slot * tok_bytes + 16 * pc, on ? 16 : 0);
        }
        dev::cp_async_commit();
        warp_arrive(bar(Geo::kBarSlotsFree + e));
        if (g > 0) {
          dev::cp_async_wait<1>();
          done(g - 1);
        }
      }
      dev::cp_async_wait<0>();
      if (ok) done(T - 1);
    } else {
      // units of (key, 16 codes) or, 4-bit, (key, 32 codes): a thread keeps its piece
      // of the row, and its keys differ by a multiple of 8, so that its offsets in
      // the swizzle are constants.  In two groups: one is loaded for the next tile
      // while the other is converted.
      constexpr int kPieces = Geo::kInt4 ? D / 32 : D / 16, kStepN = Geo::kConv / kPieces, kUnits = kN / kStepN;
      constexpr int kHalf = kUnits / 2;
      static_assert(kStepN % 8 == 0 && kN % kStepN == 0 && kUnits % 2 == 0, "units");
      // 4-bit lanes: two pieces of a 64-dim block, four keys, then the blocks and
      // further keys (a quarter-warp's stores then fall on 8 bank groups); 8-bit: the
      // pieces of a key side by side, odd 64-dim blocks storing their halves in
      // the other order
      constexpr int kBlocks = D / 64;
      const int pc = Geo::kInt4 ? 2 * ((ct >> 3) % kBlocks) + (ct & 1) : ct % kPieces;
      const int n0 = Geo::kInt4 ? ((ct >> 1) & 3) + 4 * (ct / (8 * kBlocks)) : ct / kPieces;
      const bool odd = !Geo::kInt4 && ((pc >> 2) & 1);
      const uint32_t at0 = Geo::kInt4 ? (uint32_t)((pc >> 1) * kN * 128 + n0 * 128)
                                      : (uint32_t)((pc >> 2) * kN * 128 + n0 * 128);
      const uint32_t chunk0 = Geo::kInt4 ? (uint32_t)((4 * (pc & 1)) ^ (n0 & 7))
                                         : (uint32_t)((2 * (pc & 3) + (odd ? 1 : 0)) ^ (n0 & 7));
      const uint8_t* const from = head_at + 16 * pc;
      const uint8_t* const mul = head_at + D / 2 + 4 + (D == 64 ? 4 : D == 128 ? 2 : 1) * pc;
      uint4 c[kUnits];
      uint32_t cm[Geo::kInt4 ? kUnits : 1];
      // The codes of tile g's units (its slot table is in).  Dead keys (outside the
      // range, or in a chunk without a block) read some row of the pool: their scores
      // are masked; their values are cleared, since an fp8 code may be NaN and a byte
      // that is no multiplier gives infinities (every int8 code is finite).
      auto load_units = [&](int g, auto group) {
        constexpr int i0 = decltype(group)::value * kHalf;
        const int32_t* const slots = table + (g & 3) * 16;
#pragma unroll
        for (int i = i0; i < i0 + kHalf; ++i) {
          const int nn = n0 + i * kStepN;
          const int64_t off = (int64_t)(slots[nn >> 4] + (nn & 15)) * tok_bytes;
          c[i] = dev::ldg_stream_coherent(from + off);
          if constexpr (Geo::kInt4) {
            if constexpr (D == 64) cm[i] = *reinterpret_cast<const uint32_t*>(mul + off);
            else if constexpr (D == 128) cm[i] = *reinterpret_cast<const uint16_t*>(mul + off);
            else cm[i] = *(mul + off);
          }
        }
        if constexpr (code_format(DT) != KVQ_INT8_PER_TOKEN_HEAD) {
          const uint32_t valid = (uint32_t)slots[15];
          const int lo = live_lo(g), hi = live_hi(g);
          if (for_v && (valid != kAllChunks || lo != 0 || hi != kN)) {
#pragma unroll
            for (int i = i0; i < i0 + kHalf; ++i) {
              const int nn = n0 + i * kStepN;
              if (!((valid >> (nn >> 4)) & 1u) || nn < lo || nn >= hi) {
                c[i] = make_uint4(0, 0, 0, 0);
                if constexpr (Geo::kInt4) cm[i] = 0;
              }
            }
          }
        }
      };
      auto convert = [&](uint32_t tile, auto group) {
        constexpr int i0 = decltype(group)::value * kHalf;
#pragma unroll
        for (int i = i0; i < i0 + kHalf; ++i) {
          const uint32_t at = tile + (uint32_t)(i * kStepN * 128);
          if constexpr (Geo::kInt4) {
            const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            dev::Int4Mul f[4];
            if constexpr (D == 64) {
#pragma unroll
              for (int q = 0; q < 4; ++q) f[q] = dev::int4_mul(dev::prmt(cm[i], 0x64646464u, 0x4040u + 0x101u * q));
            } else {
              f[0] = f[1] = dev::int4_mul(dev::prmt(cm[i], 0x64646464u, 0x4040u));
              f[2] = f[3] = D == 128 ? dev::int4_mul(dev::prmt(cm[i], 0x64646464u, 0x4141u)) : f[0];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t h[4];
              dev::int4_to_f16x2x4(w[q], f[q], h);
              sts128(at + ((chunk0 ^ (uint32_t)q) << 4), make_uint4(h[0], h[1], h[2], h[3]));
            }
          } else {
            sts128(at + (chunk0 << 4), codes8_to_f16<DT>(odd ? c[i].z : c[i].x, odd ? c[i].w : c[i].y));
            sts128(at + ((chunk0 ^ 1u) << 4), codes8_to_f16<DT>(odd ? c[i].x : c[i].z, odd ? c[i].y : c[i].w));
          }
        }
      };
      constexpr std::integral_constant<int, 0> first{};
      constexpr std::integral_constant<int, 1> second{};
      // Step g: convert tile g, load tile g + 1 (from step -1 on).
      for (int g = -1; g < T; ++g) {
        const int st = g & 1, e1 = (g + 1) & 3;
        const bool more = g + 1 < T;
        if (g >= 2 && !wait(bar_empty + st, (g >> 1) - 1)) break;
        const uint32_t tile = tiles + (uint32_t)(st * Geo::kTileBytes) + at0;
        if (g >= 0) convert(tile, first);
        if (more) {
          if (!wait(Geo::kBarSlots + e1, (g + 1) >> 2)) break;
          load_units(g + 1, first);
        }
        if (g >= 0) {
          convert(tile, second);
          tc::fence_async_smem();
          warp_arrive(bar(bar_full + st));
        }
        if (more) {
          load_units(g + 1, second);
          warp_arrive(bar(Geo::kBarSlotsFree + e1));
        }
      }
    }
    __syncwarp();
  } else {
    // ---- softmax -------------------------------------------------------------
    regs_up<Regs::kSoftmax>();
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float log2e = 1.4426950408889634f;
    const int head_q = kv_head * G + row_g, pos = token.y;
    const int64_t row_off = ((int64_t)token.x * p.heads_q + head_q) * D;
    float* const qscale = reinterpret_cast<float*>(sm + Geo::kOffQScale);
    float q_unscale = 1.0f;  // 2^-shift of the row's Q
    bool ok = true;
    if (two || t == 0) {
      // Q of the warp's 32 rows: copied where they belong in the operand tile (D / 8
      // lanes a row), then each thread scales its row in place.  A row enters as
      // f16 scaled by the power of two that puts its largest |q| in [2^13, 2^14):
      // exact but for elements 2^27 below that one (subnormals); bf16 rows stay as
      // they are.  The score scale's sign enters with Q, so that the softmax's
      // factor is positive.  (Short loops: unrolled loads and shuffles took 9,700
      // cycles here, most of them instruction fetches.)
      constexpr int kLpr = D / 8, kRpi = 32 / kLpr;
      const float qk_scale = Geo::kPth || Geo::kAuto ? p.sm_scale : p.sm_scale * p.k_scale;
      const uint32_t keep = qk_scale == 0.0f ? 0u : 0xFFFFFFFFu, flip = qk_scale < 0.0f ? 0x80008000u : 0u;
      const uint32_t qt = base + Geo::kOffQ + (uint32_t)(tile * Geo::kQBytes);
      const int pc = lane % kLpr, wrow = (warp & 3) * 32;
#pragma unroll 2
      for (int r0 = 0; r0 < 32; r0 += kRpi) {
        const int r = r0 + lane / kLpr;
        const int64_t off = __shfl_sync(0xffffffffu, row_off, r);
        const bool live = tile * kM + wrow + r < nrows;
        dev::cp_async_16(qt + (uint32_t)((pc >> 3) * (kM * 128) + (wrow + r) * 128 + (((pc & 7) ^ (r & 7)) << 4)),
                         p.q + off + 8 * pc, live ? 16 : 0);
      }
      dev::cp_async_commit();
      dev::cp_async_wait<0>();
      __syncwarp();
      const uint32_t mine = qt + (uint32_t)(m * 128);
      auto piece = [&](int c) { return mine + (uint32_t)((c >> 3) * (kM * 128) + (((c & 7) ^ (m & 7)) << 4)); };
      if (!Geo::kAuto || qk_scale <= 0.0f) {
        float f = 1.0f;
        if constexpr (!Geo::kAuto) {
          uint32_t big = 0;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = lds128(piece(c));
            big = dev::max_u16x2(big, dev::max_u16x2(dev::max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                                     dev::max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
          }
          const int emax = (int)(max(big & 0xFFFFu, big >> 16) >> 7);  // largest |q| < 2^(emax - 126)
          const int sh = emax == 0 ? 0 : min(140 - emax, 126);
          f = __int_as_float((127 + sh) << 23);
          q_unscale = __int_as_float((127 - sh) << 23);
          if (!two) qscale[m] = q_unscale;
        }
#pragma unroll 2
        for (int c = 0; c < D / 8; ++c) {
          uint4 x = lds128(piece(c));
          uint32_t w[4] = {(x.x & keep) ^ flip, (x.y & keep) ^ flip, (x.z & keep) ^ flip, (x.w & keep) ^ flip};
          if constexpr (!Geo::kAuto) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = dev::pack_f16x2(dev::bf16_lo(w[e]) * f, dev::bf16_hi(w[e]) * f);
          }
          sts128(piece(c), make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
      tc::fence_async_smem();
      warp_arrive(bar(Geo::kBarQFull + tile));
    }
    if (!two && t == 1) {  // (the first group's rows)
      ok = wait(Geo::kBarQFull, 0);
      if constexpr (!Geo::kAuto) q_unscale = qscale[m];
    }

    const float* const sk = reinterpret_cast<const float*>(sm + Geo::kOffSk);
    const float* const sv = reinterpret_cast<const float*>(sm + Geo::kOffSv);
    const uint32_t* const smask = reinterpret_cast<const uint32_t*>(sm + Geo::kOffSMask);
    const int32_t* const sev = reinterpret_cast<const int32_t*>(sm + Geo::kOffSMask + Geo::kSide * 4);
    const float cap = GEN ? p.soft_cap : 0.0f, cap_l2 = cap * log2e, inv_cap = cap > 0.0f ? 1.0f / cap : 0.0f;
    const float slope = GEN && p.alibi_slopes ? p.alibi_slopes[head_q] * log2e : 0.0f;
    const int row_hi = row_valid ? kv_hi : 0;  // padding rows see nothing
    const int row_lo = max(kv_lo, p.window > 0 ? pos - p.window + 1 : 0);
    // scores in log2 units (natural units under a soft cap); never zero, which times -inf is NaN
    const float signed_mul = p.sm_scale * (Geo::kInt4 ? dev::kInt4Unit : 1.0f) * q_unscale *
                             (cap > 0.0f ? 1.0f : log2e) * (Geo::kPth || Geo::kAuto ? 1.0f : p.k_scale);
    const float score_mul = fmaxf(fabsf(signed_mul), 0x1p-126f);
    // this group's items: all 64-key tiles, or one of the halves of each KV tile
    const int subs = Geo::kItems * T, count = kRT == 1 || two ? subs : subs / 2;
    const uint32_t tmem_o = tmem + Geo::kColO + (kRT == 2 ? (uint32_t)(t * D) : 0u) + lane_base;
    float m_ref = -INFINITY, l_sum = 0.0f;
    int ev = -1000;  // exponent of the value-scale reference (per-token-head)
    for (int k = 0; ok && k < count; ++k) {
      const int u = kRT == 1 || two ? k : 2 * k + t;  // 64-key tile
      const int g = u / Geo::kItems, h = u % Geo::kItems;
      const int b = 2 * t + (k & 1), sd = g & 3;
      const int kv0 = kv_first + u * Geo::kItem;
      ok = wait_bar(bar(Geo::kBarSFull + b), (uint32_t)((k >> 1) & 1), abort_flag) &&
           wait_bar(bar(Geo::kBarSide + sd), (uint32_t)((g >> 2) & 1), abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t tmem_s = tmem + (uint32_t)(Geo::kColS + b * Geo::kItem) + lane_base;
      const uint32_t cmask = (smask[sd] >> (4 * h)) & 0xFu;  // 16-key chunks of the item
      const int side = sd * kN + h * Geo::kItem;
      const int lo_n = row_lo - kv0, hi_n = row_hi - kv0;
      const bool full = __all_sync(0xffffffffu, lo_n <= 0 && hi_n >= Geo::kItem) && cmask == 0xFu;
      float alpha = 1.0f;  // factor of O
      if constexpr (Geo::kPth) {
        const int e = sev[sd];
        if (e > ev) {
          if (ev > -1000) alpha = __int_as_float((127 + max(ev - e, -127)) << 23);
          ev = e;
        }
      }
      // The row's scores, in pairs, and their maximum.
      uint64_t z[32];
      {
        uint32_t v[64];
        tc::tmem_ld32(tmem_s, *reinterpret_cast<uint32_t(*)[32]>(v));
        tc::tmem_ld32(tmem_s + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = dev::pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
      }
      if constexpr (Geo::kPth) {
        const ulonglong2* const k2 = reinterpret_cast<const ulonglong2*>(sk + side);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const ulonglong2 s2 = k2[e / 2];
          z[e] = dev::mul2(z[e], s2.x);
          z[e + 1] = dev::mul2(z[e + 1], s2.y);
        }
      }
      if constexpr (GEN) {  // final scores, in log2 units
        const int dist = kv0 - pos;  // key - position of column 0
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float2 r = dev::unpack2(z[e]);
          r.x *= score_mul;
          r.y *= score_mul;
          if (cap > 0.0f) {
            r.x = cap_l2 * dev::tanh_exp(r.x * inv_cap);
            r.y = cap_l2 * dev::tanh_exp(r.y * inv_cap);
          }
          z[e] = dev::pack2(fmaf(slope, (float)(dist + 2 * e), r.x), fmaf(slope, (float)(dist + 2 * e + 1), r.y));
        }
      }
      if (!full) {
        // masked keys by a bit each
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int lo = min(max(lo_n - 32 * q, 0), 32), hi = min(max(hi_n - 32 * q, 0), 32);
          const uint32_t cm = cmask >> (2 * q);
          uint32_t seen = hi > lo ? (0xFFFFFFFFu << lo) & (0xFFFFFFFFu >> (32 - hi)) : 0u;
          seen &= (cm & 1u ? 0xFFFFu : 0u) | (cm & 2u ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 r = dev::unpack2(z[16 * q + e]);
            z[16 * q + e] = dev::pack2((seen >> (2 * e)) & 1u ? r.x : -INFINITY, (seen >> (2 * e + 1)) & 1u ? r.y : -INFINITY);
          }
        }
      }
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float2 r = dev::unpack2(z[e]);
        mx4[e & 3] = dev::max3(mx4[e & 3], r.x, r.y);
      }
      const float mr = dev::max3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]));
      const float mx = GEN ? mr : mr * score_mul;
      if (mx > m_ref + 8.0f) {
        const float nref = ceilf(mx);
        if (m_ref != -INFINITY) {
          const float a = __int_as_float((127 + (int)fmaxf(m_ref - nref, -127.0f)) << 23);  // (an integer's power)
          alpha *= a;
          l_sum *= a;
        }
        m_ref = nref;
      }
      // A moved reference rescales O, once the group's last P V is complete: S(k + 1)
      // was issued after it; the last item's has a barrier.
      if (k > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
        ok = k + 1 < count ? wait(Geo::kBarSFull + 2 * t + ((k + 1) & 1), (k + 1) >> 1) : wait(Geo::kBarODone + t, 0);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t w[16];
          tc::tmem_ld16(tmem_o + (uint32_t)c0, w);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
          tc::tmem_st16(tmem_o + (uint32_t)c0, w);
        }
      }
      // P = 2^(z - m + 6), over the columns that the row was read from
      const float ref = m_ref == -INFINITY ? 0.0f : m_ref - 6.0f;
      const uint64_t mul2v = dev::pack2(GEN ? 1.0f : score_mul, GEN ? 1.0f : score_mul);
      const uint64_t ref2 = dev::pack2(-ref, -ref);
      uint64_t ls[2] = {0ull, 0ull};  // pairs of sums
      const ulonglong2* const v2 = reinterpret_cast<const ulonglong2*>(sv + side);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t pw[16], pl[Geo::kAuto ? 16 : 1];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          ulonglong2 s2;
          if constexpr (Geo::kPth) s2 = v2[8 * q + e / 2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float2 x = dev::unpack2(dev::fma2(z[16 * q + e + y], mul2v, ref2));
            uint64_t q2 = dev::pack2(dev::fast_exp2(x.x), dev::fast_exp2(x.y));
            ls[y] = dev::add2(ls[y], q2);
            if constexpr (Geo::kPth) q2 = dev::mul2(q2, y ? s2.y : s2.x);
            const float2 w = dev::unpack2(q2);
            if constexpr (Geo::kAuto) {
              pw[e + y] = dev::pack_bf16x2(w.x, w.y);
              pl[e + y] = dev::pack_bf16x2(w.x - dev::bf16_lo(pw[e + y]), w.y - dev::bf16_hi(pw[e + y]));
            } else {
              pw[e + y] = dev::pack_f16x2(w.x, w.y);
            }
          }
        }
        tc::tmem_st16(tmem_s + (uint32_t)(16 * q), pw);
        if constexpr (Geo::kAuto) tc::tmem_st16(tmem_s + (uint32_t)(32 + 16 * q), pl);
      }
      {
        const float2 a = dev::unpack2(dev::add2(ls[0], ls[1]));
        l_sum += a.x + a.y;
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      warp_arrive(bar(Geo::kBarPFull + b));
    }
    // ---- epilogue: O / l as fp32 partial rows or bf16 rows -------------------
    const bool join = kRT == 2 && !two && part0 < 0;  // one row tile, all its keys
    if (ok) {
      // (one row tile: the rows go out through the Q tile that both groups' MMAs read,
      // and are joined in the K tiles)
      ok = wait(Geo::kBarOFinal + t, 0) && (kRT == 1 || two || (t == 1 && !join) || wait(Geo::kBarOFinal + 1 - t, 0));
      tc::fence_after_sync();
    }
    // (rows of this group's row tile in the partials: the second group of a
    // single row tile has its own)
    const int part = part0 + (two ? tile * kM : t * part_stride);
    const int tile_rows = min(kM, nrows - tile * kM);
    {
      if (part0 < 0 && !join && p.sinks && row_valid && m_ref != -INFINITY) {
        // the sink joins the normaliser here (partial rows: in the merge)
        const float skl = p.sinks[head_q] * log2e;
        if (skl != -INFINITY) l_sum += exp2f(fminf(skl - m_ref + 6.0f, 126.0f));
      }
      // 2^ev / l in two factors, the second last: 2^ev may be at either end of
      // the exponents, and l up to 2^6 times 2^8 a key
      const int up2 = !Geo::kPth ? 0 : ev > 100 ? 20 : ev < -40 && ev > -1000 ? -60 : 0;
      const float sc = (l_sum > 0.0f ? (Geo::kInt4 ? dev::kInt4Unit : 1.0f) / l_sum : 0.0f) *
                       (Geo::kPth    ? (ev > -1000 ? __int_as_float((127 + ev - up2) << 23) : 0.0f)
                        : Geo::kAuto ? 1.0f
                                     : p.v_scale);
      const float sc2 = __int_as_float((127 + up2) << 23);
      const float lse = l_sum > 0.0f ? m_ref + log2f(l_sum) : -INFINITY;
      if (ok && part0 >= 0 && row_valid) p.part_lse[part + m] = lse;
      float own = 1.0f, other = 0.0f;  // weights of the row's two halves
      const uint32_t join_at = base + Geo::kOffK + (uint32_t)(m * D * 4);
      auto join_piece = [&](int c) { return join_at + (uint32_t)((c ^ (m & 7)) << 4); };
      if (kRT == 2 && join) {
        // the second group's normalised rows and their log-sum-exps, through the K and V
        // tiles (no longer read), to the same row's thread of the first
        float* const lse_of = reinterpret_cast<float*>(sm + Geo::kOffV);
        if (t == 1) {
          lse_of[m] = lse;
#pragma unroll 1
          for (int c0 = 0; ok && c0 < D; c0 += 32) {
            uint32_t w[32];
            tc::tmem_ld32(tmem_o + (uint32_t)c0, w);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * sc * sc2);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              sts128(join_piece((c0 + e) >> 2), make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]));
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");  // (both groups come here, whatever gave up)
        if (t == 0) {
          const float second = lse_of[m];
          const float sink = p.sinks && row_valid ? fmaf(p.sinks[head_q], log2e, 6.0f) : -INFINITY;
          const float M = dev::max3(lse, second, sink), at = M == -INFINITY ? 0.0f : M;
          own = exp2f(lse - at);
          other = exp2f(second - at);
          const float sum = own + other + exp2f(sink - at);
          const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;  // (a row that sees no key: zeros)
          own *= inv;
          other *= inv;
        }
      }
      // The warp's rows go through its part of the Q tiles (no longer read):
      // D / 2 columns a pass, 16-byte pieces swizzled by the row, then out in
      // runs of a row.
      constexpr int kCw = D / 2, kPr = kCw / 4;  // columns of a pass, 16-byte pieces of a row
      const int wr = (warp & 3) * 32;
      const uint32_t stage = base + Geo::kOffQ + (uint32_t)(t * Geo::kQBytes + (warp & 3) * 32 * kCw * 4);
#pragma unroll 1
      for (int h = ok && !(join && t == 1) ? 0 : 2; h < 2; ++h) {
#pragma unroll 1
        for (int c0 = 0; c0 < kCw; c0 += 32) {
          uint32_t w[32];
          tc::tmem_ld32(tmem_o + (uint32_t)(h * kCw + c0), w);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float f[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) f[b] = __uint_as_float(w[e + b]) * sc * sc2;
            if (kRT == 2 && join) {
              const uint4 y = lds128(join_piece((h * kCw + c0 + e) >> 2));
              f[0] = fmaf(__uint_as_float(y.x), other, f[0] * own);
              f[1] = fmaf(__uint_as_float(y.y), other, f[1] * own);
              f[2] = fmaf(__uint_as_float(y.z), other, f[2] * own);
              f[3] = fmaf(__uint_as_float(y.w), other, f[3] * own);
            }
            sts128(stage + (uint32_t)(lane * kCw * 4 + ((((c0 + e) >> 2) ^ (lane & 7)) << 4)),
                   make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
          }
        }
        __syncwarp();
        if (part0 >= 0) {
          // (the partial rows of a warp lie side by side)
          float* const to = p.part_o + (int64_t)(part + wr) * D + h * kCw;
#pragma unroll 4
          for (int x = lane; x < 32 * kPr; x += 32) {
            const int r = x / kPr, pc = x % kPr;
            const uint4 u = lds128(stage + (uint32_t)(r * kCw * 4 + ((pc ^ (r & 7)) << 4)));
            if (wr + r < tile_rows) *reinterpret_cast<uint4*>(to + r * D + 4 * pc) = u;
          }
        } else {
#pragma unroll 2
          for (int x = lane; x < 16 * kPr; x += 32) {
            const int r = x / (kPr / 2), pc = 2 * (x % (kPr / 2));
            const uint4 u = lds128(stage + (uint32_t)(r * kCw * 4 + ((pc ^ (r & 7)) << 4)));
            const uint4 v = lds128(stage + (uint32_t)(r * kCw * 4 + (((pc + 1) ^ (r & 7)) << 4)));
            const int64_t off = __shfl_sync(0xffffffffu, row_off, r);
            if (wr + r < tile_rows)
              *reinterpret_cast<uint4*>(p.out + off + h * kCw + 4 * pc) =
                  make_uint4(dev::pack_bf16x2(__uint_as_float(u.x), __uint_as_float(u.y)),
                             dev::pack_bf16x2(__uint_as_float(u.z), __uint_as_float(u.w)),
                             dev::pack_bf16x2(__uint_as_float(v.x), __uint_as_float(v.y)),
                             dev::pack_bf16x2(__uint_as_float(v.z), __uint_as_float(v.w)));
          }
        }
        __syncwarp();
      }
    }
    tc::fence_before_sync();
    __syncwarp();
  }

  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, Geo::kTmemCols);
  }
  // A unit that gave up leaves NaN in every row of its output.
  if (*abort_flag != 0u) {
    if (tid == 0) atomicExch(p.error_flag, 1);
    const int subs = kRT == 2 && !two ? 2 : 1;
    for (int x = tid; x < nrows * subs; x += Geo::kThreads) {
      const int r = x % nrows, packed = row0 + r;
      if (part0 >= 0) {
        const int64_t at = part0 + r + (int64_t)(x / nrows) * part_stride;
        for (int d = 0; d < D; ++d) p.part_o[at * D + d] = NAN;
        p.part_lse[at] = 0.0f;
      } else {
        const int2 to = __ldg(reinterpret_cast<const int2*>(rp.tokens) + tok0 + packed / G);
        uint16_t* const o = p.out + ((int64_t)to.x * p.heads_q + kv_head * G + packed % G) * D;
        for (int d = 0; d < D; ++d) o[d] = 0x7FC0u;
      }
    }
  }
}

template <int DT, int D>
int launch_rect_instance(const AttnParams& p, const RectParams& rp, cudaStream_t stream) {
  auto kern = p.soft_cap > 0.0f || p.alibi_slopes ? rect_attention_kernel<DT, D, true>
                                                  : rect_attention_kernel<DT, D, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)rect_smem_bytes(D)) != cudaSuccess)
    return KVQ_E_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rp.num_units);
  cfg.blockDim = dim3(512u);
  cfg.dynamicSmemBytes = rect_smem_bytes(D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p, rp) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_E_CUDA;
  }
  return KVQ_OK;
}

// The instances of one head_dim (a translation unit each).
template <int D>
int launch_rect_d(const AttnParams& p, const RectParams& rp, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case KVQ_AUTO: return launch_rect_instance<KVQ_AUTO, D>(p, rp, stream);
    case KVQ_FP8_E4M3: return launch_rect_instance<KVQ_FP8_E4M3, D>(p, rp, stream);
    case KVQ_FP8_E5M2: return launch_rect_instance<KVQ_FP8_E5M2, D>(p, rp, stream);
    case KVQ_INT8_PER_TOKEN_HEAD: return launch_rect_instance<KVQ_INT8_PER_TOKEN_HEAD, D>(p, rp, stream);
    case KVQ_FP8_PER_TOKEN_HEAD: return launch_rect_instance<KVQ_FP8_PER_TOKEN_HEAD, D>(p, rp, stream);
    case KVQ_FP8_E5M2_PER_TOKEN_HEAD: return launch_rect_instance<KVQ_FP8_E5M2_PER_TOKEN_HEAD, D>(p, rp, stream);
    case KVQ_INT4_PER_TOKEN_HEAD: return launch_rect_instance<KVQ_INT4_PER_TOKEN_HEAD, D>(p, rp, stream);
    default: return KVQ_E_UNSUPPORTED;
  }
}

}  // namespace kvq
