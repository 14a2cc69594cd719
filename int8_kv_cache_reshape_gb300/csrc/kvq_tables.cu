// kvq_tables.cu -- block tables and slot maps of a step, built on the GPU
// from the request lengths.  No counterpart on the pages (vLLM's scheduler
// assigns blocks on the host).
//
// What it computes: request r has L keys, the last Q of them new, and holds
// ceil((L - Q) / B) blocks; it needs ceil(L / B).  With new_r the difference
// and base_r = sum of new_i over i < r, its n-th new logical block takes
// free[count - 1 - base_r - n], and the new token at position p goes to slot
// table[r][p / B] * B + p % B.
//
// Starts that decrease leave it open whose a token is, and the searches below
// expect them sorted: every CTA looks at all of them, and where one decreases the
// whole step is left out.
//
// A token's block never depends on another thread's store: an old block comes
// from the table, a new one straight from the free list, and the thread of
// the first token in a new block stores the table entry (a new block's first
// position is always a new token).  So the work is split over tokens alone.
//
// One launch, bound by latency: 64 decode tokens move 1.3 KB.  A CTA takes a
// contiguous run of tokens and finds their requests in shared memory, among
// all the batch's requests and their prefix sum (up to kAllRequests of them,
// read and summed by every CTA for itself: two memory round trips from launch
// to slot).  Larger batches are taken in windows of kAllRequests that start
// at the run's first request, with the requests before it summed in one pass
// (every thread loads its share of the lengths at once, where a search for
// the first request takes log2 R dependent loads).  Measured, call after call:
// 3.0 us for 64 requests, 5.1 for 509 with 28,914 tokens, 8.9 for 893,000
// tokens of 37 requests (a prefix pass of its own ahead: 4.1, 10.2, 14.3).  The
// check for decreasing starts is 0.1 to 0.2 of each, as a term of the sum, a
// count of its own or a barrier that votes.
#include <cuda_runtime.h>

#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Tokens of a CTA's run, four a thread.
constexpr int kPer = 4;
constexpr int kRun = kPer * kThreads;
// Requests held in shared memory, four a thread.
constexpr int kAllRequests = kPer * kThreads;

// Added to the sum of the new blocks for a request that ends before it starts: the
// sum is then negative.  (It stays below the entries of the block table, less
// than 2^40; at most 1,024 such terms are added.)
constexpr int64_t kDecreasing = -((int64_t)1 << 44);

struct TableParams {
  const int32_t* query_start_loc;
  const int32_t* seq_lens;
  const int32_t* free_blocks;
  const int32_t* free_count;
  int32_t* block_table;
  int64_t* slot_mapping;
  int32_t* free_count_out;
  int32_t* status;
  int64_t free_capacity, num_tokens, num_blocks;
  int num_req, width, block_size;
};

struct Request {
  int64_t start, end;  // its tokens
  int first;           // position of its first new token
  int held, fresh;     // blocks it holds, blocks that begin in this step
  bool ok;
};

// Lengths that do not fit (more new tokens than keys, more blocks than the
// table's width, tokens past the buffer) leave the request out.
__device__ __forceinline__ Request load_request(const TableParams& p, int r) {
  Request q;
  q.start = p.query_start_loc[r];
  q.end = p.query_start_loc[r + 1];
  const int64_t L = p.seq_lens[r], n = q.end - q.start, B = p.block_size;
  q.ok = n >= 0 && L >= n && q.start >= 0 && q.end <= p.num_tokens && (n == 0 || L <= B * p.width);
  q.first = q.ok ? (int)(L - n) : 0;
  q.held = q.ok ? (int)((uint32_t)q.first / (uint32_t)B + ((uint32_t)q.first % (uint32_t)B != 0)) : 0;
  q.fresh = q.ok && n > 0 ? (int)((uint32_t)L / (uint32_t)B + ((uint32_t)L % (uint32_t)B != 0)) - q.held : 0;
  return q;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__global__ void __launch_bounds__(kThreads) block_tables_kernel(const TableParams p) {
  __shared__ int64_t part[kWarps], part2[kWarps], base_s[kAllRequests];
  __shared__ int32_t bad_s[kWarps];
  __shared__ int32_t start_s[kAllRequests], end_s[kAllRequests], first_s[kAllRequests], held_s[kAllRequests];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * kRun;
  const int64_t t1 = min(t0 + kRun, p.num_tokens);
  const bool last_run = blockIdx.x == gridDim.x - 1;
  // (a programmatic dependent of whatever ran before on the stream)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t count = max((int64_t)0, min((int64_t)*p.free_count, p.free_capacity));

  // large batches: the requests that end at or before this run, their new
  // blocks, and how many of them are left out
  int64_t base = 0;
  int first_req = 0, bad = 0;
  if (p.num_req > kAllRequests) {
    int64_t sum = 0;
    int n = 0, b = 0;
    bool down = false;
    for (int r = tid; r < p.num_req; r += kThreads) {
      const Request q = load_request(p, r);
      down |= q.end < q.start;
      if (q.end <= t0) {
        sum += q.fresh;
        ++n;
        b += !q.ok;
      }
    }
    sum = warp_sum(down ? kDecreasing : sum);
    const int64_t nb = warp_sum(((int64_t)b << 32) | (int64_t)n);
    if (lane == 0) {
      part[warp] = sum;
      part2[warp] = nb;
    }
    __syncthreads();
    int64_t nbs = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      base += part[w];
      nbs += part2[w];
    }
    first_req = (int)(nbs & 0xFFFFFFFF);
    bad = (int)(nbs >> 32);
    __syncthreads();
  }

  // kAllRequests requests at a time (the last run goes through all of them,
  // for the totals): thread i takes kPer consecutive ones
  int64_t t = t0;
  for (int r0 = first_req; r0 < p.num_req && (t < t1 || last_run); r0 += kAllRequests) {
    const int n = min(kAllRequests, p.num_req - r0);
    const int per = (n + kThreads - 1) / kThreads;
    int64_t local = 0, fresh[kPer];
    int bad_t = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      fresh[i] = 0;
      const int at = tid * per + i;
      if (i < per && at < n) {
        const Request q = load_request(p, r0 + at);
        start_s[at] = (int32_t)q.start;
        end_s[at] = q.ok ? (int32_t)q.end : (int32_t)q.start;  // a request left out has no tokens
        first_s[at] = q.first;
        held_s[at] = q.held;
        fresh[i] = q.fresh;
        local += q.end < q.start ? kDecreasing : q.fresh;
        bad_t += !q.ok;
      }
    }
    int64_t incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    const int bad_w = __reduce_add_sync(0xffffffffu, bad_t);
    if (lane == 31) {
      part[warp] = incl;
      bad_s[warp] = bad_w;
    }
    const int64_t next = p.query_start_loc[r0 + n];  // the window's last end
    __syncthreads();
    int64_t before = base + incl - local;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += part[w];
      base += part[w];
      bad += bad_s[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i < per && tid * per + i < n) base_s[tid * per + i] = before;
      before += fresh[i];
    }
    __syncthreads();
    const int64_t stop = base < 0 ? t : min(t1, next);  // (no token's, if the starts decrease)
    // A thread takes per_t consecutive tokens: one search for the first one's
    // request (the last that starts at or before it), steps for the others
    // (a search for each took 1.3 us more for the 893,000 tokens).
    const int per_t = (int)((stop - t + kThreads - 1) / kThreads);
    const int64_t k0 = t + (int64_t)tid * per_t;
    int lo = 0;
    for (int hi = n; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (start_s[mid] <= k0) lo = mid;
      else hi = mid;
    }
    int64_t slot[kPer];
    int32_t* entry[kPer];
    const int32_t* from[kPer];
    uint32_t off[kPer];
    bool fresh_block[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t k = k0 + i;
      from[i] = nullptr;
      entry[i] = nullptr;
      fresh_block[i] = false;
      off[i] = 0;
      if (i < per_t && k < stop) {
        if (i > 0)
          while (lo + 1 < n && start_s[lo + 1] <= k) ++lo;
        if (k >= start_s[lo] && k < end_s[lo]) {
          const uint32_t pos = (uint32_t)(first_s[lo] + (int)(k - start_s[lo]));
          const uint32_t lb = pos / (uint32_t)p.block_size;
          off[i] = pos - lb * (uint32_t)p.block_size;
          entry[i] = p.block_table + (int64_t)(r0 + lo) * p.width + lb;
          if ((int)lb < held_s[lo]) {
            from[i] = entry[i];
          } else {
            const int64_t at = base_s[lo] + (int)lb - held_s[lo];
            if (at < count) from[i] = p.free_blocks + (count - 1 - at);
            fresh_block[i] = off[i] == 0;
          }
        }
      }
    }
    int32_t id[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) id[i] = from[i] ? *from[i] : -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      slot[i] = id[i] >= 0 && id[i] < p.num_blocks ? (int64_t)id[i] * p.block_size + off[i] : -1;
      if (fresh_block[i]) *entry[i] = id[i];
    }
    if (per_t == kPer && k0 + kPer <= stop && (k0 & 1) == 0 &&
        ((uintptr_t)p.slot_mapping & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < kPer; i += 2)
        *reinterpret_cast<longlong2*>(p.slot_mapping + k0 + i) = make_longlong2(slot[i], slot[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < per_t && k0 + i < stop) p.slot_mapping[k0 + i] = slot[i];
    }
    t = max(t, stop);
    __syncthreads();
  }
  if (base < 0) {
    base = 0;
    bad = p.num_req;
  }
  for (int64_t k = t + tid; k < t1; k += kThreads) p.slot_mapping[k] = -1;

  // Totals: from the CTA of the last run.  Where free_count_out is free_count,
  // it is stored once every CTA has read that (the last to arrive does).
  if (tid == 0) {
    const int32_t left = (int32_t)max((int64_t)0, count - base);
    const bool in_place = p.free_count_out == p.free_count && gridDim.x > 1;
    if (last_run) {
      p.status[0] = (int32_t)min((int64_t)0x7FFFFFFF, max((int64_t)0, base - count));
      p.status[1] = bad;
      if (in_place) p.status[3] = left;
      else *p.free_count_out = left;
    }
    if (in_place) {
      __threadfence();
      if (atomicAdd(p.status + 2, 1) == (int)gridDim.x - 1) {
        __threadfence();
        *p.free_count_out = __ldcg(p.status + 3);
        p.status[2] = 0;
      }
    }
  }
}

}  // namespace

int launch_block_tables(int num_req, const int32_t* query_start_loc, const int32_t* seq_lens,
                        const int32_t* free_blocks, int64_t free_capacity, const int32_t* free_count,
                        int32_t* block_table, int block_table_stride, int64_t* slot_mapping,
                        int64_t num_tokens, int block_size, int64_t num_blocks,
                        int32_t* free_count_out, int32_t* status, void* stream) {
  TableParams p;
  p.query_start_loc = query_start_loc;
  p.seq_lens = seq_lens;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.block_table = block_table;
  p.slot_mapping = slot_mapping;
  p.free_count_out = free_count_out;
  p.status = status;
  p.free_capacity = free_capacity;
  p.num_tokens = num_tokens;
  p.num_blocks = num_blocks;
  p.num_req = num_req;
  p.width = block_table_stride;
  p.block_size = block_size;
  const int64_t ctas = num_tokens > kRun ? (num_tokens + kRun - 1) / kRun : 1;
  return launch_dependent(block_tables_kernel, (unsigned)ctas, kThreads, stream, p);
}

}  // namespace kvq
