// attn_plan.h -- what the two plan kernels share: one workgroup reads cu_seqlens a chunk of
// sequences at a time, numbers the chunk's tiles by a scan, and gives each thread tiles to
// place. All of it is in one workgroup because a plan is small (a few thousand items) and a
// grid-wide order would need more launches; a workgroup-wide scan takes two barriers.
#pragma once

#include "attn_common.h"

namespace attn {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

template <typename V>
struct Sum {
  typedef V type;
  static constexpr V kZero = 0;
  __device__ static V apply(V a, V b) { return a + b; }
};
typedef Sum<int32_t> AddOp;
struct MaxOp {
  typedef int32_t type;
  static constexpr int32_t kZero = INT32_MIN;
  __device__ static int32_t apply(int32_t a, int32_t b) { return a > b ? a : b; }
};

// Inclusive scan over the workgroup; buf: kPlanWaves values, free again after a barrier.
template <typename Op, typename V = typename Op::type>
__device__ inline V block_scan(V x, V* buf) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const V y = __shfl_up(x, d);
    if (lane >= d) x = Op::apply(x, y);
  }
  __syncthreads();
  if (lane == 63) buf[wave] = x;
  __syncthreads();
  V before = Op::kZero;
  for (int w = 0; w < wave; ++w) before = Op::apply(before, buf[w]);
  return Op::apply(before, x);
}

__device__ inline int32_t ceil_div(int32_t n, int32_t d) { return n / d + (n % d != 0); }

// A chunk of sequences. Slot 0 of the first chunk is an empty sequence that owns the rows
// before cu_seqlens[0]; every slot owns the rows from its sequence's start to the next one's,
// or to T, of which its sequence holds the first n.
struct SeqChunk {
  int32_t a[kPlanThreads], n[kPlanThreads], end[kPlanThreads];
  int32_t scan[kPlanWaves], last;
};

// Reads slots s0 .. s0 + kPlanThreads - 1. carry: the largest start so far. Entries count as
// clamped to [0, T], and as the largest before them where they are smaller.
__device__ inline void load_sequences(SeqChunk& c, const int32_t* cu, int32_t num_seqs, int32_t T,
                                      int32_t s0, int32_t* carry) {
  const int t = threadIdx.x;
  const int32_t slot = s0 + t;
  int32_t e = slot <= num_seqs && num_seqs > 0 ? cu[slot] : T;  // the slot's sequence ends here
  e = e < 0 ? 0 : e > T ? T : e;
  int32_t next = slot < num_seqs ? e : T;  // and the next slot's rows begin here
  next = MaxOp::apply(block_scan<MaxOp>(next, c.scan), *carry);
  c.end[t] = next;
  if (t == kPlanThreads - 1) c.last = next;
  __syncthreads();
  const int32_t a = t > 0 ? c.end[t - 1] : *carry;
  c.a[t] = a;
  c.n[t] = slot > 0 && slot <= num_seqs && e > a ? e - a : 0;
  *carry = c.last;
  __syncthreads();
  if (slot > num_seqs) c.end[t] = a;
}

// The slot of tile i: the first whose running count exceeds it.
__device__ inline int find_slot(const int32_t* running, int32_t i) {
  int lo = 0, hi = kPlanThreads - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (running[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Items are ordered by falling work in buckets; counts become first places. BUCKETS at most
// kPlanThreads.
template <int BUCKETS>
__device__ inline int32_t bucket_of(int64_t work, int64_t most) {  // more work, lower bucket
  const int64_t b = most > 0 ? work * (BUCKETS - 1) / most : 0;
  return BUCKETS - 1 - (int32_t)(b < BUCKETS ? b : BUCKETS - 1);
}
template <int BUCKETS>
__device__ inline void counts_to_places(int32_t* count, int32_t* buf) {
  const int t = threadIdx.x;
  __syncthreads();
  const int32_t own = t < BUCKETS ? count[t] : 0;
  const int32_t incl = block_scan<AddOp>(own, buf);
  if (t < BUCKETS) count[t] = incl - own;
  __syncthreads();
}

}  // namespace attn
