// kv_pages.hip -- block table, slot map and positions of a step over a paged cache, and the pages
// that finished sequences give back (include/kv_pages.h).
//
// Mathematics: with h_s = ceil(held_s / page) pages before and w_s = ceil((held_s + new_s) / page)
// - h_s more, sequence s takes the pages of the pool from sum_{r<s} w_r on; its token at position p
// lies in the (p / page - h_s)-th of them, or in one that the table names already. A new page begins
// with a new token, so whoever places that token writes the table's entry.
//
// What bounds it: latency. A chain of loads, a scan and a search is most of a step of some thousand
// tokens, so everything is one launch, without an order among its workgroups: each reads the
// lengths from the first sequence on and scans them, 4096 at a time, up to the tokens that are its
// own; one more writes what there is for each sequence. Measured: 64 sequences of one token each 5 us, 4000
// sequences with 303664 tokens 11 us.
#include "attn_plan.h"
#include "../../include/kv_pages.h"

namespace attn {
namespace {

constexpr int32_t kMostTokens = INT32_MAX - 4096;
constexpr int64_t kMost = (int64_t)1 << 30;
constexpr int32_t kTokensOfGroup = 2048;

// Tokens and pages: two sums of up to INT32_MAX, which they do not exceed.
struct PairSum {
  typedef uint64_t type;
  static constexpr uint64_t kZero = 0;
  __device__ static uint64_t apply(uint64_t a, uint64_t b) {
    const uint32_t most = INT32_MAX;
    const uint32_t lo = min((uint32_t)a + (uint32_t)b, most);
    const uint32_t hi = min((uint32_t)(a >> 32) + (uint32_t)(b >> 32), most);
    return (uint64_t)hi << 32 | lo;
  }
};

struct StepParams {
  const int32_t* new_lens;
  const int32_t* held;
  int32_t* table;
  const int32_t* ring;
  const int32_t* state;
  int32_t* cu;
  int32_t* kv_lens;
  int32_t* held_out;
  int32_t* positions;
  int64_t* slots;
  int32_t* state_out;
  int64_t table_stride;
  int32_t num_seqs, T, page_size, max_pages, num_pages;
  Div31 by_page;
};

struct CappedSum {
  typedef int32_t type;
  static constexpr int32_t kZero = 0;
  __device__ static int32_t apply(int32_t a, int32_t b) {
    return (int32_t)min((uint32_t)a + (uint32_t)b, (uint32_t)INT32_MAX);
  }
};

__device__ inline int32_t pages_of(int32_t tokens, Div31 by_page) {
  return tokens > 0 ? (int32_t)div31(tokens - 1, by_page) + 1 : 0;
}
// The ring's place `i` behind its first; both below num_pages.
__device__ inline int32_t ring_at(int32_t first, int32_t i, int32_t num_pages) {
  const int32_t x = first + i;  // < 2^31
  return x < num_pages ? x : x - num_pages;
}

// The sequence of a token: the first of a chunk whose running count exceeds it.
template <int N>
__device__ inline int find_sequence(const int32_t* upto, int32_t token) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (upto[mid] > token) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

template <int kPerThread>  // sequences
__global__ __launch_bounds__(kPlanThreads) void kv_page_step_kernel(const StepParams p) {
  constexpr int kChunk = kPerThread * kPlanThreads;
  __shared__ uint64_t scan[kPlanWaves];
  __shared__ int32_t upto[kChunk];    // tokens up to each sequence of a chunk, itself too
  __shared__ int32_t begin[kChunk];   // what it held; < 0: refused
  __shared__ int32_t fresh[kChunk];   // where its new pages begin in the ring, less those it has
  __shared__ uint64_t total;
  __shared__ int32_t used;
  const int t = threadIdx.x;
  const bool of_sequences = blockIdx.x == gridDim.x - 1;
  const int32_t first_token = blockIdx.x * kTokensOfGroup;
  const int32_t end_token = of_sequences ? 0 : min(first_token + kTokensOfGroup, p.T);
  const int32_t first = (int32_t)((uint32_t)p.state[0] % (uint32_t)p.num_pages);
  const int32_t count = min(max(p.state[1], 0), p.num_pages);
  if (t == 0) used = 0;

  uint64_t before = 0;
  int32_t most = 0;  // pages up to the last sequence that gets one
  for (int32_t s0 = 0; s0 < p.num_seqs; s0 += kChunk) {
    int32_t n[kPerThread], held[kPerThread], wants[kPerThread];
    bool fits[kPerThread];
    uint64_t mine = 0;
#pragma unroll
    for (int y = 0; y < kPerThread; ++y) {
      const int32_t s = s0 + t * kPerThread + y;
      n[y] = s < p.num_seqs ? max(p.new_lens[s], 0) : 0;
      held[y] = s < p.num_seqs ? max(p.held[s], 0) : 0;
    }
#pragma unroll
    for (int y = 0; y < kPerThread; ++y) {
      const int64_t sum = (int64_t)held[y] + n[y];
      fits[y] = sum < kMostTokens && pages_of((int32_t)sum, p.by_page) <= p.max_pages;
      wants[y] = n[y] > 0 && fits[y] ? pages_of((int32_t)sum, p.by_page) - pages_of(held[y], p.by_page) : 0;
      mine = PairSum::apply(mine, (uint64_t)wants[y] << 32 | (uint32_t)n[y]);
    }
    const uint64_t all = PairSum::apply(before, block_scan<PairSum>(mine, scan));
    if (t == kPlanThreads - 1) total = all;
    // and back to each of the thread's sequences: what is before the first of them
    uint64_t here = __shfl_up(all, 1);
    if ((t & 63) == 0) {
      here = before;
      for (int w = 0; w < t >> 6; ++w) here = PairSum::apply(here, scan[w]);
    }
#pragma unroll
    for (int y = 0; y < kPerThread; ++y) {
      const int32_t x = t * kPerThread + y, s = s0 + x;
      here = PairSum::apply(here, (uint64_t)wants[y] << 32 | (uint32_t)n[y]);
      const int32_t last_token = (int32_t)(uint32_t)here, last_page = (int32_t)(here >> 32);
      const bool served = n[y] == 0 || (fits[y] && last_token <= p.T && (wants[y] == 0 || last_page <= count));
      upto[x] = last_token;
      begin[x] = served ? held[y] : -1;
      fresh[x] = last_page - wants[y] - pages_of(held[y], p.by_page);
      if (of_sequences && s < p.num_seqs) {
        const int32_t sum = (int32_t)((uint32_t)held[y] + (uint32_t)n[y]);  // where it is served, below 2^31
        if (s == 0) p.cu[0] = 0;
        p.cu[s + 1] = min(last_token, p.T);
        p.kv_lens[s] = served ? sum : 0;
        p.held_out[s] = served && n[y] > 0 ? sum : p.held[s];
        if (served && wants[y] > 0) most = last_page;
      }
    }
    __syncthreads();
    const int32_t from = max(first_token, (int32_t)(uint32_t)before);
    const int32_t to = min(end_token, (int32_t)(uint32_t)total);
    for (int32_t token = from + t; token < to; token += kPlanThreads) {
      const int x = find_sequence<kChunk>(upto, token);
      const int32_t start = x > 0 ? upto[x - 1] : (int32_t)(uint32_t)before;
      const int32_t h = begin[x];
      int32_t pos = -1;
      int64_t slot = -1;
      if (h >= 0) {
        pos = h + (token - start);
        const int32_t at = div31(pos, p.by_page), in_page = pos - at * p.page_size;
        int32_t* entry = p.table + (int64_t)(s0 + x) * p.table_stride + at;
        int32_t page;
        if (at < pages_of(h, p.by_page)) {
          page = *entry;
        } else {
          page = p.ring[ring_at(first, fresh[x] + at, p.num_pages)];
          if (in_page == 0) *entry = page;
        }
        if (page >= 0) slot = (int64_t)page * p.page_size + in_page;
      }
      p.positions[token] = pos;
      p.slots[token] = slot;
    }
    before = total;
    if (!of_sequences && (int32_t)(uint32_t)before >= end_token) return;  // the same for all threads
    __syncthreads();
  }
  if (of_sequences) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) most = max(most, __shfl_xor(most, d));
    __syncthreads();
    if ((t & 63) == 0) atomicMax(&used, most);
    __syncthreads();
    if (t == 0) {
      if (p.num_seqs == 0) p.cu[0] = 0;
      p.state_out[0] = ring_at(first, used, p.num_pages);
      p.state_out[1] = count - used;
    }
    return;
  }
  // rows of no sequence
  for (int32_t token = max(first_token, (int32_t)(uint32_t)before) + t; token < end_token; token += kPlanThreads) {
    p.positions[token] = -1;
    p.slots[token] = -1;
  }
}

struct ReleaseParams {
  int32_t* held;
  const uint8_t* gone;
  const int32_t* table;
  int32_t* ring;
  int32_t* state;
  int64_t table_stride;
  int32_t num_seqs, max_pages, num_pages;
  Div31 by_page;
};

__global__ __launch_bounds__(kPlanThreads) void kv_page_release_kernel(const ReleaseParams p) {
  __shared__ int32_t scan[kPlanWaves], upto[kPlanThreads];
  const int t = threadIdx.x;
  const int32_t first = (int32_t)((uint32_t)p.state[0] % (uint32_t)p.num_pages);
  int32_t count = min(max(p.state[1], 0), p.num_pages);
  __syncthreads();  // read by all before it is written
  for (int32_t s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int32_t s = s0 + t;
    int32_t n = 0;
    if (s < p.num_seqs && p.gone[s] != 0) {
      n = min(pages_of(p.held[s], p.by_page), p.max_pages);
      p.held[s] = 0;
    }
    upto[t] = block_scan<CappedSum>(n, scan);
    __syncthreads();
    const int32_t total = min(upto[kPlanThreads - 1], p.num_pages - count);
    for (int32_t i = t; i < total; i += kPlanThreads) {
      const int x = find_slot(upto, i);
      const int32_t at = i - (x > 0 ? upto[x - 1] : 0);
      p.ring[ring_at(first, count + i, p.num_pages)] =
          p.table[(int64_t)(s0 + x) * p.table_stride + at];
    }
    count += total;
    __syncthreads();
  }
  if (t == 0) {
    p.state[0] = first;
    p.state[1] = count;
  }
}

bool valid_pool(int32_t num_seqs, int32_t page_size, int32_t max_pages, int64_t table_stride, int32_t num_pages) {
  return num_seqs >= 0 && num_seqs <= (1 << 24) && page_size >= 1 && page_size <= kMost && max_pages >= 0 &&
         table_stride >= 0 && table_stride <= (int64_t)1 << 40 && num_pages >= 1 && num_pages <= kMost;
}

// Whether an output of a step overlaps an input or another output; the workgroups have no order in which that
// could be right.
struct Span {
  const void* begin;
  int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = (uintptr_t)a.begin, y = (uintptr_t)b.begin;
  return a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}
template <size_t N, size_t M>
bool outputs_apart(const Span (&out)[N], const Span (&in)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return false;
    for (size_t j = 0; j < M; ++j)
      if (overlap(out[i], in[j])) return false;
  }
  return true;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int32_t kv_page_step(const int32_t* new_lens, const int32_t* held, int32_t num_seqs, int64_t T,
                     int32_t page_size, int32_t* block_table, int32_t max_pages, int64_t table_stride,
                     const int32_t* ring, int32_t num_pages, const int32_t* state, int32_t* cu_seqlens,
                     int32_t* kv_lens, int32_t* held_out, int32_t* positions, int64_t* slots,
                     int32_t* state_out, void* stream) {
  if (!valid_pool(num_seqs, page_size, max_pages, table_stride, num_pages) || T < 0 || T > kMost)
    return ROPE_EINVAL;
  if (num_seqs > 0 && (new_lens == nullptr || held == nullptr || kv_lens == nullptr || held_out == nullptr))
    return ROPE_EINVAL;
  if (num_seqs > 0 && max_pages > 0 && block_table == nullptr) return ROPE_EINVAL;
  if (T > 0 && (positions == nullptr || slots == nullptr)) return ROPE_EINVAL;
  if (ring == nullptr || state == nullptr || cu_seqlens == nullptr || state_out == nullptr) return ROPE_EINVAL;
  const int64_t n = num_seqs, rows = n > 0 && max_pages > 0 ? (n - 1) * table_stride + max_pages : 0;
  if (!outputs_apart<7, 4>({{cu_seqlens, 4 * (n + 1)}, {kv_lens, 4 * n}, {held_out, 4 * n}, {positions, 4 * T},
                            {slots, 8 * T}, {state_out, 8}, {block_table, 4 * rows}},
                           {{new_lens, 4 * n}, {held, 4 * n}, {ring, 4 * (int64_t)num_pages}, {state, 8}}))
    return ROPE_EINVAL;
  StepParams p;
  p.new_lens = new_lens;
  p.held = held;
  p.table = block_table;
  p.ring = ring;
  p.state = state;
  p.cu = cu_seqlens;
  p.kv_lens = kv_lens;
  p.held_out = held_out;
  p.positions = positions;
  p.slots = slots;
  p.state_out = state_out;
  p.table_stride = table_stride;
  p.num_seqs = num_seqs;
  p.T = (int32_t)T;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.by_page = make_div31(page_size);
  const unsigned groups = (unsigned)((T + kTokensOfGroup - 1) / kTokensOfGroup) + 1;
  // several sequences a thread, and one scan for all, where one a thread would take several
  if (num_seqs > kPlanThreads)
    hipLaunchKernelGGL((kv_page_step_kernel<4>), dim3(groups), dim3(kPlanThreads), 0,
                       static_cast<hipStream_t>(stream), p);
  else
    hipLaunchKernelGGL((kv_page_step_kernel<1>), dim3(groups), dim3(kPlanThreads), 0,
                       static_cast<hipStream_t>(stream), p);
  return launched();
}

int32_t kv_page_release(int32_t* held, const uint8_t* gone, int32_t num_seqs, int32_t page_size,
                        const int32_t* block_table, int32_t max_pages, int64_t table_stride, int32_t* ring,
                        int32_t num_pages, int32_t* state, void* stream) {
  if (!valid_pool(num_seqs, page_size, max_pages, table_stride, num_pages)) return ROPE_EINVAL;
  if (num_seqs > 0 && (held == nullptr || gone == nullptr)) return ROPE_EINVAL;
  if (num_seqs > 0 && max_pages > 0 && block_table == nullptr) return ROPE_EINVAL;
  if (ring == nullptr || state == nullptr) return ROPE_EINVAL;
  ReleaseParams p;
  p.held = held;
  p.gone = gone;
  p.table = block_table;
  p.ring = ring;
  p.state = state;
  p.table_stride = table_stride;
  p.num_seqs = num_seqs;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.by_page = make_div31(page_size);
  hipLaunchKernelGGL(kv_page_release_kernel, dim3(1), dim3(kPlanThreads), 0,
                     static_cast<hipStream_t>(stream), p);
  return launched();
}

}  // extern "C"
