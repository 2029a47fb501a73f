// attn_plan.hip -- the plan of a packed batch (attn_plan of include/attn.h): the work items
// of the attention passes, found on the device from cu_seqlens, so that no length has to
// reach the host.
//
// Layout (int32 words): a header {row items, key items, T, G, num_seqs, ...} of kHeader
// words, then the row items and the key items, 4 words each:
//   row item {start, n, row0, 0}: packed rows row0 .. row0 + 127 (row = token * G + head of
//            the group) of the sequence at rows start .. start + n - 1
//   key item {start, n, key0, 0}: keys key0 .. key0 + 127 of that sequence
//   either   {first, count, 0, 1}: rows of no sequence (at most 128)
// Items are ordered by falling work, so that the last workgroups of a launch are short
// ones: the hardware starts workgroups in order. The order of items of like work depends
// on the execution; no result depends on it.
#include "attn_common.h"

namespace attn {
namespace {

constexpr int kThreads = 1024;
constexpr int kBuckets = 1024;

struct Shared {
  int32_t scan[kThreads];
  int32_t a[kThreads], used[kThreads], end[kThreads];  // a chunk of sequences
  int32_t rows[kThreads], keys[kThreads];              // inclusive running item counts
  int32_t count[2][kBuckets];                          // items per bucket, then their place
};

// Inclusive scan over the workgroup.
template <typename Op>
__device__ int32_t block_scan(int32_t x, int32_t* buf, Op op) {
  const int t = threadIdx.x;
  buf[t] = x;
  __syncthreads();
  for (int d = 1; d < kThreads; d <<= 1) {
    const int32_t y = t >= d ? op(buf[t], buf[t - d]) : buf[t];
    __syncthreads();
    buf[t] = y;
    __syncthreads();
  }
  const int32_t r = buf[t];
  __syncthreads();
  return r;
}

struct PlanParams {
  const int32_t* cu;
  const int32_t* seqused;
  int32_t num_seqs, T, G;
  int4* row_items;
  int4* key_items;
  int32_t* header;
};

__device__ inline int32_t tiles(int32_t n, int32_t size) { return n / size + (n % size != 0); }

__device__ inline int32_t max_op(int32_t a, int32_t b) { return a > b ? a : b; }
__device__ inline int32_t add_op(int32_t a, int32_t b) { return a + b; }

// Work of an item in keys, scaled to a bucket; more work, lower bucket.
__device__ inline int32_t bucket_of(int32_t work, int32_t T) {
  const int32_t b = (int32_t)((int64_t)work * (kBuckets - 1) / (T > 0 ? T : 1));
  return kBuckets - 1 - (b < kBuckets ? b : kBuckets - 1);
}

// Sequence slot of item i of a chunk: the first slot whose running count exceeds i.
__device__ inline int find_slot(const int32_t* running, int32_t i) {
  int lo = 0, hi = kThreads - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (running[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Item i of the chunk in either list, and its work.
__device__ inline int4 make_item(const Shared& s, const int32_t* running, bool rows, int32_t i,
                                 int32_t G, int32_t* work) {
  const int slot = find_slot(running, i);
  const int32_t j = i - (slot > 0 ? running[slot - 1] : 0);
  const int32_t a = s.a[slot], n = s.used[slot];
  const int32_t of_seq = rows ? tiles(n * G, kRowTile) : tiles(n, kKeyTile);
  if (j >= of_seq) {  // rows of no sequence behind it
    const int32_t first = a + n + (j - of_seq) * kKeyTile;
    const int32_t left = s.end[slot] - first;
    *work = 0;
    return make_int4(first, left < kKeyTile ? left : kKeyTile, 0, 1);
  }
  if (rows) {
    const int32_t last = min((j + 1) * kRowTile, n * G) - 1;
    *work = last / G + 1;
    return make_int4(a, n, j * kRowTile, 0);
  }
  *work = n - j * kKeyTile;
  return make_int4(a, n, j * kKeyTile, 0);
}

// One workgroup. Slot 0 of the sequences is an empty one that owns the rows before
// cu_seqlens[0]; slot s + 1 is sequence s, and owns the rows up to the next one's start.
__global__ __launch_bounds__(kThreads) void attn_plan_kernel(const PlanParams p) {
  __shared__ Shared s;
  const int t = threadIdx.x;
  for (int i = t; i < 2 * kBuckets; i += kThreads) (&s.count[0][0])[i] = 0;
  const int32_t slots = p.num_seqs + 1;
  int32_t total[2] = {0, 0};
  for (int pass = 0; pass < 2; ++pass) {
    int32_t carry = 0;  // the largest start so far
    for (int32_t s0 = 0; s0 < slots; s0 += kThreads) {
      __syncthreads();
      const int32_t slot = s0 + t;
      // start of slot's rows: 0 for slot 0, else cu[slot - 1], and the next slot's
      int32_t next = slot < p.num_seqs ? p.cu[slot] : p.T;
      next = next < 0 ? 0 : next > p.T ? p.T : next;
      next = max_op(block_scan(next, s.scan, max_op), carry);
      s.scan[t] = next;
      __syncthreads();
      const int32_t a = t > 0 ? s.scan[t - 1] : carry;
      carry = s.scan[kThreads - 1];
      // the last sequence ends at cu[num_seqs]; the rows behind it are its gap
      int32_t n = 0;
      if (slot > 0 && slot < slots) {
        int32_t e = p.cu[slot];
        e = e < a ? a : e > p.T ? p.T : e;
        n = e - a;
        if (p.seqused != nullptr) {
          const int32_t u = p.seqused[slot - 1];
          n = u < 0 ? 0 : u < n ? u : n;
        }
      }
      const int32_t end = slot < slots ? next : a;
      s.a[t] = a;
      s.used[t] = n;
      s.end[t] = end;
      const int32_t gap = tiles(end - a - n, kKeyTile);
      __syncthreads();
      s.rows[t] = block_scan(tiles(n * p.G, kRowTile) + gap, s.scan, add_op);
      s.keys[t] = block_scan(tiles(n, kKeyTile) + gap, s.scan, add_op);
      __syncthreads();
      for (int list = 0; list < 2; ++list) {
        const int32_t* running = list == 0 ? s.rows : s.keys;
        const int32_t items = running[kThreads - 1];
        if (pass == 0) total[list] += items;
        for (int32_t i = t; i < items; i += kThreads) {
          int32_t work;
          const int4 item = make_item(s, running, list == 0, i, p.G, &work);
          const int32_t b = bucket_of(work, p.T);
          const int32_t at = atomicAdd(&s.count[list][b], 1);
          if (pass == 1) (list == 0 ? p.row_items : p.key_items)[at] = item;
        }
      }
    }
    __syncthreads();
    if (pass == 0) {  // counts to first places
      for (int list = 0; list < 2; ++list) {
        const int32_t own = s.count[list][t];
        const int32_t incl = block_scan(own, s.scan, add_op);
        s.count[list][t] = incl - own;
      }
      __syncthreads();
    }
  }
  if (t == 0) {
    p.header[0] = total[0];
    p.header[1] = total[1];
    p.header[2] = p.T;
    p.header[3] = p.G;
    p.header[4] = p.num_seqs;
  }
}

}  // namespace
}  // namespace attn

using namespace attn;

static bool valid_batch(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  return T >= 0 && T <= INT32_MAX && num_seqs >= 0 && num_seqs <= (1 << 24) &&
         valid_heads(Hq, Hkv) && T * (Hq / Hkv) <= INT32_MAX - kRowTile;
}

extern "C" {

int64_t attn_plan_ints(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  if (!valid_batch(T, num_seqs, Hq, Hkv)) return -1;
  return kHeader + 4 * (row_items(T, num_seqs, Hq / Hkv) + key_items(T, num_seqs));
}

int32_t attn_plan(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* seqused, int64_t T,
                  int32_t Hq, int32_t Hkv, int32_t* plan, int64_t plan_ints, void* stream) {
  if (!valid_batch(T, num_seqs, Hq, Hkv)) return ROPE_EINVAL;
  if (num_seqs > 0 && cu_seqlens == nullptr) return ROPE_EINVAL;
  if (plan == nullptr || !aligned16(plan)) return ROPE_EINVAL;
  if (plan_ints < attn_plan_ints(T, num_seqs, Hq, Hkv)) return ROPE_EINVAL;
  PlanParams p;
  p.cu = cu_seqlens;
  p.seqused = seqused;
  p.num_seqs = num_seqs;
  p.T = (int32_t)T;
  p.G = Hq / Hkv;
  p.header = plan;
  p.row_items = reinterpret_cast<int4*>(plan + kHeader);
  p.key_items = p.row_items + row_items(T, num_seqs, p.G);
  hipLaunchKernelGGL(attn_plan_kernel, dim3(1), dim3(kThreads), 0,
                     static_cast<hipStream_t>(stream), p);
  return launched();
}

}  // extern "C"
