// attn_plan.hip -- the plan of a packed batch (attn_plan of include/attn.h): the work items
// of the attention passes, found on the device from cu_seqlens, so that no length has to
// reach the host.
//
// Layout: a header of kHeader words {row items, key items, T, G, num_seqs, Hkv, joins}, then
// the row items, the key items and the joins (attn_packed.h). Items are ordered by falling
// work, so that the last workgroups of a launch are short ones: the hardware starts
// workgroups in order. The order of items of like work, and the slots of partial sums, depend
// on the execution; no result depends on them.
#include "attn_packed.h"
#include "attn_plan.h"

namespace attn {
namespace {

constexpr int kBuckets = 1024;

struct PlanParams {
  const int32_t* cu;
  const int32_t* seqused;
  int32_t num_seqs, T, G, Hkv;
  int32_t* header;
  RowItem* row_items;
  KeyItem* key_items;
  KeyJoin* joins;
  PackedSizes sizes;
};

struct Shared {
  SeqChunk c;
  int32_t rows[kPlanThreads], keys[kPlanThreads];  // inclusive running tile counts
  int32_t count[2][kBuckets];                      // items per bucket, then their places
  unsigned long long work;
  int32_t units, joins, items[2];
};

// One workgroup, three passes over the tiles: the work of the dK/dV pass, which gives the
// length of its splits; the number of items by work; the items.
__global__ __launch_bounds__(kPlanThreads) void attn_plan_kernel(const PlanParams p) {
  __shared__ Shared s;
  const int t = threadIdx.x;
  s.count[0][t] = s.count[1][t] = 0;
  if (t == 0) {
    s.work = 0;
    s.units = s.joins = s.items[0] = s.items[1] = 0;
  }
  __syncthreads();
  int32_t split = 1;  // row blocks of a split
  for (int pass = 0; pass < 3; ++pass) {
    int32_t carry = 0;
    for (int32_t s0 = 0; s0 <= p.num_seqs; s0 += kPlanThreads) {
      load_sequences(s.c, p.cu, p.num_seqs, p.T, s0, &carry);
      if (p.seqused != nullptr && s.c.n[t] > 0) {
        const int32_t u = p.seqused[s0 + t - 1];
        s.c.n[t] = u < 0 ? 0 : u < s.c.n[t] ? u : s.c.n[t];
      }
      const int32_t gap = ceil_div(s.c.end[t] - s.c.a[t] - s.c.n[t], kKeyTile);
      s.rows[t] = block_scan<AddOp>(ceil_div(s.c.n[t] * p.G, kRowTile) + gap, s.c.scan);
      s.keys[t] = block_scan<AddOp>(ceil_div(s.c.n[t], kKeyTile) + gap, s.c.scan);
      __syncthreads();
      const int32_t row_tiles = pass > 0 ? s.rows[kPlanThreads - 1] : 0;
      for (int32_t i = t; i < row_tiles; i += kPlanThreads) {
        const int slot = find_slot(s.rows, i);
        const int32_t j = i - (slot > 0 ? s.rows[slot - 1] : 0);
        const int32_t a = s.c.a[slot], n = s.c.n[slot], of_seq = ceil_div(n * p.G, kRowTile);
        RowItem item{a, n, j * kRowTile, 0};
        int32_t work = (min((j + 1) * kRowTile, n * p.G) - 1) / p.G + 1;  // keys
        if (j >= of_seq) {  // rows of no sequence behind it
          const int32_t first = a + n + (j - of_seq) * kKeyTile;
          item = RowItem{first, min(s.c.end[slot] - first, kKeyTile), 0, 1};
          work = 0;
        }
        const int32_t at = atomicAdd(&s.count[0][bucket_of<kBuckets>(work, p.T)], 1);
        if (pass == 1) atomicAdd(&s.items[0], 1);
        else if (at < p.sizes.rows) p.row_items[at] = item;
      }
      const int32_t key_tiles = s.keys[kPlanThreads - 1];
      for (int32_t i = t; i < key_tiles; i += kPlanThreads) {
        const int slot = find_slot(s.keys, i);
        const int32_t j = i - (slot > 0 ? s.keys[slot - 1] : 0);
        const int32_t a = s.c.a[slot], n = s.c.n[slot], of_seq = ceil_div(n, kKeyTile);
        KeyItem item{a, n, j * kKeyTile, 0, 0, 0, -1, 0};
        int32_t blocks = 0;
        if (j >= of_seq) {
          const int32_t first = a + n + (j - of_seq) * kKeyTile;
          item = KeyItem{first, min(s.c.end[slot] - first, kKeyTile), 0, 1, 0, 0, -1, 0};
        } else {
          blocks = ceil_div(n * p.G, kRowBlock) - item.key0 * p.G / kRowBlock;
        }
        if (pass == 0) {
          atomicAdd(&s.work, (unsigned long long)blocks);
          continue;
        }
        const int32_t k = max(1, ceil_div(blocks, split));
        const int32_t bucket = bucket_of<kBuckets>(ceil_div(blocks, k), split);
        const int32_t at = atomicAdd(&s.count[1][bucket], k);
        if (pass == 1) {
          atomicAdd(&s.items[1], k);
          continue;
        }
        int32_t slot0 = -1;
        if (k > 1) {
          slot0 = atomicAdd(&s.units, k);
          const int32_t join = atomicAdd(&s.joins, 1);
          if (join < p.sizes.joins) p.joins[join] = KeyJoin{a, n, item.key0, slot0, k, 0, 0, 0};
        }
        const int32_t first = item.key0 * p.G / kRowBlock;
        for (int32_t x = 0; x < k; ++x) {
          item.block0 = first + (int32_t)((int64_t)blocks * x / k);
          item.block_end = first + (int32_t)((int64_t)blocks * (x + 1) / k);
          item.slot = slot0 < 0 ? -1 : slot0 + x;
          if (at + x < p.sizes.keys) p.key_items[at + x] = item;
        }
      }
      __syncthreads();
    }
    if (pass == 0) {
      const unsigned long long want = (s.work * p.Hkv + kKeyTarget - 1) / kKeyTarget;
      split = want < kMinRowBlocks ? kMinRowBlocks : want > INT32_MAX / 2 ? INT32_MAX / 2 : (int32_t)want;
    }
    if (pass == 1) {
      counts_to_places<kBuckets>(s.count[0], s.c.scan);
      counts_to_places<kBuckets>(s.count[1], s.c.scan);
    }
  }
  if (t == 0) {
    p.header[0] = min((int64_t)s.items[0], p.sizes.rows);
    p.header[1] = min((int64_t)s.items[1], p.sizes.keys);
    p.header[2] = p.T;
    p.header[3] = p.G;
    p.header[4] = p.num_seqs;
    p.header[5] = p.Hkv;
    p.header[6] = min((int64_t)s.joins, p.sizes.joins);
  }
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int64_t attn_plan_ints(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  if (!valid_batch(T, num_seqs, Hq, Hkv)) return -1;
  const PackedSizes z = packed_sizes(T, num_seqs, Hq, Hkv);
  return kHeader + 4 * z.rows + 8 * (z.keys + z.joins);
}

int32_t attn_plan(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* seqused, int64_t T,
                  int32_t Hq, int32_t Hkv, int32_t* plan, int64_t plan_ints, void* stream) {
  if (!valid_batch(T, num_seqs, Hq, Hkv)) return ROPE_EINVAL;
  if (num_seqs > 0 && cu_seqlens == nullptr) return ROPE_EINVAL;
  if (!data_pointer(plan) || plan_ints < attn_plan_ints(T, num_seqs, Hq, Hkv)) return ROPE_EINVAL;
  PlanParams p;
  p.cu = cu_seqlens;
  p.seqused = seqused;
  p.num_seqs = num_seqs;
  p.T = (int32_t)T;
  p.G = Hq / Hkv;
  p.Hkv = Hkv;
  p.sizes = packed_sizes(T, num_seqs, Hq, Hkv);
  p.header = plan;
  p.row_items = reinterpret_cast<RowItem*>(plan + kHeader);
  p.key_items = reinterpret_cast<KeyItem*>(p.row_items + p.sizes.rows);
  p.joins = reinterpret_cast<KeyJoin*>(p.key_items + p.sizes.keys);
  hipLaunchKernelGGL(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0,
                     static_cast<hipStream_t>(stream), p);
  return launched();
}

}  // extern "C"
