// attn_plan.hip -- the plan of a packed batch (attn_plan of include/attn.h): the work items
// of the attention passes, found on the device from cu_seqlens, so that no length has to
// reach the host.
//
// Layout: a header of kHeader words {row items, key tiles, T, G, num_seqs, Hkv, work (64
// bits), kind}, then the row items and the key tiles (attn_packed.h). Row items are ordered by
// falling work, so that the last workgroups of a launch are short ones: the hardware starts
// workgroups in order. The order of items of like work depends on the execution; no result
// depends on it. Key tiles are in the order of the rows, each with the work before it, so that
// the dK/dV pass can cut the whole work into equal shares. It takes 13 us, latency of the scans,
// once a batch.
#include "attn_packed.h"
#include "attn_plan.h"

namespace attn {
namespace {

constexpr int kBuckets = 1024;

struct PlanParams {
  const int32_t* cu;
  const int32_t* seqused;
  const int32_t* prefix_lens;
  int32_t num_seqs, T, G, Hkv;
  int32_t* header;
  RowItem* row_items;
  KeyTile* key_tiles;
  PackedSizes sizes;
};

struct Shared {
  SeqChunk c;
  int32_t rows[kPlanThreads], keys[kPlanThreads];  // inclusive running tile counts
  int64_t work[kPlanThreads], scan[kPlanWaves];    // inclusive running work of the key tiles
  int32_t count[kBuckets];                         // row items per bucket, then their places
  int32_t prefix[kPlanThreads];                    // within the sequence
};

// Work of the first j key tiles of a sequence of n tokens: the sum of kTileUnits + R - 4 G i
// over i < j, R its row blocks (a tile's 128 keys are 4 G blocks of rows); the tiles that begin
// inside of the prefix have all R.
__device__ inline int64_t work_of_tiles(int32_t n, int32_t prefix, int32_t G, int64_t j) {
  const int64_t whole = min((int64_t)ceil_div(prefix, kKeyTile), j);
  return j * (ceil_div(n * G, kRowBlock) + kTileUnits) -
         (kKeyTile / kRowBlock) * (int64_t)G * (j * (j - 1) / 2 - whole * (whole - 1) / 2);
}

// One workgroup, two passes over the tiles: the number of row items by work; the items.
__global__ __launch_bounds__(kPlanThreads) void attn_plan_kernel(const PlanParams p) {
  __shared__ Shared s;
  const int t = threadIdx.x;
  s.count[t] = 0;
  __syncthreads();
  int64_t work_before = 0;
  int32_t rows_before = 0, keys_before = 0;  // of the chunks before, in the second pass
  for (int pass = 0; pass < 2; ++pass) {
    int32_t carry = 0;
    for (int32_t s0 = 0; s0 <= p.num_seqs; s0 += kPlanThreads) {
      load_sequences(s.c, p.cu, p.num_seqs, p.T, s0, &carry);
      if (p.seqused != nullptr && s.c.n[t] > 0) {
        const int32_t u = p.seqused[s0 + t - 1];
        s.c.n[t] = u < 0 ? 0 : u < s.c.n[t] ? u : s.c.n[t];
      }
      const int32_t n = s.c.n[t];
      const int32_t prefix = p.prefix_lens != nullptr && n > 0 ? min(max(p.prefix_lens[s0 + t - 1], 0), n) : 0;
      s.prefix[t] = prefix;
      const int32_t gap = ceil_div(s.c.end[t] - s.c.a[t] - n, kKeyTile);
      s.rows[t] = block_scan<AddOp>(ceil_div(n * p.G, kRowTile) + gap, s.c.scan);
      if (pass == 1) {
        s.keys[t] = block_scan<AddOp>(ceil_div(n, kKeyTile) + gap, s.c.scan);
        s.work[t] = block_scan<Sum<int64_t>>(work_of_tiles(n, prefix, p.G, ceil_div(n, kKeyTile)) + gap, s.scan);
      }
      __syncthreads();
      const int32_t row_tiles = s.rows[kPlanThreads - 1];
      for (int32_t i = t; i < row_tiles; i += kPlanThreads) {
        const int slot = find_slot(s.rows, i);
        const int32_t j = i - (slot > 0 ? s.rows[slot - 1] : 0);
        const int32_t a = s.c.a[slot], m = s.c.n[slot], of_seq = ceil_div(m * p.G, kRowTile);
        RowItem item{a, m, j * kRowTile, s.prefix[slot]};
        int32_t keys = max((min((j + 1) * kRowTile, m * p.G) - 1) / p.G + 1, s.prefix[slot]);
        if (j >= of_seq) {  // rows of no sequence behind it
          const int32_t first = a + m + (j - of_seq) * kKeyTile;
          item = RowItem{first, min(s.c.end[slot] - first, kKeyTile), 0, kGap};
          keys = 0;
        }
        const int32_t at = atomicAdd(&s.count[bucket_of<kBuckets>(keys, p.T)], 1);
        if (pass == 1 && at < p.sizes.rows) p.row_items[at] = item;
      }
      rows_before += row_tiles;
      if (pass == 1) {
        const int32_t key_tiles = s.keys[kPlanThreads - 1];
        for (int32_t i = t; i < key_tiles; i += kPlanThreads) {
          const int slot = find_slot(s.keys, i);
          const int32_t j = i - (slot > 0 ? s.keys[slot - 1] : 0);
          const int32_t a = s.c.a[slot], m = s.c.n[slot], of_seq = ceil_div(m, kKeyTile);
          const int64_t before = work_before + (slot > 0 ? s.work[slot - 1] : 0);
          const int32_t prefix = s.prefix[slot];
          KeyTile tile{a, m, j * kKeyTile, 0, before + work_of_tiles(m, prefix, p.G, j), prefix, 0};
          if (j >= of_seq) {
            const int32_t first = a + m + (j - of_seq) * kKeyTile;
            tile = KeyTile{first, min(s.c.end[slot] - first, kKeyTile), 0, 1,
                           before + work_of_tiles(m, prefix, p.G, of_seq) + (j - of_seq), 0, 0};
          }
          if (keys_before + i < p.sizes.keys) p.key_tiles[keys_before + i] = tile;
        }
        keys_before += key_tiles;
        work_before += s.work[kPlanThreads - 1];
      }
      __syncthreads();
    }
    if (pass == 0) {
      counts_to_places<kBuckets>(s.count, s.c.scan);
      rows_before = 0;
    }
  }
  if (t == 0) {
    p.header[0] = min((int64_t)rows_before, p.sizes.rows);
    p.header[1] = min((int64_t)keys_before, p.sizes.keys);
    p.header[2] = p.T;
    p.header[3] = p.G;
    p.header[4] = p.num_seqs;
    p.header[5] = p.Hkv;
    p.header[8] = kPackedPlan;
    *reinterpret_cast<int64_t*>(p.header + 6) = work_before;
  }
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int64_t attn_plan_ints(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  if (!valid_batch(T, num_seqs, Hq, Hkv)) return -1;
  const PackedSizes z = packed_sizes(T, num_seqs, Hq, Hkv);
  return kHeader + 4 * (z.rows + z.rows % 2) + 8 * z.keys;  // key tiles on 32-byte lines
}

int32_t attn_plan(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* seqused, int64_t T,
                  int32_t Hq, int32_t Hkv, int32_t* plan, int64_t plan_ints, void* stream) {
  return attn_plan_ex(cu_seqlens, num_seqs, seqused, nullptr, T, Hq, Hkv, plan, plan_ints, stream);
}

int32_t attn_plan_ex(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* seqused,
                     const int32_t* prefix_lens, int64_t T, int32_t Hq, int32_t Hkv, int32_t* plan,
                     int64_t plan_ints, void* stream) {
  if (!valid_batch(T, num_seqs, Hq, Hkv)) return ROPE_EINVAL;
  if (num_seqs > 0 && cu_seqlens == nullptr) return ROPE_EINVAL;
  if (!data_pointer(plan) || plan_ints < attn_plan_ints(T, num_seqs, Hq, Hkv)) return ROPE_EINVAL;
  PlanParams p;
  p.cu = cu_seqlens;
  p.seqused = seqused;
  p.prefix_lens = prefix_lens;
  p.num_seqs = num_seqs;
  p.T = (int32_t)T;
  p.G = Hq / Hkv;
  p.Hkv = Hkv;
  p.sizes = packed_sizes(T, num_seqs, Hq, Hkv);
  p.header = plan;
  p.row_items = reinterpret_cast<RowItem*>(plan + kHeader);
  p.key_tiles = reinterpret_cast<KeyTile*>(p.row_items + p.sizes.rows + p.sizes.rows % 2);
  hipLaunchKernelGGL(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0,
                     static_cast<hipStream_t>(stream), p);
  return launched();
}

}  // extern "C"
