// attn_paged.hip -- attention of the newest tokens of each sequence over a paged key/value
// cache (paged_plan and attn_paged of include/attn.h): one token each (decode), chunks of a
// prompt, or both in one batch.
//
// Work items come from a plan made on the device. A tile is up to 128 packed query rows
// (token-major, the heads of a group minor) of one sequence; its keys are cut into splits
// where the batch would otherwise not fill the chip, of equal length over the whole batch.
// A workgroup takes one split of one tile and one key/value head:
//  * tiles of more than 32 rows: each wave has 32 rows, and the four share key blocks
//    through LDS, as in the packed forward (bound by the matrix units);
//  * up to 32 rows (decode): the four waves have the same rows and take key blocks in turn,
//    each with its own LDS, so that none waits for another and K and V stream all the time
//    (bound by memory); their results are joined in LDS at the end.
// Splits leave (m, its rounding, l, O) in fp32, and a second, small kernel joins them in a fixed order.
//
// Keys are found through the block table: a block's page numbers arrive in LDS by an
// asynchronous copy two blocks ahead, a lane turns one key's page into its row's offset, and
// the lanes that copy that row's chunks read it from there. Rows whose page is not a page of
// the cache are hidden from every query.
//
// Measured, bf16, 32 + 8 heads of 128: 64 sequences of 512 to 16384 tokens, one new token each,
// 204 us, 5.6 TB/s (a large copy moves 5.0; reading alone goes faster); one sequence of 4099
// tokens 8.5 us, latency; four chunks of 1024 tokens over 8000 to 24000 keys 1.15 to 1.3 ms, 1.0
// PFLOP/s. The join takes 4 to 11 us, also where no tile is split, the plan 20 to 25. Head sizes
// above 128 have one workgroup on a CU, blocks of 32 keys, and keep up to 150 registers in memory (193 to 256
// columns): 64 sequences of 512 to 16388 tokens, 16 + 8 heads of 256, one new token each, still 759 us, 5.8 TB/s,
// and 777 with a cap; of 192, 635 and 644.
#include "attn_packed.h"
#include "attn_plan.h"
#include "attn_tile.h"

#ifndef ATTN_MODS  // what scores go through (attn_scores.h): this file is compiled once for each
#define ATTN_MODS 0
#endif

namespace attn {

constexpr int kBuckets = 256;
constexpr int kSplitKeys = 64;   // splits begin at multiples of this
constexpr int kMinBlocks = 4;    // of 64 keys, in a split
constexpr int kTarget = 1024;    // workgroups that a batch is split into, about
constexpr int kSmallRows = 32;   // rows of a tile whose waves share the keys out
constexpr int32_t kMostKeys = INT32_MAX - 4096;  // positions; key arithmetic stays in 32 bits

struct Item {
  int32_t q0;      // first row (token) of the sequence in q
  int32_t rows;    // its packed rows; < 0: -rows tokens of no sequence from q0 on
  int32_t row0;    // the tile's first
  int32_t before;  // position of its first token
  int32_t key0, key_end;
  int32_t seq;
  int32_t slot;    // of its partial result in units of 32 rows; < 0: the tile is not split
  int32_t prefix;  // keys that every row at a position sees, of those held
  int32_t unused[3];
};
struct Join {
  int32_t q0, row0, rows, slot, splits, units, unused0, unused1;
};

// Bounds of a plan's lists; attn_paged checks them again.
struct Sizes {
  int64_t items, joins, units;
};
inline Sizes paged_sizes(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  const int64_t G = Hq / Hkv, splits = kTarget / Hkv + 1;
  const int64_t of_tile = T * G <= kSmallRows ? 1 : kRowTile / 32;
  return {row_items(T, num_seqs, (int32_t)G) + splits, splits, 2 * splits * of_tile};
}

// ---- plan ----------------------------------------------------------------------------------

#if ATTN_MODS == 0

namespace {

struct PlanParams {
  const int32_t* cu;
  const int32_t* kv_lens;
  const int32_t* prefix_lens;
  int32_t T, num_seqs, G, Hkv;
  int32_t* header;
  Item* items;
  Join* joins;
  Sizes sizes;
};

struct PlanShared {
  SeqChunk c;
  int32_t held[kPlanThreads], prefix[kPlanThreads];
  int32_t tiles[kPlanThreads];  // inclusive running count
  int32_t count[kBuckets];      // items per bucket, then their places
  unsigned long long total;
  int32_t units, joins, items;
};

// One workgroup, three passes over the tiles: the batch's key blocks, which give the length
// of a split; the number of items by length; the items, the longest first. Slots and the
// order of equal items depend on the execution; no result depends on them.
__global__ __launch_bounds__(kPlanThreads) void paged_plan_kernel(const PlanParams p) {
  __shared__ PlanShared s;
  const int t = threadIdx.x;
  if (t < kBuckets) s.count[t] = 0;
  if (t == 0) {
    s.total = 0;
    s.units = s.joins = s.items = 0;
  }
  __syncthreads();
  int32_t split_blocks = 1;
  for (int pass = 0; pass < 3; ++pass) {
    int32_t carry = 0;
    for (int32_t s0 = 0; s0 <= p.num_seqs; s0 += kPlanThreads) {
      load_sequences(s.c, p.cu, p.num_seqs, p.T, s0, &carry);
      s.held[t] = s.c.n[t] > 0 ? p.kv_lens[s0 + t - 1] : 0;
      s.prefix[t] = p.prefix_lens != nullptr && s.c.n[t] > 0 ? min(max(p.prefix_lens[s0 + t - 1], 0), max(s.held[t], 0)) : 0;
      s.tiles[t] = block_scan<AddOp>(ceil_div(s.c.n[t] * p.G, kRowTile) +
                                         ceil_div(s.c.end[t] - s.c.a[t] - s.c.n[t], kKeyTile),
                                     s.c.scan);
      __syncthreads();
      const int32_t tiles = s.tiles[kPlanThreads - 1];
      for (int32_t i = t; i < tiles; i += kPlanThreads) {
        const int lo = find_slot(s.tiles, i);
        const int32_t j = i - (lo > 0 ? s.tiles[lo - 1] : 0);
        const int32_t rows = s.c.n[lo] * p.G;
        Item item;
        item.q0 = s.c.a[lo];
        item.seq = s0 + lo - 1;
        item.slot = -1;
        item.prefix = s.prefix[lo];
        int32_t blocks = 0, tile_rows = 0;
        if (j >= ceil_div(rows, kRowTile)) {  // rows of no sequence
          item.q0 += s.c.n[lo] + (j - ceil_div(rows, kRowTile)) * kKeyTile;
          item.rows = -min(s.c.end[lo] - item.q0, kKeyTile);
          item.row0 = item.before = item.key0 = item.key_end = 0;
        } else {
          item.rows = rows;
          item.row0 = j * kRowTile;
          tile_rows = min(kRowTile, rows - item.row0);
          // a held length below the new tokens' leaves the first of them without a key
          item.before = (int32_t)max((int64_t)s.held[lo] - s.c.n[lo], (int64_t)INT32_MIN);
          item.key0 = 0;
          const int64_t last = (int64_t)item.before + (item.row0 + tile_rows - 1) / p.G;
          item.key_end = last < 0 ? 0 : (int32_t)min(max(last + 1, (int64_t)item.prefix), (int64_t)kMostKeys);
          blocks = ceil_div(item.key_end, kSplitKeys);
        }
        if (pass == 0) {
          atomicAdd(&s.total, (unsigned long long)blocks);
          continue;
        }
        // Splits of at most that length for tiles of few rows, whose waves stream keys and have
        // little to join (4099 keys of 8 heads: 8.0 us, and 9.4 by the other rule); the nearest
        // number for larger tiles, whose split costs 64 KB of sums and a second read of them
        // (chunks of 1024 tokens over 8000 to 24000 keys: 1240 us, and 1310 by this rule).
        const int32_t up = tile_rows > kSmallRows ? (split_blocks - 1) / 2 : split_blocks - 1;
        const int32_t k = max(1, (blocks + up) / split_blocks);
        const int32_t len = ceil_div(blocks, k);
        const int32_t at = atomicAdd(&s.count[bucket_of<kBuckets>(len, split_blocks + split_blocks / 2)], k);
        if (pass == 1) {
          atomicAdd(&s.items, k);
          continue;
        }
        if (k > 1) {
          const int32_t units = ceil_div(tile_rows, 32);
          const int32_t slot0 = atomicAdd(&s.units, k * units);
          const int32_t join = atomicAdd(&s.joins, 1);
          if (join < p.sizes.joins)
            p.joins[join] = Join{item.q0, item.row0, tile_rows, slot0, k, units, 0, 0};
          item.slot = slot0;
        }
        const int32_t key_end = item.key_end, slot0 = item.slot;
        for (int32_t x = 0; x < k; ++x) {
          if (k > 1) {
            item.key0 = (int32_t)((int64_t)blocks * x / k) * kSplitKeys;
            item.key_end = min(key_end, (int32_t)((int64_t)blocks * (x + 1) / k) * kSplitKeys);
            item.slot = slot0 + x * ceil_div(tile_rows, 32);
          }
          if (at + x < p.sizes.items) p.items[at + x] = item;
        }
      }
      __syncthreads();
    }
    if (pass == 0) {
      const unsigned long long want = (s.total * p.Hkv + kTarget - 1) / kTarget;
      split_blocks = want < kMinBlocks ? kMinBlocks : want > INT32_MAX / 64 ? INT32_MAX / 64 : (int32_t)want;
    }
    if (pass == 1) counts_to_places<kBuckets>(s.count, s.c.scan);
  }
  if (t == 0) {
    p.header[0] = s.items < p.sizes.items ? s.items : (int32_t)p.sizes.items;
    p.header[1] = s.joins < p.sizes.joins ? s.joins : (int32_t)p.sizes.joins;
    p.header[2] = p.T;
    p.header[3] = p.G;
    p.header[4] = p.num_seqs;
    p.header[5] = p.Hkv;
    p.header[8] = kPagedPlan;
  }
}

}  // namespace

#endif

// ---- attention -------------------------------------------------------------------------------

struct PagedParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  void* out;
  float* lse;
  float* part_o;   // [unit][Hkv][32][D], not normalized
  float* part_ml;  // [unit][Hkv][32][4]: m in base 2, what its rounding left, l
  const int32_t* plan;
  const Item* items;
  const Join* joins;
  const int32_t* table;
  int64_t q_stride, out_stride, table_stride;
  int64_t page_bytes, slot_bytes, head_bytes;
  int64_t units;
  int32_t T, Hq, Hkv, G, D, num_seqs, num_pages, page_size, max_pages;
  float scale;  // times log2 e
  int32_t fill;
  Div31 by_hkv, by_g, by_page;
  ScoreParams scores;
};

template <int MODS>
int32_t launch_paged(const PagedParams& p, const Sizes& sizes, int32_t dtype, hipStream_t s);
template <typename T>
int32_t launch_join(const PagedParams& p, const Sizes& sizes, hipStream_t s);

namespace {

// A wave's view of the cache: rows of key blocks of BN keys, by way of the block table.
template <int BN, int CPR>
struct PagedKeys {
  const int32_t* table;  // the sequence's
  uint8_t* pages;        // LDS: 2 x 64 page numbers, of the block after the next by parity
  uint8_t* rows;         // LDS: 2 x BN row offsets (bytes, 64 bits)
  int32_t key_end;

  // Copies the page numbers of a block's keys (a lane each) into LDS.
  __device__ void fetch_pages(const PagedParams& p, int32_t key0, int parity, uint32_t lane) const {
    const uint32_t key = min(key0 + (int32_t)(lane % BN), key_end - 1);
    copy_word_to_lds(table + div31(key, p.by_page), lds_address(pages) + parity * 256);
  }
  // Page numbers that have arrived to row offsets; returns the bits of hidden keys.
  __device__ uint64_t find_rows(const PagedParams& p, int32_t key0, int parity, uint32_t lane) const {
    const uint32_t key = min(key0 + (int32_t)(lane % BN), key_end - 1);
    const int32_t page = reinterpret_cast<const int32_t*>(pages)[parity * 64 + lane];
    const bool real = page >= 0 && page < p.num_pages;
    const uint32_t slot = key - div31(key, p.by_page) * p.page_size;
    const int64_t at = real ? page * p.page_bytes + slot * p.slot_bytes : 0;
    if (BN == 64 || lane < BN) reinterpret_cast<int64_t*>(rows)[parity * BN + lane] = at;
    return __ballot(!real) & (BN == 64 ? ~0ull : (1ull << BN % 64) - 1);
  }
  __device__ const uint8_t* row(const uint8_t* base, int parity, uint32_t r) const {
    return base + reinterpret_cast<const int64_t*>(rows)[parity * BN + r];
  }
};

// This wave's reads of LDS are done: what they read may be overwritten.
__device__ inline void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

template <typename T, int DB, int MODS>
__global__ __launch_bounds__(256, DB <= 4 ? 2 : 1) void attn_paged_kernel(const PagedParams p) {
  constexpr int CPR = chunks_per_row(DB), BN = keys_per_block(DB);
  constexpr int kTileBytes = BN * CPR * 16, kSmallTile = 32 * CPR * 16;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * kTileBytes];
  __shared__ __attribute__((aligned(16))) uint8_t pages[4][512];
  __shared__ __attribute__((aligned(16))) uint8_t offsets[4][2 * 64 * 8];
  __shared__ float joined[4][3][32];

  const uint32_t index = div31(blockIdx.x, p.by_hkv);
  const uint32_t kvh = blockIdx.x - index * p.Hkv;
  if (!plan_matches(p, kPagedPlan) || (int32_t)index >= p.plan[0]) return;
  const Item item = p.items[index];
  const uint32_t tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = p.D >> 3;
  T* out = static_cast<T*>(p.out);

  if (item.rows <= 0) {  // rows of no sequence
    const int32_t n = -item.rows;
    if (!p.fill || item.q0 < 0 || n > p.T || item.q0 > p.T - n) return;
    const uint32_t per_token = p.G * chunks;
    for (uint32_t i = tid; i < n * per_token; i += 256) {
      const uint32_t t = i / per_token, c = i - t * per_token;
      *reinterpret_cast<u32x4*>(out + (int64_t)(item.q0 + t) * p.out_stride +
                                (int64_t)kvh * p.G * p.D + 8 * c) = (u32x4){0, 0, 0, 0};
    }
    for (uint32_t i = tid; i < (uint32_t)n * p.G; i += 256) {
      const uint32_t t = i / p.G, g = i - t * p.G;
      p.lse[(int64_t)(item.q0 + t) * p.Hq + kvh * p.G + g] = -__builtin_inff();
    }
    return;
  }
  if (item.q0 < 0 || item.row0 < 0 || item.row0 >= item.rows || item.seq < 0 ||
      item.seq >= p.num_seqs || item.q0 + (item.rows - 1) / p.G >= p.T || item.key0 < 0)
    return;
  const int32_t row_end = min(item.row0 + kRowTile, item.rows);
  const int32_t units = (row_end - item.row0 + 31) / 32;
  if (item.slot >= 0 && item.slot + units > p.units) return;
  const bool small = row_end - item.row0 <= kSmallRows;

  const int32_t wave_row0 = item.row0 + (small ? 0 : 32 * wave);
  const int32_t row = wave_row0 + (lane & 31);
  const bool on = row < row_end;
  const int32_t clamped = on ? row : row_end - 1;
  const int32_t token = div31(clamped, p.by_g);
  const int64_t most = min((int64_t)p.max_pages * p.page_size, (int64_t)kMostKeys);
  const int32_t key_end = (int32_t)min((int64_t)item.key_end, most);
  // visible keys of a token, 0 for none; within this split
  auto seen_by = [&](int32_t tok) __attribute__((always_inline)) {
    const int64_t s = (int64_t)item.before + tok + 1;
    return s <= 0 ? 0 : (int32_t)min(max(s, (int64_t)item.prefix), (int64_t)key_end);
  };
  const int32_t seen = seen_by(token);
  const int32_t wave_end =
      wave_row0 < row_end ? seen_by(div31(min(wave_row0 + 32, row_end) - 1, p.by_g)) : 0;
  const int32_t wave_all = seen_by(div31(min(wave_row0, row_end - 1), p.by_g));

  const int32_t* table = p.table + item.seq * p.table_stride;
  const uint8_t* kb = static_cast<const uint8_t*>(p.k_cache) + kvh * p.head_bytes;
  const uint8_t* vb = static_cast<const uint8_t*>(p.v_cache) + kvh * p.head_bytes;
  // Where this lane's row is in a tensor of token stride `stride` and `unit` values a head.
  // `anew`: formed again, so that it takes no registers in between.
  auto row_at = [&](int64_t stride, int32_t unit, bool anew) __attribute__((always_inline)) {
    int32_t c = clamped;
    if (anew) asm volatile("" : "+v"(c));
    const int32_t tok = div31(c, p.by_g);
    return (item.q0 + tok) * stride + (int64_t)(kvh * p.G + c - tok * p.G) * unit;
  };
  const int32_t head = kvh * p.G + clamped - token * p.G;
  const int32_t position = (int32_t)((uint32_t)item.before + token);  // rows before 0 see nothing
  const T* q_row = static_cast<const T*>(p.q) + row_at(p.q_stride, p.D, false);
  const int32_t keys = key_end - item.key0;
  clear_unused_chunks<CPR>(lds, 4 * BN, chunks);
  __syncthreads();  // a wave's copies may land in what another clears

  if (!small) {
    FwdTile<T, DB, BN, MODS> t;
    t.set_scores(p.scores, head, position);
    load_row<T>(t.q, q_row, half, chunks);
    const int32_t blocks = keys > 0 ? (keys + BN - 1) / BN : 0;
    const PagedKeys<BN, CPR> src{table, pages[wave], offsets[wave], key_end};
    constexpr int kLoads = BN * CPR / 256;
    uint64_t lanes[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) lanes[i] = __ballot(chunk_of<CPR, 256>(i, tid) < chunks);
    // the x-th copy of block b
    auto piece = [&](int32_t b, int x) __attribute__((always_inline)) {
      const int i = x / 2;
      const uint32_t dst = lds_address(lds) + ((b & 1) * 2 + x % 2) * kTileBytes + (i * 256 + wave * 64) * 16;
      copy_chunk_to_lds(src.row(x % 2 ? vb : kb, b & 1, row_of<CPR, 256>(i, tid)) + 16 * chunk_of<CPR, 256>(i, tid),
                        dst, lanes[i]);
    };
    constexpr int kPieces = 2 * kLoads, kPerStep = (kPieces + 2 * DB - 1) / (2 * DB);
    // Two loops, so that neither body's registers are moved for the other's sake; the first
    // ends at the first block that is not wholly seen, or that has keys on no page.
    const int32_t all = wave_end > 0 ? max(0, wave_all - item.key0) / BN : 0;
    auto walk = [&](auto mode) __attribute__((always_inline)) {
      t.clear();
      if (blocks <= 0) return;
      uint64_t hidden = 0;
      src.fetch_pages(p, item.key0, 0, lane);
      wait_copies<0>();
      uint64_t hidden_next = src.find_rows(p, item.key0, 0, lane);
      src.fetch_pages(p, item.key0 + BN, 1, lane);
#pragma unroll
      for (int x = 0; x < kPieces; ++x) piece(0, x);
      settle<T>(t.q);
      int32_t b = 0;
      // Behind the last block the last key's copies go on into the buffer that is not used.
      auto arrive = [&]() __attribute__((always_inline)) {
        const int32_t key0 = item.key0 + b * BN;
        wait_copies_and_sync<0>();  // block b has arrived, and its buffer's neighbour is free
        hidden = hidden_next;
        hidden_next = src.find_rows(p, key0 + BN, (b + 1) & 1, lane);
        src.fetch_pages(p, key0 + 2 * BN, b & 1, lane);
        return lds + (b & 1) * 2 * kTileBytes;
      };
      auto next = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int x = s * kPerStep; x < (s + 1) * kPerStep && x < kPieces; ++x) piece(b + 1, x);
      };
      for (; b < (decltype(mode)::value == kCareful && t.exact ? 0 : all) && hidden_next == 0; ++b) {
        const uint8_t* kt = arrive();
        t.template block<kWhole>(kt, kt + kTileBytes, item.key0 + b * BN, seen, 0, p.scale, lane, next);
      }
      for (; b < blocks; ++b) {
        const uint8_t* kt = arrive();
        const int32_t key0 = item.key0 + b * BN;
        if (key0 < wave_end)
          t.template block<Mode(decltype(mode)::value)>(kt, kt + kTileBytes, key0, seen, hidden, p.scale,
                                                        lane, next);
        else
#pragma unroll
          for (int s = 0; s < 2 * DB; ++s) next(s);
      }
      wait_copies<0>();
    };
    walk(Constant<kMasked>());
    const uint32_t anew = any_wave(any_nonfinite(t.o) | (uint32_t)t.large() << 1, lds);
    float low = 0.0f;
    if (anew) {
      t.exact = anew & 2;
      walk(Constant<kCareful>());
      low = t.scale_maximum(p.scale);
    }
    if (item.slot < 0) {
      const float lse = t.finish();
      store_row<T, DB>(t.o, out + row_at(p.out_stride, p.D, true), half, chunks, on);
      if (on && half == 0) p.lse[row_at(p.Hq, 1, true)] = lse;
      return;
    }
    const int64_t unit = ((int64_t)(item.slot + wave) * p.Hkv + kvh) * 32 + (lane & 31);
    const float l = half_sum(t.l);
    if (!on) return;
    if (half == 0) *reinterpret_cast<f32x4*>(p.part_ml + 4 * unit) = (f32x4){t.m, low, l, 0.0f};
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t e = 32 * d + 8 * j + 4 * half;
        if (e < (uint32_t)p.D)
          *reinterpret_cast<f32x4*>(p.part_o + unit * p.D + e) =
              (f32x4){t.o[d][4 * j], t.o[d][4 * j + 1], t.o[d][4 * j + 2], t.o[d][4 * j + 3]};
      }
    return;
  }

  // Up to 32 rows: wave w takes the 32-key blocks w, w + 4, ... A wave's LDS holds one block
  // of K and one of V (head sizes above 128: one buffer for both in turn). While a block's
  // scores are formed its V is on the way, and while its V is used the next block's K.
  constexpr bool kOneBuffer = DB > 4;
  constexpr int kLoads = 32 * CPR / 64;
  FwdTile<T, DB, 32, MODS> t;
  t.set_scores(p.scores, head, position);
  float low = 0.0f;
  load_row<T>(t.q, q_row, half, chunks);
  {
    const PagedKeys<32, CPR> src{table, pages[wave], offsets[wave], key_end};
    const uint8_t* kt = lds + wave * kTileBytes;
    const uint8_t* vt = kOneBuffer ? kt : kt + kSmallTile;
    const int32_t blocks = keys > 0 ? ((keys + 31) / 32 - (int32_t)wave + 3) / 4 : 0;
    const int32_t first = item.key0 + 32 * wave;
    uint64_t lanes[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) lanes[i] = __ballot(chunk_of<CPR, 64>(i, lane) < chunks);
    auto stage = [&](const uint8_t* base, const uint8_t* tile, int parity) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        copy_chunk_to_lds(src.row(base, parity, row_of<CPR, 64>(i, lane)) + 16 * chunk_of<CPR, 64>(i, lane),
                          lds_address(tile) + i * 1024, lanes[i]);
    };
    uint64_t hidden = 0, hidden_next = 0;
    auto round = [&](auto mode, int32_t b) __attribute__((always_inline)) {
      constexpr Mode MODE = Mode(decltype(mode)::value);
      const int32_t key0 = first + 128 * b;
      const bool more = b + 1 < blocks;
      hidden = hidden_next;
      f32x16 s[1];
      x8<T> w[2];
      wait_copies<kOneBuffer ? 0 : kLoads>();
      t.scores(s, kt, lane, [](int) {});
      reads_done();
      if (kOneBuffer) stage(vb, vt, b & 1);
      if (more) {
        hidden_next = src.find_rows(p, key0 + 128, (b + 1) & 1, lane);
        src.fetch_pages(p, key0 + 256, b & 1, lane);
        if (!kOneBuffer) stage(kb, kt, (b + 1) & 1);
      }
      t.template weights<MODE>(s, w, key0, seen, hidden, p.scale, lane);
      if (more && !kOneBuffer) wait_copies<kLoads + 1>();
      else wait_copies<0>();
      t.template accumulate<MODE>(w, vt, key0, seen, hidden, lane);
      reads_done();
      if (more) {
        if (kOneBuffer) stage(kb, kt, (b + 1) & 1);
        else stage(vb, vt, (b + 1) & 1);
      }
    };
    // blocks that every row sees whole, then the others (two loops, as above)
    const int32_t whole = max(0, wave_all - first) / 32;
    const int32_t all = wave_all >= first + 32 ? min(blocks, (whole - 1) / 4 + 1) : 0;
    auto walk = [&](auto mode) __attribute__((always_inline)) {
      t.clear();
      if (blocks <= 0) return;
      src.fetch_pages(p, first, 0, lane);
      settle<T>(t.q);
      wait_copies<0>();
      hidden_next = src.find_rows(p, first, 0, lane);
      src.fetch_pages(p, first + 128, 1, lane);
      stage(kb, kt, 0);
      if (!kOneBuffer) stage(vb, vt, 0);
      int32_t b = 0;
      for (; b < (decltype(mode)::value == kCareful && t.exact ? 0 : all) && hidden_next == 0; ++b) round(Constant<kWhole>(), b);
      for (; b < blocks; ++b) round(mode, b);
    };
    walk(Constant<kMasked>());
    t.exact = __any(t.large());  // this wave alone
    if (t.exact || __any(any_nonfinite(t.o))) {
      walk(Constant<kCareful>());
      low = t.scale_maximum(p.scale);
    }
  }

  // Join the waves: O scaled to the common maximum goes to LDS four blocks of columns at a
  // time, a wave's quarter of the tiles each, 16-byte groups swizzled by the row.
  const float l = half_sum(t.l);
  if (half == 0) {
    joined[wave][0][lane] = t.m;
    joined[wave][1][lane] = low;
    joined[wave][2][lane] = l;
  }
  __syncthreads();
  const uint32_t r = lane & 31;
  auto find_top = [&](uint32_t y, float& m, float& m_low) __attribute__((always_inline)) {
    m = joined[0][0][y];
    m_low = joined[0][1][y];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float mw = joined[w][0][y], lw = joined[w][1][y];
      const bool higher = above(mw, lw, m, m_low);
      m = higher ? mw : m;
      m_low = higher ? lw : m_low;
    }
  };
  float top, top_low;
  find_top(r, top, top_low);
  const float factor = join_factor(t.m, low, top, top_low);
  constexpr int kColumns = DB < 4 ? DB : 4;  // blocks of 32 columns a time
  constexpr int kGroups = kColumns * 8;      // 16-byte groups of a row
  const int32_t n_rows = row_end - item.row0;
#pragma unroll
  for (int d0 = 0; d0 < DB; d0 += kColumns) {
    if (on) {
#pragma unroll
      for (int d = 0; d < kColumns; ++d)
        if (d0 + d < DB) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t group = 8 * d + 2 * j + half;
            f32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = t.o[d0 + d][4 * j + e] * factor;
            *reinterpret_cast<f32x4*>(lds + wave * kTileBytes + (r * kGroups + (group ^ (r & 7))) * 16) = x;
          }
        }
    }
    __syncthreads();
    for (uint32_t i = tid; i < (uint32_t)n_rows * kGroups; i += 256) {
      const uint32_t y = i / kGroups, group = i % kGroups;
      const uint32_t e = 32 * d0 + 4 * group;
      f32x4 x = {0, 0, 0, 0};
      float m, m_low, sum = 0.0f;
      find_top(y, m, m_low);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const f32x4 part = *reinterpret_cast<const f32x4*>(
            lds + w * kTileBytes + (y * kGroups + (group ^ (y & 7))) * 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] += part[c];
        sum += joined[w][2][y] * join_factor(joined[w][0][y], joined[w][1][y], m, m_low);
      }
      if (e >= (uint32_t)p.D) continue;
      if (item.slot >= 0) {
        const int64_t unit = ((int64_t)item.slot * p.Hkv + kvh) * 32 + y;
        *reinterpret_cast<f32x4*>(p.part_o + unit * p.D + e) = x;
        if (e == 0) *reinterpret_cast<f32x4*>(p.part_ml + 4 * unit) = (f32x4){m, m_low, sum, 0.0f};
      } else {
        const int32_t packed = item.row0 + y, tok = div31(packed, p.by_g);
        const int32_t h = kvh * p.G + (packed - tok * p.G);
        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        u32x2 word = {narrow2<T>(x[0] * inv, x[1] * inv), narrow2<T>(x[2] * inv, x[3] * inv)};
        *reinterpret_cast<u32x2*>(out + (int64_t)(item.q0 + tok) * p.out_stride + (int64_t)h * p.D + e) =
            word;
        if (e == 0) p.lse[(int64_t)(item.q0 + tok) * p.Hq + h] = log_sum_exp(m, sum);
      }
    }
    __syncthreads();
  }
}

// Joins the splits of a tile: out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i, each m_i with what
// its rounding left.
#if ATTN_MODS == 0
template <typename T>
__global__ __launch_bounds__(256) void paged_join_kernel(const PagedParams p) {
  const uint32_t index = div31(blockIdx.x, p.by_hkv);
  const uint32_t kvh = blockIdx.x - index * p.Hkv, part = blockIdx.y;
  if (!plan_matches(p, kPagedPlan) || (int32_t)index >= p.plan[1]) return;
  const Join j = p.joins[index];
  if (j.q0 < 0 || j.row0 < 0 || j.rows <= 0 || j.rows > kRowTile || j.units < (j.rows + 31) / 32 ||
      j.splits < 0 || j.slot < 0 || j.slot + (int64_t)j.splits * j.units > p.units ||
      j.q0 + (j.row0 + j.rows - 1) / p.G >= p.T)
    return;
  const int32_t rows = min(32, j.rows - 32 * (int32_t)part);
  const uint32_t groups = p.D >> 2;
  const int64_t step = (int64_t)j.units * p.Hkv * 32;
  const int64_t unit0 = ((int64_t)(j.slot + part) * p.Hkv + kvh) * 32;
  for (int32_t i = threadIdx.x; i < rows * (int32_t)groups; i += 256) {
    const uint32_t y = i / groups, e = 4 * (i - y * groups);
    const float* ml = p.part_ml + 4 * (unit0 + y);
    const float* o = p.part_o + (unit0 + y) * p.D + e;
    float m = -__builtin_inff(), low = 0.0f, l = 0.0f;
    f32x4 x = {0, 0, 0, 0};
    for (int32_t s0 = 0; s0 < j.splits; s0 += 8) {  // eight splits' loads at a time
      f32x4 w[8];
      f32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t s = min(s0 + u, j.splits - 1);
        w[u] = *reinterpret_cast<const f32x4*>(ml + 4 * s * step);
        v[u] = *reinterpret_cast<const f32x4*>(o + s * step * p.D);
      }
      float top = m, top_low = low;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool higher = above(w[u][0], w[u][1], top, top_low);
        top = higher ? w[u][0] : top;
        top_low = higher ? w[u][1] : top_low;
      }
      const float f0 = join_factor(m, low, top, top_low);
      m = top;
      low = top_low;
      l *= f0;
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] *= f0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (s0 + u >= j.splits) break;
        const float f = join_factor(w[u][0], w[u][1], m, low);
        l = __builtin_fmaf(w[u][2], f, l);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = __builtin_fmaf(v[u][c], f, x[c]);
      }
    }
    const int32_t packed = j.row0 + 32 * part + y, tok = div31(packed, p.by_g);
    const int32_t h = kvh * p.G + (packed - tok * p.G);
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const u32x2 word = {narrow2<T>(x[0] * inv, x[1] * inv), narrow2<T>(x[2] * inv, x[3] * inv)};
    *reinterpret_cast<u32x2*>(static_cast<T*>(p.out) + (int64_t)(j.q0 + tok) * p.out_stride +
                              (int64_t)h * p.D + e) = word;
    if (e == 0) p.lse[(int64_t)(j.q0 + tok) * p.Hq + h] = log_sum_exp(m, l);
  }
}
#endif

template <typename T, int DB>
int32_t launch(const PagedParams& p, const Sizes& sizes, hipStream_t s) {
  hipLaunchKernelGGL((attn_paged_kernel<T, DB, ATTN_MODS>), dim3((unsigned)(sizes.items * p.Hkv)), dim3(256), 0,
                     s, p);
  const int32_t st = launched();
  return st != ROPE_OK ? st : launch_join<T>(p, sizes, s);
}

template <typename T>
int32_t launch_size(const PagedParams& p, const Sizes& sizes, hipStream_t s) {
  switch ((p.D + 31) / 32) {
    case 1: return launch<T, 1>(p, sizes, s);
    case 2: return launch<T, 2>(p, sizes, s);
    case 3: return launch<T, 3>(p, sizes, s);
    case 4: return launch<T, 4>(p, sizes, s);
    case 5:
    case 6: return launch<T, 6>(p, sizes, s);
    default: return launch<T, 8>(p, sizes, s);
  }
}

}  // namespace

template <>
int32_t launch_paged<ATTN_MODS>(const PagedParams& p, const Sizes& sizes, int32_t dtype, hipStream_t s) {
  return dtype == ROPE_BF16 ? launch_size<__bf16>(p, sizes, s) : launch_size<_Float16>(p, sizes, s);
}

#if ATTN_MODS == 0
template <typename T>
int32_t launch_join(const PagedParams& p, const Sizes& sizes, hipStream_t s) {
  hipLaunchKernelGGL((paged_join_kernel<T>), dim3((unsigned)(sizes.joins * p.Hkv), kRowTile / 32),
                     dim3(256), 0, s, p);
  return launched();
}
template int32_t launch_join<__bf16>(const PagedParams& p, const Sizes& sizes, hipStream_t s);
template int32_t launch_join<_Float16>(const PagedParams& p, const Sizes& sizes, hipStream_t s);
#endif

}  // namespace attn

#if ATTN_MODS == 0

using namespace attn;

constexpr int32_t kItemWords = 12, kJoinWords = 8;
static_assert(sizeof(Item) == 4 * kItemWords && sizeof(Join) == 4 * kJoinWords, "words");

extern "C" {

int64_t paged_plan_ints(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  if (attn_plan_ints(T, num_seqs, Hq, Hkv) < 0) return -1;
  const Sizes z = paged_sizes(T, num_seqs, Hq, Hkv);
  return kHeader + kItemWords * z.items + kJoinWords * z.joins;
}

int64_t paged_workspace_floats(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv, int32_t D) {
  if (attn_plan_ints(T, num_seqs, Hq, Hkv) < 0 || !valid_head_size(D)) return -1;
  return paged_sizes(T, num_seqs, Hq, Hkv).units * Hkv * 32 * (D + 4);
}

int32_t paged_plan(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* kv_lens, int64_t T,
                   int32_t Hq, int32_t Hkv, int32_t* plan, int64_t plan_ints, void* stream) {
  return paged_plan_ex(cu_seqlens, num_seqs, kv_lens, nullptr, T, Hq, Hkv, plan, plan_ints, stream);
}

int32_t paged_plan_ex(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* kv_lens,
                      const int32_t* prefix_lens, int64_t T, int32_t Hq, int32_t Hkv, int32_t* plan,
                      int64_t plan_ints, void* stream) {
  const int64_t need = paged_plan_ints(T, num_seqs, Hq, Hkv);
  if (need < 0 || plan_ints < need || !data_pointer(plan)) return ROPE_EINVAL;
  if (num_seqs > 0 && (cu_seqlens == nullptr || kv_lens == nullptr)) return ROPE_EINVAL;
  PlanParams p;
  p.cu = cu_seqlens;
  p.kv_lens = kv_lens;
  p.prefix_lens = prefix_lens;
  p.T = (int32_t)T;
  p.num_seqs = num_seqs;
  p.G = Hq / Hkv;
  p.Hkv = Hkv;
  p.sizes = paged_sizes(T, num_seqs, Hq, Hkv);
  p.header = plan;
  p.items = reinterpret_cast<Item*>(plan + kHeader);
  p.joins = reinterpret_cast<Join*>(p.items + p.sizes.items);
  hipLaunchKernelGGL(paged_plan_kernel, dim3(1), dim3(kPlanThreads), 0,
                     static_cast<hipStream_t>(stream), p);
  return launched();
}

int32_t attn_paged(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                   float* workspace, int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride,
                   int64_t out_stride, int32_t num_pages, int32_t page_size, int64_t page_stride,
                   int64_t slot_stride, int64_t head_stride, const int32_t* block_table,
                   int32_t max_pages, int64_t table_stride, const int32_t* plan, int32_t num_seqs,
                   double scale, int32_t dtype, int32_t fill, void* stream) {
  return attn_paged_ex(q, k_cache, v_cache, out, lse, workspace, T, Hq, Hkv, D, q_stride, out_stride,
                       num_pages, page_size, page_stride, slot_stride, head_stride, block_table, max_pages,
                       table_stride, plan, num_seqs, scale, 0.0, nullptr, dtype, fill, stream);
}

int32_t attn_paged_ex(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                      float* workspace, int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride,
                      int64_t out_stride, int32_t num_pages, int32_t page_size, int64_t page_stride,
                      int64_t slot_stride, int64_t head_stride, const int32_t* block_table,
                      int32_t max_pages, int64_t table_stride, const int32_t* plan, int32_t num_seqs,
                      double scale, double cap, const float* slopes, int32_t dtype, int32_t fill,
                      void* stream) {
  if (!valid_dtype16(dtype)) return ROPE_EUNSUPPORTED;
  if (attn_plan_ints(T, num_seqs, Hq, Hkv) < 0 || !valid_head_size(D)) return ROPE_EINVAL;
  if (!valid_scale(scale) || !valid_cap(cap, scale)) return ROPE_EINVAL;
  PagedParams p;
  if (!token_stride(q_stride, Hq, D, &p.q_stride) || !token_stride(out_stride, Hq, D, &p.out_stride))
    return ROPE_EINVAL;
  if (num_pages < 1 || page_size < 1 || max_pages < 0 || table_stride < 0 ||
      table_stride > ((int64_t)1 << 40))
    return ROPE_EINVAL;
  for (const int64_t x : {page_stride, slot_stride, head_stride})
    if (x < 0 || x % 8 != 0 || x > ((int64_t)1 << 40)) return ROPE_EINVAL;
  if (T == 0) return ROPE_OK;
  if (!data_pointer(q) || !data_pointer(k_cache) || !data_pointer(v_cache) || !data_pointer(out) ||
      !data_pointer(plan) || !data_pointer(workspace) || lse == nullptr)
    return ROPE_EINVAL;
  if (num_seqs > 0 && max_pages > 0 && block_table == nullptr) return ROPE_EINVAL;
  const Sizes z = paged_sizes(T, num_seqs, Hq, Hkv);
  if (z.items * Hkv > kMaxBlocks) return ROPE_EINVAL;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.out = out;
  p.lse = lse;
  p.part_o = workspace;
  p.part_ml = workspace + z.units * Hkv * 32 * D;
  p.plan = plan;
  p.items = reinterpret_cast<const Item*>(plan + kHeader);
  p.joins = reinterpret_cast<const Join*>(p.items + z.items);
  p.table = block_table;
  p.table_stride = table_stride;
  p.page_bytes = page_stride * 2;
  p.slot_bytes = slot_stride * 2;
  p.head_bytes = head_stride * 2;
  p.units = z.units;
  p.T = (int32_t)T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.D = D;
  p.num_seqs = num_seqs;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.scale = score_scale(scale, cap);
  p.scores = score_params(scale, cap, slopes);
  p.fill = fill;
  p.by_hkv = make_div31(Hkv);
  p.by_g = make_div31(p.G);
  p.by_page = make_div31(page_size);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (score_mods(cap, slopes)) {
    case 0: return launch_paged<0>(p, z, dtype, s);
    case kBias: return launch_paged<kBias>(p, z, dtype, s);
    case kCap: return launch_paged<kCap>(p, z, dtype, s);
    default: return launch_paged<kBias | kCap>(p, z, dtype, s);
  }
}

}  // extern "C"

#endif
