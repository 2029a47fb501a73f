// attn_packed.h -- the plan of a packed batch, as attn_plan.hip writes it and the attention
// passes read it.
#pragma once

#include "attn_common.h"

namespace attn {

// Packed query rows row0 .. row0 + 127 (row = token * G + head of the group) of the sequence
// at rows start .. start + n - 1; or, with gap set, n rows of no sequence from start on.
struct RowItem {
  int32_t start, n, row0, gap;
};

// Keys key0 .. key0 + 127 of the sequence, against its blocks block0 .. block_end - 1 of 32
// packed rows. slot: of the partial sums where a tile's rows are split, else < 0.
struct KeyItem {
  int32_t start, n, key0, gap, block0, block_end, slot, unused;
};

// A tile whose rows are split: slots slot .. slot + splits - 1.
struct KeyJoin {
  int32_t start, n, key0, slot, splits, unused[3];
};
static_assert(sizeof(RowItem) == 16 && sizeof(KeyItem) == 32 && sizeof(KeyJoin) == 32, "words");

constexpr int32_t kRowBlock = 32;      // packed rows of a step of the dK/dV pass
constexpr int32_t kMinRowBlocks = 16;  // of a split
constexpr int32_t kKeyTarget = 512;    // workgroups that its work is split into, about

struct PackedSizes {
  int64_t rows, keys, joins, units;
};
// Every split holds more than half of the work that kKeyTarget stands for, so that there are
// fewer than 2 kKeyTarget / Hkv of them, in at most kKeyTarget / Hkv tiles.
inline PackedSizes packed_sizes(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  const int64_t splits = kKeyTarget / Hkv + 1;
  return {row_items(T, num_seqs, Hq / Hkv), key_items(T, num_seqs) + splits, splits, 2 * splits};
}

inline bool valid_batch(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  return T >= 0 && T <= INT32_MAX && num_seqs >= 0 && num_seqs <= (1 << 24) &&
         valid_heads(Hq, Hkv) && T * (Hq / Hkv) <= INT32_MAX - kRowTile;
}

}  // namespace attn
