// attn_packed.h -- the plan of a packed batch, as attn_plan.hip writes it and the attention
// passes read it.
#pragma once

#include "attn_common.h"

namespace attn {

// Packed query rows row0 .. row0 + 127 (row = token * G + head of the group) of the sequence
// at rows start .. start + n - 1, all of which see its first `prefix` keys; or, with kGap in its
// place, n rows of no sequence from start on.
constexpr int32_t kGap = -1;
struct RowItem {
  int32_t start, n, row0, prefix;
};

// Keys key0 .. key0 + 127 of the sequence, against all of its blocks of 32 packed rows that
// see one; or, with gap set, n rows of no sequence. first: the work of the tiles before it.
// A tile's work is kTileUnits and one unit a block (1 in all where gap is set).
struct KeyTile {
  int32_t start, n, key0, gap;
  int64_t first;
  int32_t prefix, unused;
};
static_assert(sizeof(RowItem) == 16 && sizeof(KeyTile) == 32, "words");

constexpr int32_t kRowBlock = 32;   // packed rows of a step of the dK/dV pass
constexpr int32_t kTileUnits = 8;   // what a tile costs beside its blocks, in blocks
// Of a workgroup's share, at least. Not swept: where most samples are short a tile is about as much
// work, and most tiles are cut (61 samples of 1 to 301 tokens, 6 + 2 heads: 118 of 138).
constexpr int32_t kMinUnits = 12;

// The first row that sees a key of a sequence whose first `prefix` keys all rows see.
__host__ __device__ inline int32_t first_row_of_key(int32_t key, int32_t prefix, int32_t G) {
  return key < prefix ? 0 : key * G;
}
// Row blocks that see a key of the tile at key0 of a sequence of n tokens.
__host__ __device__ inline int32_t blocks_of_tile(int32_t n, int32_t key0, int32_t prefix, int32_t G) {
  return n * G / kRowBlock + (n * G % kRowBlock != 0) - first_row_of_key(key0, prefix, G) / kRowBlock;
}

struct PackedSizes {
  int64_t rows, keys;
};
inline PackedSizes packed_sizes(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  return {row_items(T, num_seqs, Hq / Hkv), key_items(T, num_seqs)};
}

inline bool valid_batch(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv) {
  return T >= 0 && T <= INT32_MAX && num_seqs >= 0 && num_seqs <= (1 << 24) &&
         valid_heads(Hq, Hkv) && T * (Hq / Hkv) <= INT32_MAX - kRowTile;
}

}  // namespace attn
