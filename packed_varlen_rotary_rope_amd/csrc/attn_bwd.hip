// attn_bwd.hip -- gradients of packed causal attention (attn_bwd of include/attn.h), in two
// kernels without atomics, so that results do not depend on the order of execution:
//
//  * attn_bwd_rows_kernel (dQ): a tile of 128 packed query rows walks the keys it sees, as
//    the forward does; per block S^T = K Q^T, dP^T = V dO^T, P = exp(S - lse),
//    dS = P (dP - D), dQ^T += K^T dS^T. It forms D_i = dout_i . out_i from its rows first,
//    and leaves lse * log2 e and D for the second kernel.
//  * attn_bwd_keys_kernel (dK, dV): 128 keys, 32 a wave, walk the packed rows that see
//    them, which covers every head of the group, so shared heads need no further sum; per
//    block of 32 rows S = Q K^T, dP = dO V^T, dV^T += dO^T P, dK^T += Q^T dS.
//
// In both, a wave's own rows (keys) are columns of every product: their operands stay in
// registers, P and dS come out of the matrix units as B operands of the next product, and
// the other side is shared through LDS, read along rows and, by transposing reads, along
// columns. S and dP are formed twice, 14 flops per pair and element of D instead of 10;
// the price of having no fp32 sums of dQ in memory.
//
// What bounds them: of the cycles the matrix unit is busy for 39 % (dQ) and 37 % (dK, dV), the
// vector unit for as many; the rest is waiting, for LDS and at the barrier of each block, with
// one or two waves on a SIMD to hide it (the accumulators leave no room for more). Measured,
// bf16: eight samples of 256 to 2048 tokens, 32 + 8 heads of 128: dQ 220 us, dK and dV 318, their
// join 20, which is 0.79 and 0.73 PFLOP/s of the 6 and 8 flops that each of them does; 8192 tokens
// of 16 + 2 heads of 64: 240, 340 and 20 us, 0.86 and 0.81 PFLOP/s. Rounding: P and dS go to
// the storage type before their second product, as the matrix unit takes it; a dS past 65504
// overflows in f16, as a stored dP would.
#include "attn_packed.h"
#include "attn_tile.h"

#ifndef ATTN_MODS  // what scores go through (attn_scores.h): this file is compiled once for each
#define ATTN_MODS 0
#endif

namespace attn {

struct BwdParams {
  const void* dout;
  const void* q;
  const void* k;
  const void* v;
  const void* out;
  const float* lse;
  float* lse2;   // scratch: lse * log2 e and
  float* delta;  // D_i, by key/value head and packed row: [Hkv][T * G]
  float* slope;  // kBias, the same way: slope * log2 e and
  int32_t* at;   // the token's position
  void* dq;
  void* dk;
  void* dv;
  const int32_t* plan;
  const RowItem* row_items;
  const KeyTile* key_tiles;
  float* part;  // scratch: [2 shares][dK, dV][128][D], of tiles that are cut
  int64_t dout_stride, q_stride, k_stride, v_stride, out_stride, dq_stride, dk_stride, dv_stride;
  int32_t T, Hq, Hkv, G, D, num_seqs;
  float scale, scale2;  // scale2: of what exp2 sees, times log2 e
  int32_t fill;
  Div31 by_hkv, by_g;
  ScoreParams scores;
};

template <int MODS>
int32_t launch_bwd(const BwdParams& p, const PackedSizes& z, int32_t dtype, hipStream_t s);

namespace {

// Tiles of up to so many keys form D_i = sum_j P_ij dP_ij, the others take the rounded output's
// dout_i . out_i, whose error matters where a row's weight lies on few keys: there dP_ij - D_i is small
// beside either. Capped and biased scores are such rows at any length: gradients of eight samples of 256 to
// 2048 tokens, scores of size 4 under a cap of 50, are off by 0.0024 of their norm with it, of which the
// rounding of dS and of the result is all, and by 0.0032 without (bf16, 32 + 8 heads of 128). It is paid for by a
// walk of two products, a tanh and an exponential a score, about a third of the pass.
constexpr int32_t kExactKeys = ATTN_MODS ? INT32_MAX : 256;
// dQ of changed scores takes dS in two parts, rounded and what the rounding left, up to 64 columns, where the
// vector unit is what is waited for and a product more costs 1 to 3 % of the pass (28 samples of 799 tokens,
// 32 + 8 heads of 64, cap and bias, 419 to 429 us with it): dQ is then off by the rounding of the result alone. At
// 128 columns it would be 10 % (eight samples of 256 to 2048 tokens, cap, 378 to 397 us without it).
constexpr bool two_parts(int db) { return ATTN_MODS != 0 && db <= 2; }
constexpr bool kHasCap = ATTN_MODS & kCap, kHasBias = ATTN_MODS & kBias;
// Where a batch is too small to give every workgroup of the dK/dV pass so many units, cuts that would leave
// a tile a block or none before or behind them are moved to its end: a piece without blocks costs its latency and a
// join. Measured, all kernels of a step: 24 samples of 40 to 49 tokens, 5 heads of 72, 51 us with shares of
// 12 units and every cut as it falls, 47 with such cuts moved, 39 with 9 units; 61 samples of 1 to 301
// tokens, 6 + 2 heads of 80, 70, 67, 66; moving cuts that leave 12 blocks or fewer 47 and 73, shares of 24 units
// 55 and 74. (The plain form's sums keep the order that they have always had.)
constexpr int32_t kLeastUnits = ATTN_MODS ? 9 : kMinUnits, kNearUnits = ATTN_MODS ? 1 : 0;

// Zeros to `n` rows of `heads` heads from head0.
template <typename T>
__device__ inline void clear_rows(T* x, int32_t start, int32_t n, int64_t stride, uint32_t head0,
                                  uint32_t heads, uint32_t chunks) {
  const uint32_t per_token = heads * chunks;
  for (uint32_t i = threadIdx.x; i < n * per_token; i += 256) {
    const uint32_t t = i / per_token, c = i - t * per_token;
    *reinterpret_cast<u32x4*>(x + (int64_t)(start + t) * stride + 8 * (head0 * chunks + c)) =
        (u32x4){0, 0, 0, 0};
  }
}

template <typename T, int DB, int MODS>
__global__ __launch_bounds__(256, 2) void attn_bwd_rows_kernel(const BwdParams p) {
  constexpr int CPR = chunks_per_row(DB), KS = 2 * DB, BN = DB <= 2 ? 64 : 32;
  constexpr int kTileBytes = BN * CPR * 16, kLoads = BN * CPR / 256;
  // Up to 64 columns three workgroups share a CU (3 x 48 KB of LDS), above that two (80 KB).
  constexpr int kStages = DB <= 2 ? 3 : 5;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kStages * 2 * kTileBytes];

  uint32_t kvh;
  const uint32_t index = div31(blockIdx.x, p.by_hkv);
  kvh = blockIdx.x - index * p.Hkv;
  if (!plan_matches(p, kPackedPlan) || (int32_t)index >= p.plan[0]) return;
  const RowItem item = p.row_items[index];
  const int32_t start = item.start, n = item.n;
  if (start < 0 || n <= 0 || start > p.T - n) return;
  const uint32_t tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = p.D >> 3;
  if (item.prefix == kGap) {
    if (p.fill) clear_rows(static_cast<T*>(p.dq), start, n, p.dq_stride, kvh * p.G, p.G, chunks);
    return;
  }

  const int32_t rows = n * p.G;
  const int32_t row0 = item.row0;
  if (row0 < 0 || row0 >= rows) return;
  const int32_t row_end = min(row0 + kRowTile, rows);
  const int32_t wave_row0 = row0 + 32 * wave;
  const int32_t row = wave_row0 + (lane & 31);
  const bool on = row < row_end;
  const int32_t clamped = on ? row : row_end - 1;
  const int32_t token = div31(clamped, p.by_g);
  const int32_t head = kvh * p.G + (clamped - token * p.G);
  const int32_t prefix = min(item.prefix, n);
  auto seen_by = [&](int32_t packed) __attribute__((always_inline)) {  // keys that a row sees
    return max((int32_t)div31(packed, p.by_g) + 1, prefix);
  };
  const int32_t seen = max(token + 1, prefix);
  const int32_t wave_end = wave_row0 < row_end ? seen_by(min(wave_row0 + 32, row_end) - 1) : 0;
  const int32_t wave_all = seen_by(min(wave_row0, row_end - 1));
  const int32_t key_end = seen_by(row_end - 1);

  const int64_t at_row = (int64_t)(start + token);
  x8<T> qf[KS], df[KS];
  load_row<T>(qf, static_cast<const T*>(p.q) + at_row * p.q_stride + (int64_t)head * p.D, half, chunks);
  load_row<T>(df, static_cast<const T*>(p.dout) + at_row * p.dout_stride + (int64_t)head * p.D, half,
              chunks);
  float delta = 0.0f;
  if constexpr (kExactKeys != INT32_MAX) {
    x8<T> of[KS];
    load_row<T>(of, static_cast<const T*>(p.out) + at_row * p.out_stride + (int64_t)head * p.D, half,
                chunks);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = __builtin_fmaf((float)df[s][e], (float)of[s][e], delta);
    delta = half_sum(delta);
  }
  const int64_t at_stat = at_row * p.Hq + head;
  float lse2 = p.lse[at_stat] * (float)kLog2e;
  if (lse2 == -__builtin_inff()) lse2 = 0.0f;  // every score is -inf: all weights are 0
  float slope = 0.0f;
  if constexpr (kHasBias) slope = p.scores.slopes[head] * (float)kLog2e;

  f32x16 dq[DB];
  clear_unused_chunks<CPR>(lds, kStages * 2 * BN, chunks);

  const T* k = static_cast<const T*>(p.k) + (int64_t)start * p.k_stride + (int64_t)kvh * p.D;
  const T* v = static_cast<const T*>(p.v) + (int64_t)start * p.v_stride + (int64_t)kvh * p.D;
  const int32_t blocks = (key_end + BN - 1) / BN;
  uint64_t lanes[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) lanes[i] = __ballot(chunk_of<CPR, 256>(i, tid) < chunks);
  constexpr int kPieces = 2 * kLoads, kPerStep = (kPieces + KS - 1) / KS;
  auto piece = [&](int32_t b, int x) __attribute__((always_inline)) {  // x-th copy of block b
    const int i = x / 2;
    const int64_t stride = x % 2 ? p.v_stride : p.k_stride;
    const int32_t key0 = min(b, blocks - 1) * BN;  // behind the last block, into buffers not used
    const uint32_t at = min((int32_t)row_of<CPR, 256>(i, tid), key_end - 1 - key0);
    const T* from = (x % 2 ? v : k) + (int64_t)key0 * stride;
    copy_chunk_to_lds(from + (at * (uint32_t)stride + 8 * chunk_of<CPR, 256>(i, tid)),
                      lds_address(lds) + (b % kStages * 2 + x % 2) * kTileBytes + (i * 256 + wave * 64) * 16,
                      lanes[i]);
  };

  int32_t b = 0;
  // P and dP of 32 keys of block b; the first of them begin the copies of the block
  // kStages - 1 further between their steps. What is hidden gets P = dP = 0.
  auto next = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int x = s * kPerStep; x < (s + 1) * kPerStep && x < kPieces; ++x) piece(b + kStages - 1, x);
  };
  f32x16 bent;  // kCap: tanh of the scores at hand
  auto weights = [&](auto mode, const uint8_t* kt, int32_t key0, int c, f32x16& s, f32x16& dp)
                     __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      if (c == 0) next(t);
      s = mfma(read_rows<T, CPR>(kt, 32 * c + (lane & 31), 2 * t + half), qf[t], s);
      dp = mfma(read_rows<T, CPR>(kt + kTileBytes, 32 * c + (lane & 31), 2 * t + half), df[t], dp);
    }
    if constexpr (kHasCap) {
      bend_scores(s, p.scores.bend);
      bent = s;
    }
    const float d0 = distance(key0 + 32 * c + 4 * (int32_t)half, token);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (kHasBias) {
        const float d = d0 + (float)(8 * (i / 4) + i % 4);
        s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale2, -(slope * __builtin_fabsf(d))) - lse2);
      } else {
        s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale2, -lse2));
      }
      if constexpr (decltype(mode)::value != kWhole) {
        const int32_t key = key0 + 32 * c + 8 * (i / 4) + 4 * (int32_t)half + i % 4;
        if (key >= seen) s[i] = dp[i] = 0.0f;
      }
    }
  };
  // anew: in the second walk
  auto block = [&](auto mode, auto anew, const uint8_t* kt, int32_t key0) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < BN / 32; ++c) {
      f32x16 s, dp;
      weights(mode, kt, key0, c, s, dp);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = s[i] * (dp[i] - delta);
        if constexpr (kHasCap) s[i] *= __builtin_fmaf(-bent[i], bent[i], 1.0f);
        if constexpr (decltype(mode)::value != kWhole) {  // also where D_i is not finite
          const int32_t key = key0 + 32 * c + 8 * (i / 4) + 4 * (int32_t)half + i % 4;
          if (key >= seen) s[i] = 0.0f;
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const x8<T> ds = narrow8<T>(s, t);
        x8<T> low;  // what its rounding left; nothing of a dS that it has made infinite
        if constexpr (two_parts(DB)) {
          low = rest8<T>(s, ds, t);
          if constexpr (decltype(anew)::value) low = cleaned<T>(low);
        }
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          x8<T> kc = read_columns<T, CPR>(kt, 32 * c + 16 * t, d, lane);
          // a key that is seen and not finite has made dS NaN or 0 already
          if constexpr (decltype(mode)::value == kCareful) kc = cleaned<T>(kc);
          dq[d] = mfma(kc, ds, dq[d]);
          if constexpr (two_parts(DB)) dq[d] = mfma(kc, low, dq[d]);
        }
      }
    }
  };
  auto first_stages = [&]() __attribute__((always_inline)) {
    for (int32_t i = 0; i < kStages - 1; ++i)
#pragma unroll
      for (int x = 0; x < kPieces; ++x) piece(i, x);
  };
  auto arrive = [&]() __attribute__((always_inline)) {  // block b; the buffer before it is free
    wait_copies_and_sync<(kStages - 2) * kPieces>();
    return lds + b % kStages * 2 * kTileBytes;
  };
  auto skip = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < KS; ++s) next(s);
  };
  first_stages();
  settle<T>(qf);
  settle<T>(df);
  // D_i from the rounded output errs by half a step of it, which is most where a row sees few
  // keys, and as much there as the rounding of dS. Such tiles form sum_j P_ij dP_ij first.
  if (key_end <= kExactKeys) {
    float sum = 0.0f;
    if constexpr (kExactKeys == INT32_MAX) {  // a walk worth its own loop for the blocks seen whole
      const int32_t all = wave_end > 0 ? wave_all / BN : 0;
      for (; b < all; ++b) {
        const uint8_t* kt = arrive();
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) {
          f32x16 s, dp;
          weights(Constant<kWhole>(), kt, b * BN, c, s, dp);
#pragma unroll
          for (int i = 0; i < 16; ++i) sum = __builtin_fmaf(s[i], dp[i], sum);
        }
      }
    }
    for (; b < blocks; ++b) {
      const uint8_t* kt = arrive();
      if (b * BN >= wave_end) {
        skip();
        continue;
      }
#pragma unroll
      for (int c = 0; c < BN / 32; ++c) {
        f32x16 s, dp;
        weights(Constant<kMasked>(), kt, b * BN, c, s, dp);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = __builtin_fmaf(s[i], dp[i], sum);
      }
    }
    delta = half_sum(sum);
    wait_copies_and_sync<0>();  // the last block has been read, and what came behind it is there
    b = 0;
    first_stages();
  }
  if (on && half == 0) {
    const int64_t at = ((int64_t)kvh * p.T + start) * p.G + row;
    p.lse2[at] = lse2;
    p.delta[at] = delta;
    if constexpr (kHasBias) {
      p.slope[at] = slope;
      p.at[at] = token;
    }
  }
  // two loops, and a second walk where it is needed, as in the forward
  const int32_t all = wave_end > 0 ? wave_all / BN : 0;
  auto walk = [&](auto mode) __attribute__((always_inline)) {
    constexpr Constant<decltype(mode)::value == kCareful> anew{};
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) dq[d][i] = 0.0f;
    for (; b < all; ++b) {
      const uint8_t* kt = arrive();
      block(Constant<kWhole>(), anew, kt, b * BN);
    }
    for (; b < blocks; ++b) {
      const uint8_t* kt = arrive();
      if (b * BN < wave_end) block(mode, anew, kt, b * BN);
      else skip();
    }
    wait_copies<0>();
  };
  walk(Constant<kMasked>());
  if (any_wave(any_nonfinite(dq), lds)) {
    b = 0;
    first_stages();
    walk(Constant<kCareful>());
  }
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) dq[d][i] *= p.scale;
  store_row<T, DB>(dq, static_cast<T*>(p.dq) + at_row * p.dq_stride + (int64_t)head * p.D, half,
                   chunks, on);
}

// ---- dK and dV -------------------------------------------------------------------------------
//
// The work of all tiles and key/value heads, laid end to end head by head, is cut into equal
// shares, one for each workgroup that fits the chip, wherever the cuts fall: with the tiles of
// one long sequence of few key/value heads as they are, most of the chip would wait for the
// first of them. A workgroup walks its share tile by tile; a tile that is cut leaves partial
// sums, which attn_bwd_join_kernel adds in the order of its rows.

// A place in that work: tile `index` of head `kvh`, `in_tile` units from its start.
struct Place {
  int64_t units;  // of all tiles of a head
  int64_t share;  // of a workgroup
  int64_t total;
  int32_t tiles;
  int32_t near;   // cuts so near to a tile's ends are moved there
};
// Where a cut at `pos` of a tile of `units` comes to lie.
__device__ inline int64_t place_of_cut(const Place& w, int64_t pos, int64_t units) {
  if (w.near == 0) return pos;
  return pos <= kTileUnits + w.near ? 0 : units - pos <= w.near ? units : pos;
}
__device__ inline Place place_of(const BwdParams& p, int32_t shares) {
  Place w;
  w.units = *reinterpret_cast<const int64_t*>(p.plan + 6);
  w.tiles = p.plan[1];
  w.total = w.units * p.Hkv;
  w.share = (w.total + shares - 1) / shares;
  w.near = 0;
  if (w.share < kLeastUnits) {
    w.share = kLeastUnits;
    w.near = kNearUnits;
  }
  return w;
}
// The last tile whose work begins at or before `pos` (0 <= pos < units), by 64 probes a step.
__device__ inline int32_t find_tile(const BwdParams& p, int32_t tiles, int64_t pos) {
  const int32_t lane = threadIdx.x & 63;
  int32_t lo = 0, n = tiles;  // the answer is in lo .. lo + n - 1
  while (n > 1) {
    const int32_t step = (n + 63) / 64, at = lane * step;
    const uint64_t yes = __ballot(at < n && p.key_tiles[lo + at].first <= pos);
    const int32_t last = 63 - __builtin_clzll(yes | 1);
    lo += last * step;
    n = min(step, n - last * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}
__device__ inline int64_t end_of_tile(const BwdParams& p, const Place& w, int32_t tile) {
  return tile + 1 < w.tiles ? p.key_tiles[tile + 1].first : w.units;
}

// lse and D, slope and position of a row that is none: no weight.
__device__ const float kNoRow[4] = {__builtin_inff(), 0.0f, 0.0f, 0.0f};

template <typename T, int DB, int MODS>
__global__ __launch_bounds__(256, DB <= 2 ? 2 : 1) void attn_bwd_keys_kernel(const BwdParams p) {
  constexpr int CPR = chunks_per_row(DB), KS = 2 * DB, BM = kRowBlock;
  constexpr int kTileBytes = BM * CPR * 16, kLoads = BM * CPR / 256;
  constexpr bool kPipelined = DB > 2;
  constexpr int kStatBytes = (kHasBias ? 4 : 2) * BM * 4, kStage = 2 * kTileBytes + kStatBytes, kStages = 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kStages * kStage];
  __shared__ __attribute__((aligned(16))) uint8_t flags[16];

  if (!plan_matches(p, kPackedPlan)) return;
  const Place work = place_of(p, gridDim.x);
  // workgroup i runs on die i % 8: neighbouring shares, which read the same rows, on one die
  const int32_t share = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  int64_t left = min(work.share, work.total - share * work.share);
  if (left <= 0 || work.tiles <= 0) return;
  uint32_t kvh = (uint32_t)(share * work.share / work.units);
  int64_t pos = share * work.share - kvh * work.units;
  int32_t index = find_tile(p, work.tiles, pos);
  if (work.near != 0) {  // the share begins where its cut comes to lie
    const int64_t begin = p.key_tiles[index].first, units = end_of_tile(p, work, index) - begin;
    const int64_t cut = begin + place_of_cut(work, pos - begin, units);
    left += pos - cut;
    pos = cut;
    if (cut == begin + units) ++index;
  }

  const uint32_t tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = p.D >> 3;
  for (int b = 0; b < kStages; ++b) clear_unused_chunks<CPR>(lds + b * kStage, 2 * BM, chunks);
  uint64_t lanes[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) lanes[i] = __ballot(chunk_of<CPR, 256>(i, tid) < chunks);
  // a row block further is dt tokens and dh heads on, one token more where the heads wrap
  const uint32_t dt = div31(BM, p.by_g), dh = BM - dt * p.G;
  const int64_t q_step = dt * p.q_stride + (int64_t)dh * p.D, q_wrap = p.q_stride - (int64_t)p.G * p.D;
  const int64_t g_step = dt * p.dout_stride + (int64_t)dh * p.D, g_wrap = p.dout_stride - (int64_t)p.G * p.D;

  for (; left > 0; ++index) {
    if (pos >= work.units) {
      pos = 0;
      index = 0;
      ++kvh;
    }
    const KeyTile tile = p.key_tiles[index];
    const int64_t tile_end = end_of_tile(p, work, index);
    const int64_t from = pos - tile.first;
    int64_t to = min(tile_end - tile.first, from + left);
    if (work.near != 0 && from + left < tile_end - tile.first && share * work.share + work.share < work.total) {
      to = place_of_cut(work, from + left, tile_end - tile.first);  // and so it ends
      left = to - from;
    }
    if (to <= from) return;  // also: no plan of this batch's
    const bool whole = from == 0 && to == tile_end - tile.first;
    left -= to - from;
    pos += to - from;

    const int32_t start = tile.start, n = tile.n, key0 = tile.key0;
    if (start < 0 || n <= 0 || start > p.T - n) continue;
    T* dk_out = static_cast<T*>(p.dk);
    T* dv_out = static_cast<T*>(p.dv);
    if (tile.gap != 0) {
      if (p.fill) {
        clear_rows(dk_out, start, n, p.dk_stride, kvh, 1, chunks);
        clear_rows(dv_out, start, n, p.dv_stride, kvh, 1, chunks);
      }
      continue;
    }
    if (key0 < 0 || key0 >= n) continue;

    const int32_t rows = n * p.G;
    const int32_t wave_key0 = key0 + 32 * wave;
    const int32_t key = wave_key0 + (lane & 31);
    const bool on = key < n;
    const int32_t at_key = on ? key : n - 1;
    const int32_t prefix = tile.prefix;
    const int32_t first = first_row_of_key(at_key, prefix, p.G);  // that sees this lane's key
    // and the wave's every key
    const int32_t wave_all = wave_key0 < n ? first_row_of_key(min(wave_key0 + 31, n - 1), prefix, p.G) : rows;

    x8<T> kf[KS], vf[KS];
    load_row<T>(kf, static_cast<const T*>(p.k) + (int64_t)(start + at_key) * p.k_stride +
                        (int64_t)kvh * p.D, half, chunks);
    load_row<T>(vf, static_cast<const T*>(p.v) + (int64_t)(start + at_key) * p.v_stride +
                        (int64_t)kvh * p.D, half, chunks);
    f32x16 dk[DB], dv[DB];

    // this piece's row blocks: the tile's first kTileUnits are what it costs beside them
    const int32_t block0 = (int32_t)max(from - kTileUnits, (int64_t)0);
    const int32_t blocks = min((int32_t)max(to - kTileUnits, (int64_t)0), blocks_of_tile(n, key0, prefix, p.G)) - block0;
    const int32_t row_begin = first_row_of_key(key0, prefix, p.G) / BM * BM + block0 * BM;
    auto first_row = [&](int32_t i) __attribute__((always_inline)) { return row_begin + i * BM; };

    const T* q = static_cast<const T*>(p.q) + (int64_t)start * p.q_stride + (int64_t)kvh * p.G * p.D;
    const T* g = static_cast<const T*>(p.dout) + (int64_t)start * p.dout_stride +
                 (int64_t)kvh * p.G * p.D;
    const float* stats = (half ? p.delta : p.lse2) + ((int64_t)kvh * p.T + start) * p.G;
    const float* more_stats = stats;
    if constexpr (kHasBias)
      more_stats = (half ? reinterpret_cast<const float*>(p.at) : p.slope) + ((int64_t)kvh * p.T + start) * p.G;
    // the next block's rows of this thread: head of the group, and offsets
    uint32_t heads[kLoads];
    int64_t q_at[kLoads], g_at[kLoads];
    auto seek = [&](int32_t row0) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t at = min(row0 + (int32_t)row_of<CPR, 256>(i, tid), rows - 1);
        const uint32_t t = div31(at, p.by_g);
        heads[i] = at - t * p.G;
        q_at[i] = t * p.q_stride + (heads[i] * p.D + 8 * chunk_of<CPR, 256>(i, tid));
        g_at[i] = t * p.dout_stride + (heads[i] * p.D + 8 * chunk_of<CPR, 256>(i, tid));
      }
    };
    auto advance = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        bool wrap = false;
        if (dh != 0) {
          heads[i] += dh;
          wrap = heads[i] >= (uint32_t)p.G;
          if (wrap) heads[i] -= p.G;
        }
        q_at[i] += q_step + (wrap ? q_wrap : 0);
        g_at[i] += g_step + (wrap ? g_wrap : 0);
      }
    };
    // The x-th copy of block b; blocks are begun in order, each after a call of go_to. The first
    // is of lse and D of the rows, 32 words each, by the first wave (and with a bias of slope and
    // position by the second): it waits for one copy more than it would have to, the other waves for
    // what they need.
    constexpr int kPieces = 2 * kLoads, kPerStep = (kPieces + KS - 1) / KS;
    auto go_to = [&](int32_t b) __attribute__((always_inline)) {
      if (b == 0 || first_row(b) + BM > rows) seek(first_row(b));  // also where the rows end
      else advance();
    };
    auto piece = [&](int32_t b, int x) __attribute__((always_inline)) {
      const uint32_t qd = lds_address(lds) + b % kStages * kStage, gd = qd + kTileBytes;
      const int i = x / 2;
      const uint32_t dst = (i * 256 + wave * 64) * 16;
      if (x == 0 && wave == 0) {
        const int32_t row = first_row(b) + (int32_t)(lane & 31);
        copy_word_to_lds(row < rows ? stats + row : kNoRow + half, gd + kTileBytes);
      }
      if (kHasBias && x == 0 && wave == 1) {
        const int32_t row = first_row(b) + (int32_t)(lane & 31);
        copy_word_to_lds(row < rows ? more_stats + row : kNoRow + 2 + half, gd + kTileBytes + 2 * BM * 4);
      }
      if (x % 2 == 0) copy_chunk_to_lds(q + q_at[i], qd + dst, lanes[i]);
      else copy_chunk_to_lds(g + g_at[i], gd + dst, lanes[i]);
    };

    // Above 64 columns the accumulators leave room for one wave on a SIMD, and the loop is
    // pipelined over two blocks so that every product has vector work beside it: while the matrix
    // unit forms S and dP of the next block, the vector unit turns the middle half of this one's
    // into P and dS, an operation or two per product; then dV and dK follow, beside the last
    // quarter of this block and the first one of the next. Before their last step the block after
    // the next is waited for. (With all of P and dS beside the first half of the products the
    // pass of a packed batch took 339 us, and 318 so.) Up to 64 columns two waves share a SIMD, and a
    // block is finished before the next is begun.
    f32x16 s, dp;             // of the block at hand, then of the next one (kCap: tanh of the scores)
    f32x4 lse2[4], delta[4];  // of rows 8 j + 4 half .. + 3
    f32x4 slope[4];           // kBias, and
    i32x4 places[4];          // the position that this lane's key has to them
    float wx[2], dx[2];
    uint32_t w[8], ds[8];  // P and dS of row pairs, narrowed
    x8<T> qr[KS], gr[KS];  // rows of the next block, the first two steps' from the round before
    auto buffer = [&](int32_t b) __attribute__((always_inline)) { return lds + b % kStages * kStage; };
    auto read_stats = [&](const uint8_t* qt, int j) __attribute__((always_inline)) {
      const float* stat = reinterpret_cast<const float*>(qt + 2 * kTileBytes);
      lse2[j] = *reinterpret_cast<const f32x4*>(stat + 8 * j + 4 * half);
      delta[j] = *reinterpret_cast<const f32x4*>(stat + 32 + 8 * j + 4 * half);
      if constexpr (kHasBias) {
        slope[j] = *reinterpret_cast<const f32x4*>(stat + 64 + 8 * j + 4 * half);
        places[j] = *reinterpret_cast<const i32x4*>(stat + 96 + 8 * j + 4 * half);
      }
    };
    // The u-th of 32 operations from S and dP to P (even) and dS (odd), in order.
    auto weigh = [&](auto mode, int u, const f32x16& sv, const f32x16& dpv, int32_t row0)
                     __attribute__((always_inline)) {
      constexpr int MODE = decltype(mode)::value;
      const int i = u / 2, j = i / 4, e = i % 4, c = i % 2;
      const int32_t at = row0 + 8 * j + 4 * (int32_t)half + e;
      const bool gone = MODE != kWhole && (at < first || (MODE == kCareful && at >= rows));
      if (u % 2 == 0) {
        if constexpr (kHasBias) {
          const float bias = -(slope[j][e] * __builtin_fabsf(distance(at_key, places[j][e])));
          wx[c] = __builtin_amdgcn_exp2f(__builtin_fmaf(sv[i], p.scale2, bias) - lse2[j][e]);
        } else {
          wx[c] = __builtin_amdgcn_exp2f(__builtin_fmaf(sv[i], p.scale2, -lse2[j][e]));
        }
        if (gone) wx[c] = 0.0f;
      } else {
        dx[c] = wx[c] * (dpv[i] - delta[j][e]);
        if constexpr (kHasCap) dx[c] *= __builtin_fmaf(-sv[i], sv[i], 1.0f);
        if (gone) dx[c] = 0.0f;
        if (c == 1) {
          w[i / 2] = narrow2<T>(wx[0], wx[1]);
          ds[i / 2] = narrow2<T>(dx[0], dx[1]);
        }
      }
    };
    auto read_row = [&](const uint8_t* qt, int t) __attribute__((always_inline)) {
      qr[t] = read_rows<T, CPR>(qt, lane & 31, 2 * t + half);
      gr[t] = read_rows<T, CPR>(qt + kTileBytes, lane & 31, 2 * t + half);
    };
    // S and dP of the block at `qt`, whose first two steps' rows have been read; `first(t)` and
    // `second(t)` are called in step t of KS, one before each of its two products.
    auto scores = [&](const uint8_t* qt, f32x16& s_out, f32x16& dp_out, auto first_half, auto second_half)
                      __attribute__((always_inline)) {
      f32x16 a, c;
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i] = c[i] = 0.0f;
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        step();
        if (t + 2 < KS) read_row(qt, t + 2);
        a = mfma(qr[t], kf[t], a);
        first_half(t);
        step();
        c = mfma(gr[t], vf[t], c);
        second_half(t);
      }
      step();
      if constexpr (kHasCap) bend_scores(a, p.scores.bend);
      s_out = a;
      dp_out = c;
    };
    auto round = [&](auto mode, int32_t b) __attribute__((always_inline)) {
      constexpr int MODE = decltype(mode)::value;
      const uint8_t* qt = buffer(b);
      const uint8_t* gt = qt + kTileBytes;
      const int32_t row0 = first_row(b);
      go_to(b + kStages - 1);
      if constexpr (!kPipelined) {
        wait_copies_and_sync<(kStages - 2) * kPieces>();  // block b; the buffer before it is free
#pragma unroll
        for (int j = 0; j < (kHasBias ? 1 : 4); ++j) read_stats(qt, j);
        read_row(qt, 0);
        read_row(qt, 1);
      }
      x8<T> gc[2 * DB], qc[2 * DB];  // by step: 16 rows x / DB, columns x % DB
      auto read = [&](int x) __attribute__((always_inline)) {
        gc[x] = read_columns<T, CPR>(gt, 16 * (x / DB), x % DB, lane);
        qc[x] = read_columns<T, CPR>(qt, 16 * (x / DB), x % DB, lane);
      };
      auto begin_copies = [&](int t) __attribute__((always_inline)) {
#pragma unroll
        for (int x = t * kPerStep; x < (t + 1) * kPerStep && x < kPieces; ++x) piece(b + kStages - 1, x);
      };
      f32x16 s_next, dp_next;
      // operations 8 .. 23 beside the 2 KS products of the first half
      auto middle = [&](int x) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 8 + 16 * x / (2 * KS); u < 8 + 16 * (x + 1) / (2 * KS); ++u) weigh(mode, u, s, dp, row0);
      };
      // of 4 DB in the second half: operations 24 .. 31, and 0 .. 7 of the next block
      auto rest = [&](int x) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 16 * x / (4 * DB); u < 16 * (x + 1) / (4 * DB); ++u) {
          if (u < 8) weigh(mode, 24 + u, s, dp, row0);
          else weigh(mode, u - 8, s_next, dp_next, first_row(b + 1));
        }
      };
      if constexpr (kPipelined) {
        scores(buffer(b + 1), s_next, dp_next,
               [&](int t) __attribute__((always_inline)) {
                 if (t == 0) read_stats(qt, 2);
                 if (t == KS / 2) read_stats(qt, 3);
                 middle(2 * t);
                 begin_copies(t);
               },
               [&](int t) __attribute__((always_inline)) {
                 middle(2 * t + 1);
                 if (t == KS - 1) {
                   read(0);
                   read(1);
                   read_stats(buffer(b + 1), 0);
                 }
               });
      } else {
        scores(qt, s, dp, begin_copies, [](int) {});
        read(0);
        read(1);
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          if (kHasBias && u % 8 == 0) {  // the four kinds of a row's would not all find registers
            step();
            if (u < 24) read_stats(qt, u / 8 + 1);
          }
          weigh(mode, u, s, dp, row0);
        }
      }
      x8<T> wb, db;
#pragma unroll
      for (int x = 0; x < 2 * DB; ++x) {
        step();
        if (x + 2 < 2 * DB) read(x + 2);
        if (kPipelined && x == 2 * DB - 1) {
          // all of block b has been read: block b + 2 has arrived, and b's buffer is free
          wait_copies_and_sync<kPieces>();
          read_row(buffer(b + 2), 0);
          read_row(buffer(b + 2), 1);
          read_stats(buffer(b + 1), 1);
        }
        if (x % DB == 0) {
          const int y = 4 * (x / DB);
          wb = __builtin_bit_cast(x8<T>, (u32x4){w[y], w[y + 1], w[y + 2], w[y + 3]});
          db = __builtin_bit_cast(x8<T>, (u32x4){ds[y], ds[y + 1], ds[y + 2], ds[y + 3]});
        }
        if constexpr (MODE == kCareful) {
          gc[x] = cleaned<T>(gc[x]);
          qc[x] = cleaned<T>(qc[x]);  // one that sees the key has made dS NaN or 0 already
        }
        dv[x % DB] = mfma(gc[x], wb, dv[x % DB]);
        if constexpr (kPipelined) {
          rest(2 * x);
          step();
        }
        dk[x % DB] = mfma(qc[x], db, dk[x % DB]);
        if constexpr (kPipelined) rest(2 * x + 1);
        if constexpr (MODE == kCareful)
          if (x == 2 * DB - 2)  // before the barrier
            for (int32_t j = 0; j < BM; ++j)
              add_nonfinite_row<T, DB, CPR>(dv, gt, j, row0 + j >= first && row0 + j < rows, half);
      }
      step();
      if constexpr (kPipelined) {
        s = s_next;
        dp = dp_next;
      }
    };

    const int32_t partly = min(max(blocks, 0), max(0, wave_all - row_begin + BM - 1) / BM);
    auto walk = [&](auto mode) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[d][i] = dv[d][i] = 0.0f;
      if (blocks <= 0) return;
      // Blocks behind the last are begun and scored like the others, and not used.
      for (int32_t i = 0; i < kStages - 1; ++i) {
        go_to(i);
#pragma unroll
        for (int x = 0; x < kPieces; ++x) piece(i, x);
      }
      settle<T>(kf);
      settle<T>(vf);
      if constexpr (kPipelined) {
        wait_copies_and_sync<kPieces>();  // blocks 0 and 1
        read_row(buffer(0), 0);
        read_row(buffer(0), 1);
        scores(buffer(0), s, dp, [](int) {}, [](int) {});
        read_stats(buffer(0), 0);
        read_stats(buffer(0), 1);
#pragma unroll
        for (int u = 0; u < 8; ++u) weigh(mode, u, s, dp, first_row(0));
        read_row(buffer(1), 0);
        read_row(buffer(1), 1);
      }
      // in careful mode every block is masked, for the rows behind the last
      const int32_t masked = decltype(mode)::value == kCareful ? blocks : partly;
      int32_t b = 0;
      for (; b < masked; ++b) round(mode, b);
      for (; b < blocks; ++b) round(Constant<kWhole>(), b);
      wait_copies<0>();
    };
    walk(Constant<kMasked>());
    if (any_wave(any_nonfinite(dk) || any_nonfinite(dv), flags)) {
      walk(Constant<kCareful>());
      // The next tile's first copies go into buffers that the last block was read from (behind the
      // walk above, any_wave has waited for all waves).
      wait_copies_and_sync<0>();
    }

    if (!whole) {
      float* part = p.part + (2 * (int64_t)share + (from == 0)) * 2 * kKeyTile * p.D +
                    (32 * wave + (lane & 31)) * p.D;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t e = 32 * d + 8 * j + 4 * half;
          if (!on || e >= (uint32_t)p.D) continue;
          *reinterpret_cast<f32x4*>(part + e) =
              (f32x4){dk[d][4 * j], dk[d][4 * j + 1], dk[d][4 * j + 2], dk[d][4 * j + 3]};
          *reinterpret_cast<f32x4*>(part + kKeyTile * p.D + e) =
              (f32x4){dv[d][4 * j], dv[d][4 * j + 1], dv[d][4 * j + 2], dv[d][4 * j + 3]};
        }
      continue;
    }
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) dk[d][i] *= p.scale;
    const int64_t at_row = (int64_t)(start + at_key);
    store_row<T, DB>(dk, dk_out + at_row * p.dk_stride + (int64_t)kvh * p.D, half, chunks, on);
    store_row<T, DB>(dv, dv_out + at_row * p.dv_stride + (int64_t)kvh * p.D, half, chunks, on);
  }
}

// Adds the partial sums of the tiles that are cut: workgroup x looks at the end of share x, and
// takes the tile there if that is the first cut in it; y takes 32 of its keys.
template <typename T>
__global__ __launch_bounds__(256) void attn_bwd_join_kernel(const BwdParams p) {
  if (!plan_matches(p, kPackedPlan)) return;
  const Place work = place_of(p, gridDim.x);
  const int64_t share = blockIdx.x, cut = (share + 1) * work.share;
  if (cut >= work.total || work.tiles <= 0) return;
  const uint32_t kvh = (uint32_t)(cut / work.units);
  const int64_t pos = cut - kvh * work.units;
  const int32_t index = find_tile(p, work.tiles, pos);
  const KeyTile j = p.key_tiles[index];
  const int64_t tile_begin = cut - (pos - j.first), tile_end = tile_begin - j.first + end_of_tile(p, work, index);
  if (work.near != 0) {
    const int64_t units = tile_end - tile_begin, here = pos - j.first, before = here - work.share;
    const int64_t at = place_of_cut(work, here, units);
    if (at == 0 || at == units) return;
    if (before > 0 && place_of_cut(work, before, units) != 0) return;
  } else if (pos == j.first || tile_begin < share * work.share) {
    return;
  }
  if (j.gap != 0 || j.start < 0 || j.n <= 0 || j.start > p.T - j.n || j.key0 < 0) return;
  // its pieces: the second slot of this share, then the first ones of those that follow
  const int32_t pieces = (int32_t)min((tile_end - 1 - work.near) / work.share - share + 1, (int64_t)gridDim.x - share);
  const int32_t first = 32 * blockIdx.y, keys = min(32, j.n - j.key0 - first);
  const int32_t groups = p.D >> 2, size = kKeyTile * p.D;
  for (int32_t i = threadIdx.x; i < 2 * keys * groups; i += 256) {
    const int32_t which = i >= keys * groups, of = i - which * keys * groups;
    const int32_t y = of / groups, e = 4 * (of - y * groups);
    const float* part = p.part + 2 * share * 2 * size + which * size + (first + y) * p.D + e;
    f32x4 x = {0, 0, 0, 0};
    for (int32_t s0 = 0; s0 < pieces; s0 += 8) {  // eight loads at a time
      f32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t s = min(s0 + u, pieces - 1);
        v[u] = *reinterpret_cast<const f32x4*>(part + (2 * s + (s == 0)) * 2 * size);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (s0 + u >= pieces) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] += v[u][c];
      }
    }
    const float f = which ? 1.0f : p.scale;
    T* row = static_cast<T*>(which ? p.dv : p.dk) +
             (int64_t)(j.start + j.key0 + first + y) * (which ? p.dv_stride : p.dk_stride) +
             (int64_t)kvh * p.D + e;
    *reinterpret_cast<u32x2*>(row) =
        (u32x2){narrow2<T>(x[0] * f, x[1] * f), narrow2<T>(x[2] * f, x[3] * f)};
  }
}

// Shares of the dK/dV pass: the workgroups that 256 CUs hold at once.
inline int32_t key_shares(int32_t D) { return D <= 64 ? 512 : 256; }

template <typename T, int DB>
int32_t launch(const BwdParams& p, const PackedSizes& z, hipStream_t s) {
  hipLaunchKernelGGL((attn_bwd_rows_kernel<T, DB, ATTN_MODS>), dim3((unsigned)(z.rows * p.Hkv)), dim3(256), 0, s,
                     p);
  int32_t st = launched();
  if (st != ROPE_OK) return st;
  const unsigned shares = key_shares(p.D);
  hipLaunchKernelGGL((attn_bwd_keys_kernel<T, DB, ATTN_MODS>), dim3(shares), dim3(256), 0, s, p);
  st = launched();
  if (st != ROPE_OK) return st;
  hipLaunchKernelGGL((attn_bwd_join_kernel<T>), dim3(shares, kKeyTile / 32), dim3(256), 0, s, p);
  return launched();
}

template <typename T>
int32_t launch_size(const BwdParams& p, const PackedSizes& z, hipStream_t s) {
  switch ((p.D + 31) / 32) {
    case 1: return launch<T, 1>(p, z, s);
    case 2: return launch<T, 2>(p, z, s);
    case 3: return launch<T, 3>(p, z, s);
    default: return launch<T, 4>(p, z, s);
  }
}

}  // namespace

template <>
int32_t launch_bwd<ATTN_MODS>(const BwdParams& p, const PackedSizes& z, int32_t dtype, hipStream_t s) {
  return dtype == ROPE_BF16 ? launch_size<__bf16>(p, z, s) : launch_size<_Float16>(p, z, s);
}

}  // namespace attn

#if ATTN_MODS == 0

using namespace attn;

extern "C" int64_t attn_bwd_scratch_floats(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv,
                                           int32_t D) {
  return attn_bwd_ex_scratch_floats(T, num_seqs, Hq, Hkv, D, 0);
}

extern "C" int64_t attn_bwd_ex_scratch_floats(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv,
                                              int32_t D, int32_t biased) {
  if (!valid_batch(T, num_seqs, Hq, Hkv) || !valid_head_size(D) || D > 128) return -1;
  return (int64_t)2 * key_shares(D) * 2 * kKeyTile * D + (biased ? 4 : 2) * T * Hq;
}

extern "C" int32_t attn_bwd(const void* dout, const void* q, const void* k, const void* v,
                            const void* out, const float* lse, float* scratch, void* dq, void* dk,
                            void* dv, int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                            int64_t dout_stride, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int64_t out_stride, int64_t dq_stride,
                            int64_t dk_stride, int64_t dv_stride, const int32_t* plan,
                            int32_t num_seqs, double scale, int32_t dtype, int32_t fill,
                            void* stream) {
  return attn_bwd_ex(dout, q, k, v, out, lse, scratch, dq, dk, dv, T, Hq, Hkv, D, dout_stride, q_stride,
                     k_stride, v_stride, out_stride, dq_stride, dk_stride, dv_stride, plan, num_seqs,
                     scale, 0.0, nullptr, dtype, fill, stream);
}

extern "C" int32_t attn_bwd_ex(const void* dout, const void* q, const void* k, const void* v,
                               const void* out, const float* lse, float* scratch, void* dq, void* dk,
                               void* dv, int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                               int64_t dout_stride, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, int64_t out_stride, int64_t dq_stride,
                               int64_t dk_stride, int64_t dv_stride, const int32_t* plan,
                               int32_t num_seqs, double scale, double cap, const float* slopes,
                               int32_t dtype, int32_t fill, void* stream) {
  if (!valid_dtype16(dtype)) return ROPE_EUNSUPPORTED;
  if (attn_plan_ints(T, num_seqs, Hq, Hkv) < 0 || !valid_head_size(D) || D > 128) return ROPE_EINVAL;
  if (!valid_scale(scale) || !valid_cap(cap, scale)) return ROPE_EINVAL;
  BwdParams p;
  if (!token_stride(dout_stride, Hq, D, &p.dout_stride) ||
      !token_stride(q_stride, Hq, D, &p.q_stride) || !token_stride(k_stride, Hkv, D, &p.k_stride) ||
      !token_stride(v_stride, Hkv, D, &p.v_stride) ||
      !token_stride(out_stride, Hq, D, &p.out_stride) ||
      !token_stride(dq_stride, Hq, D, &p.dq_stride) ||
      !token_stride(dk_stride, Hkv, D, &p.dk_stride) ||
      !token_stride(dv_stride, Hkv, D, &p.dv_stride))
    return ROPE_EINVAL;
  if (T == 0) return ROPE_OK;
  const void* data[] = {dout, q, k, v, out, dq, dk, dv, plan};
  for (const void* x : data)
    if (!data_pointer(x)) return ROPE_EINVAL;
  if (lse == nullptr || !data_pointer(scratch)) return ROPE_EINVAL;
  p.G = Hq / Hkv;
  const PackedSizes z = packed_sizes(T, num_seqs, Hq, Hkv);
  if (z.rows * Hkv > kMaxBlocks) return ROPE_EINVAL;
  p.dout = dout;
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.lse = lse;
  p.part = scratch;
  p.lse2 = scratch + (int64_t)2 * key_shares(D) * 2 * kKeyTile * D;
  p.delta = p.lse2 + T * Hq;
  p.slope = p.delta + T * Hq;  // with slopes only, as is the next
  p.at = reinterpret_cast<int32_t*>(p.slope + T * Hq);
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.plan = plan;
  p.row_items = reinterpret_cast<const RowItem*>(plan + kHeader);
  p.key_tiles = reinterpret_cast<const KeyTile*>(p.row_items + z.rows + z.rows % 2);
  p.T = (int32_t)T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.num_seqs = num_seqs;
  p.scale = (float)scale;
  p.scale2 = score_scale(scale, cap);
  p.scores = score_params(scale, cap, slopes);
  p.fill = fill;
  p.by_hkv = make_div31(Hkv);
  p.by_g = make_div31(p.G);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (score_mods(cap, slopes)) {
    case 0: return launch_bwd<0>(p, z, dtype, s);
    case kBias: return launch_bwd<kBias>(p, z, dtype, s);
    case kCap: return launch_bwd<kCap>(p, z, dtype, s);
    default: return launch_bwd<kBias | kCap>(p, z, dtype, s);
  }
}

#endif
