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
#include "attn_packed.h"
#include "attn_tile.h"

namespace attn {
namespace {

constexpr int32_t kExactKeys = 256;  // tiles up to here form D_i from P and dP

struct BwdParams {
  const void* dout;
  const void* q;
  const void* k;
  const void* v;
  const void* out;
  const float* lse;
  float* lse2;   // scratch: lse * log2 e
  float* delta;  // scratch: D_i
  void* dq;
  void* dk;
  void* dv;
  const int32_t* plan;
  const RowItem* row_items;
  const KeyItem* key_items;
  const KeyJoin* joins;
  float* part;    // scratch: [slot][Hkv][dK, dV][128][D], of tiles whose rows are split
  int64_t units;  // its slots
  int64_t dout_stride, q_stride, k_stride, v_stride, out_stride, dq_stride, dk_stride, dv_stride;
  int32_t T, Hq, Hkv, G, D, num_seqs;
  float scale, scale2;  // scale2: times log2 e
  int32_t fill;
  Div31 by_hkv, by_g;
};

// The item of this workgroup, or n = 0 where there is none.
template <typename I>
__device__ inline I find_item(const BwdParams& p, const I* items, int list, uint32_t* kvh) {
  const uint32_t index = div31(blockIdx.x, p.by_hkv);
  *kvh = blockIdx.x - index * p.Hkv;
  I item;
  item.n = 0;
  if (!plan_matches(p) || (int32_t)index >= p.plan[list]) return item;
  item = items[index];
  if (item.start < 0 || item.n <= 0 || item.start > p.T - item.n) item.n = 0;
  return item;
}

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

template <typename T, int DB>
__global__ __launch_bounds__(256, 2) void attn_bwd_rows_kernel(const BwdParams p) {
  constexpr int CPR = chunks_per_row(DB), KS = 2 * DB, BN = 32;
  constexpr int kTileBytes = BN * CPR * 16, kLoads = BN * CPR / 256;
  constexpr int kStages = 5;  // 80 KB at most: two workgroups on a CU
  __shared__ __attribute__((aligned(16))) uint8_t lds[kStages * 2 * kTileBytes];

  uint32_t kvh;
  const RowItem item = find_item(p, p.row_items, 0, &kvh);
  const int32_t start = item.start, n = item.n;
  if (n == 0) return;
  const uint32_t tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = p.D >> 3;
  if (item.gap != 0) {
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
  const int32_t seen = token + 1;
  const int32_t wave_end =
      wave_row0 < row_end ? (int32_t)div31(min(wave_row0 + 32, row_end) - 1, p.by_g) + 1 : 0;
  const int32_t wave_all = div31(min(wave_row0, row_end - 1), p.by_g) + 1;
  const int32_t key_end = div31(row_end - 1, p.by_g) + 1;

  const int64_t at_row = (int64_t)(start + token);
  x8<T> qf[KS], df[KS];
  load_row<T>(qf, static_cast<const T*>(p.q) + at_row * p.q_stride + (int64_t)head * p.D, half, chunks);
  load_row<T>(df, static_cast<const T*>(p.dout) + at_row * p.dout_stride + (int64_t)head * p.D, half,
              chunks);
  float delta = 0.0f;
  {
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

  f32x16 dq[DB];
  clear_unused_chunks<CPR>(lds, kStages * 2 * BN, chunks);

  const T* k = static_cast<const T*>(p.k) + (int64_t)start * p.k_stride + (int64_t)kvh * p.D;
  const T* v = static_cast<const T*>(p.v) + (int64_t)start * p.v_stride + (int64_t)kvh * p.D;
  const int32_t blocks = (key_end + BN - 1) / BN;
  auto stage = [&](int32_t b) __attribute__((always_inline)) {
    const uint32_t kd = lds_address(lds) + b % kStages * 2 * kTileBytes;
    const uint32_t vd = kd + kTileBytes;
    const int32_t key0 = b * BN;
    const T* kb = k + (int64_t)key0 * p.k_stride;
    const T* vb = v + (int64_t)key0 * p.v_stride;
    const int32_t last = key_end - 1 - key0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t c = i * 256 + tid;
      const uint32_t r = c / CPR, chunk = (c % CPR) ^ swizzle<CPR>(r);
      const uint32_t at = (uint32_t)min((int32_t)r, last);
      const uint32_t dst = (i * 256 + wave * 64) * 16;
      if (chunk < chunks) {
        copy_chunk_to_lds(kb + (at * (uint32_t)p.k_stride + 8 * chunk), kd + dst);
        copy_chunk_to_lds(vb + (at * (uint32_t)p.v_stride + 8 * chunk), vd + dst);
      }
    }
  };

  // P and dP of 32 keys; what is hidden gets P = dP = 0.
  auto weights = [&](auto mode, const uint8_t* kt, int32_t key0, f32x16& s, f32x16& dp) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      s = mfma(read_rows<T, CPR>(kt, lane & 31, 2 * t + half), qf[t], s);
      dp = mfma(read_rows<T, CPR>(kt + kTileBytes, lane & 31, 2 * t + half), df[t], dp);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale2, -lse2));
      if constexpr (decltype(mode)::value != kWhole) {
        const int32_t key = key0 + 8 * (i / 4) + 4 * (int32_t)half + i % 4;
        if (key >= seen) s[i] = dp[i] = 0.0f;
      }
    }
  };
  auto block = [&](auto mode, const uint8_t* kt, int32_t key0) __attribute__((always_inline)) {
    f32x16 s, dp;
    weights(mode, kt, key0, s, dp);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = s[i] * (dp[i] - delta);
      if constexpr (decltype(mode)::value != kWhole) {  // also where D_i is not finite
        const int32_t key = key0 + 8 * (i / 4) + 4 * (int32_t)half + i % 4;
        if (key >= seen) s[i] = 0.0f;
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const x8<T> ds = narrow8<T>(s, t);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        x8<T> kc = read_columns<T, CPR>(kt, 16 * t, d, lane);
        // a key that is seen and not finite has made dS NaN or 0 already
        if constexpr (decltype(mode)::value == kCareful) kc = cleaned<T>(kc);
        dq[d] = mfma(kc, ds, dq[d]);
      }
    }
  };

  int32_t b = 0;
  auto first_stages = [&]() __attribute__((always_inline)) {
    for (int32_t i = 0; i < min(blocks, kStages - 1); ++i) stage(i);
  };
  auto arrive = [&]() __attribute__((always_inline)) {
    wait_ring<kStages, 2 * kLoads>(blocks - 1 - b);
    if (b + kStages - 1 < blocks) stage(b + kStages - 1);
    return lds + b % kStages * 2 * kTileBytes;
  };
  first_stages();
  settle<T>(qf);
  settle<T>(df);
  // D_i from the rounded output errs by half a step of it, which is most where a row sees few
  // keys, and as much there as the rounding of dS. Such tiles form sum_j P_ij dP_ij first.
  if (key_end <= kExactKeys) {
    float sum = 0.0f;
    for (; b < blocks; ++b) {
      const uint8_t* kt = arrive();
      if (b * BN >= wave_end) continue;
      f32x16 s, dp;
      weights(Constant<kMasked>(), kt, b * BN, s, dp);
#pragma unroll
      for (int i = 0; i < 16; ++i) sum = __builtin_fmaf(s[i], dp[i], sum);
    }
    delta = half_sum(sum);
    __syncthreads();  // the last block has been read
    b = 0;
    first_stages();
  }
  if (on && half == 0) {
    p.lse2[at_stat] = lse2;
    p.delta[at_stat] = delta;
  }
  // two loops, and a second walk where it is needed, as in the forward
  const int32_t all = wave_end > 0 ? wave_all / BN : 0;
  auto walk = [&](auto mode) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) dq[d][i] = 0.0f;
    for (; b < all; ++b) {
      const uint8_t* kt = arrive();
      block(Constant<kWhole>(), kt, b * BN);
    }
    for (; b < blocks; ++b) {
      const uint8_t* kt = arrive();
      if (b * BN < wave_end) block(mode, kt, b * BN);
    }
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

template <typename T, int DB>
__global__ __launch_bounds__(256, DB <= 2 ? 2 : 1) void attn_bwd_keys_kernel(const BwdParams p) {
  constexpr int CPR = chunks_per_row(DB), KS = 2 * DB, BM = kRowBlock;
  constexpr int kTileBytes = BM * CPR * 16, kLoads = BM * CPR / 256;
  constexpr int kStatBytes = 2 * BM * 4, kStage = 2 * kTileBytes + kStatBytes, kStages = 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kStages * kStage];

  uint32_t kvh;
  const KeyItem item = find_item(p, p.key_items, 1, &kvh);
  const int32_t start = item.start, n = item.n;
  if (n == 0) return;
  const uint32_t tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = p.D >> 3;
  T* dk_out = static_cast<T*>(p.dk);
  T* dv_out = static_cast<T*>(p.dv);
  if (item.gap != 0) {
    if (p.fill) {
      clear_rows(dk_out, start, n, p.dk_stride, kvh, 1, chunks);
      clear_rows(dv_out, start, n, p.dv_stride, kvh, 1, chunks);
    }
    return;
  }
  const int32_t key0 = item.key0;
  if (key0 < 0 || key0 >= n) return;

  const int32_t rows = n * p.G;
  const int32_t wave_key0 = key0 + 32 * wave;
  const int32_t key = wave_key0 + (lane & 31);
  const bool on = key < n;
  const int32_t at_key = on ? key : n - 1;
  const int32_t first = at_key * p.G;  // the first row that sees this lane's key
  // rows that see some key, and every key, of the wave
  const int32_t wave_first = wave_key0 < n ? wave_key0 * p.G : rows;
  const int32_t wave_all = min(wave_key0 + 31, n - 1) * p.G;

  x8<T> kf[KS], vf[KS];
  load_row<T>(kf, static_cast<const T*>(p.k) + (int64_t)(start + at_key) * p.k_stride +
                      (int64_t)kvh * p.D, half, chunks);
  load_row<T>(vf, static_cast<const T*>(p.v) + (int64_t)(start + at_key) * p.v_stride +
                      (int64_t)kvh * p.D, half, chunks);
  f32x16 dk[DB], dv[DB];
  for (int b = 0; b < kStages; ++b) clear_unused_chunks<CPR>(lds + b * kStage, 2 * BM, chunks);

  const T* q = static_cast<const T*>(p.q) + (int64_t)start * p.q_stride + (int64_t)kvh * p.G * p.D;
  const T* g = static_cast<const T*>(p.dout) + (int64_t)start * p.dout_stride +
               (int64_t)kvh * p.G * p.D;
  const int64_t stat0 = (int64_t)start * p.Hq + kvh * p.G;
  if (item.block0 < 0 || item.block_end > (rows + BM - 1) / BM || item.slot >= p.units) return;
  const int32_t row_begin = item.block0 * BM;
  const int32_t blocks = item.block_end - item.block0;
  // A last block that rows end in goes first, so that the partly masked blocks of a wave (this
  // one and those on its diagonal) are a first loop and the others a second.
  const int32_t tail = blocks > 0 && item.block_end * BM > rows;
  auto first_row = [&](int32_t i) __attribute__((always_inline)) {
    return row_begin + (tail ? (i == 0 ? blocks - 1 : i - 1) : i) * BM;
  };

  auto stage = [&](int32_t b) __attribute__((always_inline)) {
    const uint32_t qd = lds_address(lds) + b % kStages * kStage, gd = qd + kTileBytes;
    const int32_t row0 = first_row(b);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t c = i * 256 + tid;
      const uint32_t r = c / CPR, chunk = (c % CPR) ^ swizzle<CPR>(r);
      const uint32_t at = min(row0 + (int32_t)r, rows - 1);
      const uint32_t t = div31(at, p.by_g), h = at - t * p.G;
      const uint32_t dst = (i * 256 + wave * 64) * 16;
      if (chunk < chunks) {
        copy_chunk_to_lds(q + (int64_t)t * p.q_stride + (h * p.D + 8 * chunk), qd + dst);
        copy_chunk_to_lds(g + (int64_t)t * p.dout_stride + (h * p.D + 8 * chunk), gd + dst);
      }
    }
    {  // lse and D of the rows, 32 words each; by every wave, for equal counts of copies
      const uint32_t at = min(row0 + (int32_t)(lane & 31), rows - 1);
      const uint32_t t = div31(at, p.by_g), h = at - t * p.G;
      copy_word_to_lds((half ? p.delta : p.lse2) + stat0 + (int64_t)t * p.Hq + h, gd + kTileBytes);
    }
  };

  // The loop is pipelined over two blocks, because a wave is alone on its SIMD: while the
  // matrix unit forms S and dP of the next block, the vector unit turns this block's into P
  // and dS, a slice of them per step; then dV and dK follow. `order()` keeps the steps apart
  // for the scheduler, with LDS read two steps ahead of its use.
  f32x16 s, dp;         // of the block at hand, then of the next one
  f32x4 lse2[4], delta[4];
  auto order = [] { __builtin_amdgcn_sched_barrier(0); };
  auto read_stats = [&](const uint8_t* qt) __attribute__((always_inline)) {
    const float* stat = reinterpret_cast<const float*>(qt + 2 * kTileBytes);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lse2[j] = *reinterpret_cast<const f32x4*>(stat + 8 * j + 4 * half);
      delta[j] = *reinterpret_cast<const f32x4*>(stat + 32 + 8 * j + 4 * half);
    }
  };
  // S and dP of the block at `qt`; `slice(t)` is called in step t of KS.
  auto scores = [&](const uint8_t* qt, f32x16& s_out, f32x16& dp_out, auto slice) __attribute__((always_inline)) {
    x8<T> qr[KS], gr[KS];
    auto read = [&](int t) __attribute__((always_inline)) {
      qr[t] = read_rows<T, CPR>(qt, lane & 31, 2 * t + half);
      gr[t] = read_rows<T, CPR>(qt + kTileBytes, lane & 31, 2 * t + half);
    };
    read(0);
    read(1);
    f32x16 a, c;
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = c[i] = 0.0f;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      order();
      if (t + 2 < KS) read(t + 2);
      slice(t);
      a = mfma(qr[t], kf[t], a);
      c = mfma(gr[t], vf[t], c);
    }
    order();
    s_out = a;
    dp_out = c;
  };
  auto round = [&](auto mode, const uint8_t* qt, const uint8_t* next, int32_t row0) __attribute__((always_inline)) {
    constexpr int MODE = decltype(mode)::value;
    const uint8_t* gt = qt + kTileBytes;
    f32x16 w, ds, s_next, dp_next;
    scores(next, s_next, dp_next, [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 16 * t / KS; i < 16 * (t + 1) / KS; ++i) {
        const int j = i / 4, e = i % 4;
        w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale2, -lse2[j][e]));
        ds[i] = w[i] * (dp[i] - delta[j][e]);
        if constexpr (MODE != kWhole) {
          const int32_t at = row0 + 8 * j + 4 * (int32_t)half + e;
          if (at < first || at >= rows) w[i] = ds[i] = 0.0f;
        }
      }
    });
    s = s_next;
    dp = dp_next;
    read_stats(next);
    x8<T> gc[2 * DB], qc[2 * DB];  // by step: 16 rows t = step / DB, columns d = step % DB
    auto read = [&](int x) __attribute__((always_inline)) {
      gc[x] = read_columns<T, CPR>(gt, 16 * (x / DB), x % DB, lane);
      qc[x] = read_columns<T, CPR>(qt, 16 * (x / DB), x % DB, lane);
    };
    read(0);
    read(1);
    x8<T> wb, db;
#pragma unroll
    for (int x = 0; x < 2 * DB; ++x) {
      order();
      if (x + 2 < 2 * DB) read(x + 2);
      if (x % DB == 0) {
        wb = narrow8<T>(w, x / DB);
        db = narrow8<T>(ds, x / DB);
      }
      if constexpr (MODE == kCareful) {
        gc[x] = cleaned<T>(gc[x]);
        qc[x] = cleaned<T>(qc[x]);  // one that sees the key has made dS NaN or 0 already
      }
      dv[x % DB] = mfma(gc[x], wb, dv[x % DB]);
      dk[x % DB] = mfma(qc[x], db, dk[x % DB]);
    }
    order();
    if constexpr (MODE == kCareful)
      for (int32_t j = 0; j < BM; ++j)
        add_nonfinite_row<T, DB, CPR>(dv, gt, j, row0 + j >= first && row0 + j < rows, half);
  };

  auto buffer = [&](int32_t b) __attribute__((always_inline)) { return lds + b % kStages * kStage; };
  // Before block b is finished its successor has arrived, and the buffer of its predecessor is
  // free. Behind the last block the scores of whatever a buffer holds are formed and not used.
  auto arrive = [&](int32_t b) __attribute__((always_inline)) {
    if (b + 1 >= blocks) return;
    wait_ring<kStages - 1, 2 * kLoads + 1>(blocks - 2 - b);
    if (b + kStages - 1 < blocks) stage(b + kStages - 1);
  };
  const int32_t masked =
      wave_first < rows ? min(blocks, tail + max(0, wave_all - row_begin + BM - 1) / BM) : blocks;
  auto walk = [&](auto mode) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) dk[d][i] = dv[d][i] = 0.0f;
    if (blocks <= 0) return;
    for (int32_t i = 0; i < min(blocks, kStages - 1); ++i) stage(i);
    settle<T>(kf);
    settle<T>(vf);
    wait_ring<kStages, 2 * kLoads + 1>(blocks - 1);
    scores(buffer(0), s, dp, [](int) {});
    read_stats(buffer(0));
    int32_t b = 0;
    for (; b < masked; ++b) {
      arrive(b);
      round(mode, buffer(b), buffer(b + 1), first_row(b));
    }
    for (; b < blocks; ++b) {
      arrive(b);
      round(Constant<kWhole>(), buffer(b), buffer(b + 1), first_row(b));
    }
  };
  walk(Constant<kMasked>());
  if (any_wave(any_nonfinite(dk) || any_nonfinite(dv), lds)) walk(Constant<kCareful>());

  if (item.slot >= 0) {
    float* part = p.part + ((int64_t)item.slot * p.Hkv + kvh) * 2 * kKeyTile * p.D +
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
    return;
  }
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) dk[d][i] *= p.scale;
  const int64_t at_row = (int64_t)(start + at_key);
  store_row<T, DB>(dk, dk_out + at_row * p.dk_stride + (int64_t)kvh * p.D, half, chunks, on);
  store_row<T, DB>(dv, dv_out + at_row * p.dv_stride + (int64_t)kvh * p.D, half, chunks, on);
}

// Adds the partial sums of a split tile, in the order of its rows: one workgroup per tile,
// key/value head and 32 keys.
template <typename T>
__global__ __launch_bounds__(256) void attn_bwd_join_kernel(const BwdParams p) {
  const uint32_t index = div31(blockIdx.x, p.by_hkv);
  const uint32_t kvh = blockIdx.x - index * p.Hkv;
  if (!plan_matches(p) || (int32_t)index >= p.plan[6]) return;
  const KeyJoin j = p.joins[index];
  if (j.start < 0 || j.n <= 0 || j.start > p.T - j.n || j.key0 < 0 || j.slot < 0 || j.splits < 0 ||
      j.slot + (int64_t)j.splits > p.units)
    return;
  const int32_t first = 32 * blockIdx.y, keys = min(32, j.n - j.key0 - first);
  const int32_t groups = p.D >> 2, size = kKeyTile * p.D;
  const int64_t step = (int64_t)p.Hkv * 2 * size;
  for (int32_t i = threadIdx.x; i < 2 * keys * groups; i += 256) {
    const int32_t which = i >= keys * groups, of = i - which * keys * groups;
    const int32_t y = of / groups, e = 4 * (of - y * groups);
    const float* part = p.part + ((int64_t)j.slot * p.Hkv + kvh) * 2 * size + which * size +
                        (first + y) * p.D + e;
    f32x4 x = {0, 0, 0, 0};
    for (int32_t s0 = 0; s0 < j.splits; s0 += 8) {  // eight loads at a time
      f32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = *reinterpret_cast<const f32x4*>(part + min(s0 + u, j.splits - 1) * step);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (s0 + u >= j.splits) break;
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

template <typename T, int DB>
int32_t launch(const BwdParams& p, const PackedSizes& z, hipStream_t s) {
  hipLaunchKernelGGL((attn_bwd_rows_kernel<T, DB>), dim3((unsigned)(z.rows * p.Hkv)), dim3(256), 0, s,
                     p);
  int32_t st = launched();
  if (st != ROPE_OK) return st;
  hipLaunchKernelGGL((attn_bwd_keys_kernel<T, DB>), dim3((unsigned)(z.keys * p.Hkv)), dim3(256), 0, s,
                     p);
  st = launched();
  if (st != ROPE_OK) return st;
  hipLaunchKernelGGL((attn_bwd_join_kernel<T>), dim3((unsigned)(z.joins * p.Hkv), kKeyTile / 32),
                     dim3(256), 0, s, p);
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
}  // namespace attn

using namespace attn;

extern "C" int64_t attn_bwd_scratch_floats(int64_t T, int32_t num_seqs, int32_t Hq, int32_t Hkv,
                                           int32_t D) {
  if (!valid_batch(T, num_seqs, Hq, Hkv) || !valid_head_size(D) || D > 128) return -1;
  return packed_sizes(T, num_seqs, Hq, Hkv).units * Hkv * 2 * kKeyTile * D + 2 * T * Hq;
}

extern "C" int32_t attn_bwd(const void* dout, const void* q, const void* k, const void* v,
                            const void* out, const float* lse, float* scratch, void* dq, void* dk,
                            void* dv, int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                            int64_t dout_stride, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int64_t out_stride, int64_t dq_stride,
                            int64_t dk_stride, int64_t dv_stride, const int32_t* plan,
                            int32_t num_seqs, double scale, int32_t dtype, int32_t fill,
                            void* stream) {
  if (!valid_dtype16(dtype)) return ROPE_EUNSUPPORTED;
  if (attn_plan_ints(T, num_seqs, Hq, Hkv) < 0 || !valid_head_size(D) || D > 128) return ROPE_EINVAL;
  if (!valid_scale(scale)) return ROPE_EINVAL;
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
  if (z.rows * Hkv > kMaxBlocks || z.keys * Hkv > kMaxBlocks) return ROPE_EINVAL;
  p.dout = dout;
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.lse = lse;
  p.part = scratch;
  p.units = z.units;
  p.lse2 = scratch + z.units * Hkv * 2 * kKeyTile * D;
  p.delta = p.lse2 + T * Hq;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.plan = plan;
  p.row_items = reinterpret_cast<const RowItem*>(plan + kHeader);
  p.key_items = reinterpret_cast<const KeyItem*>(p.row_items + z.rows);
  p.joins = reinterpret_cast<const KeyJoin*>(p.key_items + z.keys);
  p.T = (int32_t)T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.num_seqs = num_seqs;
  p.scale = (float)scale;
  p.scale2 = (float)(scale * kLog2e);
  p.fill = fill;
  p.by_hkv = make_div31(Hkv);
  p.by_g = make_div31(p.G);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == ROPE_BF16 ? launch_size<__bf16>(p, z, s) : launch_size<_Float16>(p, z, s);
}
