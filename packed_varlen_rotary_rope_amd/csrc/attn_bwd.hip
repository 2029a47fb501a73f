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
  const int4* items;
  int64_t dout_stride, q_stride, k_stride, v_stride, out_stride, dq_stride, dk_stride, dv_stride;
  int32_t T, Hq, Hkv, G, D, num_seqs;
  float scale, scale2;  // scale2: times log2 e
  int32_t fill;
  Div31 by_hkv, by_g;
};

// The item of this workgroup, or n = 0 where there is none.
__device__ inline int4 find_item(const BwdParams& p, int list, uint32_t* kvh) {
  const uint32_t index = div31(blockIdx.x, p.by_hkv);
  *kvh = blockIdx.x - index * p.Hkv;
  const int4 none = make_int4(0, 0, 0, 0);
  if (p.plan[2] != p.T || p.plan[3] != p.G || p.plan[4] != p.num_seqs) return none;
  if ((int32_t)index >= p.plan[list]) return none;
  const int4 item = p.items[index];
  return item.x < 0 || item.y <= 0 || item.x > p.T - item.y ? none : item;
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
  constexpr int CPR = chunks_per_row(DB), KS = 2 * DB, BN = 64;
  constexpr int kTileBytes = BN * CPR * 16, kLoads = BN * CPR / 256;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * kTileBytes];

  uint32_t kvh;
  const int4 item = find_item(p, 0, &kvh);
  const int32_t start = item.x, n = item.y;
  if (n == 0) return;
  const uint32_t tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = p.D >> 3;
  if (item.w != 0) {
    if (p.fill) clear_rows(static_cast<T*>(p.dq), start, n, p.dq_stride, kvh * p.G, p.G, chunks);
    return;
  }

  const int32_t rows = n * p.G;
  const int32_t row0 = item.z;
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
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) dq[d][i] = 0.0f;
  clear_unused_chunks<CPR>(lds, 4 * BN, chunks);

  const T* k = static_cast<const T*>(p.k) + (int64_t)start * p.k_stride + (int64_t)kvh * p.D;
  const T* v = static_cast<const T*>(p.v) + (int64_t)start * p.v_stride + (int64_t)kvh * p.D;
  const int32_t blocks = (key_end + BN - 1) / BN;
  auto stage = [&](int32_t b) {
    const uint32_t kd = lds_address(lds) + (b & 1) * 2 * kTileBytes;
    const uint32_t vd = kd + kTileBytes;
    const int32_t key0 = b * BN;
    const T* kb = k + (int64_t)key0 * p.k_stride;
    const T* vb = v + (int64_t)key0 * p.v_stride;
    const int32_t last = key_end - 1 - key0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t c = i * 256 + tid;
      const uint32_t r = c / CPR, chunk = (c % CPR) ^ swizzle(r);
      const uint32_t at = (uint32_t)min((int32_t)r, last);
      const uint32_t dst = (i * 256 + wave * 64) * 16;
      if (chunk < chunks) {
        copy_chunk_to_lds(kb + (at * (uint32_t)p.k_stride + 8 * chunk), kd + dst);
        copy_chunk_to_lds(vb + (at * (uint32_t)p.v_stride + 8 * chunk), vd + dst);
      }
    }
  };

  // P and dP of 32 keys; what is hidden gets P = dP = 0.
  auto weights = [&](auto masked, const uint8_t* kt, const uint8_t* vt, int32_t key0, int b, f32x16& s,
                     f32x16& dp) {
    constexpr bool MASKED = decltype(masked)::value;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      s = mfma(read_rows<T, CPR>(kt, 32 * b + (lane & 31), 2 * t + half), qf[t], s);
      dp = mfma(read_rows<T, CPR>(vt, 32 * b + (lane & 31), 2 * t + half), df[t], dp);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale2, -lse2));
      if constexpr (MASKED) {
        const int32_t key = key0 + 32 * b + 8 * (i / 4) + 4 * (int32_t)half + i % 4;
        if (key >= seen) s[i] = dp[i] = 0.0f;
      }
    }
  };
  auto block = [&](auto masked, const uint8_t* kt, int32_t key0) {
    constexpr bool MASKED = decltype(masked)::value;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x16 s, dp;
      weights(masked, kt, kt + kTileBytes, key0, b, s, dp);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = s[i] * (dp[i] - delta);
        if constexpr (MASKED) {  // also where D_i is not finite
          const int32_t key = key0 + 32 * b + 8 * (i / 4) + 4 * (int32_t)half + i % 4;
          if (key >= seen) s[i] = 0.0f;
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const x8<T> ds = narrow8<T>(s, t);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          x8<T> kc = read_columns<T, CPR>(kt, 32 * b + 16 * t, d, lane);
          // a key that is seen and not finite has made dS NaN or 0 already
          if constexpr (MASKED) kc = cleaned<T>(kc);
          dq[d] = mfma(kc, ds, dq[d]);
        }
      }
    }
  };

  stage(0);
  settle<T>(qf);
  settle<T>(df);
  int32_t b = 0;
  auto arrive = [&] {
    wait_copies_and_sync();  // block b has arrived, and its buffer's neighbour is free
    if (b + 1 < blocks) stage(b + 1);
    return lds + (b & 1) * 2 * kTileBytes;
  };
  // D_i from the rounded output errs by half a step of it, which is most where a row sees few
  // keys, and as much there as the rounding of dS. Such tiles form sum_j P_ij dP_ij first.
  if (key_end <= kExactKeys) {
    float sum = 0.0f;
    for (; b < blocks; ++b) {
      const uint8_t* kt = arrive();
      if (b * BN >= wave_end) continue;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        f32x16 s, dp;
        weights(Constant<true>(), kt, kt + kTileBytes, b * BN, c, s, dp);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = __builtin_fmaf(s[i], dp[i], sum);
      }
    }
    delta = half_sum(sum);
    __syncthreads();  // the last block has been read
    b = 0;
    stage(0);
  }
  if (on && half == 0) {
    p.lse2[at_stat] = lse2;
    p.delta[at_stat] = delta;
  }
  // two loops, as in the forward
  const int32_t all = wave_end > 0 ? wave_all / BN : 0;
  for (; b < all; ++b) {
    const uint8_t* kt = arrive();
    block(Constant<false>(), kt, b * BN);
  }
  for (; b < blocks; ++b) {
    const uint8_t* kt = arrive();
    if (b * BN < wave_end) block(Constant<true>(), kt, b * BN);
  }
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) dq[d][i] *= p.scale;
  store_row<T, DB>(dq, static_cast<T*>(p.dq) + at_row * p.dq_stride + (int64_t)head * p.D, half,
                   chunks, on);
}

template <typename T, int DB>
__global__ __launch_bounds__(256, 1) void attn_bwd_keys_kernel(const BwdParams p) {
  constexpr int CPR = chunks_per_row(DB), KS = 2 * DB, BM = 32;
  constexpr int kTileBytes = BM * CPR * 16, kLoads = BM * CPR / 256;
  constexpr int kStatBytes = 2 * BM * 4, kStage = 2 * kTileBytes + kStatBytes;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];

  uint32_t kvh;
  const int4 item = find_item(p, 1, &kvh);
  const int32_t start = item.x, n = item.y;
  if (n == 0) return;
  const uint32_t tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = p.D >> 3;
  T* dk_out = static_cast<T*>(p.dk);
  T* dv_out = static_cast<T*>(p.dv);
  if (item.w != 0) {
    if (p.fill) {
      clear_rows(dk_out, start, n, p.dk_stride, kvh, 1, chunks);
      clear_rows(dv_out, start, n, p.dv_stride, kvh, 1, chunks);
    }
    return;
  }
  const int32_t key0 = item.z;
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
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) dk[d][i] = dv[d][i] = 0.0f;
  for (int b = 0; b < 2; ++b) clear_unused_chunks<CPR>(lds + b * kStage, 2 * BM, chunks);

  const T* q = static_cast<const T*>(p.q) + (int64_t)start * p.q_stride + (int64_t)kvh * p.G * p.D;
  const T* g = static_cast<const T*>(p.dout) + (int64_t)start * p.dout_stride +
               (int64_t)kvh * p.G * p.D;
  const int64_t stat0 = (int64_t)start * p.Hq + kvh * p.G;
  const int32_t row_begin = key0 * p.G / BM * BM;
  const int32_t blocks = (rows - row_begin + BM - 1) / BM;
  // A last block that rows end in goes first, so that the partly masked blocks of a wave (this
  // one and those on its diagonal) are a first loop and the others a second.
  const int32_t tail = (rows - row_begin) % BM != 0;
  auto first_row = [&](int32_t i) {
    return row_begin + (tail ? (i == 0 ? blocks - 1 : i - 1) : i) * BM;
  };

  auto stage = [&](int32_t b) {
    const uint32_t qd = lds_address(lds) + (b & 1) * kStage, gd = qd + kTileBytes;
    const int32_t row0 = first_row(b);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t c = i * 256 + tid;
      const uint32_t r = c / CPR, chunk = (c % CPR) ^ swizzle(r);
      const uint32_t at = min(row0 + (int32_t)r, rows - 1);
      const uint32_t t = div31(at, p.by_g), h = at - t * p.G;
      const uint32_t dst = (i * 256 + wave * 64) * 16;
      if (chunk < chunks) {
        copy_chunk_to_lds(q + (int64_t)t * p.q_stride + (h * p.D + 8 * chunk), qd + dst);
        copy_chunk_to_lds(g + (int64_t)t * p.dout_stride + (h * p.D + 8 * chunk), gd + dst);
      }
    }
    if (wave == 0) {  // lse and D of the rows: 32 words each
      const uint32_t at = min(row0 + (int32_t)(lane & 31), rows - 1);
      const uint32_t t = div31(at, p.by_g), h = at - t * p.G;
      copy_word_to_lds((half ? p.delta : p.lse2) + stat0 + (int64_t)t * p.Hq + h, gd + kTileBytes);
    }
  };

  auto block = [&](auto masked, const uint8_t* qt, int32_t row0) {
    constexpr bool MASKED = decltype(masked)::value;
    const uint8_t* gt = qt + kTileBytes;
    const float* stat = reinterpret_cast<const float*>(gt + kTileBytes);
    const uint32_t r = lane & 31;
    f32x16 s, dp;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      s = mfma(read_rows<T, CPR>(qt, r, 2 * t + half), kf[t], s);
      dp = mfma(read_rows<T, CPR>(gt, r, 2 * t + half), vf[t], dp);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x4 lse2 = *reinterpret_cast<const f32x4*>(stat + 8 * j + 4 * half);
      const f32x4 delta = *reinterpret_cast<const f32x4*>(stat + 32 + 8 * j + 4 * half);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 4 * j + e;
        float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.scale2, -lse2[e]));
        float d = w * (dp[i] - delta[e]);
        if constexpr (MASKED) {
          const int32_t at = row0 + 8 * j + 4 * (int32_t)half + e;
          if (at < first || at >= rows) w = d = 0.0f;
        }
        s[i] = w;
        dp[i] = d;
      }
    }
    uint32_t bad = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const x8<T> w = narrow8<T>(s, t), ds = narrow8<T>(dp, t);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        x8<T> gc = read_columns<T, CPR>(gt, 16 * t, d, lane);
        x8<T> qc = read_columns<T, CPR>(qt, 16 * t, d, lane);
        if constexpr (MASKED) {
          bad |= nonfinite<T>(gc);
          gc = cleaned<T>(gc);
          qc = cleaned<T>(qc);  // one that sees the key has made dS NaN or 0 already
        }
        dv[d] = mfma(gc, w, dv[d]);
        dk[d] = mfma(qc, ds, dk[d]);
      }
    }
    if constexpr (MASKED) {
      if (__any(bad != 0))
        for (int32_t j = 0; j < BM; ++j)
          add_nonfinite_row<T, DB, CPR>(dv, gt, j, row0 + j >= first && row0 + j < rows, half);
    }
  };

  stage(0);
  settle<T>(kf);
  settle<T>(vf);
  int32_t b = 0;
  auto arrive = [&] {
    wait_copies_and_sync();  // block b has arrived, and its buffer's neighbour is free
    if (b + 1 < blocks) stage(b + 1);
    return lds + (b & 1) * kStage;
  };
  const int32_t masked =
      wave_first < rows ? min(blocks, tail + max(0, wave_all - row_begin + BM - 1) / BM) : blocks;
  for (; b < masked; ++b) {
    const uint8_t* qt = arrive();
    if (first_row(b) + BM > wave_first && wave_first < rows) block(Constant<true>(), qt, first_row(b));
  }
  for (; b < blocks; ++b) {
    const uint8_t* qt = arrive();
    block(Constant<false>(), qt, first_row(b));
  }
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) dk[d][i] *= p.scale;
  const int64_t at_row = (int64_t)(start + at_key);
  store_row<T, DB>(dk, dk_out + at_row * p.dk_stride + (int64_t)kvh * p.D, half, chunks, on);
  store_row<T, DB>(dv, dv_out + at_row * p.dv_stride + (int64_t)kvh * p.D, half, chunks, on);
}

template <typename T, int DB>
int32_t launch(BwdParams p, hipStream_t s) {
  const int4* rows = reinterpret_cast<const int4*>(p.plan + kHeader);
  p.items = rows;
  hipLaunchKernelGGL((attn_bwd_rows_kernel<T, DB>),
                     dim3((unsigned)(row_items(p.T, p.num_seqs, p.G) * p.Hkv)), dim3(256), 0, s, p);
  const int32_t st = launched();
  if (st != ROPE_OK) return st;
  p.items = rows + row_items(p.T, p.num_seqs, p.G);
  hipLaunchKernelGGL((attn_bwd_keys_kernel<T, DB>),
                     dim3((unsigned)(key_items(p.T, p.num_seqs) * p.Hkv)), dim3(256), 0, s, p);
  return launched();
}

template <typename T>
int32_t launch_size(const BwdParams& p, hipStream_t s) {
  switch ((p.D + 31) / 32) {
    case 1: return launch<T, 1>(p, s);
    case 2: return launch<T, 2>(p, s);
    case 3: return launch<T, 3>(p, s);
    default: return launch<T, 4>(p, s);
  }
}

}  // namespace
}  // namespace attn

using namespace attn;

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
  if (lse == nullptr || scratch == nullptr) return ROPE_EINVAL;
  p.G = Hq / Hkv;
  if (row_items(T, num_seqs, p.G) * Hkv > kMaxBlocks) return ROPE_EINVAL;
  p.dout = dout;
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.lse = lse;
  p.lse2 = scratch;
  p.delta = scratch + T * Hq;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.plan = plan;
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
  return dtype == ROPE_BF16 ? launch_size<__bf16>(p, s) : launch_size<_Float16>(p, s);
}
