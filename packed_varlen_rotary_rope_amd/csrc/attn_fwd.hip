// attn_fwd.hip -- causal attention of packed sequences, forward (attn_fwd of include/attn.h).
//
// One workgroup per item of the plan's row list and key/value head: 128 packed rows
// (token-major, the group's heads minor), so that the heads of a group share every key and
// value read and a tile spans few tokens, which wastes little above the diagonal and in
// short sequences.
//
// What bounds it: matrix and vector unit together (with 128-wide heads both are busy for more
// than half of the cycles, with 64-wide ones the exponentials for two thirds), and in long
// launches the power limit, which takes the clock from 1.9 to 1.6 GHz; with short samples also the
// start and end of workgroups (22 samples of 32 to 4096 tokens: 11 blocks of keys a workgroup, and
// 155 us where the blocks alone would take 124). Two workgroups of four
// waves share a CU (64 KB of LDS each), so that one wave's softmax runs beside another's products.
// Measured, bf16: a prompt of 16384 tokens, 32 + 8 heads of 128, 2.0 to 2.3 ms, about 1.05
// PFLOP/s (a large library product reaches 1.35); eight samples of 256 to 2048 tokens of the
// same heads 148 us, 0.79; 8192 tokens of 16 + 2 heads of 64, 181 us, 0.76. Pipelined within a
// wave over blocks of 32 keys (scores of the next beside this one's exponentials) it was 5 %
// slower: twice the barriers and address arithmetic per key.
#include "attn_packed.h"
#include "attn_tile.h"

namespace attn {
namespace {

struct FwdParams {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  const int32_t* plan;
  const RowItem* items;
  int64_t q_stride, k_stride, v_stride, out_stride;
  int32_t T, Hq, Hkv, G, D, num_seqs;
  float scale;  // times log2 e
  int32_t fill;
  Div31 by_hkv, by_g;
};

template <typename T, int DB>
__global__ __launch_bounds__(256, DB <= 4 ? 2 : 1) void attn_fwd_kernel(const FwdParams p) {
  constexpr int BN = keys_per_block(DB);
  using Tile = FwdTile<T, DB, BN>;
  constexpr int CPR = Tile::CPR, kLoads = BN * CPR / 256;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * Tile::kTileBytes];  // two blocks in flight

  const uint32_t index = div31(blockIdx.x, p.by_hkv);
  const uint32_t kvh = blockIdx.x - index * p.Hkv;
  if (!plan_matches(p, kPackedPlan)) return;
  if ((int32_t)index >= p.plan[0]) return;
  const RowItem item = p.items[index];
  const int32_t start = item.start, n = item.n;
  if (start < 0 || n <= 0 || start > p.T - n) return;
  const uint32_t tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = p.D >> 3;
  T* out = static_cast<T*>(p.out);

  if (item.gap != 0) {  // rows of no sequence
    if (!p.fill) return;
    const uint32_t per_token = p.G * chunks;
    for (uint32_t i = tid; i < n * per_token; i += 256) {
      const uint32_t t = i / per_token, c = i - t * per_token;
      *reinterpret_cast<u32x4*>(out + (int64_t)(start + t) * p.out_stride +
                                (int64_t)kvh * p.G * p.D + 8 * c) = (u32x4){0, 0, 0, 0};
    }
    for (uint32_t i = tid; i < (uint32_t)n * p.G; i += 256) {
      const uint32_t t = i / p.G, g = i - t * p.G;
      p.lse[(int64_t)(start + t) * p.Hq + kvh * p.G + g] = -__builtin_inff();
    }
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
  // keys that some row, and that every row, of the wave and of the tile sees
  const int32_t wave_end = wave_row0 < row_end ? (int32_t)div31(min(wave_row0 + 32, row_end) - 1, p.by_g) + 1 : 0;
  const int32_t wave_all = div31(min(wave_row0, row_end - 1), p.by_g) + 1;
  const int32_t key_end = div31(row_end - 1, p.by_g) + 1;

  Tile t;
  load_row<T>(t.q, static_cast<const T*>(p.q) + (int64_t)(start + token) * p.q_stride +
                       (int64_t)head * p.D, half, chunks);
  clear_unused_chunks<CPR>(lds, 4 * BN, chunks);

  const T* k = static_cast<const T*>(p.k) + (int64_t)start * p.k_stride + (int64_t)kvh * p.D;
  const T* v = static_cast<const T*>(p.v) + (int64_t)start * p.v_stride + (int64_t)kvh * p.D;
  const int32_t blocks = (key_end + BN - 1) / BN;

  // Two buffers each for K and V: while a block is worked on, the next one's copies are begun
  // one a step of its scores (all at once, they would hold the wave up).
  uint64_t lanes[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) lanes[i] = __ballot(chunk_of<CPR, 256>(i, tid) < chunks);
  auto piece = [&](int32_t b, int32_t buffer, int x) __attribute__((always_inline)) {  // x-th copy of block b
    const int i = x / 2;
    const int64_t stride = x % 2 ? p.v_stride : p.k_stride;
    const int32_t key0 = b * BN;
    const uint32_t at = min((int32_t)row_of<CPR, 256>(i, tid), key_end - 1 - key0);
    const T* from = (x % 2 ? v : k) + (int64_t)key0 * stride;
    copy_chunk_to_lds(from + (at * (uint32_t)stride + 8 * chunk_of<CPR, 256>(i, tid)),
                      lds_address(lds) + (buffer * 2 + x % 2) * Tile::kTileBytes + (i * 256 + wave * 64) * 16,
                      lanes[i]);
  };
  constexpr int kPieces = 2 * kLoads, kPerStep = (kPieces + Tile::KS - 1) / Tile::KS;
  const int32_t all = wave_end > 0 ? wave_all / BN : 0;  // blocks that every row of the wave sees
  auto walk = [&](auto mode) __attribute__((always_inline)) {
    t.clear();
#pragma unroll
    for (int x = 0; x < kPieces; ++x) piece(0, 0, x);
    settle<T>(t.q);
    int32_t b = 0;
    // behind the last block the last key's copies go on into the buffer that is not used
    auto next = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int x = s * kPerStep; x < (s + 1) * kPerStep && x < kPieces; ++x) piece(min(b + 1, blocks - 1), ~b & 1, x);
    };
    // Two loops, so that neither body's registers are moved for the other's sake. Waves may be
    // in different ones: each passes one barrier per block in either.
    for (; b < (decltype(mode)::value == kCareful && t.exact ? 0 : all); ++b) {
      wait_copies_and_sync<0>();  // block b has arrived, and the other buffers are free
      const uint8_t* kt = lds + (b & 1) * 2 * Tile::kTileBytes;
      t.template block<kWhole>(kt, kt + Tile::kTileBytes, b * BN, seen, 0, p.scale, lane, next);
    }
    for (; b < blocks; ++b) {
      wait_copies_and_sync<0>();
      const uint8_t* kt = lds + (b & 1) * 2 * Tile::kTileBytes;
      if (b * BN < wave_end)
        t.template block<Mode(decltype(mode)::value)>(kt, kt + Tile::kTileBytes, b * BN, seen, 0, p.scale,
                                                      lane, next);
      else
#pragma unroll
        for (int s = 0; s < Tile::KS; ++s) next(s);
    }
    wait_copies<0>();
  };
  walk(Constant<kMasked>());
  const uint32_t anew = any_wave(any_nonfinite(t.o) | (uint32_t)t.large() << 1, lds);
  if (anew) {
    t.exact = anew & 2;
    walk(Constant<kCareful>());
    t.scale_maximum(p.scale);
  }

  const float lse = t.finish();
  store_row<T, DB>(t.o, out + (int64_t)(start + token) * p.out_stride + (int64_t)head * p.D, half,
                   chunks, on);
  if (on && half == 0) p.lse[(int64_t)(start + token) * p.Hq + head] = lse;
}

template <typename T, int DB>
int32_t launch(const FwdParams& p, int64_t blocks, hipStream_t s) {
  hipLaunchKernelGGL((attn_fwd_kernel<T, DB>), dim3((unsigned)blocks), dim3(256), 0, s, p);
  return launched();
}

template <typename T>
int32_t launch_size(const FwdParams& p, int64_t blocks, hipStream_t s) {
  switch ((p.D + 31) / 32) {
    case 1: return launch<T, 1>(p, blocks, s);
    case 2: return launch<T, 2>(p, blocks, s);
    case 3: return launch<T, 3>(p, blocks, s);
    case 4: return launch<T, 4>(p, blocks, s);
    case 5:
    case 6: return launch<T, 6>(p, blocks, s);
    default: return launch<T, 8>(p, blocks, s);
  }
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" int32_t attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
                            int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, int64_t out_stride,
                            const int32_t* plan, int32_t num_seqs, double scale, int32_t dtype,
                            int32_t fill, void* stream) {
  if (!valid_dtype16(dtype)) return ROPE_EUNSUPPORTED;
  if (attn_plan_ints(T, num_seqs, Hq, Hkv) < 0 || !valid_head_size(D)) return ROPE_EINVAL;
  if (!valid_scale(scale)) return ROPE_EINVAL;
  FwdParams p;
  if (!token_stride(q_stride, Hq, D, &p.q_stride) || !token_stride(k_stride, Hkv, D, &p.k_stride) ||
      !token_stride(v_stride, Hkv, D, &p.v_stride) ||
      !token_stride(out_stride, Hq, D, &p.out_stride))
    return ROPE_EINVAL;
  if (T == 0) return ROPE_OK;
  if (!data_pointer(q) || !data_pointer(k) || !data_pointer(v) || !data_pointer(out) ||
      lse == nullptr || !data_pointer(plan))
    return ROPE_EINVAL;
  p.G = Hq / Hkv;
  const int64_t blocks = row_items(T, num_seqs, p.G) * Hkv;
  if (blocks > kMaxBlocks) return ROPE_EINVAL;
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.lse = lse;
  p.plan = plan;
  p.items = reinterpret_cast<const RowItem*>(plan + kHeader);
  p.T = (int32_t)T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.num_seqs = num_seqs;
  p.scale = (float)(scale * kLog2e);
  p.fill = fill;
  p.by_hkv = make_div31(Hkv);
  p.by_g = make_div31(p.G);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == ROPE_BF16 ? launch_size<__bf16>(p, blocks, s)
                            : launch_size<_Float16>(p, blocks, s);
}
