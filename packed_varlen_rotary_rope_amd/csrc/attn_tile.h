// attn_tile.h -- forward attention of one tile: 128 packed query rows (32 for each of the
// four waves of a workgroup) against a range of keys, which the waves share through LDS.
//
// Mathematics: the online softmax. Keys are walked in blocks of BN; a query row keeps its
// running maximum m, the sum l of exp(s - m) and the output O so far, and when m rises, l
// and O are scaled by exp(m_old - m). All of it is fp32, in base 2 (the scale holds log2 e).
// m is let stand while the new maximum is within 2^8 of it, which changes nothing but the
// common factor of O and l, and saves the scaling of O in all but the first few blocks.
//
// Both products are computed transposed, S^T = K Q^T and O^T = V^T P^T: a query row is a
// column of C, held by lanes l and l + 32, so that maximum and sum need one exchange
// between two lanes, scaling is by one register, and P^T is already the B operand of the
// second product (attn_common.h), never written to LDS. V^T is read by transposing LDS
// reads.
#pragma once

#include "attn_common.h"

namespace attn {

__device__ inline float log_sum_exp(float m, float l) {  // from base 2
  return l > 0.0f || l != l ? (m + __builtin_log2f(l)) * 0.693147180559945309f : -__builtin_inff();
}

constexpr float kRescale = 8.0f;  // log2 of how far a maximum may rise before O is scaled
constexpr float kLargeScore = 67108864.0f;  // 2^26, whose half steps are 4: weights up to 2^12

// One row as B operand, a column of the product: chunks past the head size are zeros.
template <typename T, int KS>
__device__ inline void load_row(x8<T> (&f)[KS], const T* row, uint32_t half, uint32_t chunks) {
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const uint32_t c = 2 * s + half;
    const u32x4 w =
        c < chunks ? *reinterpret_cast<const u32x4*>(row + 8 * c) : (u32x4){0, 0, 0, 0};
    f[s] = __builtin_bit_cast(x8<T>, w);
  }
}

// Waits for loaded operands before a loop: at their first use inside it the compiler would
// wait again in every round, for the round's copies into LDS too.
template <typename T, int KS>
__device__ inline void settle(x8<T> (&f)[KS]) {
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    u32x4 w = __builtin_bit_cast(u32x4, f[s]);
    asm volatile("" : "+v"(w));
    f[s] = __builtin_bit_cast(x8<T>, w);
  }
}

// Writes a column of C as a row, 16 bytes a store: lanes l and l + 32 hold quarters of 16
// elements in turn, and exchange them to hold halves.
template <typename T, int DB>
__device__ inline void store_row(const f32x16 (&o)[DB], T* row, uint32_t half, uint32_t chunks,
                                 bool on) {
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int g = 0; g < 2; ++g) {  // columns 32 d + 16 g .. + 15
      const uint32_t a0 = narrow2<T>(o[d][8 * g], o[d][8 * g + 1]);
      const uint32_t a1 = narrow2<T>(o[d][8 * g + 2], o[d][8 * g + 3]);
      const uint32_t b0 = narrow2<T>(o[d][8 * g + 4], o[d][8 * g + 5]);
      const uint32_t b1 = narrow2<T>(o[d][8 * g + 6], o[d][8 * g + 7]);
      const auto x = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
      const auto y = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
      const uint32_t c = 4 * d + 2 * g + half;
      if (on && c < chunks) *reinterpret_cast<u32x4*>(row + 8 * c) = (u32x4){x[0], y[0], x[1], y[1]};
    }
}

// Adds the non-finite values of row j of a tile to this lane's column of C, if it is on.
template <typename T, int DB, int CPR>
__device__ inline void add_nonfinite_row(f32x16 (&o)[DB], const uint8_t* tile, uint32_t j, bool on,
                                         uint32_t half) {
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t e = 32 * d + 8 * (i / 4) + 4 * half + i % 4;
      const T* at = reinterpret_cast<const T*>(tile + j * (CPR * 16) +
                                               (((e >> 3) ^ swizzle<CPR>(j)) << 4)) + (e & 7);
      const float v = (float)*at;
      if (on && !(__builtin_fabsf(v) < __builtin_inff())) o[d][i] += v;
    }
}

// The running state of 32 query rows of a wave, against blocks of BN keys.
template <typename T, int DB, int BN>
struct FwdTile {
  static constexpr int CPR = chunks_per_row(DB);
  static constexpr int KB = BN / 32;
  static constexpr int KS = 2 * DB;  // 16-wide steps over the head size
  static constexpr int kTileBytes = BN * CPR * 16;

  x8<T> q[KS];
  f32x16 o[DB];
  float m, l;  // m in base 2; while `exact` is set, a score as it is
  bool exact;  // read in kCareful mode only: m is subtracted before the scale, without rounding

  bool was_large;  // of the wave: some row's m was large, and has risen since

  static __device__ bool is_large(float m) {
    return __builtin_fabsf(m) > kLargeScore && __builtin_fabsf(m) < __builtin_inff();
  }
  // Whether scores are so large that scale * s - m, with m rounded, may be far from 0 for the
  // largest of them, and its weight beyond the type's range: the walk is done again in kCareful
  // mode with `exact` set, every block of it. Any m counts that the row had: the sums of an earlier
  // one may be infinite, which no later factor takes back.
  __device__ bool large() const { return was_large || is_large(m); }

  __device__ void clear() {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    m = -__builtin_inff();
    l = 0.0f;
    was_large = false;
  }

  // S^T of a block of keys, in KS steps; `piece(t)` is called in step t.
  template <typename P>
  __device__ __attribute__((always_inline)) void scores(f32x16 (&s)[KB], const uint8_t* kt,
                                                        uint32_t lane, P piece) {
    const uint32_t r = lane & 31, half = lane >> 5;
    x8<T> k[KS][KB];
    auto read = [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < KB; ++b) k[t][b] = read_rows<T, CPR>(kt, 32 * b + r, 2 * t + half);
    };
    read(0);
    read(1);
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      step();
      if (t + 2 < KS) read(t + 2);
      piece(t);
#pragma unroll
      for (int b = 0; b < KB; ++b) s[b] = mfma(k[t][b], q[t], s[b]);
    }
    step();
  }

  // Scores to weights, narrowed; m, l and o follow. Keys key0 + j at or behind `seen` (as a
  // count from key 0) are hidden unless kWhole, and those whose bit of `hidden` is set.
  template <Mode MODE>
  __device__ void weights(f32x16 (&s)[KB], x8<T> (&p)[2 * KB], int32_t key0, int32_t seen,
                          uint64_t hidden, float scale, uint32_t lane) {
    const uint32_t half = lane >> 5;
    if constexpr (MODE != kWhole) {
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int32_t j = 32 * b + 8 * (i / 4) + 4 * (int32_t)half + i % 4;
          const uint32_t bits = (uint32_t)(hidden >> (32 * b)) >> (4 * half);
          if (key0 + j >= seen || (bits >> (8 * (i / 4) + i % 4) & 1)) s[b][i] = -__builtin_inff();
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[b][i]);
    const bool as_is = MODE == kCareful && exact;
    top = as_is ? half_max(top) : half_max(top) * scale;
    const bool rises = !((as_is ? (top - m) * scale : top - m) <= kRescale);
    if (__any(rises)) {  // for the rows that need it: a row's bits do not depend on others
      was_large |= __any(rises && is_large(m));
      const float m_new = rises ? __builtin_fmaxf(m, top) : m;
      const float a = m == m_new ? 1.0f : __builtin_amdgcn_exp2f(as_is ? (m - m_new) * scale : m - m_new);
      m = m_new;
      l *= a;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= a;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m;  // a row that saw no key yet
    float sum = 0.0f;
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[b][i] = __builtin_amdgcn_exp2f(as_is ? (s[b][i] - base) * scale
                                               : __builtin_fmaf(s[b][i], scale, -base));
        sum += s[b][i];
      }
    l += sum;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      p[2 * b] = narrow8<T>(s[b], 0);
      p[2 * b + 1] = narrow8<T>(s[b], 1);
    }
  }

  // O^T += V^T P^T.
  template <Mode MODE>
  __device__ void accumulate(const x8<T> (&p)[2 * KB], const uint8_t* vt, int32_t key0, int32_t seen,
                             uint64_t hidden, uint32_t lane) {
    constexpr int N = 2 * KB * DB;  // by step: keys 16 (x / DB) .. + 15, columns 32 (x % DB) .. + 31
    x8<T> v[N];
    auto read = [&](int x) __attribute__((always_inline)) {
      v[x] = read_columns<T, CPR>(vt, 16 * (x / DB), x % DB, lane);
    };
    read(0);
    read(1);
#pragma unroll
    for (int x = 0; x < N; ++x) {
      if (x % 2 == 0) {
        step();
        if (x + 2 < N) read(x + 2);
        if (x + 3 < N) read(x + 3);
      }
      if constexpr (MODE == kCareful) v[x] = cleaned<T>(v[x]);
      o[x % DB] = mfma(v[x], p[x / DB], o[x % DB]);
    }
    step();
    // what is infinite or NaN stays so whatever its weight
    if constexpr (MODE == kCareful)
      for (int32_t j = 0; j < BN; ++j)
        add_nonfinite_row<T, DB, CPR>(o, vt, j, key0 + j < seen && !(hidden >> j & 1), lane >> 5);
  }

  template <Mode MODE, typename P>
  __device__ __attribute__((always_inline)) void block(const uint8_t* kt, const uint8_t* vt,
                                                       int32_t key0, int32_t seen, uint64_t hidden,
                                                       float scale, uint32_t lane, P piece) {
    f32x16 s[KB];
    x8<T> p[2 * KB];
    scores(s, kt, lane, piece);
    weights<MODE>(s, p, key0, seen, hidden, scale, lane);
    accumulate<MODE>(p, vt, key0, seen, hidden, lane);
  }

  // Ends a walk with `exact` set: m in base 2. Returns what its rounding leaves, without which the
  // sums of two walks cannot be joined: half a step of a large m may be any number of powers of 2.
  __device__ float scale_maximum(float scale) {
    const float s = m;
    if (exact) m = s * scale;
    return exact && __builtin_fabsf(m) < __builtin_inff() ? __builtin_fmaf(s, scale, -m) : 0.0f;
  }

  // Normalizes O and returns the row's log-sum-exp.
  __device__ float finish() {
    l = half_sum(l);
    const float r = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] *= r;
    return log_sum_exp(m, l);
  }
};

// The maxima of walks that are joined, each m + low. What the sums at (m, low) are multiplied by
// to stand at (top, top_low); with both infinite, or none seen in either, that is 1.
__device__ inline bool above(float m, float low, float m2, float low2) {
  return m > m2 || (m == m2 && low > low2);
}
__device__ inline float join_factor(float m, float low, float top, float top_low) {
  return m == top && low == top_low ? 1.0f : __builtin_amdgcn_exp2f((m - top) + (low - top_low));
}

// The chunks of a tile's rows that no load fills (head sizes below CPR chunks) are zeroed
// once: products of them with q's zeros must not be NaN.
template <int CPR>
__device__ inline void clear_unused_chunks(uint8_t* tiles, uint32_t rows, uint32_t chunks) {
  if (chunks == CPR) return;
  for (uint32_t i = threadIdx.x; i < rows * CPR; i += blockDim.x) {
    const uint32_t r = i / CPR, c = i % CPR;
    if (c >= chunks)
      *reinterpret_cast<u32x4*>(tiles + r * (CPR * 16) + ((c ^ swizzle<CPR>(r)) << 4)) =
          (u32x4){0, 0, 0, 0};
  }
}

}  // namespace attn
