// attn_scores.h -- what scores may go through before the softmax: a cap by a tanh, and a bias that
// depends on the distance of query and key.
//
// Mathematics: s = scale q.k becomes c tanh(s / c), and then s - slope_h |i - j| with i and j the
// positions of query and key. In base 2, with t = tanh(q.k bend), bend = scale / c, the score is
// t (c log2 e) - (slope_h log2 e) |i - j|: a kernel's q.k is replaced by t, its scale by c log2 e,
// and everything behind it stays as it is. The gradient gets a factor 1 - t^2, from the same t.
//
// What it costs: the vector unit, which the softmax already keeps as busy as the products do the matrix
// unit. A cap takes 8 operations of the full rate a score, beside the softmax's 8 or 9 (the exponential
// counts 4), a bias 4, and a cap whose scores come near it twice that (bend_scores). Eight samples of 256 to
// 2048 tokens, 32 + 8 heads of 128, bf16, kernel times in us (medians on three cards):
//                            forward      dQ           dK and dV
//   nothing                  147 .. 151   214 .. 225   312 .. 327
//   a bias                   163 .. 167   347 .. 351   331 .. 335
//   cap 50, scores of 4      177 .. 186   378 .. 397   381 .. 401
//   cap 50, scores of 10     220 .. 230   448 .. 467   435 .. 447   (of 16: the same)
// dQ walks the keys twice in either form (attn_bwd.hip). A bias keeps the exact distance of each pair: as one
// number a row and a multiple of the slope for each register it would take one operation or two (3 % of the
// forward), but near keys would then be differences of large products.
#pragma once

#include "attn_common.h"
#include "tanh_constants.h"

namespace attn {

enum ScoreMods : int { kBias = 1, kCap = 2 };

// What a kernel compiled with ATTN_MODS of them is given.
struct ScoreParams {
  const float* slopes;  // of each query head
  float bend;           // scale / cap
};

// cap 0: none; else positive, with scale / cap and cap log2 e well within single precision.
inline bool valid_cap(double cap, double scale) {
  return cap == 0.0 || (cap > 0.0 && cap * kLog2e < 1e30 && scale / cap > 1e-30 && scale / cap < 1e30);
}
inline int score_mods(double cap, const float* slopes) {
  return (cap != 0.0 ? kCap : 0) | (slopes != nullptr ? kBias : 0);
}
inline ScoreParams score_params(double scale, double cap, const float* slopes) {
  return {slopes, cap != 0.0 ? (float)(scale / cap) : 0.0f};
}
inline float score_scale(double scale, double cap) {  // of what the softmax sees, in base 2
  return (float)((cap != 0.0 ? cap : scale) * kLog2e);
}

// tanh(y) for |y| up to kTanhNear.
__device__ inline float tanh_near(float y) {
  const float z = y * y;
  float x = kTanhPoly[kTanhDegree];
#pragma unroll
  for (int k = kTanhDegree - 1; k >= 0; --k) x = __builtin_fmaf(x, z, kTanhPoly[k]);
  return y * x;
}

// tanh(s by) of 16 scores, within 2^-22 of it relatively: a polynomial up to kTanhNear (7 operations of
// the full rate, and exact near 0), and where one of the wave's 1024 scores is beyond it, 1 - 2 / (1 + exp(2 y))
// for all of them too (4 more, two of a quarter of the rate, and the choice). A score's result depends on no other's,
// but the time does: blocks with no score past 0.6 of the cap are all of those of normal scores of size 4 under
// a cap of 50, at size 8 some are not, and at size 10 nearly none are left. The bound is what all
// fp32 arguments give here (1.85e-7 at most, at 0.502, and 1.5e-7 beyond 0.75); from exp2 and the reciprocal
// within a step each, which is what their specification says, it would be 2.9e-7 (tanh_constants.h).
__device__ inline void bend_scores(f32x16& s, float by) {
  f32x16 y;
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = s[i] * by;
    most = __builtin_fmaxf(most, __builtin_fabsf(y[i]));
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = tanh_near(y[i]);
  if (__any(most > kTanhNear)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = __builtin_fabsf(y[i]);
      const float e = __builtin_amdgcn_exp2f(a * (float)(2.0 * kLog2e));
      const float t = __builtin_fmaf(__builtin_amdgcn_rcpf(1.0f + e), -2.0f, 1.0f);
      s[i] = a > kTanhNear ? __builtin_copysignf(t, y[i]) : s[i];
    }
  }
}

// key0 - pos as a number, where they are near enough for a key to be seen; no overflow elsewhere.
__device__ inline float distance(int32_t key, int32_t pos) {
  return (float)(int32_t)((uint32_t)key - (uint32_t)pos);
}

}  // namespace attn
