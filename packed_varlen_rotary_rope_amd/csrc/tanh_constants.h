// Generated by gen_tanh_constants.py -- do not edit. tanh(y) = y sum_i kTanhPoly[i] y^(2 i)
// for |y| <= kTanhNear, relative error 1.5e-07 as evaluated in fp32; beyond it 1 - 2 / (1 + exp(2 |y|)),
// 1.9e-07 with exp2 and the reciprocal rounded to nearest, 2.9e-07 with either off by a step.
#pragma once

namespace attn {

constexpr float kTanhNear = 6.000000238e-01f;
constexpr int kTanhDegree = 4;
constexpr float kTanhPoly[5] = {9.999999404e-01f, -3.333230317e-01f, 1.331006438e-01f, -5.209665373e-02f, 1.546875108e-02f};

}  // namespace attn
