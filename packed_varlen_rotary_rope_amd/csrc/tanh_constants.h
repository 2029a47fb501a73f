// Generated by gen_tanh_constants.py -- do not edit. tanh(y) = y sum_i kTanhPoly[i] y^(2 i)
// for |y| <= 1, relative error 9.7e-08 as evaluated in fp32.
#pragma once

namespace attn {

constexpr int kTanhDegree = 7;
constexpr float kTanhPoly[8] = {1.000000000e+00f, -3.333327770e-01f, 1.333213896e-01f, -5.386970565e-02f, 2.146141045e-02f, -7.912484929e-03f, 2.278647618e-03f, -3.523280902e-04f};

}  // namespace attn
