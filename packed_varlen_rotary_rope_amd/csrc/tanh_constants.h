// Generated by gen_tanh_constants.py -- do not edit. tanh(y) = y sum_i kTanhPoly[i] y^(2 i)
// for |y| <= kTanhNear, relative error 1.5e-07 as evaluated in fp32.
#pragma once

namespace attn {

constexpr float kTanhNear = 8.000000119e-01f;
constexpr int kTanhDegree = 5;
constexpr float kTanhPoly[6] = {9.999999404e-01f, -3.333266675e-01f, 1.332093179e-01f, -5.310926959e-02f, 1.908435300e-02f, -4.349738825e-03f};

}  // namespace attn
