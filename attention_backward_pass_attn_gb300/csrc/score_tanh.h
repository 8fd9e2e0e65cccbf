// score_tanh.h -- the polynomial that takes the place of a tanh near zero:
//
//   tanh(y) = y (c0 + c1 y^2 + ... + c4 y^8),  |y| <= 0.65
//
// with the smallest relative error that five terms reach (1.5e-7, found by
// Remez exchange), some steps of fp32.
#pragma once

namespace attn {

constexpr int kTanhTerms = 5;
constexpr double kTanhReach = 0.65;
constexpr float tanh_poly(int k) {
  constexpr float c[kTanhTerms] = {0.999999846455f, -0.333315001912f, 0.132978737432f,
                                   -0.0515179163995f, 0.0146250854857f};
  return c[k];
}

}  // namespace attn
