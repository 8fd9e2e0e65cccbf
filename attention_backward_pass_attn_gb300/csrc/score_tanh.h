// score_tanh.h -- the polynomial that takes the place of a tanh near zero:
//
//   tanh(y) = y (c0 + c1 y^2 + ... + c5 y^10),  |y| <= 0.8
//
// with the smallest relative error that six terms reach (5.8e-8, found by
// Remez exchange), as small as fp32's own steps.
#pragma once

namespace attn {

constexpr int kTanhTerms = 6;
constexpr double kTanhReach = 0.8;
constexpr float tanh_poly(int k) {
  constexpr float c[kTanhTerms] = {0.999999942083f,   -0.333326749194f, 0.133210482804f,
                                   -0.0531143154981f, 0.0190933004507f, -0.0043552995703f};
  return c[k];
}

}  // namespace attn
