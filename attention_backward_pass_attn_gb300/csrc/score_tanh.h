// score_tanh.h -- the polynomial that takes the place of a tanh near zero:
//
//   tanh(y) = y (c0 + c1 y^2 + c2 y^4 + ...)
//
// with the smallest relative error that so many terms reach, found by Remez
// exchange: five on |y| <= 0.65 and seven on |y| <= 1.1, 1.5e-7 either, two
// steps of fp32.
#pragma once

namespace attn {

constexpr int kTanhTerms = 5;
constexpr double kTanhReach = 0.65;
constexpr float tanh_poly(int k) {
  constexpr float c[kTanhTerms] = {0.999999846455f, -0.333315001912f, 0.132978737432f,
                                   -0.0515179163995f, 0.0146250854857f};
  return c[k];
}

constexpr int kTanhFarTerms = 7;
constexpr double kTanhFarReach = 1.1;
constexpr float tanh_far_poly(int k) {
  constexpr float c[kTanhFarTerms] = {0.999999849936f,   -0.333320982935f, 0.133164473669f,
                                      -0.053082114204f,  0.0195696885187f, -0.00556908130395f,
                                      0.000832431544264f};
  return c[k];
}

}  // namespace attn
