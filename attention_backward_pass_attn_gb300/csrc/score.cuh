// score.cuh -- device side of the changed scores: the cap, the visible range of
// a row, and the TMA copies of strided rows.
//
// The cap.  x = cap tanh(s / cap) for the scaled product s, in base 2.  Near
// zero, |s / cap| <= 0.65 (1.1 in the forward without a maximum), tanh is an odd
// polynomial of five (seven) terms: two scores to an instruction of the FMA pipe.
// Beyond it, tanh(y) = 1 - 2 / (1 + e^2y): an exponential and a reciprocal for
// each score, absolute error some 2^-23 of the cap.  A warp takes the polynomial for a piece of a tile
// whose scores all allow it: models that cap their scores at 30 or 50 have most
// of them well below, and the special function unit is the busier pipe of a
// softmax (figures in score_fwd.cu).  With a cap far above every score the
// polynomial is also the exact one, where 1 - 2 / (1 + e^2y) would lose the
// score in the cap's last bits.
#pragma once

#include "f32x2_arith.cuh"
#include "mask.cuh"
#include "ptx.cuh"
#include "score.h"

namespace attn {

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t f32x2(float x) { return f32x2(x, x); }

// The polynomial's factor: two capped scores in base 2 are u times it.
template <int terms>
__device__ __forceinline__ uint64_t cap_factor(const float (&c)[terms], uint64_t u) {
  const uint64_t z = mul_f32x2(u, u);
  uint64_t h = f32x2(c[terms - 1]);
#pragma unroll
  for (int k = terms - 2; k >= 0; --k) h = fma_f32x2(h, z, f32x2(c[k]));
  return h;
}
__device__ __forceinline__ uint64_t cap_poly(const ScoreMap& m, uint64_t u) {
  return mul_f32x2(u, cap_factor(m.poly, u));
}

// The largest magnitude among a thread's n raw products.
template <int n>
__device__ __forceinline__ float top_of(const uint32_t (&u)[n]) {
  float a[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) a[e] = fabsf(__uint_as_float(u[e]));
#pragma unroll
  for (int e = 4; e < n; e += 2)
    a[(e >> 1) & 3] = max3f(a[(e >> 1) & 3], fabsf(__uint_as_float(u[e])),
                            fabsf(__uint_as_float(u[e + 1])));
  return max3f(a[0], a[1], fmaxf(a[2], a[3]));
}
// Whether a polynomial holds for all of the warp's products.
__device__ __forceinline__ bool all_within(float top, float limit) {
  return __all_sync(0xffffffffu, top <= limit);
}

// 1 / (1 + e^2y) of y = u scale / cap; the capped score is cap_log2 (1 - 2 r).
__device__ __forceinline__ float cap_r(const ScoreMap& m, float u) {
  return rcp_approx(1.f + ex2(u * m.exp_scale));
}

// The row range [lo, hi) of keys that query q sees.  doc: the batch element's
// map or null; prefix: its length or 0.
struct RowMask {
  int N, causal, window;
  const int* doc;
  int prefix;
  __device__ __forceinline__ int lo(int q) const {
    return causal ? first_visible_key(q, doc, window, N) : 0;
  }
  __device__ __forceinline__ int hi(int q) const {
    return causal ? min(N, max(q + 1, prefix)) : N;
  }
};

// Tiled load and L2 prefetch through a 4-D map (head dim, row, head, batch).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int x, int y, int z,
                                                int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

}  // namespace attn
