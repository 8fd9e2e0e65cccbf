// rope.cu -- rotary positions on one to four axes, and their gradient.
//
// Pair i of a head row is (x[i], x[i + d/2]), or its neighbours (x[2i],
// x[2i+1]); it turns by theta = pos[axis(i)] * inv_freq[i]:
//
//   y_a = x_a cos(theta) - x_b sin(theta),  y_b = x_b cos(theta) + x_a sin(theta)
//
// The gradient is the inverse turn, theta -> -theta, so one kernel serves
// both.  Bound by HBM: every value is read and written once (4 bytes a
// value), with 3 FLOPs a value.  Video's 16,384 tokens of 32 heads, d=128, out
// of a fused projection: 46 us (5.9 TB/s).
//
// The angle.  pos * inv_freq in fp32 would be off by pos * inv_freq * 2^-24
// radians, 0.06 at position 10^6.  What matters is the angle modulo one turn,
// so each pair's frequency is written as a 64-bit fraction of a turn,
// F = inv_freq / (2 pi) * 2^64 mod 2^64, from the 24-bit integer and the
// exponent of inv_freq (integer arithmetic, no FP64, whose rate on this chip
// is two operations per clock and SM), and pos * F mod 2^64 is the turn:
// an error of at most (|pos| inv_freq + |pos|) * 2^-64 turns.  Its upper 32
// bits are a quarter turn and a remainder of at most an eighth, x <= pi / 4 in
// radians, whose sine and cosine are Taylor's polynomials to x^9 and x^8: off
// by x^11 / 11! < 2^-29 and x^10 / 10! < 2^-25.
//
// A block turns its frequencies into fractions once, takes a tile of tokens (a
// thread owns 8 pairs, two 16-byte pieces, of one of them), forms their sines
// and cosines once and runs over a group of heads of q and k with them.  Blocks
// that follow one another take tiles that follow one another of the same
// heads, so that the GPU moves through memory in order: 32,768 tokens of 32
// heads, d=128, take 85 us (6.3 TB/s, 93 % of a copy).  Blocks that walk all
// heads of their tile took 91; sincospif and a fraction per thread 87.
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"
#include "serving.h"

namespace attn {
namespace {

constexpr int kThreads = 64;
constexpr int kPairs = 8;  // per thread
constexpr int kBlocksPerSm = 20;  // resident
constexpr int kHeadsPerBlock = 8;  // fewer where that leaves the GPU idle

// floor(2^64 / (2 pi)): the turn of one radian.
constexpr uint64_t kTurnPerRadian = 0x28BE60DB9391054Aull;

// inv_freq / (2 pi) as a fraction of a turn, times 2^64 (mod 2^64).
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int e = int((bits >> 23) & 0xFF);
  const uint64_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int shift = 150 - (e ? e : 1);  // f = +-m 2^-shift
  const uint64_t lo = m * kTurnPerRadian, hi = __umul64hi(m, kTurnPerRadian);
  uint64_t r;
  if (shift >= 128) r = 0;
  else if (shift >= 64) r = hi >> (shift - 64);
  else if (shift > 0) r = (hi << (64 - shift)) | (lo >> shift);
  else r = shift > -64 ? lo << -shift : 0;
  return (bits >> 31) ? 0ull - r : r;
}

// Sine and cosine of turn / 2^32 of a turn.
__device__ __forceinline__ void sin_cos_of_turn(uint32_t turn, float* s, float* c) {
  constexpr float kRadians = 1.46291807926715968e-9f;  // 2 pi / 2^32
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = float(int32_t(turn - (quarter << 30))) * kRadians, x2 = x * x;
  float p = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
  p = fmaf(p, x2, 1.f / 120.f);
  p = fmaf(p, x2, -1.f / 6.f);
  const float sn = fmaf(p * x2, x, x);
  float q = fmaf(x2, 1.f / 40320.f, -1.f / 720.f);
  q = fmaf(q, x2, 1.f / 24.f);
  q = fmaf(q, x2, -0.5f);
  const float cs = fmaf(q, x2, 1.f);
  // a quarter turn on: (s, c) -> (c, -s)
  const float a = quarter & 1 ? cs : sn, b = quarter & 1 ? sn : cs;
  *s = __uint_as_float(__float_as_uint(a) ^ (quarter & 2) << 30);
  *c = __uint_as_float(__float_as_uint(b) ^ ((quarter + 1) & 2) << 30);
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) rope_kernel(const RopeArgs a,
                                                                      int head_group) {
  constexpr int kPerToken = D / 2 / kPairs;  // threads of a token
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint64_t fraction[D / 2];
  static_assert(kThreads >= D / 2, "a thread for every frequency");
  if (threadIdx.x < D / 2) fraction[threadIdx.x] = turn_fraction(__ldg(a.inv_freq + threadIdx.x));
  __syncthreads();
  const int64_t token = int64_t(blockIdx.x) * (kThreads / kPerToken) + threadIdx.x / kPerToken;
  if (token >= int64_t(a.B) * a.N) return;
  const int part = threadIdx.x % kPerToken;
  const int b = int(fast_div(unsigned(token), a.N_div)), n = int(token) - b * a.N;

  float c[kPairs], s[kPairs];
  {
    const int* pp = a.pos + b * a.pos_batch + n;
    int p[kMaxAxes];
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) p[x] = x < a.axes ? __ldg(pp + x * a.pos_axis) : 0;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int i = part * kPairs + j;
      const int at = i < a.axis_end[0] ? p[0] : i < a.axis_end[1] ? p[1]
                     : i < a.axis_end[2] ? p[2] : p[3];
      const uint64_t turn = uint64_t(int64_t(at)) * fraction[i];
      sin_cos_of_turn(uint32_t(turn >> 32), &s[j], &c[j]);
      if (a.backward) s[j] = -s[j];
    }
  }

  const int off0 = INTERLEAVED ? part * 2 * kPairs : part * kPairs;
  const int off1 = INTERLEAVED ? off0 + 8 : off0 + D / 2;
  const int first = blockIdx.y * head_group;
  const int last = min(first + head_group, a.heads[0] + a.heads[1]);
#pragma unroll 4
  for (int h = first; h < last; ++h) {
    const int w = h >= a.heads[0];
    const int hh = w ? h - a.heads[0] : h;
    const uint16_t* x = static_cast<const uint16_t*>(a.x[w]) + b * a.sb[w] + hh * a.sh[w] +
                        n * a.sn[w];
    uint16_t* y = static_cast<uint16_t*>(a.y[w]) + ((int64_t(b) * a.heads[w] + hh) * a.N + n) * D;
    const uint4 u = *reinterpret_cast<const uint4*>(x + off0);
    const uint4 v = *reinterpret_cast<const uint4*>(x + off1);
    const uint32_t ui[4] = {u.x, u.y, u.z, u.w}, vi[4] = {v.x, v.y, v.z, v.w};
    uint32_t uo[4], vo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (INTERLEAVED) {  // word k of u is pair k, of v pair 4 + k
        const float a0 = bf16lo_to_f32(ui[k]), b0 = bf16hi_to_f32(ui[k]);
        const float a1 = bf16lo_to_f32(vi[k]), b1 = bf16hi_to_f32(vi[k]);
        uo[k] = pack_bf16x2(a0 * c[k] - b0 * s[k], b0 * c[k] + a0 * s[k]);
        vo[k] = pack_bf16x2(a1 * c[4 + k] - b1 * s[4 + k], b1 * c[4 + k] + a1 * s[4 + k]);
      } else {  // word k holds halves of pairs 2k and 2k + 1
        const float a0 = bf16lo_to_f32(ui[k]), a1 = bf16hi_to_f32(ui[k]);
        const float b0 = bf16lo_to_f32(vi[k]), b1 = bf16hi_to_f32(vi[k]);
        uo[k] = pack_bf16x2(a0 * c[2 * k] - b0 * s[2 * k], a1 * c[2 * k + 1] - b1 * s[2 * k + 1]);
        vo[k] = pack_bf16x2(b0 * c[2 * k] + a0 * s[2 * k], b1 * c[2 * k + 1] + a1 * s[2 * k + 1]);
      }
    }
    st_global_v4(y + off0, uo[0], uo[1], uo[2], uo[3]);
    st_global_v4(y + off1, vo[0], vo[1], vo[2], vo[3]);
  }
}

template <int D, bool INTERLEAVED>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  constexpr int kTokens = kThreads / (D / 2 / kPairs);
  const int64_t tiles = (int64_t(a.B) * a.N + kTokens - 1) / kTokens;
  const int64_t heads = int64_t(a.heads[0]) + a.heads[1];
  // Eight heads share a thread's sines; with few tokens, fewer, down to one,
  // until every SM has six blocks (4,094 tokens of 32 heads, d=64: 7.5 us with
  // eight, 9.2 with four; 800 tokens of 40 heads, d=128: 5.1 us with eight, 4.5
  // with four).
  int64_t group = kHeadsPerBlock;
  while (group > 1 && tiles * ((heads + group - 1) / group) < 6 * int64_t(device_sm_count()))
    group /= 2;
  group = std::max(group, (heads + 65534) / 65535);
  return launch_kernel(rope_kernel<D, INTERLEAVED>,
                       dim3(unsigned(tiles), unsigned((heads + group - 1) / group)),
                       dim3(kThreads), 0, stream, a, int(group));
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.d == 64) return a.interleaved ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
  return a.interleaved ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
}

}  // namespace attn
