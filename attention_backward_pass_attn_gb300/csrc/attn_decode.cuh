// attn_decode.cuh -- attention of one new token per sequence over its pages: the
// kernel, instantiated in attn_decode.cu (bf16 and e4m3 caches),
// attn_decode_int4.cu and attn_decode_score.cu (changed scores).
//
//   s_j = scale <q, k_j>,  o = sum_j softmax(s)_j v_j,  l = logsumexp(s)
//
// over the visible positions j.  Bound by HBM: each cached row is read once,
// for all query heads that share it, and 4 d FLOPs per head and key are far
// below the tensor cores' rate at that speed.  So the kernel is built to keep
// loads in flight and to need few instructions per byte:
//
// - Work is cut into units of 64 to 256 keys of one (sequence, key head) and
//   dealt out in contiguous, even shares to one wave of thread blocks,
//   whatever the lengths of the sequences: every block reads the same number
//   of bytes and all end together.  A share that begins or ends inside a
//   sequence leaves a partial result (running maximum, sum, unnormalised
//   output) in the workspace, and the last of a sequence's blocks to arrive
//   joins them, in the order of their keys: results repeat bit for bit.
// - The keys of a unit are split over the block's four warps, each with its
//   own running maximum, sum and output, joined in shared memory once per
//   sequence and share.  In the loop warps do not wait for one another.
// - Rows go from global memory straight into the registers that the tensor
//   core instruction wants them in; no shared memory, no barrier.  With
//   mma.m16n8k16 the keys (for S^T = K Q^T) or output columns (for O^T = V^T
//   P^T) are the 16 rows and up to 8 query heads the 8 columns; the order of
//   the contracted index is free as long as both operands use the same one,
//   so a thread's 16-byte load of a K row is four or eight consecutive k
//   indices, and the 2 x 2 transposes of V are byte permutes.  128 keys (or
//   output columns) would fill a tile of tcgen05.mma as well, but its operands
//   lie in shared memory and its results in tensor memory: two trips more for
//   every row in a kernel that HBM bounds, whose tensor pipe is 12 to 21 % busy.
// - K of the next keys is loaded while the current scores are weighted, V of
//   the next keys while the next scores are formed: 4 to 8 KB in flight per
//   warp, 12 warps per SM.
//
// Measured (one call among others in a graph): 131,072 positions, 8 key heads
// x 4, d=128, bf16: 84 us, 6.4 TB/s, of which the walk over the keys is 76; 32
// sequences of up to 8,192, 8 key heads x 8, e4m3: 52 us for 264 MB; 500
// positions of 16 heads: 7.2 us, 2.7 of them from the arrivals on.  256
// sequences of up to 256, 8 key heads x 4, bound by the changes of sequence:
// e4m3 32 us for 67 MB, bf16 37 us for 131 MB.  With 16 heads to a key head (two
// blocks to an SM) 16 sequences of up to 8,192, 2 key heads, take 21 us for 31 MB
// in e4m3 and 22 us for 60 MB in bf16, bound by latency (issue slots 24 to 30 %,
// DRAM 16 to 31 %): eight warps an SM hide less than twelve, and 16 heads of
// partial output are written, read back and joined where there were 8.
//
// A 4-bit cache (int4.cuh) is bound by instructions, not by HBM: the 131,072
// positions above take 43 us for 151 MB (e4m3: 50 for 277), 345 warp instructions
// for 16 keys, of which 144 make bf16 numbers of nibbles (a mask and a
// multiply-add a pair, a shift for four) for the tensor core's 24; issue slots
// 49 %, ALU 41 %.  (With the pairs of int4_pair, four instructions each, 46 us.)
// Sixteen warps to an SM were slower (58 us), as they are with bf16.
//
// Changed scores (a cap, a bias) cost 1 to 3 % with bf16 and e4m3, 9 to 13 % with
// 4-bit rows.
//
// Rounding.  Scores, maxima, sums and outputs are fp32.  The weights p (times
// V's factor of an e4m3 row) meet V as a sum of two bf16 numbers, 16 bits in
// all (2^-16), so the result's only rounding that counts is the last one to
// bf16.  The second instruction costs nothing with a bf16 cache and 2 % with
// an e4m3 one, where one fp16 number would do if the factors were known to be
// of similar size.  An e4m3 K is widened to fp16 (exact) and meets a q scaled by
// a power of two into fp16's range, where that is exact too: where the head's
// nonzero elements lie within 31 binades.  Where they do not, K is widened to
// bf16 (exact) and meets q's own numbers, scaled clear of overflow: exact down
// to 2^-222 of the head's largest element.  fp16 is the faster of the two, one
// conversion for a pair of keys' values where bf16 takes four.  V is widened to
// bf16 (exact).  The choice is made for a run of keys at a time: every head in
// bf16 takes the batch above to 56 us, telling the two apart costs it 0.5 %, and
// 1.5 % of the 256 short sequences.  A choice for every product took 58 us.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "f32x2.cuh"
#include "int4.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "score_tanh.h"
#include "serving.h"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLn2 = 0.69314718055994531f;

// How many binades below a head's largest element, scaled into [2^14, 2^15),
// fp16 holds all 8 bits of a bf16 number: those of 2^-17 end at 2^-24.
constexpr uint32_t kFp16Span = 31;

// D, the cache's type (CacheType) and the number of 8-head column tiles (1 or
// 2) fix the rest: KT runs of 16 keys per warp and step, so that a step's K
// (and its V) is eight 16-byte loads per thread.  A 4-bit row takes half the
// runs that would make: its step, 690 instructions for two runs, is bound by
// them, and with four (of 840 for two, then) the loop no longer fitted the
// instruction caches (131,072 positions, 8 key heads x 4, d=128: 67 us in place
// of 51).
template <int D, int TYPE>
struct Cfg {
  static constexpr int kRow = TYPE == kCacheInt4 ? D / 2 : TYPE == kCacheE4m3 ? D : 2 * D;  // bytes
  static constexpr int KT = TYPE == kCacheInt4 ? 2 : 256 / kRow;  // 1, 2, 2, 4, 2, 2
  static constexpr int kUnit = kWarps * KT * 16;                  // keys of a unit
  static constexpr int kWords = kRow / 16;  // 32-bit words of K per row and thread,
  static constexpr int kChunks = kWords < 4 ? 1 : kWords / 4;  // in this many loads
  static constexpr int kVWords = kRow / 32;  // 32-bit words of V per row and thread
};

__device__ __forceinline__ void ld_stream(uint32_t (&r)[4], const uint8_t* p) {
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "l"(p));
}

// D[16 x 8] += A[16 x 16] B[16 x 8], fp32 accumulators.
template <bool F16>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held one row of two columns
// per thread (row = lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two e4m3 values (low 16 bits) as fp16 and as bf16; both exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
  return h;
}
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Magnitudes of two bf16 numbers compare as integers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t add_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Reduction over the lanes that hold different keys of the same head.
__device__ __forceinline__ float keys_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float keys_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// The blocks that share a head block count their arrivals in a word of the
// workspace: the call's tag (48 bits) and the count.  open_count, which every
// one of them runs before its work, makes the word the call's own: what an
// earlier call or another owner left there has another tag, and the first to
// replace it wins.  arrive is true for the last of `parts`, which leaves the
// count at zero for a replay of the same launch.  One addition per block: a
// compare-and-swap loop here cost 30 us where 57 blocks end together.
__device__ __forceinline__ void fence_acq_rel_gpu() {
  asm volatile("fence.acq_rel.gpu;" ::: "memory");
}
__device__ __forceinline__ void open_count(unsigned long long* word, unsigned long long tag) {
  const unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(word);
  if ((old >> 16) != tag) atomicCAS(word, old, tag << 16);
}
__device__ __forceinline__ bool arrive(unsigned long long* word, unsigned long long tag,
                                       int parts) {
  const unsigned long long old = atomicAdd(word, 1ull);
  const bool last = int(old & 0xFFFFull) + 1 == parts;
  if (last) atomicExch(word, tag << 16);
  return last;
}

// A head block that this block has a part of.
struct SharedPiece : Piece {
  int heads;
  int64_t out;  // its first output row
};

// A run of units of one head block, and where it stands.  Kept in shared
// memory while the keys are walked, whose loop needs the registers.
struct Work {
  int64_t left;        // units of the block's share from this run's first on
  int64_t first_unit;  // the head block's first unit among all units
  int b, h, u, n;      // sequence, head block, first unit of the run, units of the head block
  int lo, len;         // visible positions of the sequence
  __device__ __forceinline__ int units() const { return int(left < n - u ? left : n - u); }
};

// Units of sequence b, and its visible positions.
template <int U>
__device__ __forceinline__ int sequence_units(const DecodeArgs& a, int b, int* lo, int* len) {
  *len = clamp_length(__ldg(a.lens + b), a.c.capacity);
  *lo = first_visible_position(*len, a.window);
  return units_of(*lo, *len, U);
}

template <int D, int TYPE, int NG, bool MOD>
struct Warp {
  using C = Cfg<D, TYPE>;
  static constexpr bool FP8 = TYPE == kCacheE4m3, INT4 = TYPE == kCacheInt4;
  static constexpr int KT = C::KT;
  const DecodeArgs& a;
  const int lane, r, q;  // r = lane / 4: key or output row; q = lane % 4: column pair
  uint32_t kw[KT * 2 * C::kChunks][4];
  uint32_t vw[KT][4][C::kVWords];
  float kd[FP8 ? KT : 1][2], vd[FP8 ? KT : 1][2];
  // INT4: factors, as bf16, of the thread's group of two K rows and four V rows
  uint16_t kf[INT4 ? KT : 1][2], vf[INT4 ? KT : 1][4];
  bool wide;  // FP8: q is held in bf16, see kFp16Span; INT4: factors of any size
  uint32_t seen;  // INT4: two largest factors less kInt4LowFactor, wrapped, as bf16 bits
  uint32_t qf[NG][D / 16][2];
  float factor[NG][2];
  float slope[MOD ? NG : 1][2];  // of distance, base 2
  float m[NG][2], l[NG][2];
  float acc[NG][D / 16][4];

  __device__ __forceinline__ Warp(const DecodeArgs& args)
      : a(args), lane(threadIdx.x % 32), r(lane / 4), q(lane % 4) {}

  // q's fragments for heads hq0 .. hq0 + heads - 1 of sequence b, as they lie.
  __device__ __forceinline__ void load_q(int b, int hq0, int heads) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int head = g * 8 + r;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(a.q) + (int64_t(b) * a.Hq + hq0 + head) * D);
      const bool live = head < heads;
      if (MOD && a.score.slopes) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
          slope[g][y] = g * 8 + 2 * q + y < heads
                            ? __ldg(a.score.slopes + hq0 + g * 8 + 2 * q + y) * 1.4426950408889634f
                            : 0.f;
      }
      if constexpr (INT4) {  // elements p and p + 4 of eight, as int4_pair takes them
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint4 x = live ? __ldg(src + (D / 32) * q + w) : make_uint4(0, 0, 0, 0);
          qf[g][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);
          qf[g][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);
          qf[g][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);
          qf[g][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);
        }
      } else {
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
          for (int x = 0; x < (FP8 ? 2 : 1); ++x) {
            const uint4 w =
                live ? __ldg(src + (4 * c + q) * (FP8 ? 2 : 1) + x) : make_uint4(0, 0, 0, 0);
            const int step = FP8 ? 4 * c + 2 * x : 2 * c;
            qf[g][step][0] = w.x;
            qf[g][step][1] = w.y;
            qf[g][step + 1][0] = w.z;
            qf[g][step + 1][1] = w.w;
          }
      }
    }
  }

  // The running state's start; q in the products' type, and what turns a
  // product into a score.
  __device__ __forceinline__ void begin(bool any_factor) {
    uint32_t top[NG];
    wide = INT4 && any_factor;
    seen = 0;
    if (FP8) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        // Largest finite and smallest nonzero magnitude, as bf16 bits, two at a
        // time, the latter less one: a zero becomes the largest number.
        // Infinities and NaN, which would sort above, are rare and sorted out
        // apart.
        uint32_t hi = 0, lo = 0xFFFFFFFFu;
#pragma unroll
        for (int s = 0; s < D / 8; ++s) {
          const uint32_t w = qf[g][s / 2][s % 2] & 0x7FFF7FFFu;
          hi = max_u16x2(hi, w);
          lo = min_u16x2(lo, add_u16x2(w, 0xFFFFFFFFu));
        }
        if (((hi & 0xFFFFu) >= 0x7F80u) | (hi >= 0x7F800000u)) {
          hi = 0;
#pragma unroll
          for (int s = 0; s < D / 8; ++s) {
            const uint32_t w = qf[g][s / 2][s % 2] & 0x7FFF7FFFu;
            hi = max_u16x2(hi, ((w & 0xFFFFu) < 0x7F80u ? w & 0xFFFFu : 0u) |
                                   (w < 0x7F800000u ? w & 0xFFFF0000u : 0u));
          }
        }
        hi = max_u16x2(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
        hi = max_u16x2(hi, __shfl_xor_sync(0xffffffffu, hi, 2));
        top[g] = max(hi & 0xFFFFu, hi >> 16) >> 7;
        lo = min(lo & 0xFFFFu, lo >> 16) >> 7;
        wide |= top[g] > lo + kFp16Span;
      }
      wide = __any_sync(0xffffffffu, wide);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float f = a.scale_log2;
      if (INT4 && !wide) f *= kInt4Up;  // K's values come times 2^-16
      if (FP8) {
        // 2^e puts the largest element into [2^14, 2^15) for fp16, into
        // [2^96, 2^97) where bf16 has to hold the row.
        const int e = min((wide ? 96 : 14) + 127 - int(top[g]), 126);
        const uint32_t up = uint32_t(e + 127) * 0x00800080u;  // as two bf16
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t w = mul_bf16x2(qf[g][s][x], up);
            qf[g][s][x] = wide ? w : pack_f16x2(bf16lo_to_f32(w), bf16hi_to_f32(w));
          }
        f *= pow2f(-e);
      }
      // the lane of head 2q (+1) holds that column's factor
      factor[g][0] = __shfl_sync(0xffffffffu, f, 8 * q);
      factor[g][1] = __shfl_sync(0xffffffffu, f, 8 * q + 4);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[g][x] = -INFINITY;
        l[g][x] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[g][i][x] = 0.f;
    }
  }

  // The cache row of the first key of run lane % KT of the step at key `tile`,
  // or of the last run below len; -1 on a bad page.
  __device__ __forceinline__ int64_t find(const int* table, int kvh, int tile, int len) {
    const int pos = min(tile + 16 * (lane % KT), (len - 1) & ~(kPageQuantum - 1));
    const int pi = int(fast_div(pos, a.c.page_div));
    const int page = __ldg(table + pi);
    if (!page_in_range(page, a.c.num_pages)) {
      report_error(a.err, kDevBadIndex, kSiteDecodePage);
      return -1;
    }
    return cache_row(page, a.c.Hkv, kvh, a.c.page_size, pos - pi * a.c.page_size);
  }

  // Whether every key of the step is visible and its pages are good.
  __device__ __forceinline__ bool full(int64_t rows, int tile, int lo, int len) const {
    return tile >= lo && tile + 16 * KT <= len && __all_sync(0xffffffffu, rows >= 0);
  }
  __device__ __forceinline__ static bool sees(int64_t row, int key, int lo, int len) {
    return row >= 0 && key >= lo && key < len;
  }

  // The loads of a step have no conditions: a run that is only partly visible
  // is read whole (it lies on one page), one past the length reads the last
  // run again, one on a bad page row 0, and what must not count is masked
  // where it is used.  A branch here made the registers that wait for the
  // loads meet at its end, and the loop wait with them (the e4m3 batch above:
  // 62 us became 76).
  __device__ __forceinline__ void load_k(int64_t rows) {
    const uint8_t* cache = static_cast<const uint8_t*>(a.c.kc);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int64_t row = __shfl_sync(0xffffffffu, rows < 0 ? 0 : rows, t) + r;
      const uint8_t* base = cache + row * C::kRow + q * (C::kWords < 4 ? 8 : 16);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (C::kWords < 4) {
          uint32_t(&w)[4] = kw[2 * t + x];
          asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.b32 {%0, %1}, [%2];"
                       : "=r"(w[0]), "=r"(w[1])
                       : "l"(base + x * 8 * C::kRow));
        } else {
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            ld_stream(kw[(2 * t + x) * C::kChunks + c], base + x * 8 * C::kRow + c * 64);
        }
        if constexpr (INT4)
          kf[t][x] = __ldg(a.c.kf + (row + 8 * x) * (D / kInt4Group) + (D / 4) * q / kInt4Group);
        if (FP8) {
          kd[t][x] = __ldg(a.c.kd + row + 8 * x);
          vd[t][x] = __ldg(a.c.vd + row + 8 * x);
        }
      }
    }
  }

  // Row j of a thread's four: key 2q + (j & 1) + 8 (j >> 1) of the run.
  __device__ __forceinline__ void load_v(int64_t rows) {
    const uint8_t* cache = static_cast<const uint8_t*>(a.c.vc);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int64_t row = __shfl_sync(0xffffffffu, rows < 0 ? 0 : rows, t) + 2 * q;
      const uint8_t* base = cache + row * C::kRow + r * (C::kVWords < 4 ? 4 * C::kVWords : 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* p = base + ((j & 1) + 8 * (j >> 1)) * C::kRow;
        uint32_t(&w)[C::kVWords] = vw[t][j];
        if constexpr (INT4)
          vf[t][j] = __ldg(a.c.vf + (row + (j & 1) + 8 * (j >> 1)) * (D / kInt4Group) +
                           (D / 8) * r / kInt4Group);
        if (C::kVWords == 1) {
          asm volatile("ld.global.nc.L1::no_allocate.L2::256B.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
        } else if (C::kVWords == 2) {
          asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.b32 {%0, %1}, [%2];"
                       : "=r"(w[0]), "=r"(w[C::kVWords - 1])
                       : "l"(p));
        } else {
#pragma unroll
          for (int i = 0; i < C::kVWords; i += 4)
            asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[(i + 2) % C::kVWords]),
                           "=r"(w[(i + 3) % C::kVWords])
                         : "l"(p + i * 32));
        }
      }
    }
  }

  // Of a step that is not full: scores of what is not visible become -inf,
  // V's rows there zero, or their factors 1 (they may hold anything, NaN
  // included).
  __device__ __forceinline__ void mask(float (&s)[KT][NG][4], int64_t rows, int tile, int lo,
                                       int len) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int64_t row = __shfl_sync(0xffffffffu, rows, t);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (sees(row, tile + 16 * t + 8 * x + r, lo, len)) continue;
        if (FP8) vd[t][x] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) s[t][g][2 * x] = s[t][g][2 * x + 1] = -INFINITY;
      }
    }
  }
  // INT4: what is not visible has factors of 1 in K too, before they are noted:
  // an unwritten row's, zero or NaN, would have the run walked a second time.
  __device__ __forceinline__ void mask_k(int64_t rows, int tile, int lo, int len) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int64_t row = __shfl_sync(0xffffffffu, rows, t);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (!sees(row, tile + 16 * t + 8 * x + r, lo, len)) kf[t][x] = 0x3F80;
    }
  }
  __device__ __forceinline__ void mask_v(int64_t rows, int tile, int lo, int len) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int64_t row = __shfl_sync(0xffffffffu, rows, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sees(row, tile + 16 * t + 2 * q + (j & 1) + 8 * (j >> 1), lo, len)) continue;
        if constexpr (INT4) {
          vf[t][j] = 0x3F80;  // 1: values of weight 0, finite
        } else {
#pragma unroll
          for (int i = 0; i < C::kVWords; ++i) vw[t][j][i] = 0;
        }
      }
    }
  }

  // S^T of one run of 16 keys.
  template <bool WIDE>
  __device__ __forceinline__ void scores_int4(int t, float (&s)[NG][4]) {
#pragma unroll
    for (int g = 0; g < NG; ++g) s[g][0] = s[g][1] = s[g][2] = s[g][3] = 0.f;
    const Int4Factor f0 = int4_factor(kf[t][0] * 0x00010001u),
                     f1 = int4_factor(kf[t][1] * 0x00010001u);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint32_t x = kw[2 * t][w], y = kw[2 * t + 1][w];
#pragma unroll
      for (int p = 0; p < 4; p += 2) {
        const uint32_t a0 = int4_value<WIDE>(x, p, f0), a2 = int4_value<WIDE>(x, p + 1, f0);
        const uint32_t a1 = int4_value<WIDE>(y, p, f1), a3 = int4_value<WIDE>(y, p + 1, f1);
#pragma unroll
        for (int g = 0; g < NG; ++g)
          mma_16x8x16<false>(s[g], a0, a1, a2, a3, qf[g][2 * w + p / 2][0],
                             qf[g][2 * w + p / 2][1]);
      }
    }
  }
  template <bool WIDE>
  __device__ __forceinline__ void scores(int t, float (&s)[NG][4]) {
#pragma unroll
    for (int g = 0; g < NG; ++g) s[g][0] = s[g][1] = s[g][2] = s[g][3] = 0.f;
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c) {
      const uint32_t(&x)[4] = kw[(2 * t) * C::kChunks + c];
      const uint32_t(&y)[4] = kw[(2 * t + 1) * C::kChunks + c];
      if (FP8) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (WIDE) {
            const uint32_t a0 = e4m3x2_to_bf16x2(x[w]), a2 = e4m3x2_to_bf16x2(x[w] >> 16);
            const uint32_t a1 = e4m3x2_to_bf16x2(y[w]), a3 = e4m3x2_to_bf16x2(y[w] >> 16);
#pragma unroll
            for (int g = 0; g < NG; ++g)
              mma_16x8x16<false>(s[g], a0, a1, a2, a3, qf[g][4 * c + w][0], qf[g][4 * c + w][1]);
            continue;
          }
          const uint32_t a0 = e4m3x2_to_f16x2(x[w]), a2 = e4m3x2_to_f16x2(x[w] >> 16);
          const uint32_t a1 = e4m3x2_to_f16x2(y[w]), a3 = e4m3x2_to_f16x2(y[w] >> 16);
#pragma unroll
          for (int g = 0; g < NG; ++g)
            mma_16x8x16<true>(s[g], a0, a1, a2, a3, qf[g][4 * c + w][0], qf[g][4 * c + w][1]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int g = 0; g < NG; ++g)
            mma_16x8x16<false>(s[g], x[2 * w], y[2 * w], x[2 * w + 1], y[2 * w + 1],
                               qf[g][2 * c + w][0], qf[g][2 * c + w][1]);
      }
    }
  }

  // Scores in base 2 capped by a tanh, and less the bias of their distance
  // from the newest position (see score.cuh and score_tanh.h; here a step's
  // scores take the polynomial when the warp's are all near zero, else both
  // ways, each score its own).
  __device__ __forceinline__ void change(float (&s)[KT][NG][4], int tile, int len) {
    if (a.score.cap_log2 > 0.f) {
      float top = 0.f;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int g = 0; g < NG; ++g)
          top = max3f(max3f(top, fabsf(s[t][g][0]), fabsf(s[t][g][1])), fabsf(s[t][g][2]),
                      fabsf(s[t][g][3]));
      const bool far = __any_sync(0xffffffffu, !(top <= a.score.reach));
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float u = s[t][g][x], y = u * a.score.inv_cap_log2, z = y * y;
            float h = tanh_poly(kTanhTerms - 1);
#pragma unroll
            for (int k = kTanhTerms - 2; k >= 0; --k) h = fmaf(h, z, tanh_poly(k));
            float v = u * h;
            if (far && !(fabsf(u) <= a.score.reach)) {
              float e;  // 1 / (1 + e^2y)
              asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(1.f + ex2(u * a.score.exp_scale)));
              v = fmaf(e, -2.f * a.score.cap_log2, a.score.cap_log2);
            }
            s[t][g][x] = v;
          }
    }
    if (a.score.slopes) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float dist = float(len - 1 - (tile + 16 * t + 8 * x + r));
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            s[t][g][2 * x] = fmaf(-slope[g][0], dist, s[t][g][2 * x]);
            s[t][g][2 * x + 1] = fmaf(-slope[g][1], dist, s[t][g][2 * x + 1]);
          }
        }
    }
  }

  // Weight the scores of the step's keys: running maximum and sum, rescaled
  // accumulators, and P^T as two bf16 parts in the tensor core's layout.
  template <bool WIDE>
  __device__ __forceinline__ void weigh(float (&s)[KT][NG][4], bool full, int64_t rows, int tile,
                                        int lo, int len, uint32_t (&p)[KT][NG][2][2]) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          s[t][g][x] *= FP8 ? factor[g][x & 1] * kd[t][x / 2] : factor[g][x & 1];
    if (MOD) change(s, tile, len);
    if (!full) mask(s, rows, tile, lo, len);
    bool grown = false;
    float ref[NG][2], alpha[NG][2];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float mx = -INFINITY;
#pragma unroll
        for (int t = 0; t < KT; ++t) mx = max3f(mx, s[t][g][y], s[t][g][2 + y]);
        mx = fmaxf(m[g][y], keys_max(mx));
        ref[g][y] = mx == -INFINITY ? 0.f : mx;
        alpha[g][y] = ex2(m[g][y] - ref[g][y]);
        grown |= mx != m[g][y];
        m[g][y] = mx;
      }
    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        l[g][0] *= alpha[g][0];
        l[g][1] *= alpha[g][1];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[g][i][x] *= alpha[g][x & 1];
      }
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float w0 = ex2(s[t][g][2 * x] - ref[g][0]), w1 = ex2(s[t][g][2 * x + 1] - ref[g][1]);
          l[g][0] += w0;
          l[g][1] += w1;
          if (INT4 && !WIDE) {
            w0 *= kInt4Up;
            w1 *= kInt4Up;
          }
          if (FP8) {
            w0 *= vd[t][x];
            w1 *= vd[t][x];
          }
          const uint32_t hi = pack_bf16x2(w0, w1);
          p[t][g][0][x] = transpose_8x8(hi);
          p[t][g][1][x] =
              transpose_8x8(pack_bf16x2(w0 - bf16lo_to_f32(hi), w1 - bf16hi_to_f32(hi)));
        }
      }
  }

  // INT4: the walk with int4_pair_down takes note of every visible factor, and the
  // run is walked once more with int4_pair if one of them was outside its range,
  // which takes the warp's run twice its time (131,072 positions whose last run
  // has such a factor: 61 us in place of 43).  (A
  // choice for every step took 131,072 positions from 41 us to 46: its branches
  // part the loads from their use.)
  template <int runs, int n>
  __device__ __forceinline__ void note(const uint16_t (&f)[runs][n]) {
#pragma unroll
    for (int t = 0; t < runs; ++t)
#pragma unroll
      for (int j = 0; j < n; j += 2)
        seen = max_u16x2(seen, add_u16x2(f[t][j] | uint32_t(f[t][j + 1]) << 16,
                                         (0x10000u - kInt4LowFactor) * 0x00010001u));
  }
  __device__ __forceinline__ bool out_of_range() const {
    return __any_sync(0xffffffffu, max(seen & 0xFFFFu, seen >> 16) >= kInt4Factors);
  }
  // One of int4.cuh's two forms of a pair.
  template <bool WIDE>
  __device__ __forceinline__ static uint32_t int4_value(uint32_t w, int p, const Int4Factor& f) {
    return WIDE ? int4_pair(w, p, f.f) : int4_pair_down(w, p, f);
  }

  // One step's keys; MORE: with the loads of the next step's among it.
  template <bool MORE, bool WIDE>
  __device__ __forceinline__ void step(int64_t rows, bool full, int tile, int lo, int len,
                                       int64_t next_rows) {
    float s[KT][NG][4];
    if constexpr (INT4 && !WIDE) {
      if (!full) mask_k(rows, tile, lo, len);
      note(kf);
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      if constexpr (INT4)
        scores_int4<WIDE>(t, s[t]);
      else
        scores<WIDE>(t, s[t]);
    }
    uint32_t p[KT][NG][2][2];
    weigh<WIDE>(s, full, rows, tile, lo, len, p);
    if (MORE) load_k(next_rows);
    if (!full) mask_v(rows, tile, lo, len);
    if constexpr (INT4 && !WIDE) note(vf);
    add<WIDE>(p);
    if (MORE) load_v(next_rows);
  }

  // O^T += V^T P^T over the step's keys.  Accumulator i of a thread covers
  // output columns column(i) and the next one.
  __device__ __forceinline__ int column(int i) const {
    return FP8 || INT4 ? (D / 8) * r + 2 * i : (i / 4) * 64 + 8 * r + 2 * (i % 4);
  }
  template <bool WIDE>
  __device__ __forceinline__ void add(const uint32_t (&p)[KT][NG][2][2]) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      // INT4: factors of keys 2q, 2q + 1, and of those eight further
      Int4Factor f0, f1;
      if constexpr (INT4) {
        f0 = int4_factor(vf[t][0] | uint32_t(vf[t][1]) << 16);
        f1 = int4_factor(vf[t][2] | uint32_t(vf[t][3]) << 16);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a0, a1, a2, a3;
        if constexpr (INT4) {  // columns 2i, 2i + 1 are byte i % 4 of word i / 4
          const uint32_t sel = i & 2 ? 0x7632u : 0x5410u;
          const uint32_t u = __byte_perm(vw[t][0][i / 4], vw[t][1][i / 4], sel);
          const uint32_t v = __byte_perm(vw[t][2][i / 4], vw[t][3][i / 4], sel);
          a0 = int4_value<WIDE>(u, 2 * (i & 1), f0);
          a1 = int4_value<WIDE>(u, 2 * (i & 1) + 1, f0);
          a2 = int4_value<WIDE>(v, 2 * (i & 1), f1);
          a3 = int4_value<WIDE>(v, 2 * (i & 1) + 1, f1);
        } else if (FP8) {  // columns 2i, 2i + 1 are bytes of word i / 2
          const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
          const uint32_t u = __byte_perm(vw[t][0][i / 2], vw[t][1][i / 2], sel);
          const uint32_t v = __byte_perm(vw[t][2][i / 2], vw[t][3][i / 2], sel);
          a0 = e4m3x2_to_bf16x2(u);
          a1 = e4m3x2_to_bf16x2(u >> 16);
          a2 = e4m3x2_to_bf16x2(v);
          a3 = e4m3x2_to_bf16x2(v >> 16);
        } else {
          a0 = __byte_perm(vw[t][0][i], vw[t][1][i], 0x5410);
          a1 = __byte_perm(vw[t][0][i], vw[t][1][i], 0x7632);
          a2 = __byte_perm(vw[t][2][i], vw[t][3][i], 0x5410);
          a3 = __byte_perm(vw[t][2][i], vw[t][3][i], 0x7632);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            mma_16x8x16<false>(acc[g][i], a0, a1, a2, a3, p[t][g][x][0], p[t][g][x][1]);
      }
    }
  }
};

// Joining the parts of a head block, all threads of the block together.  With
// four warps on the SM and nothing to hide them, what counts is how many reads
// follow one another: all heads' maxima and sums are one, then IT x KP rows of
// every thread.  w: the weights, kDecodeHeads x kPartsStride of shared memory.
// `out` < 0: the result is a part of the second step, in slot ps.slot0, its
// maximum and sum in an array of their own.
constexpr int kPartsStride = 40;  // a multiple of 8
static_assert(kPartsStride >= max_join_parts(kDecodeMaxBlocks), "room for the parts of one join");

__device__ __forceinline__ void join_weights(const DecodeArgs& a, const Parts& ps, int heads,
                                             int64_t out, float* w) {
  constexpr int kLanes = kThreads / kDecodeHeads, kEach = kPartsStride / kLanes;
  const float2* ml = reinterpret_cast<const float2*>(ps.stride == 1 ? a.part_ml : a.part_ml2);
  const int head = min(int(threadIdx.x) / kLanes, heads - 1), lane = threadIdx.x % kLanes;
  const int last = ps.parts - 1;
  float2 x[kEach];
  float M = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    x[i] = __ldcg(ml + ps.slot(min(lane + kLanes * i, last)) * kDecodeHeads + head);
#pragma unroll
  for (int i = 0; i < kEach; ++i) M = fmaxf(M, x[i].x);
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
  const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    // What does not count is told by its index, not by its weight: a part whose
    // scores are all NaN has no maximum, weight 0, and a sum that must show.
    const bool counts = lane + kLanes * i <= last;
    x[i].x = counts ? ex2(x[i].x - ref) : 0.f;
    sum += counts ? x[i].x * x[i].y : 0.f;
  }
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  const float unit = out < 0 ? 1.f : (sum == 0.f ? 0.f : 1.f / sum);
#pragma unroll
  for (int i = 0; i < kEach; ++i) w[head * kPartsStride + lane + kLanes * i] = x[i].x * unit;
  if (lane == 0) {
    if (out >= 0)
      a.lse[out + head] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    else
      reinterpret_cast<float2*>(a.part_ml2)[ps.slot0 * kDecodeHeads + head] = make_float2(M, sum);
  }
}

template <int D, int IT, int KP>
__device__ __forceinline__ void join_rows(const DecodeArgs& a, const Parts& ps, int heads,
                                          int64_t out, float* w) {
  const int items = heads * (D / 4), last = ps.parts - 1;
  float4 v[KP][IT];
  auto load = [&](int i0, int k0) {
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const float* src = a.part_o + ps.slot(min(k0 + j, last)) * (kDecodeHeads * D);
#pragma unroll
      for (int n = 0; n < IT; ++n)
        v[j][n] = __ldcg(reinterpret_cast<const float4*>(src) + min(i0 + n * kThreads, items - 1));
    }
  };
  load(threadIdx.x, 0);  // ahead of the weights, which need a read of their own
  join_weights(a, ps, heads, out, w);
  __syncthreads();
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < items; i0 += IT * kThreads) {
    float4 acc[IT];
#pragma unroll
    for (int n = 0; n < IT; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 <= last; k0 += KP) {
      if (k0 || i0 >= kThreads) load(i0, k0);
#pragma unroll
      for (int j = 0; j < KP; ++j)  // parts past the last have weight 0
#pragma unroll
        for (int n = 0; n < IT; ++n) {
          const float e = w[min(i0 + n * kThreads, items - 1) / (D / 4) * kPartsStride + k0 + j];
          acc[n].x += e * v[j][n].x;
          acc[n].y += e * v[j][n].y;
          acc[n].z += e * v[j][n].z;
          acc[n].w += e * v[j][n].w;
        }
    }
#pragma unroll
    for (int n = 0; n < IT; ++n) {
      const int i = i0 + n * kThreads;
      if (i >= items) continue;
      if (out >= 0)
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + out * D)[i] =
            make_uint2(pack_bf16x2(acc[n].x, acc[n].y), pack_bf16x2(acc[n].z, acc[n].w));
      else
        reinterpret_cast<float4*>(a.part_o + ps.slot0 * (kDecodeHeads * D))[i] = acc[n];
    }
  }
}

template <int D>
__device__ __forceinline__ void join_parts(const DecodeArgs& a, const Parts& ps, int heads,
                                           int64_t out, float* w) {
  if (heads * (D / 4) <= kThreads)
    join_rows<D, 1, 20>(a, ps, heads, out, w);
  else
    join_rows<D, 4, 8>(a, ps, heads, out, w);
  __syncthreads();
}

template <int D, int TYPE, int NG, bool MOD>
__global__ void __launch_bounds__(kThreads, NG == 1 ? 3 : 2) decode_kernel(const DecodeArgs a) {
  using C = Cfg<D, TYPE>;
  constexpr int U = C::kUnit;
  constexpr int kHeadStride = D + 8;
  __shared__ __align__(16) float sh_o[kWarps][NG * 8][kHeadStride];
  __shared__ __align__(8) float sh_ml[kWarps][NG * 8][2];
  static_assert(kWarps == 4, "the joins below take four warps' results");
  __shared__ int64_t sh_scan[kWarps];
  __shared__ int64_t sh_W;
  __shared__ Work sh_work[2];
  __shared__ bool sh_last[2];
  __shared__ SharedPiece sh_piece[2];

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  grid_dep_wait();
  grid_dep_launch();

  // Units of all sequences: each thread counts a contiguous part of the
  // batch, then a scan over the block.
  const int per = (a.c.B + kThreads - 1) / kThreads;
  const int b_begin = min(tid * per, a.c.B), b_end = min(b_begin + per, a.c.B);
  int64_t mine = 0;
  for (int b = b_begin; b < b_end; ++b) {
    int lo, len;
    mine += sequence_units<U>(a, b, &lo, &len);
    if (blockIdx.x == 0 && __ldg(a.lens + b) != len)
      report_error(a.err, kDevBadIndex, kSiteLength);
  }
  int64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += x;
  }
  if (lane == 31) sh_scan[warp] = scan;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) scan += sh_scan[w];
    total += sh_scan[w];
  }
  const int64_t W = total * a.head_blocks;
  const int G = int(W < int64_t(gridDim.x) ? W : int64_t(gridDim.x));

  // Sequences with nothing to see.
  for (int b = blockIdx.x; b < a.c.B; b += gridDim.x) {
    int lo, len;
    if (sequence_units<U>(a, b, &lo, &len)) continue;
    uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + int64_t(b) * a.Hq * D);
    for (int64_t i = tid; i < int64_t(a.Hq) * (D / 2); i += kThreads) o[i] = 0;
    for (int i = tid; i < a.Hq; i += kThreads) a.lse[int64_t(b) * a.Hq + i] = -INFINITY;
  }

  if (int(blockIdx.x) >= G) return;

  // The sequence that holds the share's first unit: its thread's part of the
  // batch holds it.
  {
    const int64_t w0 = split_begin(blockIdx.x, W, G);
    if (w0 >= (scan - mine) * a.head_blocks && w0 < scan * a.head_blocks) {
      Work w;
      int64_t prefix = scan - mine;
      for (w.b = b_begin;; ++w.b) {
        w.n = sequence_units<U>(a, w.b, &w.lo, &w.len);
        if (w0 < (prefix + w.n) * a.head_blocks) break;
        prefix += w.n;
      }
      const int64_t x = w0 - prefix * a.head_blocks;
      w.h = int(x / w.n);
      w.u = int(x - int64_t(w.h) * w.n);
      w.first_unit = w0 - w.u;
      w.left = split_begin(blockIdx.x + 1, W, G) - w0;
      sh_work[0] = w;
      sh_W = W;
    }
  }
  __syncthreads();

  Warp<D, TYPE, NG, MOD> wp(a);
  int64_t rows;
  // A run's first loads.
  auto key_head = [&](int h) { return int(fast_div(h, a.block_div)); };
  auto heads_of = [&](int h) {
    return min(a.block_heads, a.group - (h - key_head(h) * a.group_blocks) * a.block_heads);
  };
  auto first_head = [&](int h) {
    return key_head(h) * a.group + (h - key_head(h) * a.group_blocks) * a.block_heads;
  };
  auto first_tile = [&](const Work& w) {
    return (w.lo & ~(kPageQuantum - 1)) + w.u * U + warp * C::KT * 16;
  };
  auto enter = [&](const Work& w) {
    rows = wp.find(a.c.table + int64_t(w.b) * a.c.max_pages, key_head(w.h), first_tile(w),
                   w.len);
    wp.load_q(w.b, first_head(w.h), heads_of(w.h));
    wp.load_k(rows);
    wp.load_v(rows);
  };
  enter(sh_work[0]);
  int pieces = 0;
  for (int turn = 0;; ++turn) {
    {
      const Work w = sh_work[turn & 1];
      const int units = w.units();
      if (tid == 0 && units != w.n) {
        const int64_t W = sh_W;
        const int G = int(W < int64_t(gridDim.x) ? W : int64_t(gridDim.x));
        const SharedPiece pc = {split_piece(w.first_unit, w.n, W, G), heads_of(w.h),
                                int64_t(w.b) * a.Hq + first_head(w.h)};
        sh_piece[pieces] = pc;
        open_count(a.arrivals + pc.group(blockIdx.x).slot0, a.tag);
        if (!pc.direct()) open_count(a.arrivals2 + pc.slot0, a.tag);
      }
      // (2^16 times the scale must be finite)
      wp.begin(a.scale_log2 > 1e33f);
      const int* table = a.c.table + int64_t(w.b) * a.c.max_pages;
      const int kvh = key_head(w.h);
      auto walk = [&](auto wide) {
        constexpr bool kWide = decltype(wide)::value;
        int tile = first_tile(w);
        bool full = wp.full(rows, tile, w.lo, w.len);
        // The last step stands apart: it has nothing to load.
        for (int i = 1; i < units; ++i) {
          const int64_t next_rows = wp.find(table, kvh, tile + U, w.len);
          wp.template step<true, kWide>(rows, full, tile, w.lo, w.len, next_rows);
          tile += U;
          rows = next_rows;
          full = wp.full(rows, tile, w.lo, w.len);
        }
        // ... and a warp past the end of a sequence no keys
        if (tile < w.len) wp.template step<false, kWide>(rows, full, tile, w.lo, w.len, 0);
      };
      // The bf16 walk is the branch not expected: laid out the other way, its
      // instructions cost an e4m3 call of 18 us (caches cold) 6 us more, not 2.
      for (;;) {
        if (TYPE == kCacheBf16 || __builtin_expect(!wp.wide, 1)) {
          walk(std::false_type());
          if (TYPE != kCacheInt4 || __builtin_expect(!wp.out_of_range(), 1)) break;
          enter(w);
          wp.begin(true);
        } else {
          walk(std::true_type());
          break;
        }
      }
    }

    // The run's results leave the registers; the next run's first loads are
    // under way while they are joined.
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int head = g * 8 + 2 * wp.q + y;
        const float sum = keys_sum(wp.l[g][y]);
        if (wp.r == 0) {
          sh_ml[warp][head][0] = wp.m[g][y];
          sh_ml[warp][head][1] = sum;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(&sh_o[warp][head][wp.column(i)]) =
              make_float2(wp.acc[g][i][y], wp.acc[g][i][2 + y]);
      }
    __syncthreads();
    const volatile Work& seen = sh_work[turn & 1];
    const int units = int(seen.left < seen.n - seen.u ? seen.left : seen.n - seen.u);
    const bool whole = units == seen.n, more = seen.left > units;
    if (more) {
      Work w;
      w.left = seen.left - units;
      w.first_unit = seen.first_unit + seen.n;
      w.u = 0;
      w.b = seen.b;
      w.h = seen.h + 1;
      w.n = seen.n;
      w.lo = seen.lo;
      w.len = seen.len;
      if (w.h == a.head_blocks) {
        w.h = 0;
        do w.n = sequence_units<U>(a, ++w.b, &w.lo, &w.len);
        while (w.n == 0);
      }
      if (tid == 0) sh_work[(turn & 1) ^ 1] = w;
      enter(w);
    }
    const int heads = heads_of(seen.h);
    const int64_t out = int64_t(seen.b) * a.Hq + first_head(seen.h);
    const int slot = part_slot(blockIdx.x, turn);
    for (int i = tid; i < heads * (D / 4); i += kThreads) {
      const int head = i / (D / 4), c = 4 * (i % (D / 4));
      float2 ml[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ml[w] = *reinterpret_cast<float2*>(sh_ml[w][head]);
      const float M = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
      const float ref = M == -INFINITY ? 0.f : M;
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float e = ex2(ml[w].x - ref);
        const float4 v = *reinterpret_cast<const float4*>(&sh_o[w][head][c]);
        sum += e * ml[w].y;
        o.x += e * v.x;
        o.y += e * v.y;
        o.z += e * v.z;
        o.w += e * v.w;
      }
      if (whole) {
        const int64_t row = out + head;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * D + c) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (c == 0) a.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
      } else {
        const int64_t at = int64_t(slot) * kDecodeHeads + head;
        *reinterpret_cast<float4*>(a.part_o + at * D + c) = o;
        if (c == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(M, sum);
      }
    }
    if (!whole) ++pieces;  // at most twice: a share's first and last head block
    __syncthreads();       // the shared tiles are free again, the parts are written
    if (!more) break;
  }

  // Both pieces' arrivals at once, after one fence; then the second step of
  // those that take two.
  bool waits = tid < pieces;  // this thread has an arrival to make
#pragma unroll 1
  for (int step = 0; pieces; ++step) {
    if (tid < 2) {
      bool last = false;
      if (waits) {
        const SharedPiece pc = sh_piece[tid];
        fence_acq_rel_gpu();
        last = step ? arrive(a.arrivals2 + pc.slot0, a.tag, pc.groups().parts)
                    : arrive(a.arrivals + pc.group(blockIdx.x).slot0, a.tag,
                             pc.group(blockIdx.x).parts);
        fence_acq_rel_gpu();
        waits = last && step == 0 && !pc.direct();
      }
      sh_last[tid] = last;
    }
    __syncthreads();
    bool again = false;
#pragma unroll 1
    for (int x = 0; x < pieces; ++x) {
      if (!sh_last[x]) continue;
      const SharedPiece pc = sh_piece[x];
      const bool whole = step || pc.direct();
      again |= !whole;
      join_parts<D>(a, step ? pc.groups() : pc.group(blockIdx.x), pc.heads, whole ? pc.out : -1,
                    &sh_o[0][0][0]);
    }
    if (!again) break;
  }
}

template <int D, int TYPE, int NG, bool MOD>
cudaError_t launch(const DecodeArgs& a, cudaStream_t stream) {
  using C = Cfg<D, TYPE>;
  constexpr int kPerSm = NG == 1 ? 3 : 2;  // resident blocks: see __launch_bounds__
  // at most as many blocks as there can be units
  const int seen = a.window > 0 && a.window < a.c.capacity ? a.window : a.c.capacity;
  const int64_t units = int64_t(a.c.B) * a.head_blocks * (seen / C::kUnit + 2);
  int64_t grid = int64_t(device_sm_count()) * kPerSm;
  if (grid > kDecodeMaxBlocks) grid = kDecodeMaxBlocks;
  if (grid > units) grid = units;
  return launch_kernel(decode_kernel<D, TYPE, NG, MOD>, dim3(unsigned(grid)), dim3(kThreads), 0,
                       stream, a);
}

template <int TYPE, bool MOD>
cudaError_t launch_type(const DecodeArgs& a, cudaStream_t stream) {
  if (a.c.d == 64)
    return a.block_heads <= 8 ? launch<64, TYPE, 1, MOD>(a, stream)
                              : launch<64, TYPE, 2, MOD>(a, stream);
  return a.block_heads <= 8 ? launch<128, TYPE, 1, MOD>(a, stream)
                            : launch<128, TYPE, 2, MOD>(a, stream);
}

}  // namespace
}  // namespace attn
