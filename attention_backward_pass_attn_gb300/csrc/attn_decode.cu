// attn_decode.cu -- attention of one new token per sequence over its pages.
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
//   output) in the workspace; a second kernel joins those of each sequence in
//   the order of their keys, so results repeat bit for bit.
// - The keys of a unit are split over the block's four warps, each with its
//   own running maximum, sum and output, joined in shared memory once per
//   sequence and share.  In the loop warps do not wait for one another.
// - Rows go from global memory straight into the registers that the tensor
//   core instruction wants them in; no shared memory, no barrier.  With
//   mma.m16n8k16 the keys (for S^T = K Q^T) or output columns (for O^T = V^T
//   P^T) are the 16 rows and up to 8 query heads the 8 columns; the order of
//   the contracted index is free as long as both operands use the same one,
//   so a thread's 16-byte load of a K row is four or eight consecutive k
//   indices, and the 2 x 2 transposes of V are byte permutes.  A tile of 128
//   rows in tensor memory (tcgen05.mma) would waste 120 of its 128 rows on
//   absent heads and cost a trip through shared memory.
// - K of the next keys is loaded while the current scores are weighted, V of
//   the next keys while the next scores are formed: 4 to 8 KB in flight per
//   warp, 16 warps per SM.
//
// Rounding.  Scores, maxima, sums and outputs are fp32.  The weights p go to
// the tensor core as a sum of two bf16 numbers, 16 bits in all (2^-16; a
// second instruction that costs nothing here), so the result's only rounding
// that counts is the last one to bf16.  For an e4m3 cache, K is widened to
// fp16 (exact) and meets a q scaled by a power of two into fp16's range
// (exact down to 2^-29 of its largest element); V is widened to bf16 (exact)
// and its factors multiply p in fp32.
#include <cuda_fp16.h>

#include "f32x2.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "serving.h"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLn2 = 0.69314718055994531f;

// D, the cache's type and the number of 8-head column tiles (1 or 2) fix the
// rest: KT runs of 16 keys per warp and step, so that a step's K (and its V)
// is eight 16-byte loads per thread in every case.
template <int D, bool FP8>
struct Cfg {
  static constexpr int kRow = D * (FP8 ? 1 : 2);  // bytes
  static constexpr int KT = 512 / kRow / 2;       // 1, 2, 2, 4
  static constexpr int kUnit = kWarps * KT * 16;  // keys of a unit
  static constexpr int kChunks = kRow / 64;       // 16-byte K loads per row and thread
  static constexpr int kVWords = kRow / 32;       // 32-bit words of V per row and thread
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

// Two e4m3 values (low 16 bits) as fp16, and as bf16; both exact.
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

// Query heads of a key head, cut into blocks of at most kDecodeHeads.
struct HeadSplit {
  int blocks;  // per key head
  int heads;   // per block (the last may have fewer)
};
__host__ __device__ inline HeadSplit split_heads(int group) {
  const int nb = (group + kDecodeHeads - 1) / kDecodeHeads;
  return {nb, (group + nb - 1) / nb};
}

// What the joining kernel needs to know of the split, in the workspace's
// meta section: entry i = the unit block i starts with, {b, head block, unit
// within it, units in it}; a block that starts with unit 0 has nothing to
// join to.  Entry 0 also carries the number of units in all, W.
struct Start {
  int b, h, u, n;
};

// Units of sequence b, and its visible positions.
template <int U>
__device__ __forceinline__ int sequence_units(const DecodeArgs& a, int b, int* lo, int* len) {
  *len = clamp_length(__ldg(a.lens + b), a.c.capacity);
  *lo = first_visible_position(*len, a.window);
  return units_of(*lo, *len, U);
}

template <int D, bool FP8, int NG>
struct Warp {
  using C = Cfg<D, FP8>;
  static constexpr int KT = C::KT;
  const DecodeArgs& a;
  const int lane, r, q;  // r = lane / 4: key or output row; q = lane % 4: column pair
  uint32_t kw[KT * 2 * C::kChunks][4];
  uint32_t vw[KT][4][C::kVWords];
  float kd[FP8 ? KT : 1][2], vd[FP8 ? KT : 1][2];
  uint32_t qf[NG][D / 16][2];
  float factor[NG][2];
  float m[NG][2], l[NG][2];
  float acc[NG][D / 16][4];

  __device__ __forceinline__ Warp(const DecodeArgs& args)
      : a(args), lane(threadIdx.x % 32), r(lane / 4), q(lane % 4) {}

  // q's fragments for heads hq0 .. hq0 + heads - 1 of sequence b, and the
  // running state's start.
  __device__ __forceinline__ void begin(int b, int hq0, int heads) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int head = g * 8 + r;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(a.q) + (int64_t(b) * a.Hq + hq0 + head) * D);
      const bool live = head < heads;
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < C::kChunks; ++c) {
#pragma unroll
        for (int x = 0; x < (FP8 ? 2 : 1); ++x) {
          const uint4 w = live ? src[(4 * c + q) * (FP8 ? 2 : 1) + x] : make_uint4(0, 0, 0, 0);
          const int step = FP8 ? 4 * c + 2 * x : 2 * c;
          qf[g][step][0] = w.x;
          qf[g][step][1] = w.y;
          qf[g][step + 1][0] = w.z;
          qf[g][step + 1][1] = w.w;
        }
      }
      float f = a.scale_log2;
      if (FP8) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float u = fabsf(bf16lo_to_f32(qf[g][s][x]));
            const float v = fabsf(bf16hi_to_f32(qf[g][s][x]));
            if (u < INFINITY) amax = fmaxf(amax, u);
            if (v < INFINITY) amax = fmaxf(amax, v);
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^e puts the largest element into [2^14, 2^15)
        const int e = min(14 - (int(__float_as_uint(amax) >> 23) - 127), 126);
        const float up = __int_as_float((e + 127) << 23);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const __half2 h = __floats2half2_rn(bf16lo_to_f32(qf[g][s][x]) * up,
                                                bf16hi_to_f32(qf[g][s][x]) * up);
            qf[g][s][x] = *reinterpret_cast<const uint32_t*>(&h);
          }
        f *= __int_as_float((127 - e) << 23);
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

  // The cache row of the first key of run `lane` (lanes below KT) of the step
  // at key `tile`; -1 where there is none to read.
  __device__ __forceinline__ int64_t find(const int* table, int kvh, int tile, int len) {
    const int pos = tile + 16 * lane;
    if (lane >= KT || pos >= len) return -1;
    const int pi = int(unsigned(pos) / unsigned(a.c.page_size));
    const int page = __ldg(table + pi);
    if (!page_in_range(page, a.c.num_pages)) {
      report_error(a.err, kDevBadIndex, kSiteDecodePage);
      return -1;
    }
    return cache_row(page, a.c.Hkv, kvh, a.c.page_size, pos - pi * a.c.page_size);
  }

  __device__ __forceinline__ bool sees(int64_t row, int key, int lo, int len) const {
    return row >= 0 && key >= lo && key < len;
  }

  __device__ __forceinline__ void load_k(int64_t rows, int tile, int lo, int len) {
    const uint8_t* cache = static_cast<const uint8_t*>(a.c.kc);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int64_t row = __shfl_sync(0xffffffffu, rows, t);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool ok = sees(row, tile + 16 * t + 8 * x + r, lo, len);
        const int64_t at = row + 8 * x + r;
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) {
          uint32_t(&w)[4] = kw[(2 * t + x) * C::kChunks + c];
          w[0] = w[1] = w[2] = w[3] = 0;
          if (ok) ld_stream(w, cache + at * C::kRow + c * 64 + q * 16);
        }
        if (FP8) {
          kd[t][x] = ok ? __ldg(a.c.kd + at) : 0.f;
          vd[t][x] = ok ? __ldg(a.c.vd + at) : 0.f;
        }
      }
    }
  }

  // Row j of a thread's four: key 2q + (j & 1) + 8 (j >> 1) of the run.
  __device__ __forceinline__ void load_v(int64_t rows, int tile, int lo, int len) {
    const uint8_t* cache = static_cast<const uint8_t*>(a.c.vc);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int64_t row = __shfl_sync(0xffffffffu, rows, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 2 * q + (j & 1) + 8 * (j >> 1);
        const bool ok = sees(row, tile + 16 * t + k, lo, len);
        const uint8_t* p = cache + (row + k) * C::kRow;
        uint32_t(&w)[C::kVWords] = vw[t][j];
#pragma unroll
        for (int i = 0; i < C::kVWords; ++i) w[i] = 0;
        if (ok) {
          if (C::kVWords == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + r * 8));
            w[0] = v.x;
            w[1] = v.y;
          } else {
#pragma unroll
            for (int i = 0; i < C::kVWords / 4; ++i) {
              uint32_t v[4];
              ld_stream(v, p + i * 128 + r * 16);
#pragma unroll
              for (int x = 0; x < 4; ++x) w[4 * i + x] = v[x];
            }
          }
        }
      }
    }
  }

  // S^T of one run of 16 keys.
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

  // Weight the scores of the step's keys: running maximum and sum, rescaled
  // accumulators, and P^T as two bf16 parts in the tensor core's layout.
  __device__ __forceinline__ void weigh(float (&s)[KT][NG][4], int64_t rows, int tile, int lo,
                                        int len, uint32_t (&p)[KT][NG][2][2]) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int64_t row = __shfl_sync(0xffffffffu, rows, t);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool ok = sees(row, tile + 16 * t + 8 * x + r, lo, len);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float& v = s[t][g][2 * x + y];
            const float f = FP8 ? factor[g][y] * kd[t][x] : factor[g][y];
            v = ok ? v * f : -INFINITY;
          }
      }
    }
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
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float w0 = ex2(s[t][g][2 * x] - ref[g][0]), w1 = ex2(s[t][g][2 * x + 1] - ref[g][1]);
          l[g][0] += w0;
          l[g][1] += w1;
          if (FP8) {
            w0 *= vd[t][x];
            w1 *= vd[t][x];
          }
          const uint32_t hi = pack_bf16x2(w0, w1);
          const uint32_t lo2 = pack_bf16x2(w0 - bf16lo_to_f32(hi), w1 - bf16hi_to_f32(hi));
          p[t][g][0][x] = transpose_8x8(hi);
          p[t][g][1][x] = transpose_8x8(lo2);
        }
  }

  // O^T += V^T P^T over the step's keys.  Accumulator i of a thread covers
  // output columns column(i) and the next one.
  __device__ __forceinline__ int column(int i) const {
    return FP8 ? (D / 8) * r + 2 * i : (i / 4) * 64 + 8 * r + 2 * (i % 4);
  }
  __device__ __forceinline__ void add(const uint32_t (&p)[KT][NG][2][2]) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a0, a1, a2, a3;
        if (FP8) {  // columns 2i, 2i + 1 are bytes of word i / 2
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
};

template <int D, bool FP8, int NG>
__global__ void __launch_bounds__(kThreads, NG == 1 ? 3 : 2) decode_kernel(const DecodeArgs a) {
  using C = Cfg<D, FP8>;
  constexpr int U = C::kUnit;
  constexpr int kHeadStride = D + 8;
  __shared__ float sh_o[kWarps][NG * 8][kHeadStride];
  __shared__ float sh_ml[kWarps][NG * 8][2];
  __shared__ int64_t sh_scan[kWarps];
  __shared__ int64_t sh_prefix;
  __shared__ int sh_b;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const HeadSplit split = split_heads(a.Hq / a.c.Hkv);
  const int Hn = a.c.Hkv * split.blocks;  // head blocks of a sequence
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
  const int64_t W = total * Hn;
  const int G = int(W < int64_t(gridDim.x) ? W : int64_t(gridDim.x));

  // Sequences with nothing to see.
  for (int b = blockIdx.x; b < a.c.B; b += gridDim.x) {
    int lo, len;
    if (sequence_units<U>(a, b, &lo, &len)) continue;
    uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + int64_t(b) * a.Hq * D);
    for (int i = tid; i < a.Hq * D / 2; i += kThreads) o[i] = 0;
    for (int i = tid; i < a.Hq; i += kThreads) a.lse[int64_t(b) * a.Hq + i] = -INFINITY;
  }

  Start* starts = reinterpret_cast<Start*>(a.meta);
  if (int(blockIdx.x) >= G) {
    if (tid == 0) starts[blockIdx.x] = {0, 0, 0, 0};
    return;
  }
  const int64_t w0 = split_begin(blockIdx.x, W, G);
  int64_t left = split_begin(blockIdx.x + 1, W, G) - w0;

  // The sequence that holds unit w0: its thread's part holds it.
  {
    const int64_t first = (scan - mine) * Hn;
    if (w0 >= first && w0 < scan * Hn) {
      int64_t prefix = scan - mine;
      int b = b_begin;
      for (;; ++b) {
        int lo, len;
        const int n = sequence_units<U>(a, b, &lo, &len);
        if (w0 < (prefix + n) * Hn) break;
        prefix += n;
      }
      sh_b = b;
      sh_prefix = prefix;
    }
  }
  __syncthreads();
  int b = sh_b, lo, len;
  int n = sequence_units<U>(a, b, &lo, &len);
  int h, u;
  {
    const int64_t x = w0 - sh_prefix * Hn;
    h = int(x / n);
    u = int(x - int64_t(h) * n);
  }
  if (tid == 0) {
    starts[blockIdx.x] = {b, h, u, n};
    if (blockIdx.x == 0) *reinterpret_cast<int64_t*>(starts + kDecodeMaxBlocks) = W;
  }

  Warp<D, FP8, NG> wp(a);
  bool first_segment = true;
  while (true) {
    const int units = int(left < n - u ? left : n - u);
    const int kvh = h / split.blocks, hb = h % split.blocks;
    const int group = a.Hq / a.c.Hkv;
    const int hq0 = kvh * group + hb * split.heads;
    const int heads = min(split.heads, group - hb * split.heads);
    const int* table = a.c.table + int64_t(b) * a.c.max_pages;
    wp.begin(b, hq0, heads);

    int tile = (lo & ~(kPageQuantum - 1)) + u * U + warp * C::KT * 16;
    int64_t rows = wp.find(table, kvh, tile, len);
    wp.load_k(rows, tile, lo, len);
    wp.load_v(rows, tile, lo, len);
    for (int i = 0; i < units; ++i) {
      // past the last step nothing is read: its keys are not below len
      const bool more = i + 1 < units;
      const int next_tile = tile + U;
      const int next_len = more ? len : 0;
      const int64_t next_rows = wp.find(table, kvh, next_tile, next_len);
      float s[C::KT][NG][4];
#pragma unroll
      for (int t = 0; t < C::KT; ++t) wp.scores(t, s[t]);
      uint32_t p[C::KT][NG][2][2];
      wp.weigh(s, rows, tile, lo, len, p);
      wp.load_k(next_rows, next_tile, lo, next_len);
      wp.add(p);
      wp.load_v(next_rows, next_tile, lo, next_len);
      tile = next_tile;
      rows = next_rows;
    }

    // Join the four warps.
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
    const bool whole = u == 0 && units == n;
    const int slot = 2 * blockIdx.x + (first_segment ? 0 : 1);
    for (int i = tid; i < heads * (D / 2); i += kThreads) {
      const int head = i / (D / 2), c = 2 * (i % (D / 2));
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh_ml[w][head][0]);
      const float ref = M == -INFINITY ? 0.f : M;
      float sum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float e = ex2(sh_ml[w][head][0] - ref);
        sum += e * sh_ml[w][head][1];
        o0 += e * sh_o[w][head][c];
        o1 += e * sh_o[w][head][c + 1];
      }
      if (whole) {
        const int64_t out = int64_t(b) * a.Hq + hq0 + head;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + out * D + c) =
            pack_bf16x2(o0 * inv, o1 * inv);
        if (c == 0) a.lse[out] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
      } else {
        const int64_t at = int64_t(slot) * kDecodeHeads + head;
        *reinterpret_cast<float2*>(a.part_o + at * D + c) = make_float2(o0, o1);
        if (c == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(M, sum);
      }
    }

    left -= units;
    if (left == 0) break;
    __syncthreads();  // the shared tiles are free again
    first_segment = false;
    u = 0;
    if (++h == Hn) {
      h = 0;
      do n = sequence_units<U>(a, ++b, &lo, &len);
      while (n == 0);
    }
  }
}

// Joins the parts of every head block that more than one block worked on.
// Grid block (j, head): if block j of the split began inside a head block,
// and is the first to do so there, its predecessor holds that head block's
// first part, and the parts up to the owner of its last unit are joined.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const DecodeArgs a) {
  constexpr int kCols = D / 4;            // threads across the output
  constexpr int kLanes = 256 / kCols;     // parts added at once
  __shared__ float4 sh[kLanes][kCols];
  grid_dep_wait();
  grid_dep_launch();
  const Start* starts = reinterpret_cast<const Start*>(a.meta);
  const int j = blockIdx.x + 1;
  const int4 st = __ldg(reinterpret_cast<const int4*>(starts + j));
  const Start s = {st.x, st.y, st.z, st.w};
  if (s.u == 0) return;
  const int64_t W = *reinterpret_cast<const int64_t*>(starts + kDecodeMaxBlocks);
  const int blocks = gridDim.x + 1;
  const int G = int(W < blocks ? W : blocks);
  const int64_t begin = split_begin(j, W, G) - s.u;
  const int i0 = split_owner(begin, W, G);
  if (i0 != j - 1) return;
  const int i1 = split_owner(begin + s.n - 1, W, G);
  const int group = a.Hq / a.c.Hkv;
  const HeadSplit split = split_heads(group);
  const int hb = s.h % split.blocks;
  const int head = blockIdx.y;
  if (head >= min(split.heads, group - hb * split.heads)) return;

  // part k: block i0 + k; its first piece of work, except that the first
  // block may have come to this head block after another one
  const int parts = i1 - i0 + 1;
  const int slot0 = 2 * i0 + (split_begin(i0, W, G) < begin ? 1 : 0);
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  auto at = [&](int k) {
    return int64_t(k == 0 ? slot0 : 2 * (i0 + k)) * kDecodeHeads + head;
  };
  const int lane = threadIdx.x % 32;
  float M = -INFINITY;
  for (int k = lane; k < parts; k += 32) M = fmaxf(M, ml[at(k)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
  float sum = 0.f;
  for (int k = lane; k < parts; k += 32) {
    const float2 x = ml[at(k)];
    sum += ex2(x.x - ref) * x.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);

  const int col = threadIdx.x % kCols, part = threadIdx.x / kCols;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = part; k < parts; k += kLanes) {
    const float e = ex2(ml[at(k)].x - ref);
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + at(k) * D + col * 4);
    acc.x += e * x.x;
    acc.y += e * x.y;
    acc.z += e * x.z;
    acc.w += e * x.w;
  }
  sh[part][col] = acc;
  __syncthreads();
  if (part) return;
#pragma unroll
  for (int k = 1; k < kLanes; ++k) {
    const float4 x = sh[k][col];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  const int64_t out = int64_t(s.b) * a.Hq + (s.h / split.blocks) * group + hb * split.heads + head;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + out * D + col * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (col == 0) a.lse[out] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
}

template <int D, bool FP8, int NG>
cudaError_t launch(const DecodeArgs& a, int heads, cudaStream_t stream) {
  using C = Cfg<D, FP8>;
  constexpr int kPerSm = NG == 1 ? 3 : 2;  // resident blocks: see __launch_bounds__
  // at most as many blocks as there can be units
  const HeadSplit split = split_heads(a.Hq / a.c.Hkv);
  const int seen = a.window > 0 && a.window < a.c.capacity ? a.window : a.c.capacity;
  const int64_t units = int64_t(a.c.B) * a.c.Hkv * split.blocks * (seen / C::kUnit + 2);
  int64_t grid = int64_t(device_sm_count()) * kPerSm;
  if (grid > kDecodeMaxBlocks) grid = kDecodeMaxBlocks;
  if (grid > units) grid = units;
  cudaError_t e = launch_kernel(decode_kernel<D, FP8, NG>, dim3(unsigned(grid)), dim3(kThreads), 0,
                                stream, a);
  if (e != cudaSuccess || grid == 1) return e;
  return launch_kernel(join_kernel<D>, dim3(unsigned(grid - 1), unsigned(heads)), dim3(256), 0,
                       stream, a);
}

template <int D, bool FP8>
cudaError_t launch_heads(const DecodeArgs& a, cudaStream_t stream) {
  const int heads = split_heads(a.Hq / a.c.Hkv).heads;
  return heads <= 8 ? launch<D, FP8, 1>(a, heads, stream) : launch<D, FP8, 2>(a, heads, stream);
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream) {
  if (a.c.d == 64)
    return a.c.kd ? launch_heads<64, true>(a, stream) : launch_heads<64, false>(a, stream);
  return a.c.kd ? launch_heads<128, true>(a, stream) : launch_heads<128, false>(a, stream);
}

}  // namespace attn
