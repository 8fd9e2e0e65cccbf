// kv_cache_int4.cu -- the paged key/value cache in four bits (int4.cuh), as it is
// written and as it is read back.
//
// Of a group of 32 values, amax its largest finite magnitude:
//
//   f = amax / 7 rounded to five significant bits, ties to even; at least
//       2^-120; 1 where amax = 0; NaN where the group holds a NaN
//   c = round(x / f), ties to even, clamped to -7 .. 7
//
// f is within 1/33 of amax / 7, so the largest value still rounds to 7 and no
// finite one is clamped.  Both roundings are of the exact quotient.  amax / 7
// is a fp32 division, whose result is a tie of five bits only if the quotient
// is (a quotient of a bf16 number by 7 that is not one lies at least 2^-12 of
// itself away).  x / f, a division for every value, is a product with the
// reciprocal and Markstein's correction (P. Markstein, 1990: with r = 1 / f
// rounded to nearest and q = x r, q + r (x - q f) is the quotient rounded to
// nearest), which ties need: x r alone misses 7.5 by a last bit.  Adding
// 1.5 2^23 + 8 rounds it to a whole number, ties to even, and leaves c + 8 in
// the low bits; eight of them join by multiplications.
//
// A value that is read back, c f, is a bf16 number: no rounding at all.
//
// A written row is read once (2 d bytes) and written once (d / 2 and d / 16 of
// factors); reading back is the reverse.  Reading is at a copy's speed (32,768
// rows of 16 heads, 20,480 of them held, d=128: 49 us, 6.5 TB/s); writing issues
// in 70 % of all slots and reaches 5.2 TB/s (a padded batch of 4 x 8,192 tokens
// of 16 heads, mean of three sets of lengths: 42 us).
#include "f32x2_arith.cuh"
#include "int4.cuh"
#include "kv_rows.cuh"

namespace attn {
namespace {

// Largest magnitude of a lane's eight values as bf16 bits.
__device__ __forceinline__ uint32_t amax8(const uint4& x) {
  const uint32_t m = max_u16x2(max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                               max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

// Two bf16 values without infinities and NaN, which are rare: those become the
// largest finite number (clamped, later, to +-7) and zero.  *nan is set if
// there was one, and *top is the largest magnitude of the finite ones.
__device__ __forceinline__ uint32_t tame2(uint32_t w, uint32_t* top, bool* nan) {
  uint32_t out = 0;
#pragma unroll
  for (int shift = 0; shift < 32; shift += 16) {
    const uint32_t v = w >> shift & 0x7FFFu, sign = w >> shift & 0x8000u;
    if (v < 0x7F80u) *top = max(*top, v);
    *nan |= v > 0x7F80u;
    out |= (v < 0x7F80u ? sign | v : v > 0x7F80u ? 0u : sign | 0x7F7Fu) << shift;
  }
  return out;
}

// The group's factor from amax's bf16 bits.
__device__ __forceinline__ float factor_of(uint32_t amax) {
  if (amax == 0) return 1.f;
  uint32_t q = __float_as_uint(__uint_as_float(amax << 16) / 7.f);
  q += 0x3FFFFu + ((q >> 19) & 1u);  // to five significant bits, ties to even
  return fmaxf(__uint_as_float(q & ~0x7FFFFu), 7.5231638452626401e-37f /* 2^-120 */);
}

// Eight finite values as nibbles; r = 1 / f, rounded to nearest.  CLAMP: they
// may be beyond 7.5 f (an infinity's stand-in).
template <bool CLAMP>
__device__ __forceinline__ uint32_t codes8(const uint4& v, float f, float r) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint64_t rr = f32x2(r, r), nf = f32x2(-f, -f);
  const uint64_t bias = f32x2(12582920.f, 12582920.f);  // 1.5 2^23 + 8
  uint32_t out = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float x0 = bf16lo_to_f32(w[k]), x1 = bf16hi_to_f32(w[k]);
    if (CLAMP) {
      x0 = fminf(fmaxf(x0, -7.f * f), 7.f * f);
      x1 = fminf(fmaxf(x1, -7.f * f), 7.f * f);
    }
    const uint64_t x = f32x2(x0, x1), q = mul_f32x2(x, rr);
    float a, b;
    f32x2_split(add_f32x2(fma_f32x2(fma_f32x2(q, nf, x), rr, q), bias), a, b);
    out += __float_as_uint(a) * (1u << (8 * k)) + __float_as_uint(b) * (16u << (8 * k));
  }
  return out - 0x4B400000u * 0x11111111u;  // the bits of 1.5 2^23, eight times
}

// As kv_cache.cu's e4m3 rows: D / 16 lanes take a row of K and of V, eight
// values of either half each.  Four lanes share a group in either half of
// either row; each of them works out one of the four factors, whose divisions
// would otherwise be a third of the kernel's instructions.  Six blocks to an SM,
// at 40 registers a thread: with the 58 that the compiler took unasked a padded
// batch of 4 x 8,192 tokens, 16 heads, d=128 (one set of lengths), took 45 us in
// place of 40.
template <int D>
__global__ void __launch_bounds__(kThreads, 6)
    kv_write_int4_kernel(const CacheArgs c, const CacheRows r, unsigned rows, int* err) {
  constexpr int kLanes = D / 16, kGroups = kThreads / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % kLanes;
  const unsigned i = blockIdx.x * kGroups + threadIdx.x / kLanes;
  uint4 x[4] = {};  // K's halves, V's halves
  int64_t dst = -1;
  if (i < rows) {
    const Row w = row_of(i, c, r);
    dst = locate(c, r, w, kSiteWritePage, lane, err);
    if (dst >= 0) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.x[s]) +
                                                          w.b * r.sb[s] + w.h * r.sh[s] +
                                                          w.t * r.st[s]);
        x[2 * s] = __ldg(src + lane);
        x[2 * s + 1] = __ldg(src + kLanes + lane);
      }
    }
  }
  if (!__any_sync(0xffffffffu, dst >= 0)) return;  // a padded batch's filling
  uint32_t top[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) top[g] = amax8(x[g]);
  const uint32_t most = max(max(top[0], top[1]), max(top[2], top[3]));
  const bool odd = __any_sync(0xffffffffu, most >= 0x7F80u);
  uint32_t nans = 0;  // a bit per group
  if (odd) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      bool nan = false;
      top[g] = 0;
      x[g].x = tame2(x[g].x, &top[g], &nan);
      x[g].y = tame2(x[g].y, &top[g], &nan);
      x[g].z = tame2(x[g].z, &top[g], &nan);
      x[g].w = tame2(x[g].w, &top[g], &nan);
      nans |= uint32_t(nan) << g;
    }
    nans |= __shfl_xor_sync(0xffffffffu, nans, 1);
    nans |= __shfl_xor_sync(0xffffffffu, nans, 2);
  }
  uint32_t lo = top[0] | top[1] << 16, hi = top[2] | top[3] << 16;
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) {
    lo = max_u16x2(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_u16x2(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const int mine = lane % 4;  // this lane's group of the four
  const uint32_t both = mine & 2 ? hi : lo;
  const float f = factor_of(mine & 1 ? both >> 16 : both & 0xFFFFu), inv = 1.f / f;
  uint32_t codes[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float fg = __shfl_sync(0xffffffffu, f, g, 4), rg = __shfl_sync(0xffffffffu, inv, g, 4);
    codes[g] = odd ? codes8<true>(x[g], fg, rg) : codes8<false>(x[g], fg, rg);
  }
  if (dst < 0) return;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(g < 2 ? c.kc : c.vc) +
                                dst * (D / 2))[(g & 1) * kLanes + lane] = codes[g];
  (mine < 2 ? c.kf : c.vf)[dst * (D / kInt4Group) + ((mine & 1) * kLanes + lane) / 4] =
      nans >> mine & 1 ? 0x7FFFu : uint16_t(__float_as_uint(f) >> 16);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    kv_read_int4_kernel(const CacheArgs c, const CacheRows r, unsigned rows, int* err) {
  constexpr int kLanes = D / 16, kGroups = kThreads / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % kLanes;
  const unsigned i = blockIdx.x * kGroups + threadIdx.x / kLanes;
  if (i >= rows) return;
  uint4 y[2][2] = {};
  const int64_t src = locate(c, r, row_of(i, c, r), kSiteReadPage, lane, err);
  if (src >= 0) {
    uint32_t u[2][2], f[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(
          static_cast<const uint8_t*>(s ? c.vc : c.kc) + src * (D / 2));
      const uint16_t* factors = (s ? c.vf : c.kf) + src * (D / kInt4Group);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        u[s][half] = __ldg(codes + half * kLanes + lane);
        f[s][half] = __ldg(factors + (half * kLanes + lane) / 4) * 0x00010001u;
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // elements p and p + 4, put back in order
        uint32_t z[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) z[p] = int4_pair(u[s][half], p, f[s][half]);
        y[s][half] = make_uint4(__byte_perm(z[0], z[1], 0x5410), __byte_perm(z[2], z[3], 0x5410),
                                __byte_perm(z[0], z[1], 0x7632), __byte_perm(z[2], z[3], 0x7632));
      }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {  // the output is contiguous: row i of [B][Hkv][T]
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(r.x[s]) + int64_t(i) * D);
    out[lane] = y[s][0];
    out[kLanes + lane] = y[s][1];
  }
}

}  // namespace

cudaError_t launch_kv_write_int4(const CacheArgs& c, const CacheRows& r, int* err,
                                 cudaStream_t stream) {
  return c.d == 64 ? launch(kv_write_int4_kernel<64>, c, r, err, stream)
                   : launch(kv_write_int4_kernel<128>, c, r, err, stream);
}

cudaError_t launch_kv_read_int4(const CacheArgs& c, const CacheRows& r, int* err,
                                cudaStream_t stream) {
  return c.d == 64 ? launch(kv_read_int4_kernel<64>, c, r, err, stream)
                   : launch(kv_read_int4_kernel<128>, c, r, err, stream);
}

}  // namespace attn
