// kv_cache.cu -- the paged key/value cache as it is written (rounded to e4m3
// on the way, if that is what it holds) and as it is read back.
//
// An e4m3 row (the d values of one token and head) has a factor of its own,
// descale = the smallest power of two with amax <= 448 descale (1 for a row of
// zeros), amax taken over the row's finite values, and holds
// e4m3(x / descale), ties to even; an infinity saturates to +-448 and a NaN
// stays one.  A power of two makes the division exact, so the row's only
// rounding is the one to e4m3 (half a step, 2^-4 of the value), and a
// floating-point row loses nothing by it that amax / 448 would keep but the
// last bit of its smallest subnormals.  The exponent is kept at or above -126,
// where 1 / descale is still finite.
//
// Bound by HBM: a written row is read once (2 d bytes) and written once (2 d,
// or d + 4 in e4m3); reading back is the reverse.  32,768 tokens of 16 heads,
// d=128: 61 us to e4m3, 81 us to bf16, 80 us back from bf16 (6.6 to 6.7 TB/s,
// a copy's speed).
#include <cuda_fp16.h>

#include "kv_rows.cuh"

namespace attn {
namespace {

// Largest magnitude among a lane's 16 values, as bf16 bits; of the finite ones
// when there are others.
__device__ __forceinline__ uint32_t amax_bits(const uint4 (&x)[2]) {
  const uint32_t w[8] = {x[0].x & 0x7FFF7FFFu, x[0].y & 0x7FFF7FFFu, x[0].z & 0x7FFF7FFFu,
                         x[0].w & 0x7FFF7FFFu, x[1].x & 0x7FFF7FFFu, x[1].y & 0x7FFF7FFFu,
                         x[1].z & 0x7FFF7FFFu, x[1].w & 0x7FFF7FFFu};
  uint32_t m = w[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) m = max_u16x2(m, w[k]);
  m = max(m & 0xFFFFu, m >> 16);
  if (m >= 0x7F80u) {  // an infinity or a NaN
    m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t lo = w[k] & 0xFFFFu, hi = w[k] >> 16;
      m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
  }
  return m;
}

// Exponent of the row's descale from amax's bf16 bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ int descale_exponent(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = int(amax >> 7) - 127 - 8 + ((amax & 0x7Fu) > 0x60u ? 1 : 0);
  return e < -126 ? -126 : e;
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// D / 16 lanes take a row of K and of V, 8 values of either half each: finding
// the row is shared by 64 bytes a lane.  With 32 bytes a lane and 64-bit
// divisions this kernel was bound by its instructions (the ALU 71 % busy): 76 us
// for a padded batch of 17,600 tokens (4 x 8,192 with their filling) that now
// takes 36, with 32 at a copy's speed.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(const CacheArgs c, const CacheRows r, unsigned rows, int* err) {
  constexpr int kLanes = D / 16, kGroups = kThreads / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % kLanes;
  const unsigned i = blockIdx.x * kGroups + threadIdx.x / kLanes;
  uint4 x[2][2] = {};
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
        x[s][0] = __ldg(src + lane);
        x[s][1] = __ldg(src + kLanes + lane);
      }
    }
  }
  if (!__any_sync(0xffffffffu, dst >= 0)) return;  // a padded batch's filling
  uint32_t amax = 0;  // K's in the low half, V's in the high one
  if (FP8) {
    amax = amax_bits(x[0]) | amax_bits(x[1]) << 16;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      amax = max_u16x2(amax, __shfl_xor_sync(0xffffffffu, amax, o, kLanes));
  }
  if (dst < 0) return;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint8_t* cache = static_cast<uint8_t*>(s ? c.vc : c.kc) + dst * (D * (FP8 ? 1 : 2));
    if (!FP8) {
      reinterpret_cast<uint4*>(cache)[lane] = x[s][0];
      reinterpret_cast<uint4*>(cache)[kLanes + lane] = x[s][1];
      continue;
    }
    const int e = descale_exponent(s ? amax >> 16 : amax & 0xFFFFu);
    // 1 / descale as two bf16: x / descale is exact, or below every e4m3
    // value's half and rounded to zero either way
    const uint32_t inv = uint32_t(127 - e) * 0x00800080u;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 v = x[s][half];
      const uint32_t w[4] = {mul_bf16x2(v.x, inv), mul_bf16x2(v.y, inv), mul_bf16x2(v.z, inv),
                             mul_bf16x2(v.w, inv)};
      reinterpret_cast<uint2*>(cache)[half * kLanes + lane] =
          make_uint2(pack_e4m3x4(bf16lo_to_f32(w[0]), bf16hi_to_f32(w[0]), bf16lo_to_f32(w[1]),
                                 bf16hi_to_f32(w[1])),
                     pack_e4m3x4(bf16lo_to_f32(w[2]), bf16hi_to_f32(w[2]), bf16lo_to_f32(w[3]),
                                 bf16hi_to_f32(w[3])));
    }
    if (lane == 0) (s ? c.vd : c.kd)[dst] = pow2f(e);
  }
}

// Two e4m3 values (low 16 bits) as floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(const CacheArgs c, const CacheRows r, unsigned rows, int* err) {
  constexpr int kLanes = D / 16, kGroups = kThreads / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % kLanes;
  const unsigned i = blockIdx.x * kGroups + threadIdx.x / kLanes;
  if (i >= rows) return;
  uint4 y[2][2] = {};
  const int64_t src = locate(c, r, row_of(i, c, r), kSiteReadPage, lane, err);
  if (src >= 0) {
    uint2 u[2][2];
    float f[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint8_t* cache =
          static_cast<const uint8_t*>(s ? c.vc : c.kc) + src * (D * (FP8 ? 1 : 2));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (FP8)
          u[s][half] = __ldg(reinterpret_cast<const uint2*>(cache) + half * kLanes + lane);
        else
          y[s][half] = __ldg(reinterpret_cast<const uint4*>(cache) + half * kLanes + lane);
      }
      if (FP8) f[s] = __ldg((s ? c.vd : c.kd) + src);
    }
    if (FP8) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 g =
                e4m3x2_to_f32((k < 2 ? u[s][half].x : u[s][half].y) >> (k & 1 ? 16 : 0));
            o[k] = pack_bf16x2(g.x * f[s], g.y * f[s]);
          }
          y[s][half] = make_uint4(o[0], o[1], o[2], o[3]);
        }
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

cudaError_t launch_kv_write(const CacheArgs& c, const CacheRows& r, int* err,
                            cudaStream_t stream) {
  if (c.type == kCacheInt4) return launch_kv_write_int4(c, r, err, stream);
  if (c.d == 64)
    return c.kd ? launch(kv_write_kernel<64, true>, c, r, err, stream)
                : launch(kv_write_kernel<64, false>, c, r, err, stream);
  return c.kd ? launch(kv_write_kernel<128, true>, c, r, err, stream)
              : launch(kv_write_kernel<128, false>, c, r, err, stream);
}

cudaError_t launch_kv_read(const CacheArgs& c, const CacheRows& r, int* err,
                           cudaStream_t stream) {
  if (c.type == kCacheInt4) return launch_kv_read_int4(c, r, err, stream);
  if (c.d == 64)
    return c.kd ? launch(kv_read_kernel<64, true>, c, r, err, stream)
                : launch(kv_read_kernel<64, false>, c, r, err, stream);
  return c.kd ? launch(kv_read_kernel<128, true>, c, r, err, stream)
              : launch(kv_read_kernel<128, false>, c, r, err, stream);
}

}  // namespace attn
