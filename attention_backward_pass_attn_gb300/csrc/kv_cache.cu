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
// or d + 4 in e4m3); reading back is the reverse.  D / 8 lanes hold a row,
// 16 bytes of bf16 each.
#include <cuda_fp16.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "serving.h"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Largest magnitude among a lane's 8 values, as bf16 bits; of the finite ones
// when there are others.
__device__ __forceinline__ uint32_t amax_bits(const uint4& x) {
  const uint32_t w[4] = {x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu, x.z & 0x7FFF7FFFu,
                         x.w & 0x7FFF7FFFu};
  uint32_t m = max_u16x2(max_u16x2(w[0], w[1]), max_u16x2(w[2], w[3]));
  m = max(m & 0xFFFFu, m >> 16);
  if (m >= 0x7F80u) {  // an infinity or a NaN
    m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
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

struct Row {
  int b, h, t;
};
__device__ __forceinline__ Row row_of(unsigned i, const CacheArgs& c, const CacheRows& r) {
  const unsigned bh = fast_div(i, r.T_div), b = fast_div(bh, r.head_div);
  return {int(b), int(bh - b * c.Hkv), int(i - bh * r.T)};
}

// Where row w of the call lies in the cache, or -1 (recorded by `lane` 0).
__device__ __forceinline__ int64_t locate(const CacheArgs& c, const CacheRows& r, const Row& w,
                                          int site, int lane, int* err) {
  if (w.t >= (r.count ? __ldg(r.count + w.b) : r.T)) return -1;
  const int64_t pos = int64_t(__ldg(r.start + w.b)) + w.t;
  if (pos < 0 || pos >= c.capacity) {
    if (lane == 0) report_error(err, kDevBadIndex, kSiteLength);
    return -1;
  }
  const unsigned p = unsigned(pos), pi = fast_div(p, c.page_div);
  const int page = __ldg(c.table + int64_t(w.b) * c.max_pages + pi);
  if (!page_in_range(page, c.num_pages)) {
    if (lane == 0) report_error(err, kDevBadIndex, site);
    return -1;
  }
  return cache_row(page, c.Hkv, w.h, c.page_size, int(p - pi * c.page_size));
}

// Each group of D / 8 lanes takes R rows, their loads issued together.
template <int D, bool FP8, int R>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(const CacheArgs c, const CacheRows r, unsigned rows, int* err) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % kLanes;
  const unsigned first = blockIdx.x * (kGroups * R) + threadIdx.x / kLanes;
  int64_t dst[R];
  uint4 x[R][2];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const unsigned i = first + j * kGroups;
    dst[j] = -1;
    x[j][0] = x[j][1] = make_uint4(0, 0, 0, 0);
    if (i >= rows) continue;
    const Row w = row_of(i, c, r);
    dst[j] = locate(c, r, w, kSiteWritePage, lane, err);
    if (dst[j] < 0) continue;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      x[j][s] = __ldg(reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(r.x[s]) + w.b * r.sb[s] + w.h * r.sh[s] + w.t * r.st[s] +
          lane * 8));
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    uint32_t amax = 0;  // K's in the low half, V's in the high one
    if (FP8) {
      amax = amax_bits(x[j][0]) | amax_bits(x[j][1]) << 16;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)  // all lanes: shuffles
        amax = max_u16x2(amax, __shfl_xor_sync(0xffffffffu, amax, o, kLanes));
    }
    if (dst[j] < 0) continue;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint8_t* cache = static_cast<uint8_t*>(s ? c.vc : c.kc);
      if (!FP8) {
        *reinterpret_cast<uint4*>(cache + (dst[j] * D + lane * 8) * 2) = x[j][s];
        continue;
      }
      const int e = descale_exponent(s ? amax >> 16 : amax & 0xFFFFu);
      // 1 / descale as two bf16: x / descale is exact, or below every e4m3
      // value's half and rounded to zero either way
      const uint32_t inv = uint32_t(127 - e) << 7 | uint32_t(127 - e) << 23;
      const uint32_t w[4] = {mul_bf16x2(x[j][s].x, inv), mul_bf16x2(x[j][s].y, inv),
                             mul_bf16x2(x[j][s].z, inv), mul_bf16x2(x[j][s].w, inv)};
      uint32_t o[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        o[k] = pack_e4m3x4(bf16lo_to_f32(w[2 * k]), bf16hi_to_f32(w[2 * k]),
                           bf16lo_to_f32(w[2 * k + 1]), bf16hi_to_f32(w[2 * k + 1]));
      *reinterpret_cast<uint2*>(cache + dst[j] * D + lane * 8) = make_uint2(o[0], o[1]);
      if (lane == 0) (s ? c.vd : c.kd)[dst[j]] = pow2f(e);
    }
  }
}

// Two e4m3 values (low 16 bits) as floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

template <int D, bool FP8, int R>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(const CacheArgs c, const CacheRows r, unsigned rows, int* err) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % kLanes;
  const unsigned first = blockIdx.x * (kGroups * R) + threadIdx.x / kLanes;
  uint4 x[R][2];  // e4m3: the first two words
  float f[R][2];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const unsigned i = first + j * kGroups;
    x[j][0] = x[j][1] = make_uint4(0, 0, 0, 0);
    f[j][0] = f[j][1] = 0.f;
    if (i >= rows) continue;
    const int64_t src = locate(c, r, row_of(i, c, r), kSiteReadPage, lane, err);
    if (src < 0) continue;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint8_t* cache = static_cast<const uint8_t*>(s ? c.vc : c.kc);
      if (FP8) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(cache + src * D + lane * 8));
        x[j][s].x = u.x;
        x[j][s].y = u.y;
        f[j][s] = __ldg((s ? c.vd : c.kd) + src);
      } else {
        x[j][s] = __ldg(reinterpret_cast<const uint4*>(cache + (src * D + lane * 8) * 2));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const unsigned i = first + j * kGroups;
    if (i >= rows) continue;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint4 y = x[j][s];
      if (FP8) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 g = e4m3x2_to_f32((k < 2 ? y.x : y.y) >> (k & 1 ? 16 : 0));
          o[k] = pack_bf16x2(g.x * f[j][s], g.y * f[j][s]);
        }
        y = make_uint4(o[0], o[1], o[2], o[3]);
      }
      // the output is contiguous: row i of [B][Hkv][T]
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(r.x[s]) + int64_t(i) * D + lane * 8) = y;
    }
  }
}

// Rows per group of lanes: one while that leaves the GPU short of blocks.
template <typename K>
cudaError_t launch(K one, K several, const CacheArgs& c, const CacheRows& r, int* err,
                   cudaStream_t stream) {
  const unsigned rows = unsigned(int64_t(c.B) * c.Hkv * r.T);
  const unsigned groups = kThreads / (c.d / 8);
  const unsigned blocks = (rows + groups - 1) / groups;
  if (blocks <= unsigned(device_sm_count()) * 8)
    return launch_kernel(one, dim3(blocks), dim3(kThreads), 0, stream, c, r, rows, err);
  return launch_kernel(several, dim3((blocks + kRows - 1) / kRows), dim3(kThreads), 0, stream, c, r,
                       rows, err);
}

}  // namespace

cudaError_t launch_kv_write(const CacheArgs& c, const CacheRows& r, int* err,
                            cudaStream_t stream) {
  if (c.d == 64)
    return c.kd ? launch(kv_write_kernel<64, true, 1>, kv_write_kernel<64, true, kRows>, c, r, err, stream)
                : launch(kv_write_kernel<64, false, 1>, kv_write_kernel<64, false, kRows>, c, r, err, stream);
  return c.kd ? launch(kv_write_kernel<128, true, 1>, kv_write_kernel<128, true, kRows>, c, r, err, stream)
              : launch(kv_write_kernel<128, false, 1>, kv_write_kernel<128, false, kRows>, c, r, err, stream);
}

cudaError_t launch_kv_read(const CacheArgs& c, const CacheRows& r, int* err,
                           cudaStream_t stream) {
  if (c.d == 64)
    return c.kd ? launch(kv_read_kernel<64, true, 1>, kv_read_kernel<64, true, kRows>, c, r, err, stream)
                : launch(kv_read_kernel<64, false, 1>, kv_read_kernel<64, false, kRows>, c, r, err, stream);
  return c.kd ? launch(kv_read_kernel<128, true, 1>, kv_read_kernel<128, true, kRows>, c, r, err, stream)
              : launch(kv_read_kernel<128, false, 1>, kv_read_kernel<128, false, kRows>, c, r, err, stream);
}

}  // namespace attn
