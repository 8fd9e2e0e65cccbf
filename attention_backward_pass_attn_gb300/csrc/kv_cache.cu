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

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Largest finite magnitude of a row as bf16 bits, over the row's lanes.
template <int LANES>
__device__ __forceinline__ uint32_t row_amax_bits(const uint4& x) {
  uint32_t m = 0;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t mag = w[k] & 0x7FFF7FFFu;
    if ((mag & 0xFFFFu) >= 0x7F80u) mag &= 0xFFFF0000u;
    if ((mag >> 16) >= 0x7F80u) mag &= 0x0000FFFFu;
    m = max_u16x2(m, mag);
  }
  m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o, LANES));
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
__device__ __forceinline__ Row row_of(int64_t i, int T, int Hkv) {
  const int64_t bh = i / T;
  return {int(bh / Hkv), int(bh % Hkv), int(i - bh * T)};
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(const CacheArgs c, const CacheRows r, int64_t rows, int* err) {
  constexpr int kLanes = D / 8;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % kLanes;
  const int64_t i = int64_t(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const bool live = i < rows;
  const Row w = live ? row_of(i, r.T, c.Hkv) : Row{0, 0, 0};
  bool ok = live && w.t < (r.count ? __ldg(r.count + w.b) : r.T);
  int64_t dst = 0;
  if (ok) {
    const int64_t pos = int64_t(__ldg(r.start + w.b)) + w.t;
    ok = pos >= 0 && pos < c.capacity;
    if (!ok && lane == 0) report_error(err, kDevBadIndex, kSiteLength);
    if (ok) {
      const int pi = int(pos) / c.page_size;
      const int page = __ldg(c.table + int64_t(w.b) * c.max_pages + pi);
      ok = page_in_range(page, c.num_pages);
      if (!ok && lane == 0) report_error(err, kDevBadIndex, kSiteWritePage);
      dst = cache_row(page, c.Hkv, w.h, c.page_size, int(pos) - pi * c.page_size);
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (ok)
      x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.x[s]) + w.b * r.sb[s] +
                                          w.h * r.sh[s] + w.t * r.st[s] + lane * 8);
    uint8_t* cache = static_cast<uint8_t*>(s ? c.vc : c.kc);
    if (!FP8) {
      if (ok) *reinterpret_cast<uint4*>(cache + (dst * D + lane * 8) * 2) = x;
    } else {
      const int e = descale_exponent(row_amax_bits<kLanes>(x));  // all lanes: shuffles
      if (!ok) continue;
      const float inv = pow2f(-e);
      const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = bf16lo_to_f32(w4[k]) * inv;
        f[2 * k + 1] = bf16hi_to_f32(w4[k]) * inv;
      }
      *reinterpret_cast<uint2*>(cache + dst * D + lane * 8) =
          make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
      if (lane == 0) (s ? c.vd : c.kd)[dst] = pow2f(e);
    }
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
    kv_read_kernel(const CacheArgs c, const CacheRows r, int64_t rows, int* err) {
  constexpr int kLanes = D / 8;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % kLanes;
  const int64_t i = int64_t(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (i >= rows) return;
  const Row w = row_of(i, r.T, c.Hkv);
  bool ok = w.t < (r.count ? __ldg(r.count + w.b) : r.T);
  int64_t src = 0;
  if (ok) {
    const int64_t pos = int64_t(__ldg(r.start + w.b)) + w.t;
    ok = pos >= 0 && pos < c.capacity;
    if (!ok && lane == 0) report_error(err, kDevBadIndex, kSiteLength);
    if (ok) {
      const int pi = int(pos) / c.page_size;
      const int page = __ldg(c.table + int64_t(w.b) * c.max_pages + pi);
      ok = page_in_range(page, c.num_pages);
      if (!ok && lane == 0) report_error(err, kDevBadIndex, kSiteReadPage);
      src = cache_row(page, c.Hkv, w.h, c.page_size, int(pos) - pi * c.page_size);
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint4 y = make_uint4(0, 0, 0, 0);
    const uint8_t* cache = static_cast<const uint8_t*>(s ? c.vc : c.kc);
    if (ok) {
      if (!FP8) {
        y = *reinterpret_cast<const uint4*>(cache + (src * D + lane * 8) * 2);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(cache + src * D + lane * 8);
        const float f = (s ? c.vd : c.kd)[src];
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 g = e4m3x2_to_f32((k < 2 ? u.x : u.y) >> (k & 1 ? 16 : 0));
          o[k] = pack_bf16x2(g.x * f, g.y * f);
        }
        y = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(r.x[s]) + w.b * r.sb[s] + w.h * r.sh[s] +
                              w.t * r.st[s] + lane * 8) = y;
  }
}

template <typename K>
cudaError_t launch(K kernel, const CacheArgs& c, const CacheRows& r, int* err,
                   cudaStream_t stream) {
  const int64_t rows = int64_t(c.B) * c.Hkv * r.T;
  const int per_block = kThreads / (c.d / 8);
  return launch_kernel(kernel, dim3(unsigned((rows + per_block - 1) / per_block)), dim3(kThreads),
                       0, stream, c, r, rows, err);
}

}  // namespace

cudaError_t launch_kv_write(const CacheArgs& c, const CacheRows& r, int* err,
                            cudaStream_t stream) {
  if (c.d == 64)
    return c.kd ? launch(kv_write_kernel<64, true>, c, r, err, stream)
                : launch(kv_write_kernel<64, false>, c, r, err, stream);
  return c.kd ? launch(kv_write_kernel<128, true>, c, r, err, stream)
              : launch(kv_write_kernel<128, false>, c, r, err, stream);
}

cudaError_t launch_kv_read(const CacheArgs& c, const CacheRows& r, int* err,
                           cudaStream_t stream) {
  if (c.d == 64)
    return c.kd ? launch(kv_read_kernel<64, true>, c, r, err, stream)
                : launch(kv_read_kernel<64, false>, c, r, err, stream);
  return c.kd ? launch(kv_read_kernel<128, true>, c, r, err, stream)
              : launch(kv_read_kernel<128, false>, c, r, err, stream);
}

}  // namespace attn
