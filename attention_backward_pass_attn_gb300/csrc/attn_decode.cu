// attn_decode.cu -- attention of one new token per sequence over its pages.
//
//   s_j = scale <q, k_j>,  o = sum_j softmax(s)_j v_j,  l = logsumexp(s)
//
// over the visible positions j of the sequence, one thread block for each
// (sequence, query head): a thread per key forms the scores of 128 keys at a
// time, a running maximum and sum are kept over the runs of 128 keys, and a
// thread per output column adds the weighted values.
#include <cuda_fp16.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "serving.h"

namespace attn {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Eight consecutive values of a cache row.
template <bool FP8>
__device__ __forceinline__ void load8(const void* cache, int64_t at, float (&f)[8]) {
  if (FP8) {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + at);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 g = e4m3x2_to_f32((k < 2 ? u.x : u.y) >> (k & 1 ? 16 : 0));
      f[2 * k] = g.x;
      f[2 * k + 1] = g.y;
    }
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cache) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = bf16lo_to_f32(w[k]);
      f[2 * k + 1] = bf16hi_to_f32(w[k]);
    }
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) decode_kernel(const DecodeArgs a) {
  __shared__ float q[D];
  __shared__ float p[kThreads];
  __shared__ int64_t row[kThreads];
  __shared__ float red[4];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x;
  const int hq = blockIdx.x % a.Hq, b = blockIdx.x / a.Hq;
  const int h = hq / (a.Hq / a.c.Hkv);
  const int raw = a.lens[b];
  const int len = clamp_length(raw, a.c.capacity);
  if (raw != len && tid == 0 && hq == 0) report_error(a.err, kDevBadIndex, kSiteLength);
  const int lo = first_visible_position(len, a.window);
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (int64_t(b) * a.Hq + hq) * D;
  for (int i = tid; i < D; i += kThreads)
    q[i] = __uint_as_float(uint32_t(qp[i]) << 16) * a.scale_log2;
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = lo; j0 < len; j0 += kThreads) {
    const int j = j0 + tid;
    float s = -INFINITY;
    int64_t at = -1;
    if (j < len) {
      const int pi = j / a.c.page_size;
      const int page = a.c.table[int64_t(b) * a.c.max_pages + pi];
      if (page_in_range(page, a.c.num_pages))
        at = cache_row(page, a.c.Hkv, h, a.c.page_size, j - pi * a.c.page_size);
      else
        report_error(a.err, kDevBadIndex, kSiteDecodePage);
    }
    if (at >= 0) {
      float dot = 0.f;
      for (int c = 0; c < D; c += 8) {
        float f[8];
        load8<FP8>(a.c.kc, at * D + c, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) dot += f[k] * q[c + k];
      }
      s = FP8 ? dot * a.c.kd[at] : dot;
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (tid % 32 == 0) red[tid / 32] = mx;
    __syncthreads();
    const float mn = fmaxf(fmaxf(m, fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - ref);
    m = mn;
    const float pj = exp2f(s - ref);
    l = l * alpha + pj;
    p[tid] = FP8 && at >= 0 ? pj * a.c.vd[at] : pj;
    row[tid] = at;
    __syncthreads();
    acc *= alpha;
    if (tid < D)
      for (int k = 0; k < kThreads && j0 + k < len; ++k) {
        if (row[k] < 0) continue;
        float f;
        if (FP8)
          f = e4m3x2_to_f32(static_cast<const uint8_t*>(a.c.vc)[row[k] * D + tid]).x;
        else
          f = __uint_as_float(
              uint32_t(static_cast<const uint16_t*>(a.c.vc)[row[k] * D + tid]) << 16);
        acc += p[k] * f;
      }
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (tid % 32 == 0) red[tid / 32] = l;
  __syncthreads();
  l = red[0] + red[1] + red[2] + red[3];
  const int64_t out = int64_t(b) * a.Hq + hq;
  if (tid < D)
    static_cast<__nv_bfloat16*>(a.o)[out * D + tid] =
        __float2bfloat16_rn(l == 0.f ? 0.f : acc / l);
  if (tid == 0) a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int D, bool FP8>
cudaError_t launch(const DecodeArgs& a, cudaStream_t stream) {
  return launch_kernel(decode_kernel<D, FP8>, dim3(unsigned(a.c.B) * a.Hq), dim3(kThreads), 0,
                       stream, a);
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream) {
  if (a.c.d == 64) return a.c.kd ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
  return a.c.kd ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
}

}  // namespace attn
