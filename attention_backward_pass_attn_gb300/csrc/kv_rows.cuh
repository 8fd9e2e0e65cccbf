// kv_rows.cuh -- what writing and reading rows of the paged cache have in common:
// which row of the call lies where.
#pragma once

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "serving.h"

namespace attn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

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

template <typename K>
cudaError_t launch(K kernel, const CacheArgs& c, const CacheRows& r, int* err,
                   cudaStream_t stream) {
  const unsigned rows = unsigned(int64_t(c.B) * c.Hkv * r.T);
  const unsigned per_block = kThreads / (c.d / 16);
  return launch_kernel(kernel, dim3((rows + per_block - 1) / per_block), dim3(kThreads), 0, stream,
                       c, r, rows, err);
}

}  // namespace
}  // namespace attn
