// paged.cuh -- index arithmetic of the paged key/value cache, and of the split
// of the single-token attention's work over thread blocks.  Plain integer
// functions with no CUDA dependency, the same on host and device, so that
// every bound they promise is checked on the CPU by brute force.
//
// The cache is [num_pages][Hkv][page_size][d]: the rows of one (page, head)
// are contiguous, so a run of 16 positions is one contiguous piece.  Position
// p of sequence b lives in page table[b][p / page_size], row p % page_size.
// page_size is a multiple of 16: a run of 16 positions that starts at a
// multiple of 16 never crosses a page.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define ATTN_HD __host__ __device__ __forceinline__
#else
#define ATTN_HD inline
#endif

namespace attn {

constexpr int kPageQuantum = 16;  // page sizes are multiples of this

// A sequence length clamped into what its page table can address.
ATTN_HD int clamp_length(int len, int capacity) {
  return len < 0 ? 0 : (len > capacity ? capacity : len);
}

// Whether a page-table entry names a page of the cache.
ATTN_HD bool page_in_range(int page, int num_pages) {
  return uint32_t(page) < uint32_t(num_pages);
}

// Row of the cache (in units of d values) of row r of (page, head).  64 bits:
// a 280 GB cache of short 8-bit rows has more than 2^31 of them.
ATTN_HD int64_t cache_row(int page, int Hkv, int head, int page_size, int r) {
  return (int64_t(page) * Hkv + head) * page_size + r;
}

// The positions the newest token of a sequence sees: [lo, len).
ATTN_HD int first_visible_position(int len, int window) {
  return window > 0 && len > window ? len - window : 0;
}

// Work units (of `unit` positions, the first starting at lo rounded down to
// 16) of a sequence that sees [lo, len).
ATTN_HD int units_of(int lo, int len, int unit) {
  const int base = lo & ~(kPageQuantum - 1);
  return len > lo ? int((int64_t(len) - base + unit - 1) / unit) : 0;
}

// W units in a row, cut into G contiguous shares as even as possible: share i
// is [split_begin(i), split_begin(i + 1)).  0 < G <= W.
ATTN_HD int64_t split_begin(int i, int64_t W, int G) { return int64_t(i) * W / G; }

// The share that holds unit x: the last i with split_begin(i) <= x.  From
// i W / G < x + 1  <=>  i < (x + 1) G / W.
ATTN_HD int split_owner(int64_t x, int64_t W, int G) { return int(((x + 1) * G - 1) / W); }

// Division of 0 <= n < 2^31 by a fixed d >= 1, as a multiplication: with
// s = ceil(log2 d) and mul = floor(2^(31 + s) / d) + 1 < 2^32, the product
// exceeds n 2^(31 + s) / d by less than n <= 2^31, too little to reach the next
// quotient.  A division by a number that the compiler does not know takes
// some twenty instructions, this two.
struct FastDiv {
  uint32_t mul;    // 0: d = 1
  uint32_t shift;
};
inline FastDiv make_fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return s == 0 ? FastDiv{0, 0} : FastDiv{uint32_t((uint64_t(1) << (31 + s)) / d + 1), s - 1};
}
ATTN_HD uint32_t fast_div(uint32_t n, const FastDiv& f) {
  return f.mul ? uint32_t((uint64_t(n) * f.mul) >> 32) >> f.shift : n;
}

}  // namespace attn
