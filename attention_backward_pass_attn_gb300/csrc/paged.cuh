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

// A head block (the units of one sequence and block of heads) that several
// shares cover leaves a partial result in each.  A share has two slots for
// them: `turn` counts the head blocks it has come through, and only its first
// and its last can be shared with others.
ATTN_HD int part_slot(int share, int turn) { return 2 * share + (turn ? 1 : 0); }

// Partial results to be joined: part 0 lies in slot0, part k >= 1 in the first
// slot of share share1 + (k - 1) stride.
struct Parts {
  int slot0, share1, stride, parts;
  ATTN_HD int slot(int k) const {
    return k == 0 ? slot0 : part_slot(share1 + (k - 1) * stride, 0);
  }
};

// More than kDirect parts of a head block are joined in two steps: first those
// of each kGroup consecutive shares (share / kGroup), into the slot of the
// first of them, then those results.  One block alone would read hundreds of
// parts for longer than it computed.
constexpr int kDirect = 32, kGroup = 16;

// The most parts that one join has, of either step, with G shares.
constexpr int max_join_parts(int G) {
  return (G - 1) / kGroup + 1 > kDirect ? (G - 1) / kGroup + 1 : kDirect;
}

// A head block with shares i0 .. i1; its first part lies in slot0.
struct Piece {
  int i0, i1, slot0;
  ATTN_HD bool direct() const { return i1 - i0 < kDirect; }
  // The parts joined together with share i's.
  ATTN_HD Parts group(int i) const {
    const int g = i / kGroup * kGroup;
    const int from = direct() || g < i0 ? i0 : g;
    const int to = direct() || g + kGroup - 1 > i1 ? i1 : g + kGroup - 1;
    return {from == i0 ? slot0 : part_slot(from, 0), from + 1, 1, to - from + 1};
  }
  // The groups' results.
  ATTN_HD Parts groups() const {
    const int g = i0 / kGroup;
    return {slot0, (g + 1) * kGroup, kGroup, i1 / kGroup - g + 1};
  }
};

// The head block of units first .. first + n - 1, of W units in G shares.
ATTN_HD Piece split_piece(int64_t first, int n, int64_t W, int G) {
  const int i0 = split_owner(first, W, G);
  // its first share may have come to it after another head block
  return {i0, split_owner(first + n - 1, W, G), part_slot(i0, split_begin(i0, W, G) < first)};
}

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
