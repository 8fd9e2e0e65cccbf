"""The index arithmetic of the paged cache and of the single-token attention's
split (``csrc/paged.cuh``), compiled for the host and checked by brute force:
every position maps to the row its definition says, no page outside the cache
passes, and the shares cover all work once.  CPU only."""

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "attention_backward_pass_attn_gb300", "csrc")

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "paged.cuh"
using namespace attn;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  // pages: below zero, past the end, the extremes
  for (int n : {1, 7, INT_MAX}) {
    CHECK(!page_in_range(-1, n) && !page_in_range(INT_MIN, n) && page_in_range(0, n));
    CHECK(page_in_range(n - 1, n) && (n == INT_MAX || !page_in_range(n, n)));
    CHECK(n == INT_MAX || !page_in_range(INT_MAX, n));
  }
  CHECK(clamp_length(-5, 64) == 0 && clamp_length(INT_MIN, 64) == 0 && clamp_length(65, 64) == 64);
  CHECK(clamp_length(INT_MAX, 64) == 64 && clamp_length(64, 64) == 64 && clamp_length(3, 64) == 3);
  // rows: in order, distinct, within the cache; 64 bits where 32 overflow
  const int P = 5, H = 3;
  for (int ps : {16, 48, 256}) {
    int64_t next = 0;
    for (int p = 0; p < P; ++p)
      for (int h = 0; h < H; ++h)
        for (int r = 0; r < ps; ++r) CHECK(cache_row(p, H, h, ps, r) == next++);
    CHECK(next == int64_t(P) * H * ps);
  }
  CHECK(cache_row(1 << 24, 16, 15, 256, 255) == ((int64_t(1) << 24) * 16 + 15) * 256 + 255);
  // a run of 16 positions from a multiple of 16 stays on one page
  for (int ps = 16; ps <= 512; ps += 16)
    for (int p = 0; p < 4096; p += 16) CHECK(p / ps == (p + 15) / ps);
  // visible positions and their units
  for (int unit : {64, 128, 256})
    for (int window : {0, 1, 5, 64, 100, 1000})
      for (int len = 0; len < 700; ++len) {
        const int lo = first_visible_position(len, window);
        CHECK(lo >= 0 && lo <= len && (window == 0 ? lo == 0 : len - lo == (len < window ? len : window)));
        const int n = units_of(lo, len, unit), base = lo & ~15;
        CHECK((n == 0) == (len == lo));
        if (n) {
          CHECK(base <= lo && base + int64_t(n) * unit >= len && base + int64_t(n - 1) * unit < len);
        }
      }
  CHECK(units_of(0, INT_MAX, 64) == (INT_MAX / 64) + 1);
  CHECK(first_visible_position(INT_MAX, INT_MAX) == 0);
  // shares: in order, as even as possible, the owner of each unit is the share that holds it
  for (int G = 1; G <= 40; ++G)
    for (int64_t W = G; W <= 3 * G + 7; ++W) {
      CHECK(split_begin(0, W, G) == 0 && split_begin(G, W, G) == W);
      for (int i = 0; i < G; ++i) {
        const int64_t a = split_begin(i, W, G), b = split_begin(i + 1, W, G);
        CHECK(b > a && b - a <= W / G + 1 && b - a >= W / G);
        for (int64_t x = a; x < b; ++x) CHECK(split_owner(x, W, G) == i);
      }
    }
  const int64_t W = int64_t(1) << 42;  // products stay inside 64 bits at the largest sizes
  for (int G : {1, 455, 456}) {
    for (int i = 0; i < G; ++i) CHECK(split_owner(split_begin(i, W, G), W, G) == i);
    CHECK(split_owner(W - 1, W, G) == G - 1);
  }
  // division by multiplication: every small case, and the edges of every quotient
  // near the ends of the range
  for (uint32_t d = 1; d <= 300; ++d) {
    const FastDiv f = make_fast_div(d);
    for (uint32_t n = 0; n < 5000; ++n) CHECK(fast_div(n, f) == n / d);
  }
  uint32_t rnd = 12345;
  for (int i = 0; i < 200000; ++i) {
    rnd = rnd * 1664525u + 1013904223u;
    const uint32_t d = (rnd >> (i % 31)) % 0x7FFFFFFFu + 1;
    const FastDiv f = make_fast_div(d);
    const uint32_t q = 0x7FFFFFFFu / d;
    for (uint32_t n : {0u, d - 1, q * d - 1, q * d, 0x7FFFFFFFu, q / 2 * d, (q / 2 + 1) * d - 1})
      if (n <= 0x7FFFFFFFu) CHECK(fast_div(n, f) == n / d);
  }
  for (uint32_t d : {0x7FFFFFFFu, 0x7FFFFFFEu, 0x40000000u, 0x40000001u}) {
    const FastDiv f = make_fast_div(d);
    for (uint32_t n : {0u, 1u, d - 1, d, 0x7FFFFFFFu}) CHECK(fast_div(n, f) == n / d);
  }
  return 0;
}
"""


def test_paged_index_arithmetic(tmp_path):
    src = tmp_path / "paged_check.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "paged_check"
    # -ftrapv: a signed overflow aborts the program
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, p.stdout + p.stderr
