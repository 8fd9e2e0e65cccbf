"""Who leaves which partial result of the single-token attention where, and who
joins it (``csrc/paged.cuh``), walked on the host as the kernel's blocks walk
it, with the blocks arriving in random order: no two parts share a slot, no two
counts a word, and every head block's parts are joined once each, in the order
of their keys.  CPU only."""

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "attention_backward_pass_attn_gb300", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <map>
#include <numeric>
#include <random>
#include <vector>
#include "paged.cuh"
using namespace attn;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

std::mt19937 rng(1);

// units[h]: units of head block h, all at least 1
int walk(const std::vector<int>& units, int grid) {
  const int64_t W = std::accumulate(units.begin(), units.end(), int64_t(0));
  const int G = int(std::min<int64_t>(W, grid));
  std::vector<int64_t> first(units.size());
  for (size_t h = 1; h < units.size(); ++h) first[h] = first[h - 1] + units[h - 1];

  struct Mine { int h; Piece pc; };
  std::vector<std::vector<Mine>> pieces(G);
  std::map<int, int> slot_owner;   // slot -> head block
  // a slot's parts, as the head block's ranges of units
  std::map<int, std::vector<std::pair<int64_t, int64_t>>> parts;
  std::vector<int> done(units.size(), 0);

  for (int i = 0; i < G; ++i) {
    const int64_t w0 = split_begin(i, W, G), w1 = split_begin(i + 1, W, G);
    CHECK(w1 > w0);
    int64_t at = w0;
    for (int turn = 0; at < w1; ++turn) {
      const int h = int(std::upper_bound(first.begin(), first.end(), at) - first.begin()) - 1;
      const int64_t end = std::min(w1, first[h] + units[h]);
      if (end - at == units[h]) {
        ++done[h];  // whole: written at once
      } else {
        const Piece pc = split_piece(first[h], units[h], W, G);
        CHECK(pc.i0 <= i && i <= pc.i1 && pc.i0 < pc.i1 && pc.i1 < G);
        CHECK(pieces[i].size() < 2);
        pieces[i].push_back({h, pc});
        const int slot = part_slot(i, turn);
        CHECK(slot >= 0 && slot < 2 * G && !slot_owner.count(slot));
        slot_owner[slot] = h;
        parts[slot] = {{at, end}};
        // the slot is one that the join looks into, in its place
        const Parts ps = pc.group(i);
        int found = 0;
        for (int k = 0; k < ps.parts; ++k) found += ps.slot(k) == slot;
        CHECK(found == 1 && ps.parts >= 1 && ps.parts <= max_join_parts(G));
      }
      at = end;
    }
  }

  // arrivals: one count per group of a piece, then one per piece
  std::map<int, int> word_owner, count, word_owner2, count2;
  std::vector<std::pair<int, int>> events;
  for (int i = 0; i < G; ++i)
    for (int x = 0; x < int(pieces[i].size()); ++x) events.push_back({i, x});
  std::shuffle(events.begin(), events.end(), rng);
  auto join = [&](const Parts& ps, int h) {
    std::vector<std::pair<int64_t, int64_t>> all;
    for (int k = 0; k < ps.parts; ++k) {
      const int s = ps.slot(k);
      if (!slot_owner.count(s) || slot_owner[s] != h || parts[s].empty()) return 1;
      all.insert(all.end(), parts[s].begin(), parts[s].end());
      parts[s].clear();  // taken: nothing may take it again
    }
    for (size_t k = 1; k < all.size(); ++k)
      if (all[k].first != all[k - 1].second) return 1;  // in the order of the keys
    parts[ps.slot0] = all;
    return 0;
  };
  auto complete = [&](int slot, int h) {
    const auto& p = parts[slot];
    return !p.empty() && p.front().first == first[h] && p.back().second == first[h] + units[h];
  };
  for (const auto& e : events) {
    const Mine& m = pieces[e.first][e.second];
    const Parts ps = m.pc.group(e.first);
    if (!word_owner.count(ps.slot0)) word_owner[ps.slot0] = m.h;
    CHECK(word_owner[ps.slot0] == m.h);
    if (++count[ps.slot0] < ps.parts) continue;
    CHECK(count[ps.slot0] == ps.parts);
    CHECK(join(ps, m.h) == 0);
    if (m.pc.direct()) {
      CHECK(complete(ps.slot0, m.h));
      ++done[m.h];
      continue;
    }
    const Parts gs = m.pc.groups();
    CHECK(gs.parts >= 2 && gs.parts <= max_join_parts(G));
    if (!word_owner2.count(m.pc.slot0)) word_owner2[m.pc.slot0] = m.h;
    CHECK(word_owner2[m.pc.slot0] == m.h && m.pc.slot0 == gs.slot0);
    if (++count2[m.pc.slot0] < gs.parts) continue;
    CHECK(join(gs, m.h) == 0 && complete(gs.slot0, m.h));
    ++done[m.h];
  }
  for (int n : done) CHECK(n == 1);
  return 0;
}

int main() {
  for (int grid : {1, 2, 3, 15, 16, 17, 31, 32, 33, 34, 47, 48, 49, 304, 456}) {
    for (int n = 1; n <= 3 * grid + 40; ++n) {
      if (walk({n}, grid)) return 1;
      if (walk({n, 1, n}, grid)) return 1;
    }
    for (int t = 0; t < 300; ++t) {
      std::vector<int> units(1 + rng() % 40);
      const int most = 1 << rng() % 13;
      for (int& n : units) n = 1 + rng() % (rng() % 4 ? most : 3);
      if (walk(units, grid)) { std::printf("grid %d\n", grid); return 1; }
    }
  }
  CHECK(max_join_parts(456) <= 40);
  return 0;
}
"""


def test_parts_of_shares_are_joined_once(tmp_path):
    src = tmp_path / "split_check.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "split_check"
    # -ftrapv: a signed overflow aborts the program
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout + p.stderr
