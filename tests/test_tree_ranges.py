"""Host-side index logic of the drafted-token attention, compiled with g++ and run on the CPU: every query row has
one column of one chunk and back, columns and shared memory stay within their limits, the CTAs' shares cover every
tile of every item once and in order, partials never share a slot and are all written, and a tile's values stand
where the order of a segment's loads has them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_decoding_saga_b200", "csrc")

PROGRAM = r"""
#define __host__
#define __device__
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <vector>
#include "saga_tree.h"
using namespace saga;

static int fails = 0;
#define CHECK(c, ...) do { if (!(c)) { ++fails; if (fails < 20) { std::printf(__VA_ARGS__); std::printf("\n"); } } } while (0)

static const int Ts[] = {1, 2, 3, 4, 5, 7, 8, 12, 16, 31, 32, 33, 48, 63, 64};
static void plans() {
  for (int h_k = 1; h_k <= 8; ++h_k) for (int h_v = 1; h_v <= 32; ++h_v) for (int d = 64; d <= 128; d += 64)
    for (int h_q = 1; h_q <= 64; ++h_q) {
      if (h_q % h_k || h_q % h_v || (h_v % h_k && h_k % h_v) || h_q / h_k > (d == 64 ? 64 : 32)) continue;
      if (h_v > h_k && h_v / h_k > 32) continue;
      for (int T : Ts) {
        for (int which = 0; which < 3; ++which) {  // columns, columns of 8-bit weights, rows
          const bool by_rows = which == 2;
          const TreePlan p = by_rows ? tree_plan_rows(h_q, h_k, h_v, d, T) : tree_plan(h_q, h_k, h_v, T, which == 1);
          // 8-bit weights come as columns only where a chunk by rows has fewer than 56 rows
          if (which == 1) {
            if (tree_live_rows(tree_plan_rows(h_q, h_k, h_v, d, T)) >= 56) continue;
            const int pieces = tree_piece_cols(p.groups);
            CHECK(pieces <= 256 && pieces >= 24 * p.groups && 2 * p.cols + p.nv * pieces <= 512, "pieces");
          }
          const int G = h_q / h_k;
          CHECK(p.cols <= kTreeMaxCols && p.cols % 16 == 0 && p.nv * p.nvp <= p.cols, "cols");
          if (by_rows) CHECK(p.nv * d <= 256 && tree_live_rows(p) <= 128, "rows");
          else CHECK(p.nvp % 16 == 0 && p.groups * 8 <= p.nvp && p.groups >= 1, "groups");
          CHECK(p.hpv * p.nvh == G, "heads");
          std::map<std::pair<int, int>, int> seen;
          for (int jj = 0; jj < G; ++jj) for (int t = 0; t < T; ++t) {
            const TreeSpot s = tree_spot(p, T, jj, t);
            CHECK(s.chunk >= 0 && s.chunk < p.chunks && s.col >= 0 && s.col < p.nv * p.nvp, "spot of %d %d", jj, t);
            const int uses = ++seen[std::make_pair(s.chunk, s.col)];
            CHECK(uses == 1, "two rows in one column");
            int j2 = -1, t2 = -1;
            CHECK(tree_row(p, T, s.chunk, s.col, &j2, &t2) && j2 == jj && t2 == t, "row of column");
            // its value head is the one whose columns these are
            const int vl = s.col / p.nvp, v0 = p.rsplit == 1 ? s.chunk * p.nv : s.chunk / p.rsplit;
            CHECK(((v0 + vl) * p.hpv) / (h_q / h_v) == jj / (h_q / h_v), "value head");
          }
          int live = 0;
          for (int c = 0; c < p.chunks; ++c) for (int col = 0; col < p.cols; ++col) {
            int a, b;
            live += tree_row(p, T, c, col, &a, &b);
          }
          CHECK(live == G * T, "live columns %d of %d", live, G * T);
          for (int e = 0; e < 2; ++e) {
            if (which < 2 && e != which) continue;
            const TreeSmem s = tree_smem(p, d, e != 0, by_rows != 0);
            // rows: what the stages of a tile's values held before is older than the tile's keys
            if (by_rows) CHECK(s.stages >= 2 * p.nv + 1, "stages %d of %d value heads", s.stages, p.nv);
            CHECK(s.stages >= 3 && s.stages <= kTreeMaxStages && s.total <= 227 * 1024, "smem %d stages %d", s.total, s.stages);
            CHECK(s.ones % 1024 == 0 && s.q % 1024 == 0 && s.p % 1024 == 0 && s.m % 16 == 0 && s.f % 16 == 0 && s.bars % 8 == 0, "smem alignment");
          }
        }
      }
    }
}

static void lines() {
  int by_items = 0;
  std::srand(1);
  for (int round = 0; round < 3000; ++round) {
    const int B = 1 + std::rand() % 40, items = 1 + std::rand() % 9, T = 1 + std::rand() % 64, cap = 64 + std::rand() % 3000;
    const int most = (round % 3 == 0) ? 148 : (round % 3 == 1) ? 600 : 1 + std::rand() % 20, nv = 1 + std::rand() % 5;
    std::vector<int> prefix(B), counts(B);
    for (int b = 0; b < B; ++b) {
      prefix[b] = std::rand() % 5 == 0 ? 0 : std::rand() % (cap + 50) - 20;
      counts[b] = std::rand() % 4 == 0 ? 0 : std::rand() % (T + 3) - 1;
    }
    const TreeLine line{prefix.data(), round % 2 ? counts.data() : nullptr, T, cap, items};
    TreeCut cut{0, most, false};
    for (int b = 0; b < B; ++b) {
      int P, n;
      tree_lens(line, b, &P, &n);
      CHECK(P >= 0 && n >= 0 && P + n <= cap, "lens");
      cut.total += items * tree_tiles(P, n);
    }
    bool can = cut.total > 0;
    int longest = 0;
    for (int b = 0; b < B; ++b) {
      int P, n;
      tree_lens(line, b, &P, &n);
      const int tiles = tree_tiles(P, n);
      if (tiles == 0) continue;
      const int k = tree_item_ctas(cut, tiles);
      can = can && k > 0;
      if (k > 0 && tree_longest(tiles, k) > longest) longest = tree_longest(tiles, k);
    }
    cut.by_items = can && (round % 4 < 2);
    by_items += cut.by_items;
    std::vector<int> before(B + 1, 0), tiles_before(B + 1, 0);
    for (int b = 0; b < B; ++b) {
      int P, n;
      tree_lens(line, b, &P, &n);
      before[b + 1] = before[b] + tree_extent(line, cut, tree_tiles(P, n));
      tiles_before[b + 1] = tiles_before[b] + items * tree_tiles(P, n);
    }
    CHECK(!cut.by_items || before[B] <= most, "by items: %d CTAs of %d", before[B], most);
    int x = 0, longest_seen = 0;
    std::set<long long> slots;
    std::map<int, std::pair<int, int>> held;  // item -> first and last CTA
    std::map<int, int> told;                   // item -> what its first CTA says is its last
    for (int i = 0; i < most; ++i) {
      const int at = tree_start(cut, i);
      if (at < 0 || at >= before[B]) continue;
      int b = 0;
      while (before[b + 1] <= at) ++b;
      int P, n;
      tree_lens(line, b, &P, &n);
      TreeWalk w = tree_walk_begin(line, cut, i, b, at - before[b], P, n);
      CHECK(w.left >= 1, "empty run");
      if (w.left > longest_seen) longest_seen = w.left;
      bool more = true;
      while (more) {
        CHECK(w.t0 < w.t1 && w.t1 <= w.tiles && w.hc < items && w.t1 - w.t0 <= w.left, "segment");
        CHECK(w.item == w.b * items + w.hc, "item");
        CHECK(slots.insert((long long)i + w.item).second, "slot used twice");
        CHECK(i + w.item < most + (long long)B * items, "slot out of range");
        if (!held.count(w.item)) held[w.item] = std::make_pair(i, i);
        CHECK(held[w.item].second >= i - 1, "a CTA between has no partial");
        held[w.item].second = i;
        if (w.t0 == 0) told[w.item] = tree_last_holder(cut, i, w.tiles, tiles_before[w.b] + w.hc * w.tiles);
        CHECK(told.count(w.item) == 1, "an item's first tile comes first");
        CHECK(w.t1 == w.tiles ? told[w.item] == i : told[w.item] > i, "last holder %d, CTA %d", told[w.item], i);
        for (int t = w.t0; t < w.t1; ++t, ++x)
          CHECK(x == tiles_before[w.b] + w.hc * w.tiles + t, "tile order");
        // the loads: K(t0), then K(t + 1), V(t, ...)
        std::vector<std::pair<int, int>> want;
        want.push_back({w.t0, -1});
        for (int t = w.t0; t < w.t1; ++t) {
          if (t + 1 < w.t1) want.push_back({t + 1, -1});
          CHECK((int)want.size() == tree_value_place(t - w.t0, w.t1 - w.t0, nv), "place of the values");
          for (int v = 0; v < nv; ++v) want.push_back({t, v});
        }
        more = tree_walk_next(line, w);
      }
    }
    CHECK(x == cut.total, "tiles covered %d of %d", x, cut.total);
    if (cut.by_items) CHECK(longest_seen == longest, "longest run");
    else CHECK(cut.total == 0 || longest_seen == tree_longest_even(cut), "longest even run");
  }
  CHECK(by_items > 100, "few lines cut by items: %d", by_items);
}

int main() {
  plans();
  lines();
  std::printf(fails ? "%d failures\n" : "ok\n", fails);
  return fails != 0;
}
"""


def test_plan_shares_and_feed(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src = tmp_path / "t.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "t"
    subprocess.run(["g++", "-O1", "-std=c++17", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
