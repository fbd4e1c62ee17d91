// saga_tree.h - how attention of drafted tokens is laid out over columns,
// tiles and CTAs.  Host and device; not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace saga {

constexpr int kTreeTile = 128;     // cache rows per tile (the M of the score product)
constexpr int kTreeMaxCols = 128;  // query columns of one CTA's products
constexpr int kTreeMaxStages = 12;

// The query rows of one (batch row, key head) are its G = h_q / h_k heads by T
// tokens, one column of the products each.  Columns that share a value head
// are neighbours and padded to the product's column unit; a chunk is as many
// value heads as fit 128 columns, or a part of one value head's columns.
// Column r of a value head is head r / T, token r % T.
struct TreePlan {
  int nvh;     // value heads of a key head's group (1 where several key heads share a value head)
  int hpv;     // query heads of the group per value head
  int rows;    // hpv * T columns of a value head, before padding
  int nv;      // value heads per chunk (the last chunk of a group may have fewer)
  int rsplit;  // chunks that one value head is cut into (nv == 1), else 1
  int rpc;     // columns of a value head per chunk, before padding
  int nvp;     // the same, padded
  int chunks;  // chunks per key head
  int cols;    // columns of a chunk: nv * nvp
  int groups;  // 8-column groups with a live column, per value head of a chunk
};

// 8-bit weights: the columns of a value head in the second product, which are
// its column groups in three pieces one after the other, padded.
__host__ __device__ inline int tree_piece_cols(int groups) { return (3 * 8 * groups + 15) / 16 * 16; }

// 8-bit: the accumulators, which have a column per piece, and two buffers of
// scores fit the 512 columns of TMEM.
__host__ __device__ inline TreePlan tree_plan(int h_q, int h_k, int h_v, int T, bool e4m3) {
  TreePlan p;
  const int G = h_q / h_k, per_v = h_q / h_v;
  p.hpv = per_v < G ? per_v : G;
  p.nvh = G / p.hpv;
  p.rows = p.hpv * T;
  const int unit = 16;  // columns that a product with M = 128 is made of
  const int padded = (p.rows + unit - 1) / unit * unit;
  if (padded <= kTreeMaxCols) {
    int per = kTreeMaxCols / padded;
    const int room = 512 / (2 * padded + tree_piece_cols((p.rows + 7) / 8));
    if (e4m3 && per > room) per = room > 0 ? room : 1;
    p.chunks = (p.nvh + per - 1) / per;
    p.nv = (p.nvh + p.chunks - 1) / p.chunks;
    p.chunks = (p.nvh + p.nv - 1) / p.nv;
    p.rsplit = 1;
    p.rpc = p.rows;
    p.nvp = padded;
  } else {
    p.rsplit = (p.rows + kTreeMaxCols - 1) / kTreeMaxCols;
    p.rpc = (p.rows + p.rsplit - 1) / p.rsplit;
    p.rsplit = (p.rows + p.rpc - 1) / p.rpc;
    p.nvp = (p.rpc + unit - 1) / unit * unit;
    p.nv = 1;
    p.chunks = p.nvh * p.rsplit;
  }
  p.cols = p.nv * p.nvp;
  p.groups = (p.rpc + 7) / 8;
  return p;
}

// The same with queries as the rows of the products (M = 128) and cache rows as
// their columns: a chunk is up to 128 query rows without padding, of as many
// value heads as have room for their d columns of sums in TMEM (256).
__host__ __device__ inline TreePlan tree_plan_rows(int h_q, int h_k, int h_v, int d, int T) {
  TreePlan p;
  const int G = h_q / h_k, per_v = h_q / h_v;
  p.hpv = per_v < G ? per_v : G;
  p.nvh = G / p.hpv;
  p.rows = p.hpv * T;
  if (p.rows <= kTreeMaxCols) {
    int per = kTreeMaxCols / p.rows;
    if (per > 256 / d) per = 256 / d;
    p.chunks = (p.nvh + per - 1) / per;
    p.nv = (p.nvh + p.chunks - 1) / p.chunks;
    p.chunks = (p.nvh + p.nv - 1) / p.nv;
    p.rsplit = 1;
    p.rpc = p.rows;
  } else {
    p.rsplit = (p.rows + kTreeMaxCols - 1) / kTreeMaxCols;
    p.rpc = (p.rows + p.rsplit - 1) / p.rsplit;
    p.rsplit = (p.rows + p.rpc - 1) / p.rpc;
    p.nv = 1;
    p.chunks = p.nvh * p.rsplit;
  }
  p.nvp = p.rpc;
  p.cols = kTreeMaxCols;
  p.groups = 0;
  return p;
}
// Query rows of a chunk of that plan.
__host__ __device__ inline int tree_live_rows(const TreePlan& p) { return p.nv * p.rpc; }

// The work is a line of tiles: batch rows in order, in each its `items`
// (key head, chunk) items in order, in each its tiles.  It is cut in one of
// two ways.  Evenly: CTA i takes the i-th of `ctas` runs of tiles whose lengths
// differ by one at most, wherever items begin and end.  By items: each item of
// batch row b gets a whole number of CTAs, in proportion to its tiles, so that
// no CTA has to change items; a change costs about as much as five tiles (Q and
// the references anew, the sums written out), so this is taken where its
// longest run is not longer than the even one by more.  No CTA has a run
// without tiles between two that have some.  CTA i's partial of item k lies in
// slot i + k: along the line one of the two grows from one partial to the next,
// so no two share a slot.
constexpr int kTreeChange = 5;
constexpr int kTreeMaxCtas = 240;

struct TreeLine {
  const int* prefix;
  const int* counts;  // nullable
  int tokens, l_cap;
  int items;  // of each batch row
};

// The prefix and the tokens of batch row b; false if the prefix was clamped.
__host__ __device__ inline bool tree_lens(const TreeLine& l, int b, int* P, int* n) {
  int c = l.counts != nullptr ? l.counts[b] : l.tokens;
  c = c < 0 ? 0 : c > l.tokens ? l.tokens : c;
  const int given = l.prefix[b];
  *n = c;
  *P = given < 0 ? 0 : given > l.l_cap - c ? l.l_cap - c : given;
  return *P == given;
}
__host__ __device__ inline int tree_tiles(int prefix, int n) { return n > 0 ? (prefix + n + kTreeTile - 1) / kTreeTile : 0; }

// How the line of `total` tiles is cut into runs for `most` <= kTreeMaxCtas
// CTAs.  32 bits hold the tiles (cache rows are below 2^31, chunks of a key
// head at most 64) and the products of an item's tiles with a number of CTAs.
struct TreeCut {
  int total, most;
  bool by_items;
};
// CTAs of each item of a batch row of `tiles` tiles; 0: too few CTAs to cut by items.
__host__ __device__ inline int tree_item_ctas(const TreeCut& c, int tiles) {
  const int x = (int)((unsigned)c.most * (unsigned)tiles / (unsigned)c.total);
  return x < tiles ? x : tiles;
}
// The longest run of such an item.
__host__ __device__ inline int tree_longest(int tiles, int ctas) { return (tiles + ctas - 1) / ctas; }
__host__ __device__ inline int tree_longest_even(const TreeCut& c) { return (c.total + c.most - 1) / c.most; }

// Even runs: the first tile of CTA i, and the CTA of tile x.
__host__ __device__ inline int tree_even_ctas(const TreeCut& c) { return c.total < c.most ? c.total : c.most; }
__host__ __device__ inline int tree_even_first(const TreeCut& c, int i) {
  const int n = tree_even_ctas(c), base = c.total / n, more = c.total - base * n;
  return i * base + (i < more ? i : more);
}
__host__ __device__ inline int tree_even_cta(const TreeCut& c, int x) {
  const int n = tree_even_ctas(c), base = c.total / n, more = c.total - base * n, longer = more * (base + 1);
  return x < longer ? x / (base + 1) : more + (x - longer) / base;
}

// One segment of a CTA's run: tiles [t0, t1) of item `hc` of batch row b.
struct TreeWalk {
  int b, hc, t0, t1, tiles, P, n;
  int left;  // tiles of the run from t0 on
  int item;
};

// What a batch row takes of the axis along which runs are found: CTAs (by
// items) or tiles (even).
__host__ __device__ inline int tree_extent(const TreeLine& l, const TreeCut& c, int tiles) {
  return tiles == 0 ? 0 : l.items * (c.by_items ? tree_item_ctas(c, tiles) : tiles);
}
// Where CTA i starts on that axis; -1: it has nothing (by items, that shows when no batch row holds it).
__host__ __device__ inline int tree_start(const TreeCut& c, int i) {
  if (c.total == 0) return -1;
  return c.by_items ? i : i < tree_even_ctas(c) ? tree_even_first(c, i) : -1;
}
// CTA i's first segment, `place` units into what batch row b takes.
__host__ __device__ inline TreeWalk tree_walk_begin(const TreeLine& l, const TreeCut& c, int i, int b, int place, int P,
                                                    int n) {
  TreeWalk w;
  w.b = b;
  w.P = P;
  w.n = n;
  w.tiles = tree_tiles(P, n);
  if (c.by_items) {
    const int k = tree_item_ctas(c, w.tiles);
    w.hc = place / k;
    const int part = place - w.hc * k;
    w.t0 = (int)((unsigned)part * (unsigned)w.tiles / (unsigned)k);
    w.t1 = (int)((unsigned)(part + 1) * (unsigned)w.tiles / (unsigned)k);
    w.left = w.t1 - w.t0;
  } else {
    w.left = tree_even_first(c, i + 1) - tree_even_first(c, i);
    w.hc = place / w.tiles;
    w.t0 = place - w.hc * w.tiles;
    w.t1 = w.tiles - w.t0 < w.left ? w.tiles : w.t0 + w.left;
  }
  w.item = b * l.items + w.hc;
  return w;
}

__host__ __device__ inline bool tree_walk_next(const TreeLine& l, TreeWalk& w) {
  w.left -= w.t1 - w.t0;
  if (w.left == 0) return false;
  w.t0 = 0;
  if (++w.hc == l.items) {
    w.hc = 0;
    do {  // ends: tiles of the run are left, so a later batch row has some
      ++w.b;
      tree_lens(l, w.b, &w.P, &w.n);
      w.tiles = tree_tiles(w.P, w.n);
    } while (w.tiles == 0);
  }
  w.t1 = w.tiles < w.left ? w.tiles : w.left;
  w.item = w.b * l.items + w.hc;
  return true;
}

// The last CTA of the item whose first tile is CTA i's first segment's (its
// first CTA: t0 == 0) or begins within CTA i's run.  `place`: the item's first
// tile on the line, for even runs.
__host__ __device__ inline int tree_last_holder(const TreeCut& c, int i, int tiles, int place) {
  return c.by_items ? i + tree_item_ctas(c, tiles) - 1 : tree_even_cta(c, place + tiles - 1);
}

// The order of a segment's loads: K(t0), then for every t: K(t + 1) if there
// is one, V(t, 0), V(t, 1), ...  Where V(t0 + i, 0) stands in that order:
__host__ __device__ inline int tree_value_place(int i, int tiles, int nv) { return 1 + i * nv + (i + 1 < tiles ? i + 1 : tiles - 1); }

// Where a query row (head jj of its key head's group, token t) sits.
struct TreeSpot {
  int chunk, col;
};
__host__ __device__ inline TreeSpot tree_spot(const TreePlan& p, int T, int jj, int t) {
  const int v = jj / p.hpv, r = (jj - v * p.hpv) * T + t;
  TreeSpot s;
  if (p.rsplit == 1) {
    s.chunk = v / p.nv;
    s.col = (v - s.chunk * p.nv) * p.nvp + r;
  } else {
    s.chunk = v * p.rsplit + r / p.rpc;
    s.col = r % p.rpc;
  }
  return s;
}

// The query row of a chunk's column: false for padding.
__host__ __device__ inline bool tree_row(const TreePlan& p, int T, int chunk, int col, int* jj, int* t) {
  const int vl = col / p.nvp, c = col - vl * p.nvp;
  int v, r;
  if (p.rsplit == 1) {
    v = chunk * p.nv + vl;
    r = c;
  } else {
    v = chunk / p.rsplit;
    r = (chunk - v * p.rsplit) * p.rpc + c;
  }
  if (vl >= p.nv || v >= p.nvh || c >= p.rpc || r >= p.rows) return false;
  *jj = v * p.hpv + r / T;
  *t = r - r / T * T;
  return true;
}

// Shared memory of the kernel: the tile ring, ones (the operand that adds bf16
// weights up), Q (bf16, or two 8-bit pieces one after the other), two P buffers
// (bf16, or three 8-bit pieces), per-column words, and for 8-bit caches the rows'
// scales of two tiles and the sums of weights.
struct TreeSmem {
  int stages, stage_bytes;
  int ones, q, p, p_bytes, mask, m, tau, cs, f, row, words, sums, scales, bars, total;
};
__host__ __device__ inline TreeSmem tree_smem(const TreePlan& p, int d, bool e4m3, bool by_rows) {
  TreeSmem s;
  s.stage_bytes = kTreeTile * d * (e4m3 ? 1 : 2);
  const int budget = 227 * 1024 - 1024;  // less the slack that aligns the base to 1024 bytes
  const int q_bytes = p.cols * d * 2;
  // by rows the weights are in TMEM
  s.p_bytes = by_rows ? 0 : kTreeTile * (e4m3 ? p.nv * tree_piece_cols(p.groups) : p.cols * 2);
  const int words = p.cols * (8 + 5 * 4 + 4 * 4);
  const int sums = by_rows || !e4m3 ? 0 : 2 * p.cols * 4 * 4;
  const int eight = e4m3 ? sums + 2 * (by_rows ? 1 : 2) * (1 + p.nv) * kTreeTile * 4 : 0;
  const int bar_bytes = 8 * (3 * kTreeMaxStages + 16) + 16 + (int)(sizeof(TreeWalk) + sizeof(TreeCut));
  const int fixed = 2048 + q_bytes + 2 * s.p_bytes + words + eight + bar_bytes;
  s.stages = (budget - fixed) / s.stage_bytes;
  if (s.stages > kTreeMaxStages) s.stages = kTreeMaxStages;
  s.ones = s.stages * s.stage_bytes;
  s.q = s.ones + 2048;
  s.p = s.q + q_bytes;
  s.mask = s.p + 2 * s.p_bytes;
  s.m = s.mask + p.cols * 8;
  s.tau = s.m + p.cols * 4;
  s.cs = s.tau + p.cols * 4;
  s.f = s.cs + p.cols * 4;
  s.row = s.f + p.cols * 4;
  s.words = s.row + p.cols * 4;
  s.sums = s.words + p.cols * 16;
  s.scales = s.sums + sums;
  s.bars = s.words + p.cols * 16 + eight;
  s.total = s.bars + bar_bytes + 1024;
  return s;
}

}  // namespace saga
