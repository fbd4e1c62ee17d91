// saga_tree.cu - attention of drafted tokens (a tree, a chain or one token)
// over a bf16 or 8-bit cache: saga_tree_attn.
//
// The query rows of a key head are the columns of two products per tile of 128
// cache rows (saga_tree.h):
//   S[row, col]  = K[row, :] . q[col, :]             tcgen05, M = 128 rows of the tile
//   O[d, col]   += sum_row V[row, d] P[row, col]     tcgen05, M = d, the tile as the inner dimension
// Cache rows are the lanes and queries the columns, so that few queries cost
// little (columns are padded to 8 or 16, rows never), a tile's value heads each
// take their own columns of P (a value head with its own rows is the case that
// SAGA's h_k < h_v brings), and what belongs to a cache row (its scale, whether
// a drafted token sees it) is a thread's own.  V as it lies in memory is the
// transposed operand, so nothing is transposed.
//
// P = 2^(x - m) with x the score in powers of two and m a reference per column.
// The softmax needs no exact maximum: any m within the range of the weights'
// exponents gives the same quotient.  So m comes from the first tile and is
// moved only when a score rises too far above it, which one comparison per
// score and one vote per tile watch for; then the accumulators are rescaled and
// the tile is done again.
//
// bf16 caches: weights are rounded to bf16, and what they are divided by is the
// sum of the rounded weights: a row of ones beside V in the second product adds
// them up in fp32.  Where a value head has at most 8 columns, half of its 16 are
// padding, and what a weight lost in rounding goes there as a second bf16 number:
// the same products then give outputs as exact as fp32 weights do.
//
// 8-bit caches: the codes go to the tensor cores as they are (kind::f8f6f4), so
// a tile is read once, by TMA, and nothing is widened.  The other operands are
// given in pieces: q, scaled by a power of two that brings the row's largest
// element into [128, 256), as the sum of two e4m3 numbers (4 + 4 of bf16's 8 bits:
// exact down to 2^-9 of 128, smaller elements off by at most 2^-17 of it), whose
// products add up in the same accumulators; the weights as the sum of three e5m2
// numbers (each off by 2^-3 of what is left: 2^-9; with two the error of an output
// over a long cache was twice that of rounding it).  e5m2 ends at 2^-16, and the
// largest weight of a segment's first tile is put at 2^10: weights below 2^-18 of
// it have fewer bits, and those below 2^-27 of it are left out of the products,
// though not of the sum that they are divided by.  With
// queries as columns the pieces are columns of one product, added at a segment's
// end: a product of 48 columns takes little longer than one of 16 (one token
// over 128K rows 34.9 -> 30.7 us).
// A key row's scale multiplies its scores and a value row's scale its weights,
// both in fp32 and before any rounding; the sums of weights are fp32 sums of the
// unrounded ones (so a NaN score, whose pieces would be zeros, still shows).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "saga_device.cuh"
#include "saga_launch.cuh"
#include "saga_serve.h"

namespace saga {
namespace {

constexpr float kUnset = -1e37f;      // a column's reference before any kept score
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kEpiWarp0 = 4, kEpiAll = 256, kTreeThreads = kEpiWarp0 * 32 + kEpiAll;
// How far (in powers of two) a weight may rise above its column's reference:
// bf16 has fp32's exponents; e5m2 ends below 2^16.
constexpr float kOverBf16 = 32.f, kOverE5m2 = 15.f;
// Where the first tile's largest weight is put: e5m2's smallest numbers are
// 2^-16, so rows down to 2^-26 of the largest still count.
constexpr float kTopE5m2 = 10.f;
constexpr float kMinScale = 8.271806125530277e-25f;  // 2^-80: smaller value scales do not lower the reference

// ------------------------------------------------------------------ the line of tiles
__device__ __forceinline__ TreeLine line_of(const TreeParams& p) {
  return TreeLine{p.prefix_lens, p.counts, p.tokens, p.l_cap, p.h_k * p.plan.chunks};
}

__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }
__device__ __forceinline__ int warp_scan(int x) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane_id() >= o) x += y;
  }
  return x;
}

// The cut of the line (a whole warp calls; the same in every warp of both kernels).
__device__ __forceinline__ TreeCut cut_of(const TreeLine& line, int batch, int most, bool* clamped) {
  TreeCut c{0, most, false};
  int P = 0, n = 0;
  for (int b = lane_id(); b < batch; b += 32) {
    if (!tree_lens(line, b, &P, &n)) *clamped = true;
    c.total += line.items * tree_tiles(P, n);
  }
  c.total = warp_sum(c.total);
  *clamped = __any_sync(0xffffffffu, *clamped);
  if (c.total == 0) return c;
  int fewest = 1 << 30, longest = 0;
  for (int b = lane_id(); b < batch; b += 32) {
    if (batch > 32) tree_lens(line, b, &P, &n);  // else it is the one just read
    const int tiles = tree_tiles(P, n);
    if (tiles == 0) continue;
    const int k = tree_item_ctas(c, tiles);
    fewest = min(fewest, k);
    if (k > 0) longest = max(longest, tree_longest(tiles, k));
  }
  fewest = __reduce_min_sync(0xffffffffu, fewest);
  longest = __reduce_max_sync(0xffffffffu, longest);
  c.by_items = fewest > 0 && longest <= tree_longest_even(c) + kTreeChange;
  return c;
}

// Heads of a segment.
struct Heads {
  int kh, chunk, nv;  // key head, chunk, value heads here
  size_t key, value;  // cache row 0 of the key head and of the first value head (the others follow, l_cap rows apart)
};
__device__ __forceinline__ Heads heads_of(const TreeParams& p, const TreeWalk& w) {
  Heads h;
  h.kh = w.hc / p.plan.chunks;
  h.chunk = w.hc - h.kh * p.plan.chunks;
  const int v0 = p.plan.rsplit == 1 ? h.chunk * p.plan.nv : h.chunk / p.plan.rsplit;  // of the group
  h.nv = p.plan.rsplit == 1 ? min(p.plan.nv, p.plan.nvh - v0) : 1;
  h.key = ((size_t)w.b * p.h_k + h.kh) * p.l_cap;
  const int vh = p.h_v > p.h_k ? h.kh * p.plan.nvh + v0 : h.kh * p.h_v / p.h_k;
  h.value = ((size_t)w.b * p.h_v + vh) * p.l_cap;
  return h;
}

// Drafted tokens that any present token sees (the whole warp calls).
__device__ __forceinline__ unsigned long long seen_by_any(const TreeParams& p, const TreeWalk& w) {
  const unsigned long long all = w.n >= 64 ? ~0ull : (1ull << w.n) - 1ull;
  if (p.mask == nullptr) return all;
  unsigned long long u = 0;
  for (int t = lane_id(); t < w.n; t += 32) u |= p.mask[(size_t)w.b * p.tokens + t];
  const unsigned lo = __reduce_or_sync(0xffffffffu, (unsigned)u), hi = __reduce_or_sync(0xffffffffu, (unsigned)(u >> 32));
  return all & ((unsigned long long)hi << 32 | lo);
}

// Whether a cache row is one that some token of the batch row sees.
__device__ __forceinline__ bool row_seen(const TreeWalk& w, unsigned long long seen, int row) {
  return row < w.P || (row < w.P + w.n && (seen >> (row - w.P) & 1ull));
}

// ------------------------------------------------------------------ tcgen05 pieces beyond saga_device.cuh
// Shared-memory matrix descriptors (addresses, distances in bytes).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride, uint32_t layout) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)layout << 61);
}
constexpr uint32_t kLayoutPlain = 0, kLayout128 = 2, kLayout64 = 4;
// K tile and Q: rows of the inner dimension, 8-row groups 8 rows apart.
template <int D, bool E4M3>
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
  return E4M3 && D == 64 ? smem_desc(addr, 16, 512, kLayout64) : smem_desc(addr, 16, 1024, kLayout128);
}
// V tile: the product's M (d) dense, 8-row groups of the inner dimension one
// after the other.  bf16: 64-element blocks `block` bytes apart; for d = 64 the
// second block of the M = 128 product is the ones.
template <int D, bool E4M3>
__device__ __forceinline__ uint64_t desc_v(uint32_t addr, uint32_t block) {
  return E4M3 && D == 64 ? smem_desc(addr, block, 512, kLayout64) : smem_desc(addr, block, 1024, kLayout128);
}
// P: N (columns) dense in 16-byte groups; the 8-row blocks of a column group
// lie 128 bytes apart, column groups 2048 bytes.
__device__ __forceinline__ uint64_t desc_p(uint32_t addr) { return smem_desc(addr, 128, 2048, kLayoutPlain); }

// Instruction descriptor: fp32 sums; a, b: operand formats of the kind.
__host__ __device__ constexpr uint32_t idesc(uint32_t a, uint32_t b, int M, int N, bool transposed) {
  return (1u << 4) | (a << 7) | (b << 10) | (transposed ? 3u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kBf16 = 1;            // kind::f16
constexpr uint32_t kE4m3 = 0, kE5m2 = 1; // kind::f8f6f4

__device__ __forceinline__ void umma_8bit(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(id), "r"(accumulate)
      : "memory");
}

// 8 columns of this thread's lane: the load, and the wait after which they may be read.
__device__ __forceinline__ void tmem_ld8_start(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8_end(uint32_t* r, float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  tmem_ld8_start(taddr, r);
  tmem_ld8_end(r, v);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(__float_as_uint(v[0])),
      "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
      "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(taddr)
      : "memory");
}

// One lane of a converged warp.  Code under it issues tensor-core and copy
// instructions from uniform registers: under a test of the lane number each
// product took about 150 clocks to issue, under this about 40.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A threshold that is no number keeps nothing.
__device__ __forceinline__ float threshold(float tau) { return tau == tau ? tau : INFINITY; }

// What a row's products are multiplied by, from the sum of its weights: 0 where
// nothing was kept, and NaN where the sum is no number, so that a NaN among what
// the row sees shows in its output.
__device__ __forceinline__ float inverse_of(float sum) { return sum == 0.f ? 0.f : sum < INFINITY ? 1.f / sum : NAN; }

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return reinterpret_cast<const __half2&>(x); }
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t&>(h);
}
// Two weights as three e5m2 numbers each, in the upper bytes of the halves.  An
// e5m2 number is the upper byte of a half-precision one, so a piece is that
// byte rounded and the rest an exact subtraction away: no conversions, which
// were half of a tile's time.
__device__ __forceinline__ void pieces_of(float a, float b, uint32_t& first, uint32_t& second, uint32_t& third) {
  const uint32_t all = pack_half(a, b);
  first = (all + 0x00800080u) & 0xff00ff00u;
  __half2 rest = __hsub2(as_half2(all), as_half2(first));
  second = (reinterpret_cast<const uint32_t&>(rest) + 0x00800080u) & 0xff00ff00u;
  rest = __hsub2(rest, as_half2(second));
  third = reinterpret_cast<const uint32_t&>(rest) + 0x00800080u;
}
// Two numbers as an 8-bit format each, in the low 16 bits, and back.
__device__ __forceinline__ uint32_t pack_8bit(float a, float b, __nv_fp8_interpretation_t f) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, f);
}
__device__ __forceinline__ float2 unpack_8bit(uint32_t x, __nv_fp8_interpretation_t f) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)x, f);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t&>(h);
}

__device__ __forceinline__ void cp_async4_zfill(void* smem_dst, const void* gsrc, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(smem_dst)),
               "l"(reinterpret_cast<uint64_t>(gsrc)), "r"(valid ? 4 : 0)
               : "memory");
}

// A position in the tile ring.
struct Ring {
  int st = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void step(int stages) {
    if (++st == stages) {
      st = 0;
      ++round;
    }
  }
  __device__ __forceinline__ void jump(int by, int stages) {
    const int x = st + by;
    round += x / stages;
    st = x % stages;
  }
};

struct Bars {
  uint64_t *full, *empty, *vfix;       // per stage
  uint64_t *s_full, *s_empty;          // per score buffer
  uint64_t *p_full, *pv_done;          // per P buffer
  uint64_t *q_full, *drain;
};

// The column groups (8 live columns or fewer, the rest padding) of a
// warpgroup: `count` of them from `col` on, `groups` to a value head of `nvp`
// columns, the first of them the `at`-th of its value head; v counts the value
// heads from the warpgroup's first on.
// pcol: the group's first column among the 8-bit weights' first pieces.
struct Groups {
  int col, at, v, count, groups, nvp, pcol, pcols;
  __device__ __forceinline__ void step() {
    col += 8;
    pcol += 8;
    if (++at == groups) {
      at = 0;
      ++v;
      col += nvp - groups * 8;
      pcol += pcols - groups * 8;
    }
  }
};

// What a thread's cache row is to the columns of a tile.
struct Row {
  float f;                 // score factor, without the columns'
  bool all;                // every column sees the row
  bool live;               // some column does
  unsigned long long bit;  // else the drafted token in it (0: none)
  const float* scale;      // 8-bit: value scales of the row, the v-th kTreeTile words on
};

// The columns' words: the reference, negated; the threshold and the score
// factor (8-bit: both in powers of two); which drafted rows the column sees.
struct Columns {
  float *m, *tau, *cs;
  unsigned long long* mask;
};

__device__ __forceinline__ void load8(const float* from, float* to) {
  *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(from);
  *reinterpret_cast<float4*>(to + 4) = *reinterpret_cast<const float4*>(from + 4);
}

// Two fp32 products (and sums) at once: the weights of a tile are bound by the
// instructions issued for them.
__device__ __forceinline__ unsigned long long two(float a, float b) {
  unsigned long long x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ void untwo(unsigned long long x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long x;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
  return x;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long x;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(a), "l"(b), "l"(c));
  return x;
}

// Scores of 8 columns in powers of two, less the columns' references with
// RELATIVE; with TEST -inf where the row is hidden or the score below the
// threshold (a row of the prefix is hidden from nobody: no masks are read).
// bf16 compares fl(product * scale) with the threshold, as the decode calls do.
template <bool E4M3, bool TEST, bool RELATIVE>
__device__ __forceinline__ void exponents(float* s, const Row& r, int col, const Columns& c) {
  float mm[8], cc[8], tt[8];
  if (RELATIVE) load8(c.m + col, mm);
  if (E4M3) load8(c.cs + col, cc);
  if (TEST) load8(c.tau + col, tt);
  unsigned seen = 0xffu;
  if (TEST && !r.all) {
    seen = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(c.mask + col + 2 * i);
      if ((x.x & r.bit) != 0ull) seen |= 1u << (2 * i);
      if ((x.y & r.bit) != 0ull) seen |= 2u << (2 * i);
    }
  }
  const float f = E4M3 || TEST ? r.f : r.f * kLog2e;
  const unsigned long long ff = two(f, f), ll = two(kLog2e, kLog2e);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    unsigned long long x = two(s[i], s[i + 1]);
    bool keep0 = true, keep1 = true;
    if (TEST) {
      x = mul2(x, ff);
      if (E4M3) x = mul2(x, two(cc[i], cc[i + 1]));
      float a, b;
      untwo(x, a, b);
      keep0 = !(a < tt[i]) && (seen >> i & 1u) != 0u;  // a NaN stays, so that it shows
      keep1 = !(b < tt[i + 1]) && (seen >> i & 2u) != 0u;
      if (RELATIVE) x = fma2(x, E4M3 ? two(1.f, 1.f) : ll, two(mm[i], mm[i + 1]));
      else if (!E4M3) x = mul2(x, ll);
    } else if (E4M3) {
      x = mul2(x, ff);
      x = RELATIVE ? fma2(x, two(cc[i], cc[i + 1]), two(mm[i], mm[i + 1])) : mul2(x, two(cc[i], cc[i + 1]));
    } else {
      x = RELATIVE ? fma2(x, ff, two(mm[i], mm[i + 1])) : mul2(x, ff);
    }
    untwo(x, s[i], s[i + 1]);
    if (TEST) {
      s[i] = keep0 ? s[i] : -INFINITY;
      s[i + 1] = keep1 ? s[i + 1] : -INFINITY;
    }
  }
}

// 8 columns' sums over the 32 lanes; lane 4 c holds column octet_column(lane).
__device__ __forceinline__ int octet_column(int lane) { return (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1); }
__device__ __forceinline__ float octet_sum(const float* v, int lane) {
  float a[4], b[2], c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float mine = lane & 16 ? v[4 + i] : v[i], other = lane & 16 ? v[i] : v[4 + i];
    a[i] = mine + __shfl_xor_sync(0xffffffffu, other, 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float mine = lane & 8 ? a[2 + i] : a[i], other = lane & 8 ? a[i] : a[2 + i];
    b[i] = mine + __shfl_xor_sync(0xffffffffu, other, 8);
  }
  {
    const float mine = lane & 4 ? b[1] : b[0], other = lane & 4 ? b[0] : b[1];
    c = mine + __shfl_xor_sync(0xffffffffu, other, 4);
  }
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  c += __shfl_xor_sync(0xffffffffu, c, 1);
  return c;
}

// Weights of a tile into P; returns the largest exponent of the thread's.
// bf16: a row of P is 16 bytes per 8 columns.  8-bit: 8 bytes per 8 columns of
// each of three pieces, which are columns of their own; and the weights' sums
// over the warp's rows into here[column] (a tile that is done again overwrites them).
template <bool E4M3, bool TEST>
__device__ __forceinline__ float weigh(uint32_t s_tmem, uint8_t* p_row, float* here, Groups g, const Row& r,
                                       const Columns& c) {
  float top = -INFINITY;
  const int lane = lane_id();
  uint32_t raw[8];
  if (g.count > 0) tmem_ld8_start(s_tmem + g.col, raw);
#pragma unroll 1
  for (int n = g.count; n > 0; --n) {
    float s[8];
    tmem_ld8_end(raw, s);
    const int col = g.col, pcol = g.pcol;
    const float vs = E4M3 && r.live ? r.scale[g.v * kTreeTile] : 0.f;
    g.step();
    if (n > 1) tmem_ld8_start(s_tmem + g.col, raw);  // the next group's scores, while this one's are weighed
    exponents<E4M3, TEST, true>(s, r, col, c);
    if (!E4M3) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        top = fmaxf(top, s[i]);
        s[i] = ex2(s[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16(s[2 * i], s[2 * i + 1]);
      *reinterpret_cast<uint4*>(p_row + (col >> 3) * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
      if (g.groups == 1) {  // what was rounded off, into the padding
        uint32_t z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          z[i] = pack_bf16(s[2 * i] - __uint_as_float(w[i] << 16), s[2 * i + 1] - __uint_as_float(w[i] & 0xffff0000u));
        *reinterpret_cast<uint4*>(p_row + ((col >> 3) + 1) * 2048) = make_uint4(z[0], z[1], z[2], z[3]);
      }
    } else {
      float most = s[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) most = fmaxf(most, s[i]);
      top = fmaxf(top, most + __log2f(fmaxf(vs, kMinScale)));
      uint32_t w[4], z[4], y[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = ex2(s[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        untwo(mul2(two(s[2 * i], s[2 * i + 1]), two(vs, vs)), a, b);
        pieces_of(a, b, w[i], z[i], y[i]);
      }
      auto put = [&](int c, const uint32_t* x) {
        *reinterpret_cast<uint2*>(p_row + (c >> 4) * 2048 + (c & 8)) = make_uint2(__byte_perm(x[0], x[1], 0x7531), __byte_perm(x[2], x[3], 0x7531));
      };
      put(pcol, w);
      put(pcol + g.groups * 8, z);
      put(pcol + g.groups * 16, y);
      const float sum = octet_sum(s, lane);
      if ((lane & 3) == 0) here[col + octet_column(lane)] = sum;
    }
  }
  return top;
}

// The columns' largest weights over the warp's rows, in powers of two, into
// the column's word of this warp.
template <bool E4M3>
__device__ __forceinline__ void maxima(uint32_t s_tmem, float* words, Groups g, const Row& r, const Columns& c) {
#pragma unroll 1
  for (int n = g.count; n > 0; --n, g.step()) {
    float s[8];
    tmem_ld8(s_tmem + g.col, s);
    exponents<E4M3, true, false>(s, r, g.col, c);
    // (the scale of a row that no token sees may be anything, an infinity too)
    const float lv = E4M3 && r.live ? __log2f(fmaxf(r.scale[g.v * kTreeTile], kMinScale)) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t k = __reduce_max_sync(0xffffffffu, float_key(s[i] + lv));
      if (lane_id() == 0) words[(g.col + i) * 4 + (threadIdx.x >> 5 & 3)] = key_float(k);
    }
  }
}

// ------------------------------------------------------------------ parts of both kernels
// A CTA's shared memory by name, and its place.
struct Block {
  uint8_t* smem;
  Bars bar;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  TreeWalk* share;  // left == 0: this CTA has no tiles
  TreeCut* share_cut;
  int warp, lane;
};

__device__ __forceinline__ Block block_of(const TreeParams& p, uint8_t* smem_raw) {
  Block k;
  k.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bar = k.bar;
  bar.full = reinterpret_cast<uint64_t*>(k.smem + p.smem.bars);
  bar.empty = bar.full + kTreeMaxStages;
  bar.vfix = bar.empty + kTreeMaxStages;
  bar.s_full = bar.vfix + kTreeMaxStages;
  bar.s_empty = bar.s_full + 2;
  bar.p_full = bar.s_empty + 2;
  bar.pv_done = bar.p_full + 2;
  bar.q_full = bar.pv_done + 2;
  bar.drain = bar.q_full + 1;
  k.tmem_slot = reinterpret_cast<uint32_t*>(bar.drain + 1);
  k.abort_flag = reinterpret_cast<volatile int*>(k.tmem_slot + 1);
  k.share = reinterpret_cast<TreeWalk*>(k.tmem_slot + 2);
  k.share_cut = reinterpret_cast<TreeCut*>(k.share + 1);
  k.warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  k.lane = threadIdx.x & 31;
  return k;
}

// Barriers, TMEM, and after the dependency wait this CTA's run of the line.
template <int D>
__device__ __forceinline__ void block_start(const TreeParams& p, const Block& k, const CUtensorMap* kmap,
                                            const CUtensorMap* vmap, uint32_t tmem_cols) {
  const Bars& bar = k.bar;
  const int warp = k.warp, lane = k.lane;
  if (threadIdx.x == 0) {
    *k.abort_flag = 0;
    for (int i = 0; i < p.smem.stages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
      mbar_init(&bar.vfix[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.s_empty[i], 8);
      mbar_init(&bar.p_full[i], 8);
      mbar_init(&bar.pv_done[i], 1);
    }
    mbar_init(bar.q_full, 8);
    mbar_init(bar.drain, 32);
    mbar_init_fence();
    tma_prefetch_desc(kmap);
    tma_prefetch_desc(vmap);
  }
  if (warp == 1) {
    tmem_alloc(k.tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  if (warp == 3) {
    // lines that the start needs, into L2 before the dependency wait: a prefetch moves no values
    if (lane == 0) prefetch_l2_line(p.prefix_lens);
    if (lane == 1 && p.counts != nullptr) prefetch_l2_line(p.counts);
    const long long q_lines = (long long)p.batch * p.tokens * p.h_q * D / 64;
    for (long long i = (long long)blockIdx.x * 32 + lane; i < q_lines; i += (long long)gridDim.x * 32) prefetch_l2_line(p.q + i * 64);
    if (p.mask != nullptr)
      for (int i = blockIdx.x * 32 + lane; i < p.batch * p.tokens / 16; i += gridDim.x * 32) prefetch_l2_line(p.mask + i * 16);
    if (p.tau != nullptr)
      for (int i = blockIdx.x * 32 + lane; i < p.batch * p.h_q / 32; i += gridDim.x * 32) prefetch_l2_line(p.tau + i * 32);
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 0) {
    // this CTA's run of the line of tiles
    const TreeLine line = line_of(p);
    bool clamped = false;
    const TreeCut cut = cut_of(line, p.batch, p.ctas, &clamped);
    if (blockIdx.x == 0 && clamped) flag_status(p.status, SAGA_STATUS_LEN_CLAMPED);
    const int at = tree_start(cut, blockIdx.x);
    if (lane == 0) k.share->left = 0;
    __syncwarp();
    int base = 0;
    for (int b0 = 0; b0 < p.batch && at >= 0; b0 += 32) {
      int P = 0, n = 0;
      if (b0 + lane < p.batch) tree_lens(line, b0 + lane, &P, &n);
      const int mine = tree_extent(line, cut, tree_tiles(P, n));
      const int incl = warp_scan(mine);
      const unsigned hit = __ballot_sync(0xffffffffu, base + incl > at);
      if (hit != 0u) {
        if (lane == __ffs(hit) - 1) {
          *k.share = tree_walk_begin(line, cut, blockIdx.x, b0 + lane, at - (base + incl - mine), P, n);
          *k.share_cut = cut;
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

// Warp 0: the tiles' loads.  Returns how many were issued.
template <int D, bool E4M3>
__device__ __forceinline__ int load_tiles(const TreeParams& p, const Block& k, const CUtensorMap* kmap,
                                          const CUtensorMap* vmap, TreeWalk w) {
  int issued = 0;
  Ring r;
  bool ok = true;
  auto load = [&](const CUtensorMap* map, size_t row) {
    if (!ok) return;
    if (r.round > 0) ok = __all_sync(0xffffffffu, mbar_wait(&k.bar.empty[r.st], (r.round - 1) & 1, k.abort_flag));
    if (!ok) return;
    if (elect_one()) {
      mbar_arrive_expect_tx(&k.bar.full[r.st], (uint32_t)p.smem.stage_bytes);
#pragma unroll
      for (int h = 0; h < (E4M3 ? 1 : D / 64); ++h)
        tma_load_2d(k.smem + r.st * p.smem.stage_bytes + h * (kTreeTile * 128), map, &k.bar.full[r.st], h * 64, (int)row);
    }
    __syncwarp();
    r.step(p.smem.stages);
    ++issued;
  };
  do {
    const Heads h = heads_of(p, w);
    load(kmap, h.key + (size_t)w.t0 * kTreeTile);
    for (int t = w.t0; t < w.t1; ++t) {
      if (t + 1 < w.t1) load(kmap, h.key + (size_t)(t + 1) * kTreeTile);
      for (int v = 0; v < h.nv; ++v) load(vmap, h.value + (size_t)v * p.l_cap + (size_t)t * kTreeTile);
    }
  } while (ok && tree_walk_next(line_of(p), w));
  return issued;
}

// The first warpgroup, after its part of a tile with rows past the prefix: value
// rows that no token sees may hold anything, so they become zeros before the
// product reads them.  `bad`: this thread's row is one; vr: the ring's place of
// the tile's first value head.
template <int D, bool E4M3>
__device__ __forceinline__ void zero_unseen(const TreeParams& p, const Block& k, Ring vr, int nv, int r, bool bad) {
  for (int v = 0; v < nv; ++v) {
    if (!__all_sync(0xffffffffu, mbar_wait(&k.bar.full[vr.st], vr.round & 1, k.abort_flag))) break;
    if (bad) {
#pragma unroll
      for (int i = 0; i < (E4M3 ? D / 16 : D / 8); ++i) {  // neighbouring rows at different banks
        uint8_t* line = k.smem + vr.st * p.smem.stage_bytes +
                        (E4M3 ? r * D + ((i + r) & (D / 16 - 1)) * 16
                              : (i >> 3) * (kTreeTile * 128) + r * 128 + ((i + r) & 7) * 16);
        *reinterpret_cast<uint4*>(line) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_shared();
    }
    __syncwarp();
    if (k.lane == 0) mbar_arrive(&k.bar.vfix[vr.st]);
    vr.step(p.smem.stages);
  }
  __syncwarp();
}

// Everything has come to its end, or to a wait that gave up: then what is in
// flight lands before the memory is given back.
__device__ __forceinline__ void block_end(const TreeParams& p, const Block& k, int issued, uint32_t tmem, uint32_t tmem_cols) {
  tc_fence_before();
  __syncthreads();
  if (*k.abort_flag != 0) {
    cp_async_wait_all();  // scales of a tile that is not taken any more
    if (threadIdx.x == 0) {
      flag_status(p.status, SAGA_STATUS_TIMEOUT);
      // loads still in flight land before the shared memory is given up
      for (int x = issued > p.smem.stages ? issued - p.smem.stages : 0; x < issued; ++x)
        mbar_wait_drain(&k.bar.full[x % p.smem.stages], (x / p.smem.stages) & 1);
    }
    if (k.warp == 1) {  // and so do the products (every lane may have issued some)
      umma_commit(k.bar.drain);
      mbar_wait_drain(k.bar.drain, 0);
    }
  }
  __syncthreads();
  if (k.warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// 8-bit caches: 8 elements of a query (D / 8 neighbouring lanes hold it) as two
// e4m3 numbers each, scaled by the power of two that brings the query's largest
// into [128, 256), in a layout of `count` rows of D swizzled bytes; and the
// query's score factor in powers of two.  Whole warps call; rows past the end
// are not stored.
template <int D>
__device__ __forceinline__ void put_q8(uint8_t* at, int count, int row, int c, const uint4& x, float* factor, float scale) {
  float f[8];
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(u[k] << 16);
    f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    amax = fmaxf(amax, fmaxf(fabsf(f[2 * k]), fabsf(f[2 * k + 1])));
  }
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int ex = min(max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -126), 126);  // 2^ex and 2^-ex are normal
  const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
  uint32_t y[4], z[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = f[2 * k] * down, b = f[2 * k + 1] * down;
    y[k] = pack_8bit(a, b, __NV_E4M3);
    const float2 had = unpack_8bit(y[k], __NV_E4M3);
    z[k] = pack_8bit(a - had.x, b - had.y, __NV_E4M3);
  }
  if (row >= count) return;
  // half a 16-byte piece of the row
  at += row * D + (c & 1) * 8 + (((c >> 1) ^ (D == 64 ? row >> 1 & 3 : row & 7)) << 4);
  *reinterpret_cast<uint2*>(at) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
  *reinterpret_cast<uint2*>(at + count * D) = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
  if (c == 0) factor[row] = __uint_as_float((uint32_t)(127 + ex) << 23) * (scale * kLog2e);
}

// ------------------------------------------------------------------ the kernel
// Warp 0: TMA loads of the tiles.  Warp 1: the products, issued by one lane.
// Warps 4 .. 11: two warpgroups, each half of the column groups of every tile.
// Ring order: K of tile 0, then for each tile K of the next one and its own
// value heads, so that the next tile's scores are there while a tile's weights
// are computed.
// A tile of few columns is bound by its loads and one chain (scores, weights,
// products); about 8 us go before the first product and to the end of the
// join.  12/1/4 heads of 128 over 128K rows: one token from an 8-bit cache
// (87 MB) 31 us, 4 tokens under thresholds from a bf16 cache (168 MB) 41 us,
// 4.1 TB/s; 4 tokens over 1K rows of 8/1/8 heads of 64 16 us.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kTreeThreads, 1)
    saga_tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  const Block k = block_of(p, smem_raw);
  const Bars& bar = k.bar;
  uint8_t* const smem = k.smem;
  volatile int* const abort_flag = k.abort_flag;
  const TreeSmem& L = p.smem;
  const int warp = k.warp, lane = k.lane;
  const int stages = L.stages;
  const int cols = p.plan.cols;
  const int pcols = tree_piece_cols(p.plan.groups);
  // two score buffers, the accumulators, and bf16 weights' sums (d = 64: lanes 64 .. 127 of the accumulators)
  const int used = E4M3 ? 2 * cols + p.plan.nv * pcols : (D == 64 ? 3 : 4) * cols;
  const uint32_t tmem_cols = used <= 64 ? 64u : used <= 128 ? 128u : used <= 256 ? 256u : 512u;
  if (warp == 2 || warp == 3) {
    for (int i = threadIdx.x - 64; i < 2048 / 16; i += 64)
      *reinterpret_cast<uint4*>(smem + L.ones + i * 16) = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    fence_proxy_async_shared();
  }
  block_start<D>(p, k, &kmap, &vmap, tmem_cols);
  const uint32_t tmem = *k.tmem_slot;
  const uint32_t o_tmem = tmem + 2 * cols, l_tmem = tmem + 3 * cols;
  int issued = 0;  // TMA loads (warp 0)
  TreeWalk w = *k.share;
  const bool any = w.left > 0;

  if (warp == 0) {
    if (any) issued = load_tiles<D, E4M3>(p, k, &kmap, &vmap, w);
  } else if (warp == 1) {
    if (any && (p.test_wait_ns == 0u || mbar_wait(bar.drain, 0, abort_flag, p.test_wait_ns))) {
      const uint32_t id_s = E4M3 ? idesc(kE4m3, kE4m3, kTreeTile, cols, false) : idesc(kBf16, kBf16, kTreeTile, cols, false);
      const uint32_t id_o = E4M3 ? idesc(kE4m3, kE5m2, D, pcols, true) : idesc(kBf16, kBf16, 128, p.plan.nvp, true);
      const uint32_t id_l = idesc(kBf16, kBf16, 64, cols, true);
      const uint32_t ones = smem_u32(smem + L.ones), ring0 = smem_u32(smem);
      const uint64_t q_desc = desc_rows<D, E4M3>(smem_u32(smem + L.q));
      const uint64_t l_desc = desc_v<128, false>(ones, 0);
      Ring r;
      uint32_t fixed = 0;  // parity of each stage's vfix barrier
      int gs = 0, gp = 0, seg = 0;  // score products, value products, segments so far
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag)); };
      auto scores = [&]() {
        if (!wait(&bar.full[r.st], r.round & 1)) return false;
        if (gs >= 2 && !wait(&bar.s_empty[gs & 1], ((gs >> 1) - 1) & 1)) return false;
        tc_fence_after();
        const uint64_t k_desc = desc_rows<D, E4M3>(ring0 + r.st * L.stage_bytes);
        const uint32_t d = tmem + (gs & 1) * cols;
        if (elect_one()) {
          if (E4M3) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) umma_8bit(d, k_desc + k * 2, q_desc + k * 2, id_s, k > 0);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) umma_8bit(d, k_desc + k * 2, q_desc + cols * (D / 16) + k * 2, id_s, 1u);
          } else {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)  // 64-column halves: K of the tile 16 KB apart, Q cols * 128 bytes
              umma_bf16(d, k_desc + (k >> 2) * (kTreeTile * 128 / 16) + (k & 3) * 2,
                        q_desc + (k >> 2) * (cols * 8) + (k & 3) * 2, id_s, k > 0);
          }
          umma_commit(&bar.empty[r.st]);
          umma_commit(&bar.s_full[gs & 1]);
        }
        __syncwarp();
        r.step(stages);
        ++gs;
        return true;
      };
      do {
        const Heads h = heads_of(p, w);
        ok = wait(bar.q_full, seg & 1);
        ++seg;
        tc_fence_after();
        ok = ok && scores();
        for (int t = w.t0; ok && t < w.t1; ++t) {
          if (t + 1 < w.t1) ok = scores();
          ok = ok && wait(&bar.p_full[gp & 1], (gp >> 1) & 1);
          const uint64_t p_desc = desc_p(smem_u32(smem + L.p + (gp & 1) * L.p_bytes));
          const bool fix = (t + 1) * kTreeTile > w.P;
          const uint32_t first = t > w.t0 ? 1u : 0u;
          for (int v = 0; ok && v < h.nv; ++v) {
            ok = wait(&bar.full[r.st], r.round & 1);
            if (ok && fix) {
              ok = wait(&bar.vfix[r.st], fixed >> r.st & 1);
              fixed ^= 1u << r.st;
            }
            if (!ok) break;
            tc_fence_after();
            const uint32_t a0 = ring0 + r.st * L.stage_bytes, d = o_tmem + v * (E4M3 ? pcols : p.plan.nvp);
            // bf16, d = 64: the block of ones stays where it is while the tile's rows go by
            const uint64_t a = desc_v<D, E4M3>(a0, E4M3 ? 0 : D == 64 ? ones - a0 : kTreeTile * 128);
            const uint64_t b = p_desc + v * (E4M3 ? pcols >> 4 : p.plan.nvp >> 3) * 128;
            constexpr uint64_t kStep = D == 64 ? 128ull - (128ull << 16) : 128ull;
            if (elect_one()) {
              if (E4M3) {  // 32 rows a step: 4 groups of 8
#pragma unroll
                for (int k = 0; k < kTreeTile / 32; ++k)
                  umma_8bit(d, a + k * (D * 2), b + k * 32, id_o, k > 0 ? 1u : first);
              } else {
#pragma unroll
                for (int k = 0; k < kTreeTile / 16; ++k)
                  umma_bf16(d, a + k * kStep, b + k * 16, id_o, k > 0 ? 1u : first);
              }
              umma_commit(&bar.empty[r.st]);
            }
            __syncwarp();
            r.step(stages);
          }
          if (!ok) break;
          if (elect_one()) {
            if (D == 128 && !E4M3) {  // the sums of weights, which d = 64 has beside the values
#pragma unroll
              for (int k = 0; k < kTreeTile / 16; ++k) umma_bf16(l_tmem, l_desc, p_desc + k * 16, id_l, k > 0 ? 1u : first);
            }
            umma_commit(&bar.pv_done[gp & 1]);
          }
          __syncwarp();
          ++gp;
        }
      } while (ok && tree_walk_next(line_of(p), w));
    }
  } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + 8) {
    const int wg = (warp - kEpiWarp0) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;        // cache row of the tile
    const int et = threadIdx.x - kEpiWarp0 * 32;  // 0 .. 255
    Columns cw;
    cw.m = reinterpret_cast<float*>(smem + L.m);
    cw.tau = reinterpret_cast<float*>(smem + L.tau);
    cw.cs = reinterpret_cast<float*>(smem + L.cs);
    cw.mask = reinterpret_cast<unsigned long long*>(smem + L.mask);
    float* fac = reinterpret_cast<float*>(smem + L.f);
    int* out_row = reinterpret_cast<int*>(smem + L.row);
    float* words = reinterpret_cast<float*>(smem + L.words);
    float* sums = reinterpret_cast<float*>(smem + L.sums) + quarter * cols;  // 8-bit: this quarter's rows,
    float* sums_here = sums + 4 * cols;                                      // and those of the tile in hand
    constexpr float kOver = E4M3 ? kOverE5m2 : kOverBf16;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const int G = p.h_q / p.h_k;
    int gt = 0;  // tiles so far
    Ring seg_ring;  // ring position of the segment's first load
    bool ok = true;
    if (any) do {
      const Heads h = heads_of(p, w);
      // column groups of this warpgroup: half of the live ones
      Groups mine;
      mine.groups = p.plan.groups;
      mine.nvp = p.plan.nvp;
      const int live = h.nv * mine.groups, g0 = wg == 0 ? 0 : (live + 1) >> 1;
      mine.count = wg == 0 ? (live + 1) >> 1 : live >> 1;
      mine.at = g0 % mine.groups;
      mine.v = 0;
      const int v_first = g0 / mine.groups;
      mine.col = v_first * mine.nvp + mine.at * 8;
      mine.pcols = pcols;
      mine.pcol = v_first * pcols + mine.at * 8;
      const int nt = w.t1 - w.t0;
      // 8-bit: the scales of this thread's row, of the key head and of the warpgroup's value heads, a tile ahead
      const int v_count = mine.count > 0 ? (g0 + mine.count - 1) / mine.groups - v_first + 1 : 0;
      const int scale_slot = 2 * (1 + p.plan.nv) * kTreeTile;
      float* scales = reinterpret_cast<float*>(smem + L.scales) + wg * (1 + p.plan.nv) * kTreeTile + r;
      auto fetch_scales = [&](int i) {  // of the segment's tile i
        if (!E4M3) return;
        float* dst = scales + (i & 1) * scale_slot;
        const int row = (w.t0 + i) * kTreeTile + r;
        const bool there = row < w.P + w.n;
        const size_t safe = there ? row : 0;
        cp_async4_zfill(dst, p.k_scale + h.key + safe, there);
        for (int v = 0; v < v_count; ++v)
          cp_async4_zfill(dst + (1 + v) * kTreeTile, p.v_scale + h.value + (size_t)(v_first + v) * p.l_cap + safe, there);
        cp_async_commit();
      };
      fetch_scales(0);
      // the columns' words, then Q with every load in flight before the first is used
      int my_row = -1;  // of the output: thread et's column
      float my_tau = INFINITY;
      unsigned long long my_mask = 0ull;
      if (et < cols) {
        int jj, t;
        if (tree_row(p.plan, p.tokens, h.chunk, et, &jj, &t) && t < w.n) {
          my_row = (w.b * p.tokens + t) * p.h_q + h.kh * G + jj;
          my_tau = p.tau != nullptr ? threshold(p.tau[w.b * p.h_q + h.kh * G + jj]) : -INFINITY;
          my_mask = p.mask != nullptr ? p.mask[(size_t)w.b * p.tokens + t] : (2ull << t) - 1ull;
        }
      }
      named_bar_sync(3, kEpiAll);  // the last segment's words and Q are no longer read
      if (et < cols) {
        cw.m[et] = my_row >= 0 ? -kUnset : kUnset;  // padding: weights of zero whatever its scores
        out_row[et] = my_row;
      }
      named_bar_sync(3, kEpiAll);
      constexpr int LPR = D / 8, STEP = kEpiAll / LPR, FLIGHT = 4;
      const int c = et % LPR;
#pragma unroll 1
      for (int col0 = et / LPR; col0 - et / LPR < cols; col0 += FLIGHT * STEP) {
        uint4 x[FLIGHT];
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
          const int row = col0 + i * STEP < cols ? out_row[col0 + i * STEP] : -1;
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (row >= 0) x[i] = *reinterpret_cast<const uint4*>(p.q + (size_t)row * D + c * 8);
        }
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
          const int col = col0 + i * STEP;
          if (E4M3) {
            put_q8<D>(smem + L.q, cols, col, c, x[i], cw.cs, p.scale);
          } else if (col < cols) {
            *reinterpret_cast<uint4*>(smem + L.q + (c >> 3) * (cols * 128) + col * 128 + (((c & 7) ^ (col & 7)) << 4)) = x[i];
          }
        }
      }
      if (E4M3)
        for (int i = et; i < 4 * cols; i += kEpiAll) reinterpret_cast<float*>(smem + L.sums)[i] = 0.f;
      if (et < cols) {
        cw.tau[et] = E4M3 ? my_tau * kLog2e : my_tau;
        cw.mask[et] = my_mask;
      }
      fence_proxy_async_shared();
      named_bar_sync(3, kEpiAll);
      if (lane == 0) mbar_arrive(bar.q_full);
      // for the join: the CTAs that hold the item (even runs: the line's tile at which it begins is the run's first
      // and what the run has done so far)
      if (et == 0 && w.t0 == 0) {
        const TreeCut cut = *k.share_cut;
        const int place = cut.by_items ? 0 : tree_even_first(cut, blockIdx.x) + gt;
        p.holders[w.item] = make_int2(blockIdx.x, tree_last_holder(cut, blockIdx.x, w.tiles, place));
      }
      unsigned long long seen = 0;
      if (w.t1 * kTreeTile > w.P) seen = seen_by_any(p, w);

      for (int i = 0; i < nt; ++i, ++gt) {
        const int buf = gt & 1;
        const uint32_t s_tmem = tmem + buf * cols + lanes;
        uint8_t* p_buf = smem + L.p + buf * L.p_bytes;
        const int row = (w.t0 + i) * kTreeTile + r;
        Row rw;
        rw.all = row < w.P;
        rw.live = row_seen(w, seen, row);
        rw.bit = !rw.all && row < w.P + w.n ? 1ull << (row - w.P) : 0ull;
        const bool tail = (w.t0 + i + 1) * kTreeTile > w.P;
        const bool test = tail || p.tau != nullptr;
        if (E4M3) {
          cp_async_wait_all();  // this thread's own copies
          rw.scale = scales + (i & 1) * scale_slot + kTreeTile;
          rw.f = rw.scale[-kTreeTile];
          if (i + 1 < nt) fetch_scales(i + 1);
        } else {
          rw.f = p.scale;
          rw.scale = nullptr;
        }
        ok = mbar_wait(&bar.s_full[buf], (gt >> 1) & 1, abort_flag) &&
             (gt < 2 || mbar_wait(&bar.pv_done[buf], ((gt >> 1) - 1) & 1, abort_flag));
        tc_fence_after();
        // A segment's first tile.  bf16: any score that every column sees is a good enough reference, so the tile's
        // first row's; where that is a drafted row, the exact maxima.  8-bit weights want the maxima.
        const bool common = !E4M3 && (w.t0 + i) * kTreeTile < w.P;
        if (i == 0 && common) {
          if (quarter == 0) {
            Groups g = mine;
#pragma unroll 1
            for (int n = g.count; n > 0; n -= 2) {
              uint32_t raw[2][8];
              const int col = g.col;
              tmem_ld8_start(s_tmem + g.col, raw[0]);
              g.step();
              const int next = g.col;
              if (n > 1) tmem_ld8_start(s_tmem + g.col, raw[1]);
              g.step();
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if (k >= n) break;
                float s[8];
                tmem_ld8_end(raw[k], s);
                const int at = k == 0 ? col : next;
                exponents<E4M3, false, false>(s, rw, at, cw);
                if (lane == 0) {
                  float old[8];
                  load8(cw.m + at, old);  // padding keeps its own
#pragma unroll
                  for (int x = 0; x < 8; ++x) cw.m[at + x] = old[x] == -kUnset ? -s[x] : old[x];
                }
              }
            }
          }
          named_bar_sync(1 + wg, 128);
        }
        // One place for the weights' code (a kernel's first tiles pay for fetching it): a tile is weighed against the
        // references as they are, and again after moving them if a score is too far above.
        bool redo = i == 0 && !common;
        if (redo && named_bar_or(3, kEpiAll, !ok || *abort_flag != 0)) {
          ok = false;
          break;
        }
        while (true) {
          if (redo) {
            // the general test serves every tile here: rows of a tile without drafted ones are seen by all
            maxima<E4M3>(s_tmem, words, mine, rw, cw);
            named_bar_sync(1 + wg, 128);
            for (int c = et & 127; c < mine.count * 8; c += 128) {
              const int ag = g0 + (c >> 3), col = ag / mine.groups * mine.nvp + ag % mine.groups * 8 + (c & 7);
              const float4 x = *reinterpret_cast<const float4*>(words + col * 4);
              const float now = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) - (E4M3 ? kTopE5m2 : 0.f);
              const float old = -cw.m[col], next = now > -INFINITY ? fmaxf(old, now) : old;
              cw.m[col] = -next;
              fac[col] = old == kUnset ? 0.f : ex2(old - next);
            }
            if (i > 0) {
              // the products so far must be in the accumulators (a wait that gives up sets the abort flag, which the
              // next tile sees)
              mbar_wait(&bar.pv_done[buf ^ 1], ((gt - 1) >> 1) & 1, abort_flag);
              tc_fence_after();
            }
            named_bar_sync(1 + wg, 128);
            if (i > 0) {
              Groups g = mine;
#pragma unroll 1
              for (int n = g.count; n > 0; --n, g.step()) {
#pragma unroll
                for (int part = 0; part < (E4M3 ? 3 : D == 64 ? 2 : 4); ++part) {
                  if (!E4M3 && (part & 1) != 0 && g.groups > 1) continue;
                  const uint32_t at = lanes + (E4M3 ? o_tmem + g.pcol + part * g.groups * 8
                                                    : (part < 2 ? o_tmem : l_tmem) + g.col + (part & 1) * 8);
                  float o[8];
                  tmem_ld8(at, o);
#pragma unroll
                  for (int x = 0; x < 8; ++x) o[x] *= fac[g.col + x];
                  tmem_st8(at, o);
                }
                if (E4M3 && lane < 8) sums[g.col + lane] *= fac[g.col + lane];
              }
            }
          }
          uint8_t* at = p_buf + r * 16;
          const float top = test ? weigh<E4M3, true>(s_tmem, at, sums_here, mine, rw, cw)
                                 : weigh<E4M3, false>(s_tmem, at, sums_here, mine, rw, cw);
          if (redo) break;
          if (!named_bar_or(3, kEpiAll, top > kOver || !ok || *abort_flag != 0)) break;
          // new references, or the end of it all: the 256 threads meet at the same barriers, so they go together
          if (named_bar_or(3, kEpiAll, !ok || *abort_flag != 0)) {
            ok = false;
            break;
          }
          redo = true;
        }
        if (!ok) break;
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.p_full[buf]);
          mbar_arrive(&bar.s_empty[buf]);
        }
        if (E4M3) {  // while the products run
          Groups g = mine;
          for (int n = g.count; n > 0; --n, g.step())
            if (lane < 8) sums[g.col + lane] += sums_here[g.col + lane];
        }
        if (tail && wg == 0) {
          // a barrier's phase is known by its parity only, so what its stage held before must have been read: the
          // values of the tile before, and the keys of the next
          if (i > 0) mbar_wait(&bar.pv_done[buf ^ 1], ((gt - 1) >> 1) & 1, abort_flag);
          if (i + 1 < nt) mbar_wait(&bar.s_full[buf ^ 1], ((gt + 1) >> 1) & 1, abort_flag);
          __syncwarp();
          Ring vr = seg_ring;
          vr.jump(tree_value_place(i, nt, h.nv), stages);
          zero_unseen<D, E4M3>(p, k, vr, h.nv, r, !row_seen(w, seen, row));
        }
      }
      if (!ok) break;
      seg_ring.jump(nt * (1 + h.nv), stages);
      // the segment's sums: written out, or left as a partial
      ok = mbar_wait(&bar.pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1, abort_flag);
      if (named_bar_or(3, kEpiAll, !ok || *abort_flag != 0)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.tiles;
      const size_t slot = (size_t)blockIdx.x + w.item;
      // the sums of weights: lanes 64 .. 127 of the accumulators (bf16, d = 64), lane 0 of their own columns (d = 128),
      // or the four warps' (8-bit)
      if (E4M3) {
        named_bar_sync(1 + wg, 128);
        for (int c = et & 127; c < mine.count * 8; c += 128) {
          const int ag = g0 + (c >> 3), col = ag / mine.groups * mine.nvp + ag % mine.groups * 8 + (c & 7);
          const float* x = reinterpret_cast<const float*>(smem + L.sums) + col;
          const float sum = (x[0] + x[cols]) + (x[2 * cols] + x[3 * cols]);
          if (whole) {
            fac[col] = inverse_of(sum);
          } else {
            p.part_l[slot * cols + col] = sum;
            p.part_m[slot * cols + col] = -cw.m[col];
          }
        }
      } else if (quarter == (D == 64 ? 2 : 0)) {
        Groups g = mine;
#pragma unroll 1
        for (int n = g.count; n > 0; --n, g.step()) {
          float l[8];
          tmem_ld8((D == 64 ? o_tmem : l_tmem) + lanes + g.col, l);
          if (g.groups == 1) {
            float more[8];
            tmem_ld8((D == 64 ? o_tmem : l_tmem) + lanes + g.col + 8, more);
#pragma unroll
            for (int k = 0; k < 8; ++k) l[k] += more[k];
          }
          float sum = l[0];
#pragma unroll
          for (int k = 1; k < 8; ++k) sum = lane == k ? l[k] : sum;
          if (lane < 8) {
            if (whole) {
              fac[g.col + lane] = inverse_of(sum);
            } else {
              p.part_l[slot * cols + g.col + lane] = sum;
              p.part_m[slot * cols + g.col + lane] = -cw.m[g.col + lane];
            }
          }
        }
      }
      if (whole) named_bar_sync(1 + wg, 128);
      // lane of the accumulators: d where M = 128; 16 of each warp's 32 where M = 64 (8-bit, d = 64)
      const int dd = E4M3 && D == 64 ? quarter * 16 + lane : r;
      const bool has_d = E4M3 && D == 64 ? lane < 16 : D == 128 || quarter < 2;
      if (__any_sync(0xffffffffu, has_d)) {
        Groups g = mine;
#pragma unroll 1
        for (int n = g.count; n > 0; --n, g.step()) {
          float o[8];
          tmem_ld8(o_tmem + lanes + (E4M3 ? g.pcol : g.col), o);
          const int parts = E4M3 ? 3 : g.groups == 1 ? 2 : 1;
#pragma unroll 1
          for (int part = 1; part < parts; ++part) {
            float more[8];
            tmem_ld8(o_tmem + lanes + (E4M3 ? g.pcol : g.col) + part * g.groups * 8, more);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] += more[k];
          }
          if (!has_d) continue;
          if (!whole) {  // padding too: nobody reads it
            float* dst = p.part_o + (slot * cols + g.col) * D + dd;
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k * D] = o[k];
            continue;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = out_row[g.col + k];
            if (row < 0) continue;
            const float f = fac[g.col + k], y = f == 0.f ? 0.f : o[k] * f;
            if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[(size_t)row * D + dd] = __float2bfloat16(y);
            else static_cast<float*>(p.out)[(size_t)row * D + dd] = y;
          }
        }
      }
      tc_fence_before();
    } while (tree_walk_next(line_of(p), w));
  }

  block_end(p, k, issued, tmem, tmem_cols);
}

// ------------------------------------------------------------------ queries as rows
// For chunks with many query rows: the products the other way
// round,
//   S[query, row] = q . K      M = 128 queries, N = 128 rows of the tile
//   O[query, d]  += P V        P from TMEM, where it takes its scores' place,
// so that a thread has a query and its reference, threshold and sum in
// registers, no column words are read, and the weights never go through shared
// memory, which the products' operands fill by then: with 128 columns the
// kernel above takes 1.6 us per tile of d = 64, two thirds of it the weights'.
// Each value head of the chunk takes all 128 rows of P and a share of the
// columns of O, of which its own rows are kept; that costs products, of which
// there is room.  Two warpgroups, each half of the tile's rows.  8-bit caches in
// the same pieces as above; the scales of a tile's rows come to shared memory a
// tile ahead and are read by all threads alike, and the sums of weights are
// each thread's own.
// A tile takes 1.1 us here (bf16, d = 64) or 2.3 (8-bit, d = 128, three pieces):
// the chain in a warp from its scores to its weights, at a third of the issue
// slots, 41 % of the exponentials' pipe and 21 % of the tensor pipe.  Leaving out
// the exponentials, the sums or the products changes it by less than 5 %; twice
// the warps with half of the scores each take 8 % more (bf16; 8-bit ones spill).
// 64 tokens over 8 ragged rows of up to 16K of 32/8/8 heads of 64: 106 us; 16
// tokens over 128K 8-bit rows of 12/1/4 heads of 128: 55 us.

__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_8bit_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(id), "r"(accumulate)
      : "memory");
}

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A thread's query.
struct Query {
  float nm;                // its reference, negated
  float tau;               // its threshold (8-bit: in powers of two)
  float scale;             // its score factor (8-bit: in powers of two)
  unsigned long long sees; // of the 64 cache rows in hand, with TEST
  const float *ks, *vs;    // 8-bit: the scales of those rows as keys, and as values of its value head
};

// N scores from the `first`-th of the 64 on into exponents relative to the
// reference (RELATIVE) or not.
template <bool E4M3, bool TEST, bool RELATIVE, int N>
__device__ __forceinline__ void row_exponents(float* s, const Query& q, int first) {
  const uint32_t bits = (uint32_t)(q.sees >> first);
  const float f = E4M3 || TEST ? q.scale : q.scale * kLog2e, nm = RELATIVE ? q.nm : 0.f;
  const unsigned long long ff = two(f, f), ll = two(kLog2e, kLog2e), mm = two(nm, nm);
#pragma unroll
  for (int g = 0; g < N / 4; ++g) {
    float4 ks;
    if (E4M3) ks = reinterpret_cast<const float4*>(q.ks + first)[g];
#pragma unroll
    for (int i = 4 * g; i < 4 * g + 4; i += 2) {
      unsigned long long x = two(s[i], s[i + 1]);
      if (E4M3) x = mul2(x, i & 2 ? two(ks.z, ks.w) : two(ks.x, ks.y));
      if (TEST) {
        x = mul2(x, ff);
        float a, b;
        untwo(x, a, b);
        const bool keep0 = !(a < q.tau) && (bits >> i & 1u) != 0u, keep1 = !(b < q.tau) && (bits >> i & 2u) != 0u;
        if (E4M3) x = RELATIVE ? fma2(x, two(1.f, 1.f), mm) : x;
        else x = RELATIVE ? fma2(x, ll, mm) : mul2(x, ll);
        untwo(x, s[i], s[i + 1]);
        s[i] = keep0 ? s[i] : -INFINITY;
        s[i + 1] = keep1 ? s[i + 1] : -INFINITY;
      } else {
        x = RELATIVE ? fma2(x, ff, mm) : mul2(x, ff);
        untwo(x, s[i], s[i + 1]);
      }
    }
  }
}

// 64 scores into words of weights (bf16: 32; 8-bit: 16 for each of three
// pieces); their sum, and how far the largest is above what it may be (over 0).
template <bool E4M3, bool TEST>
__device__ __forceinline__ void row_weights(uint32_t s_tmem, const Query& q, uint32_t* w, float* sum, float* over) {
  float most = E4M3 ? 0.f : -INFINITY;
  unsigned long long add[2] = {0ull, 0ull};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float s[32];
    tmem_ld32(s_tmem + h * 32, s);
    row_exponents<E4M3, TEST, true, 32>(s, q, h * 32);
    if (!E4M3) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        most = fmaxf(most, s[i]);
        s[i] = ex2(s[i]);
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint32_t y = pack_bf16(s[i], s[i + 1]);
        w[h * 16 + (i >> 1)] = y;
        // the sum of the rounded weights, as the other kernel's row of ones gives it
        add[i >> 1 & 1] = fma2(two(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u)), two(1.f, 1.f), add[i >> 1 & 1]);
      }
    } else {
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float4 vs = reinterpret_cast<const float4*>(q.vs + h * 32)[g];
        uint32_t p1[2], p2[2], p3[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const unsigned long long x = two(ex2(s[4 * g + 2 * i]), ex2(s[4 * g + 2 * i + 1]));
          add[i] = fma2(x, two(1.f, 1.f), add[i]);
          float a, b;
          untwo(mul2(x, i ? two(vs.z, vs.w) : two(vs.x, vs.y)), a, b);
          most = fmaxf(most, fmaxf(a, b));
          pieces_of(a, b, p1[i], p2[i], p3[i]);
        }
        w[h * 8 + g] = __byte_perm(p1[0], p1[1], 0x7531);
        w[16 + h * 8 + g] = __byte_perm(p2[0], p2[1], 0x7531);
        w[32 + h * 8 + g] = __byte_perm(p3[0], p3[1], 0x7531);
      }
    }
  }
  float a, b, c, d;
  untwo(add[0], a, b);
  untwo(add[1], c, d);
  *sum = (a + b) + (c + d);
  // 8-bit: a row whose scale lies far below the others' does not show among the scaled weights, but in the sum
  *over = E4M3 ? (*sum < 1e34f ? most - 32768.f : INFINITY) : most - kOverBf16;
}

// The largest of the 64, in powers of two.  Once per segment, so its code is
// kept short: a kernel's first tile waits for it to be fetched.
template <bool E4M3>
__device__ __forceinline__ float row_maximum(uint32_t s_tmem, const Query& q) {
  float most = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < 64; h += 8) {
    float s[8];
    tmem_ld8(s_tmem + h, s);
    row_exponents<E4M3, true, false, 8>(s, q, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, E4M3 ? s[i] + __log2f(fmaxf(q.vs[h + i], kMinScale)) : s[i]);
  }
  return most;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kTreeThreads, 1)
    saga_tree_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  const Block k = block_of(p, smem_raw);
  const Bars& bar = k.bar;
  uint8_t* const smem = k.smem;
  volatile int* const abort_flag = k.abort_flag;
  const TreeSmem& L = p.smem;
  const int warp = k.warp, lane = k.lane, stages = L.stages;
  block_start<D>(p, k, &kmap, &vmap, 512);
  const uint32_t tmem = *k.tmem_slot;
  const uint32_t o_tmem = tmem + 2 * kTreeTile;  // after two score buffers: d columns for each value head
  int issued = 0;                                // TMA loads (warp 0)
  TreeWalk w = *k.share;
  const bool any = w.left > 0;

  if (warp == 0) {
    if (any) issued = load_tiles<D, E4M3>(p, k, &kmap, &vmap, w);
  } else if (warp == 1) {
    if (any && (p.test_wait_ns == 0u || mbar_wait(bar.drain, 0, abort_flag, p.test_wait_ns))) {
      const uint32_t id_s = E4M3 ? idesc(kE4m3, kE4m3, 128, kTreeTile, false) : idesc(kBf16, kBf16, 128, kTreeTile, false);
      // V as it lies: its rows are the inner dimension
      const uint32_t id_o = (E4M3 ? idesc(kE5m2, kE4m3, 128, D, false) : idesc(kBf16, kBf16, 128, D, false)) | 1u << 16;
      const uint32_t ring0 = smem_u32(smem);
      const uint64_t q_desc = desc_rows<D, E4M3>(smem_u32(smem + L.q));
      Ring r;
      uint32_t fixed = 0;  // parity of each stage's vfix barrier
      int gs = 0, gp = 0, seg = 0;  // score products, value products, segments so far
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag)); };
      auto scores = [&]() {
        if (!wait(&bar.full[r.st], r.round & 1)) return false;
        // the buffer held the weights of two tiles before, until their product was done
        if (gs >= 2 && !wait(&bar.pv_done[gs & 1], ((gs >> 1) - 1) & 1)) return false;
        tc_fence_after();
        const uint64_t k_desc = desc_rows<D, E4M3>(ring0 + r.st * L.stage_bytes);
        if (elect_one()) {
          const uint32_t d = tmem + (gs & 1) * kTreeTile;
          if (E4M3) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) umma_8bit(d, q_desc + i * 2, k_desc + i * 2, id_s, i > 0);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) umma_8bit(d, q_desc + kTreeMaxCols * (D / 16) + i * 2, k_desc + i * 2, id_s, 1u);
          } else {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {  // 64-column halves 16 KB apart in both
              const uint32_t at = (i >> 2) * (kTreeTile * 128 / 16) + (i & 3) * 2;
              umma_bf16(d, q_desc + at, k_desc + at, id_s, i > 0);
            }
          }
          umma_commit(&bar.empty[r.st]);
          umma_commit(&bar.s_full[gs & 1]);
        }
        __syncwarp();
        r.step(stages);
        ++gs;
        return true;
      };
      do {
        const Heads h = heads_of(p, w);
        ok = wait(bar.q_full, seg & 1);
        ++seg;
        tc_fence_after();
        ok = ok && scores();
        for (int t = w.t0; ok && t < w.t1; ++t) {
          if (t + 1 < w.t1) ok = scores();
          // the values first, which come early (the ring holds a tile's: at most 4 of 8 stages, or 2 of 4), then the
          // weights: the products of a tile then follow one another without a pause
          const bool fix = (t + 1) * kTreeTile > w.P;
          Ring at = r;
          for (int v = 0; ok && v < h.nv; ++v) {
            ok = wait(&bar.full[at.st], at.round & 1);
            if (ok && fix) {
              ok = wait(&bar.vfix[at.st], fixed >> at.st & 1);
              fixed ^= 1u << at.st;
            }
            at.step(stages);
          }
          ok = ok && wait(&bar.p_full[gp & 1], (gp >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t first = t > w.t0 ? 1u : 0u, a = tmem + (gp & 1) * kTreeTile;
          for (int v = 0; v < h.nv; ++v) {
            const uint64_t b = desc_v<D, E4M3>(ring0 + r.st * L.stage_bytes, kTreeTile * 128);
            if (elect_one()) {
              // each warpgroup's 64 rows of weights lie 64 columns apart: 32 columns of bf16, or 16 for each piece
              if (E4M3) {
#pragma unroll
                for (int piece = 0; piece < 3; ++piece)
#pragma unroll
                  for (int i = 0; i < kTreeTile / 32; ++i)
                    umma_8bit_ts(o_tmem + v * D, a + (i >> 1) * 64 + (i & 1) * 8 + piece * 16, b + i * (D * 2), id_o,
                                 piece + i > 0 ? 1u : first);
              } else {
#pragma unroll
                for (int i = 0; i < kTreeTile / 16; ++i)
                  umma_bf16_ts(o_tmem + v * D, a + (i >> 2) * 64 + (i & 3) * 8, b + i * 128, id_o, i > 0 ? 1u : first);
              }
              umma_commit(&bar.empty[r.st]);
            }
            __syncwarp();
            r.step(stages);
          }
          if (elect_one()) umma_commit(&bar.pv_done[gp & 1]);
          __syncwarp();
          ++gp;
        }
      } while (ok && tree_walk_next(line_of(p), w));
    }
  } else if (warp >= kEpiWarp0) {
    const int wg = (warp - kEpiWarp0) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;            // query row, and the cache row of a tile that this thread may zero
    const int et = threadIdx.x - kEpiWarp0 * 32;  // 0 .. 255
    int* out_row = reinterpret_cast<int*>(smem + L.row);
    float* words = reinterpret_cast<float*>(smem + L.words);  // [2][128]
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const int G = p.h_q / p.h_k;
    int gt = 0;  // tiles so far
    Ring seg_ring;
    bool ok = true;
    if (any) do {
      const Heads h = heads_of(p, w);
      const int nt = w.t1 - w.t0;
      const unsigned long long all = w.n >= 64 ? ~0ull : (1ull << w.n) - 1ull;
      int my_row = -1;
      float my_tau = INFINITY;
      unsigned long long my_mask = 0ull;
      {
        int jj, t;
        if (tree_row(p.plan, p.tokens, h.chunk, r, &jj, &t) && t < w.n) {
          my_row = (w.b * p.tokens + t) * p.h_q + h.kh * G + jj;
          my_tau = p.tau != nullptr ? threshold(p.tau[w.b * p.h_q + h.kh * G + jj]) : -INFINITY;
          my_mask = all & (p.mask != nullptr ? p.mask[(size_t)w.b * p.tokens + t] : (2ull << t) - 1ull);
        }
      }
      unsigned long long seen = 0;
      if (w.t1 * kTreeTile > w.P) seen = seen_by_any(p, w);
      // 8-bit: the scales of a tile's rows, of the key head and of the chunk's value heads, a tile ahead; rows that no
      // token sees get zeros
      float* scales = reinterpret_cast<float*>(smem + L.scales);
      const int scale_slot = (1 + p.plan.nv) * kTreeTile;
      auto fetch_scales = [&](int i) {  // of the segment's tile i
        if (!E4M3) return;
        float* dst = scales + (i & 1) * scale_slot;
        for (int x = et; x < (1 + h.nv) * kTreeTile; x += kEpiAll) {
          const int which = x / kTreeTile, row = (w.t0 + i) * kTreeTile + x % kTreeTile;
          const bool there = row_seen(w, seen, row);
          const float* src = which == 0 ? p.k_scale + h.key : p.v_scale + h.value + (size_t)(which - 1) * p.l_cap;
          cp_async4_zfill(dst + x, src + (there ? row : 0), there);
        }
        cp_async_commit();
      };
      fetch_scales(0);
      const bool idle = !__any_sync(0xffffffffu, my_row >= 0);  // a warp without queries: its rows of O are garbage
      if (wg == 0) out_row[r] = my_row;  // read below only, since the last segment's barriers
      named_bar_sync(3, kEpiAll);
      constexpr int LPR = D / 8, STEP = kEpiAll / LPR, FLIGHT = 4;
      static_assert(kTreeMaxCols % (FLIGHT * STEP) == 0, "no row past the last is looked up");
      const int c = et % LPR;
#pragma unroll 1
      for (int row0 = et / LPR; row0 - et / LPR < kTreeMaxCols; row0 += FLIGHT * STEP) {
        uint4 x[FLIGHT];
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
          const int row = out_row[row0 + i * STEP];
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (row >= 0) x[i] = *reinterpret_cast<const uint4*>(p.q + (size_t)row * D + c * 8);
        }
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
          const int row = row0 + i * STEP;
          if (E4M3) put_q8<D>(smem + L.q, kTreeMaxCols, row, c, x[i], reinterpret_cast<float*>(smem + L.cs), p.scale);
          else *reinterpret_cast<uint4*>(smem + L.q + (c >> 3) * (kTreeMaxCols * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = x[i];
        }
      }
      fence_proxy_async_shared();
      named_bar_sync(3, kEpiAll);
      if (lane == 0) mbar_arrive(bar.q_full);
      if (E4M3) cp_async_wait_all();  // the first tile's scales, seen by all after its first barrier
      if (et == 0 && w.t0 == 0) {  // for the join, as above
        const TreeCut cut = *k.share_cut;
        const int place = cut.by_items ? 0 : tree_even_first(cut, blockIdx.x) + gt;
        p.holders[w.item] = make_int2(blockIdx.x, tree_last_holder(cut, blockIdx.x, w.tiles, place));
      }
      Query q;
      q.nm = my_row >= 0 ? -kUnset : kUnset;  // rows without a query: weights of zero whatever their scores
      q.tau = E4M3 ? my_tau * kLog2e : my_tau;
      q.scale = E4M3 ? reinterpret_cast<const float*>(smem + L.cs)[r] : p.scale;
      const int my_head = min(r / p.plan.rpc, h.nv - 1);  // of the chunk's value heads
      float l = 0.f;

      for (int i = 0; i < nt; ++i, ++gt) {
        const int buf = gt & 1, t0 = (w.t0 + i) * kTreeTile;
        const uint32_t s_tmem = tmem + buf * kTreeTile + wg * 64 + lanes;
        const bool tail = t0 + kTreeTile > w.P, test = tail || p.tau != nullptr;
        // of the 64 cache rows in hand: those of the prefix, then the drafted ones that the query sees
        const int rel = w.P - (t0 + wg * 64);
        q.sees = rel >= 64 ? ~0ull : rel > 0 ? (~0ull >> (64 - rel)) | my_mask << rel : rel > -64 ? my_mask >> -rel : 0ull;
        if (my_row < 0) q.sees = 0ull;
        if (E4M3) {
          q.ks = scales + (i & 1) * scale_slot + wg * 64;
          q.vs = q.ks + (1 + my_head) * kTreeTile;
          if (i + 1 < nt) fetch_scales(i + 1);
        }
        ok = mbar_wait(&bar.s_full[buf], (gt >> 1) & 1, abort_flag);
        tc_fence_after();
        constexpr int WORDS = E4M3 ? 48 : 32;
        uint32_t weights[WORDS];
        float sum = 0.f, over = -INFINITY;
        // A tile is weighed against the references as they are, and again after moving them if a score is too far
        // above; a segment's first tile, which has none, after taking them from its maxima.
        auto weigh_rows = [&]() {
          if (!idle) {
            if (test) row_weights<E4M3, true>(s_tmem, q, weights, &sum, &over);
            else row_weights<E4M3, false>(s_tmem, q, weights, &sum, &over);
          }
          if (E4M3) cp_async_wait_all();  // the next tile's scales, seen by all after the vote
        };
        auto move_references = [&]() {
          if (!idle) words[wg * 128 + r] = row_maximum<E4M3>(s_tmem, q);
          named_bar_sync(3, kEpiAll);
          const float now = fmaxf(words[r], words[128 + r]) - (E4M3 ? kTopE5m2 : 0.f), old = -q.nm;
          const float next = !idle && now > -INFINITY ? fmaxf(old, now) : old;
          const float f = old == kUnset ? 0.f : ex2(old - next);
          q.nm = -next;
          l *= f;
          if (i > 0) {
            // the products so far must be in the accumulators (a wait that gives up sets the abort flag, which the
            // next tile sees)
            mbar_wait(&bar.pv_done[buf ^ 1], ((gt - 1) >> 1) & 1, abort_flag);
            tc_fence_after();
            const int half = h.nv * (D / 2);
#pragma unroll 1
            for (int x = wg * half; x < (wg + 1) * half; x += 8) {
              float o[8];
              tmem_ld8(o_tmem + lanes + x, o);
#pragma unroll
              for (int y = 0; y < 8; ++y) o[y] *= f;
              tmem_st8(o_tmem + lanes + x, o);
            }
          }
        };
        // the 256 threads meet at the same barriers, so they give up together
        auto given_up = [&]() { return named_bar_or(3, kEpiAll, !ok || *abort_flag != 0); };
        auto vote = [&]() { return named_bar_or(3, kEpiAll, over > 0.f || !ok || *abort_flag != 0); };
        if (!E4M3) {
          if (i > 0) weigh_rows();
          else over = INFINITY;
          if (vote()) {
            if (given_up()) {
              ok = false;
              break;
            }
            move_references();
            weigh_rows();
            named_bar_sync(3, kEpiAll);  // the words are read before they are written again
          }
        } else {
          // one place for the weights' code, long as it is: the first tiles pay for fetching it (60 -> 57 us for a tree
          // of 16 over 128K rows; with bf16 the same costs 5 %)
          bool moved = i == 0;
          if (moved && given_up()) {
            ok = false;
            break;
          }
          while (true) {
            if (moved) move_references();
            weigh_rows();
            if (moved) {
              named_bar_sync(3, kEpiAll);
              break;
            }
            if (!vote()) break;
            if (given_up()) {
              ok = false;
              break;
            }
            moved = true;
          }
          if (!ok) break;
        }
        if (!idle) {
          l += sum;
#pragma unroll
          for (int x = 0; x < WORDS; x += 16) tmem_st16(s_tmem + x, weights + x);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[buf]);
        if (tail && wg == 0) {
          // (the ring has at least 2 nv + 1 stages here, so these stages held something before this tile's keys, which
          // have been read, and their barriers' phases cannot be mistaken)
          Ring vr = seg_ring;
          vr.jump(tree_value_place(i, nt, h.nv), stages);
          zero_unseen<D, E4M3>(p, k, vr, h.nv, r, !row_seen(w, seen, t0 + r));
        }
      }
      if (!ok) break;
      seg_ring.jump(nt * (1 + h.nv), stages);
      // the segment's sums: written out, or left as a partial
      words[wg * 128 + r] = l;
      ok = mbar_wait(&bar.pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1, abort_flag);
      if (named_bar_or(3, kEpiAll, !ok || *abort_flag != 0)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.tiles;
      const size_t slot = (size_t)blockIdx.x + w.item;
      const float total = words[r] + words[128 + r];
      if (!whole && wg == 0 && my_row >= 0) {
        p.part_l[slot * kTreeMaxCols + r] = total;
        p.part_m[slot * kTreeMaxCols + r] = -q.nm;
      }
      const float inv = inverse_of(total);
      if (!idle) {
        const int mine = r / p.plan.rpc;  // this row's value head of the chunk
        const int v_lo = (quarter * 32) / p.plan.rpc, v_hi = min((quarter * 32 + 31) / p.plan.rpc, h.nv - 1);
#pragma unroll 1
        for (int v = v_lo; v <= v_hi; ++v)
#pragma unroll 1
          for (int x = wg * (D / 2); x < (wg + 1) * (D / 2); x += 32) {
            float o[32];
            tmem_ld32(o_tmem + lanes + v * D + x, o);
            if (my_row < 0 || v != mine) continue;
            if (!whole) {
              float4* dst = reinterpret_cast<float4*>(p.part_o + (slot * kTreeMaxCols + r) * D + x);
#pragma unroll
              for (int y = 0; y < 8; ++y) dst[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
              continue;
            }
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = inv == 0.f ? 0.f : o[y] * inv;
            if (p.out_bf16) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)my_row * D + x);
#pragma unroll
              for (int y = 0; y < 4; ++y)
                dst[y] = make_uint4(pack_bf16(o[8 * y], o[8 * y + 1]), pack_bf16(o[8 * y + 2], o[8 * y + 3]),
                                    pack_bf16(o[8 * y + 4], o[8 * y + 5]), pack_bf16(o[8 * y + 6], o[8 * y + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + (size_t)my_row * D + x);
#pragma unroll
              for (int y = 0; y < 8; ++y) dst[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
            }
          }
      }
      tc_fence_before();
    } while (tree_walk_next(line_of(p), w));
  }

  block_end(p, k, issued, tmem, 512);
}

// ------------------------------------------------------------------ the join
// The partials of the CTAs that shared a query row's item, each relative to
// its own power of two.  A row whose item one CTA held is there already.
// WARPS warps per row, each with every WARPS-th partial: 8 where an item is
// spread over many CTAs (a CTA per row and 32 of its elements), 1 where items
// are many and have few partials each (8 rows per CTA).  With 8 for all, the
// rows of 64 tokens in a batch of 8 took 150 us to join; with 1 they take 12
// from cold caches.
constexpr int kJoinThreads = 256;

template <int WARPS, int COLS>
__global__ void __launch_bounds__(kJoinThreads) saga_tree_join_kernel(const TreeParams p, const int d) {
  constexpr int LANES = COLS / 4, AT_ONCE = 32 / LANES;  // lanes of a partial (16 bytes each), partials per load
  constexpr int BATCH = WARPS == 8 ? 5 : 4;              // loads in flight
  __shared__ float4 acc[kJoinThreads];
  __shared__ float sums[8], tops[8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long at_row = WARPS == 8 ? blockIdx.x : (long long)blockIdx.x * 8 + warp;
  if (at_row >= (long long)p.batch * p.tokens * p.h_q) return;  // WARPS == 1: the warp's own
  const int row = (int)at_row;
  const int j = row % p.h_q, bt = row / p.h_q, b = bt / p.tokens, t = bt - b * p.tokens;
  const TreeSpot spot = tree_spot(p.plan, p.tokens, j % (p.h_q / p.h_k), t);
  const int item = (b * p.h_k + j / (p.h_q / p.h_k)) * p.plan.chunks + spot.chunk;
  const int2 held = p.holders[item];  // not written where the batch row has no tokens
  if (p.counts != nullptr && t >= p.counts[b]) return;
  // (within the CTAs even where a call that gave up wrote none)
  const int c0 = min(max(held.x, 0), p.ctas - 1), c1 = min(max(held.y, 0), p.ctas - 1);
  if (c0 >= c1) return;
  const int w = WARPS == 8 ? warp : 0;
  const int parts = c1 - c0 >= w ? (c1 - c0 - w) / WARPS + 1 : 0;  // this warp's: w, w + WARPS, ...
  const size_t slot0 = (size_t)c0 + item + w;
  const int sub = lane / LANES, l4 = lane % LANES;
  const size_t step = (size_t)WARPS * p.plan.cols;
  const float4* src = reinterpret_cast<const float4*>(p.part_o + (slot0 * p.plan.cols + spot.col) * d + blockIdx.y * COLS) + l4;
  const size_t step4 = step * d / 4;
  float top = kUnset, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < parts; base += 32) {
    const int here = min(32, parts - base);
    float4 x[BATCH];  // the first loads do not wait for the weights
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = k * AT_ONCE + sub;
      x[k] = i < here ? src[(size_t)(base + i) * step4] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float pm = kUnset, pl = 0.f;
    if (lane < here) {
      pm = p.part_m[slot0 * p.plan.cols + spot.col + (base + lane) * step];
      pl = p.part_l[slot0 * p.plan.cols + spot.col + (base + lane) * step];
    }
    const float now = fmaxf(top, warp_max(pl != 0.f ? pm : kUnset));
    const float f = ex2(top - now), wt = pl != 0.f ? ex2(pm - now) : 0.f;
    top = now;
    float add = wt * pl;
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) add += __shfl_xor_sync(0xffffffffu, add, y);
    sum = sum * f + add;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
    for (int i0 = 0; i0 < here; i0 += AT_ONCE * BATCH) {
      if (i0 > 0) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int i = i0 + k * AT_ONCE + sub;
          x[k] = i < here ? src[(size_t)(base + i) * step4] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int i = i0 + k * AT_ONCE + sub;
        const float fw = __shfl_sync(0xffffffffu, wt, i & 31);
        if (i < here && fw != 0.f) {  // a partial without weights may hold anything
          o.x = fmaf(fw, x[k].x, o.x);
          o.y = fmaf(fw, x[k].y, o.y);
          o.z = fmaf(fw, x[k].z, o.z);
          o.w = fmaf(fw, x[k].w, o.w);
        }
      }
    }
  }
#pragma unroll
  for (int x = LANES; x < 32; x <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
  }
  if (WARPS == 8) {
    if (lane == 0) {
      sums[warp] = sum;
      tops[warp] = top;
    }
    acc[threadIdx.x] = o;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, tops[i]);
    sum = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = ex2(tops[i] - top);
      const float4 x = acc[i * 32 + lane];
      sum = fmaf(f, sums[i], sum);
      o.x = fmaf(f, x.x, o.x);
      o.y = fmaf(f, x.y, o.y);
      o.z = fmaf(f, x.z, o.z);
      o.w = fmaf(f, x.w, o.w);
    }
  }
  if (lane >= LANES) return;
  const float inv = inverse_of(sum);
  const size_t at = (size_t)row * d + blockIdx.y * COLS + l4 * 4;
  if (p.out_bf16) {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
}

// ------------------------------------------------------------------ host
constexpr size_t kTreeStatusBytes = 256;

int validate_tree(const saga_shape* s, int tokens) {
  int rc = api_validate_shape(s);
  if (rc) return rc;
  if (tokens < 1 || tokens > SAGA_TREE_MAX_TOKENS)
    return api_fail(SAGA_ERR_ARG, "tokens=%d outside [1, %d]", tokens, SAGA_TREE_MAX_TOKENS);
  if (tokens > s->l_cap) return api_fail(SAGA_ERR_ARG, "tokens=%d exceeds l_cap=%d", tokens, s->l_cap);
  if ((long long)s->batch * s->h_q * tokens >= (1ll << 31))
    return api_fail(SAGA_ERR_UNSUPPORTED, "batch * h_q * tokens too large");
  return SAGA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct TreeSizes {
  size_t slots, part_m, part_l, holders, total;  // byte offsets; the sums follow the status word
};

TreeSizes tree_sizes(const saga_shape* s, const TreePlan& plan, int ctas) {
  TreeSizes z;
  z.slots = (size_t)ctas + (size_t)s->batch * s->h_k * plan.chunks;
  z.part_m = kTreeStatusBytes + z.slots * plan.cols * s->d * 4;
  z.part_l = z.part_m + z.slots * plan.cols * 4;
  z.holders = z.part_l + z.slots * plan.cols * 4;
  z.total = z.holders + (size_t)s->batch * s->h_k * plan.chunks * 8;
  return z;
}

// Queries as rows from so many live rows a chunk on.  On caches of up to 42 MB,
// which stay in the L2 from call to call: a tree of T tokens over 32K rows of
// 32/2/8 heads of 64 (16 T live rows up to 128), as columns and as rows: bf16
// T = 4 20.3 and 20.8 us, T = 6 21.9 and 21.3; 8-bit T = 2 21.7 and 25.5, T = 4
// 26.4 and 26.2.  Over 16K rows of 32/8/8 heads (4 T live rows): bf16 T = 16 23.3
// and 23.8, T = 24 29.0 and 26.9; 8-bit T = 12 32.3 and 32.8, T = 16 37.2 and 33.4.
constexpr int kTreeRowsBf16 = 80, kTreeRowsE4m3 = 56;
bool by_rows(const TreePlan& rows, bool e4m3) { return tree_live_rows(rows) >= (e4m3 ? kTreeRowsE4m3 : kTreeRowsBf16); }

typedef void (*TreeKernel)(CUtensorMap, CUtensorMap, TreeParams);

}  // namespace
}  // namespace saga

using namespace saga;

extern "C" {

size_t saga_tree_workspace_bytes(const saga_shape* s, int tokens) {
  if (validate_tree(s, tokens)) return 0;
  int sms = 0;
  if (api_device_sms(&sms)) return 0;
  const int ctas = std::min(sms, kTreeMaxCtas);
  size_t most = 0;  // of calls with fewer tokens too (padding makes some of them the larger), of either format
  for (int t = 1; t <= tokens; ++t) {
    for (bool e4m3 : {false, true}) most = std::max(most, tree_sizes(s, tree_plan(s->h_q, s->h_k, s->h_v, t, e4m3), ctas).total);
    const TreePlan rows = tree_plan_rows(s->h_q, s->h_k, s->h_v, s->d, t);
    if (by_rows(rows, true)) most = std::max(most, tree_sizes(s, rows, ctas).total);
  }
  return most;
}

int saga_tree_attn(const saga_shape* s, int tokens, const void* q, const saga_cache* cache, const int* prefix_lens,
                   const int* counts, const unsigned long long* tree_mask, const float* tau, void* out, int out_dtype,
                   void* workspace, size_t ws_bytes, void* stream) {
  int rc = validate_tree(s, tokens);
  if (rc) return rc;
  rc = api_check_cache(s, cache);
  if (rc) return rc;
  if (!q || !out || !prefix_lens) return api_fail(SAGA_ERR_ARG, "NULL tensor pointer");
  if (!aligned16(q) || !aligned16(out)) return api_fail(SAGA_ERR_ARG, "q and out must be 16-byte aligned");
  if (out_dtype != SAGA_OUT_F32 && out_dtype != SAGA_OUT_BF16) return api_fail(SAGA_ERR_ARG, "bad out_dtype %d", out_dtype);
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return api_fail(SAGA_ERR_WORKSPACE, "workspace must be a 256-byte aligned device buffer");
  int sms = 0;
  rc = api_device_sms(&sms);
  if (rc) return rc;
  TreeParams p{};
  const bool e4m3 = cache->format == SAGA_CACHE_E4M3;
  const TreePlan rows_plan = tree_plan_rows(s->h_q, s->h_k, s->h_v, s->d, tokens);
  const bool as_rows = by_rows(rows_plan, e4m3);
  p.plan = as_rows ? rows_plan : tree_plan(s->h_q, s->h_k, s->h_v, tokens, e4m3);
  const TreeSizes z = tree_sizes(s, p.plan, std::min(sms, kTreeMaxCtas));
  if (ws_bytes < z.total) return api_fail(SAGA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, z.total);
  p.smem = tree_smem(p.plan, s->d, e4m3, as_rows);
  p.q = static_cast<const uint16_t*>(q);
  p.k = cache->k;
  p.v = cache->v;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.prefix_lens = prefix_lens;
  p.counts = counts;
  p.mask = tree_mask;
  p.tau = tau;
  p.out = out;
  p.status = static_cast<unsigned*>(workspace);
  p.scale = (float)(1.0 / sqrt((double)s->d));
  p.out_bf16 = out_dtype == SAGA_OUT_BF16;
  p.batch = s->batch;
  p.tokens = tokens;
  p.h_q = s->h_q;
  p.h_k = s->h_k;
  p.h_v = s->h_v;
  p.l_cap = s->l_cap;
  p.ctas = std::min(sms, kTreeMaxCtas);
  p.test_wait_ns = api_take_test_wait();
  char* base = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(base + kTreeStatusBytes);
  p.part_m = reinterpret_cast<float*>(base + z.part_m);
  p.part_l = reinterpret_cast<float*>(base + z.part_l);
  p.holders = reinterpret_cast<int2*>(base + z.holders);
  CUtensorMap km{}, vm{};
  rc = api_rows_map(&km, cache->k, (long long)s->batch * s->h_k * s->l_cap, s->d, e4m3);
  if (rc) return rc;
  rc = api_rows_map(&vm, cache->v, (long long)s->batch * s->h_v * s->l_cap, s->d, e4m3);
  if (rc) return rc;
  const TreeKernel kernel = as_rows      ? (s->d == 64 ? (e4m3 ? saga_tree_rows_kernel<64, true> : saga_tree_rows_kernel<64, false>)
                                                       : (e4m3 ? saga_tree_rows_kernel<128, true> : saga_tree_rows_kernel<128, false>))
                            : s->d == 64 ? (e4m3 ? saga_tree_kernel<64, true> : saga_tree_kernel<64, false>)
                                         : (e4m3 ? saga_tree_kernel<128, true> : saga_tree_kernel<128, false>);
  static std::atomic<uint64_t> done[8], done_join[3];
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), 227 * 1024,
                                 done[(as_rows ? 4 : 0) + (e4m3 ? 2 : 0) + (s->d == 64 ? 0 : 1)]);
  if (e == cudaSuccess)
    e = launch_pdl(kernel, dim3(p.ctas), dim3(kTreeThreads), p.smem.total, st, km, vm, p);
  if (e != cudaSuccess) return api_cuda_fail(e, "drafted-token attention launch");
  // partials of an item: about ctas / items of them, and one more
  const unsigned rows = (unsigned)s->batch * tokens * s->h_q;
  const bool few = 4ll * s->batch * s->h_k * p.plan.chunks >= p.ctas;
  auto join = !few ? saga_tree_join_kernel<8, 32> : s->d == 64 ? saga_tree_join_kernel<1, 64> : saga_tree_join_kernel<1, 128>;
  e = prepare_kernel(reinterpret_cast<const void*>(join), 0, done_join[!few ? 0 : s->d == 64 ? 1 : 2]);
  if (e == cudaSuccess)
    e = launch_pdl(join, few ? dim3((rows + 7) / 8) : dim3(rows, s->d / 32), dim3(kJoinThreads), 0, st, p, s->d);
  if (e != cudaSuccess) return api_cuda_fail(e, "drafted-token join launch");
  return api_ok();
}

}  // extern "C"
