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
// The softmax needs no exact maximum: any m within the range of the 16-bit
// weights gives the same quotient.  So m is taken from the first tile's maximum
// and moved only when a score rises above what the weights can hold, which one
// comparison per score and one vote per tile watch for; then sums and
// accumulators are rescaled and the tile is done again.  Sums of weights are
// kept per thread and column in registers and added across rows once at the
// end of a segment.
//
// 8-bit caches: the codes are widened to half precision (exactly) on their way
// into the same tile ring; a key row's scale multiplies its scores and a value
// row's scale its weights, in fp32, before the rounding of P.  q goes to half
// precision scaled by a power of two, exact for all that matters of bf16.
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
constexpr float kMinScale = 8.271806125530277e-25f;  // 2^-80: value scales below it do not lower the reference
constexpr int kEpiWarp0 = 4, kConvWarp0 = 12;
constexpr int kEpiAll = 256;

template <bool E4M3>
constexpr int kTreeThreads = E4M3 ? 512 : 384;

// ------------------------------------------------------------------ the line of tiles
__device__ __forceinline__ TreeLine line_of(const TreeParams& p) {
  return TreeLine{p.prefix_lens, p.counts, p.tokens, p.l_cap, p.h_k * p.plan.chunks};
}

// Heads of a segment.
struct Heads {
  int kh, chunk, v0, nv;  // first value head of the group, value heads here
};
__device__ __forceinline__ Heads heads_of(const TreeParams& p, const TreeWalk& w) {
  Heads h;
  h.kh = w.hc / p.plan.chunks;
  h.chunk = w.hc - h.kh * p.plan.chunks;
  h.v0 = p.plan.rsplit == 1 ? h.chunk * p.plan.nv : h.chunk / p.plan.rsplit;
  h.nv = p.plan.rsplit == 1 ? min(p.plan.nv, p.plan.nvh - h.v0) : 1;
  return h;
}
__device__ __forceinline__ size_t key_row(const TreeParams& p, const TreeWalk& w, const Heads& h) {
  return ((size_t)w.b * p.h_k + h.kh) * p.l_cap;
}
__device__ __forceinline__ size_t value_row(const TreeParams& p, const TreeWalk& w, const Heads& h, int v) {
  const int j = h.kh * (p.h_q / p.h_k) + (h.v0 + v) * p.plan.hpv;  // the value head's first query head
  return ((size_t)w.b * p.h_v + j / (p.h_q / p.h_v)) * p.l_cap;
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
// Matrix descriptors.  V tile: 128-byte swizzle, the product's M (d) dense:
// 64-element blocks `block` bytes apart, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_v(uint32_t addr, uint32_t block) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// P: no swizzle, N (columns) dense in 16-byte groups of 8; the 8 x 8 blocks of
// a column group lie 128 bytes apart along the rows, column groups 2048 bytes.
__device__ __forceinline__ uint64_t desc_p(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 16) | ((uint64_t)(2048u >> 4) << 32) |
         ((uint64_t)1u << 46);
}
// Instruction descriptor: fp32 sums of bf16 (1) or half (0) operands.
__host__ __device__ constexpr uint32_t idesc16(bool half, int M, int N, bool transposed) {
  return (1u << 4) | ((half ? 0u : 1u) << 7) | ((half ? 0u : 1u) << 10) | (transposed ? 3u << 15 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(__float_as_uint(v[0])),
      "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
      "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool E4M3>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (E4M3) {
    const __half2 h = __floats2half2_rn(a, b);
    return reinterpret_cast<const uint32_t&>(h);
  }
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

template <int M>
struct Mode {
  static constexpr int value = M;
};

// The epilogue's view of one tile.
template <int D, bool E4M3>
struct Tile {
  uint32_t s_tmem;      // scores of this warp's lanes
  uint8_t* p_buf;       // the P buffer
  uint8_t* p_row;       // this thread's 16 bytes of column group 0 in it
  const float* sc;      // 8-bit: this row's scales, [0] key, [1 + v - v_first] value (stride kTreeTile)
  bool all;             // every column sees the row
  unsigned long long bit;  // else the drafted token of the row (0: none)
  float scale;
};

enum { kAccumulate, kUndo, kMax };

// Words for exchanging a column group's values between the four warps of its
// warpgroup: the group's part of a P buffer while that holds no weights.
__device__ __forceinline__ float* column_words(uint8_t* p_buf, int col) {
  return reinterpret_cast<float*>(p_buf + (col >> 3) * 2048);
}

// One pass over this warpgroup's columns of a tile.  kAccumulate: weights into
// P and the sums, true if a score is above what its column's reference allows.
// kUndo: takes the same weights out of the sums again.  kMax: the columns'
// maxima over the warp's rows into column_words.
template <int D, bool E4M3, int MAXG, bool MASKED, int MODE>
__device__ __forceinline__ bool tile_pass(const TreeParams& p, const Tile<D, E4M3>& t, int g0, int ng, int gpv,
                                          const float* m, const float* tau, const float* cs,
                                          const unsigned long long* mask, float* l) {
  bool over = false;
  const float ks = E4M3 ? t.sc[0] : t.scale;
  const int v_first = E4M3 ? g0 / gpv : 0;
#pragma unroll
  for (int g = 0; g < MAXG; ++g) {
    if (g < ng) {
      const int vl = (g0 + g) / gpv, col = vl * p.plan.nvp + (g0 + g - vl * gpv) * 8;
      float s[8];
      tmem_ld8(t.s_tmem + col, s);
      float vs = 1.f, lv = 0.f, lim = 32.f;
      if (E4M3) {
        vs = t.sc[(1 + vl - v_first) * kTreeTile];
        lv = __log2f(fmaxf(vs, kMinScale));
        lim = 15.f - lv;
      }
      float e[8], mm[8];
      *reinterpret_cast<float4*>(mm) = *reinterpret_cast<const float4*>(m + col);
      *reinterpret_cast<float4*>(mm + 4) = *reinterpret_cast<const float4*>(m + col + 4);
      if (!MASKED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = (E4M3 ? ks * cs[col + i] : ks) * kLog2e;
          e[i] = MODE == kMax ? s[i] * f : fmaf(s[i], f, -mm[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = s[i] * (E4M3 ? ks * cs[col + i] : ks);
          const bool keep = (t.all || (mask[col + i] & t.bit) != 0ull) && a >= tau[col + i];
          e[i] = keep ? (MODE == kMax ? a * kLog2e : fmaf(a, kLog2e, -mm[i])) : -INFINITY;
        }
      }
      if (MODE == kMax) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t k = __reduce_max_sync(0xffffffffu, float_key(e[i] + lv));
          if (lane_id() == 0) column_words(t.p_buf, col)[(threadIdx.x >> 5 & 3) * 8 + i] = key_float(k);
        }
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          over |= e[i] > lim;
          e[i] = ex2(fminf(e[i], lim));
          if (MODE == kAccumulate) l[g * 8 + i] += e[i];
          else l[g * 8 + i] -= e[i];
        }
        if (MODE == kAccumulate) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = E4M3 ? pack2<E4M3>(e[2 * i] * vs, e[2 * i + 1] * vs) : pack2<E4M3>(e[2 * i], e[2 * i + 1]);
          *reinterpret_cast<uint4*>(t.p_row + (col >> 3) * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  return over;
}

// 8 columns' sums over the 32 lanes: lane 4 c holds column
// (bit 2 of c) * 4 + (bit 1) * 2 + bit 0 of its octet.
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

// ------------------------------------------------------------------ 8-bit tiles into the ring
// The loads of a CTA's share in ring order, with where each comes from.
template <int D>
struct Feed {
  TreeWalk w;
  TreeFeed at;
  Heads h;
  unsigned long long seen;
  bool live;
  __device__ __forceinline__ void segment(const TreeParams& p) {
    h = heads_of(p, w);
    at = tree_feed(w);
    seen = w.t1 * kTreeTile > w.P ? seen_by_any(p, w) : 0ull;
  }
  __device__ __forceinline__ void next(const TreeParams& p) {
    if (tree_feed_next(w, h.nv, at)) return;
    live = tree_walk_next(line_of(p), w);
    if (live) segment(p);
  }
  __device__ __forceinline__ const uint8_t* base(const TreeParams& p) const {
    return static_cast<const uint8_t*>(at.v < 0 ? p.k : p.v) +
           ((at.v < 0 ? key_row(p, w, h) : value_row(p, w, h, at.v)) + (size_t)at.t * kTreeTile) * D;
  }
  __device__ __forceinline__ int rows() const {  // rows of the tile that hold anything
    return min(kTreeTile, w.P + w.n - at.t * kTreeTile);
  }
};

// 16 codes as 16 half-precision values.
__device__ __forceinline__ void widen16(const uint4& u, uint4* a, uint4* b) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> 16), __NV_E4M3);
    y[2 * i] = reinterpret_cast<const uint32_t&>(lo);
    y[2 * i + 1] = reinterpret_cast<const uint32_t&>(hi);
  }
  *a = make_uint4(y[0], y[1], y[2], y[3]);
  *b = make_uint4(y[4], y[5], y[6], y[7]);
}

// 128 threads: 16-byte pieces of the tile's codes, loaded one tile ahead into
// registers, widened into the 128-byte swizzle that the products read.  Rows
// that no token sees become zeros.  One lane asks L2 for the tiles further on.
constexpr int kFeedAhead = 6;

template <int D>
__device__ void widen_tiles(const TreeParams& p, const TreeWalk& w0, uint8_t* smem, const Bars& bar, volatile int* abort_flag) {
  constexpr int CPR = D / 16;                      // pieces per row
  constexpr int PER = kTreeTile * CPR / 128;       // pieces per thread
  constexpr int RSTEP = 128 / CPR;                 // rows between a thread's pieces
  const int tid = threadIdx.x - kConvWarp0 * 32, lane = threadIdx.x & 31;
  const int c = tid % CPR, r0 = tid / CPR;
  const TreeSmem& L = p.smem;
  Feed<D> f, far;
  f.w = w0;
  f.live = true;
  f.segment(p);
  far = f;
  auto ask = [&]() {
    if (!far.live) return;
    const int rows = far.rows();
    if (tid == 0 && rows > 0) prefetch_l2_bulk(far.base(p), (uint32_t)rows * D);
    far.next(p);
  };
  uint4 x[PER];
  auto fetch = [&]() {
    const uint8_t* src = f.base(p) + (size_t)r0 * D + c * 16;
    const int row0 = f.at.t * kTreeTile + r0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      x[i] = row_seen(f.w, f.seen, row0 + i * RSTEP)
                 ? __ldg(reinterpret_cast<const uint4*>(src + (size_t)i * RSTEP * D))
                 : make_uint4(0u, 0u, 0u, 0u);
  };
  if (tid < 32)
    for (int i = 0; i < kFeedAhead; ++i) ask();
  fetch();
  Ring r;
  while (true) {
    if (tid < 32) ask();
    bool ok = r.round == 0 || mbar_wait(&bar.empty[r.st], (r.round - 1) & 1, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) break;
    uint8_t* dst = smem + r.st * L.stage_bytes + ((c * 16) >> 6) * (kTreeTile * 128);
    const int j = (c & 3) * 2;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      uint4 a, b;
      widen16(x[i], &a, &b);
      const int row = r0 + i * RSTEP;
      uint8_t* at = dst + row * 128;
      *reinterpret_cast<uint4*>(at + ((j ^ (row & 7)) << 4)) = a;
      *reinterpret_cast<uint4*>(at + (((j + 1) ^ (row & 7)) << 4)) = b;
    }
    f.next(p);
    if (f.live) fetch();
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.full[r.st]);
    r.step(L.stages);
    if (!f.live) break;
  }
}

// ------------------------------------------------------------------ the kernel
// Warp 0: TMA loads of the tiles (bf16 caches).  Warp 1: the products, issued
// by one lane.  Warps 4 .. 11: two warpgroups, each half of the column groups
// of every tile.  Warps 12 .. 15: widening of 8-bit tiles into the ring.
// Ring order: K of tile 0, then for each tile K of the next one and its own
// value heads, so that the next tile's scores are there while a tile's weights
// are computed.
template <int D, bool E4M3, int MAXG>
__global__ void __launch_bounds__(kTreeThreads<E4M3>, 1)
    saga_tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const TreeSmem& L = p.smem;
  Bars bar;
  bar.full = reinterpret_cast<uint64_t*>(smem + L.bars);
  bar.empty = bar.full + kTreeMaxStages;
  bar.vfix = bar.empty + kTreeMaxStages;
  bar.s_full = bar.vfix + kTreeMaxStages;
  bar.s_empty = bar.s_full + 2;
  bar.p_full = bar.s_empty + 2;
  bar.pv_done = bar.p_full + 2;
  bar.q_full = bar.pv_done + 2;
  bar.drain = bar.q_full + 1;
  long long* share = reinterpret_cast<long long*>(bar.drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(share + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = L.stages;
  const int cols = p.plan.cols;
  const uint32_t tmem_cols = 3 * cols <= 64 ? 64u : 3 * cols <= 128 ? 128u : 3 * cols <= 256 ? 256u : 512u;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < stages; ++i) {
      mbar_init(&bar.full[i], E4M3 ? 4 : 1);
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
    mbar_init(bar.drain, 1);
    mbar_init_fence();
    if (!E4M3) {
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 0) {
    // this CTA's share of the line of tiles
    const TreeLine line = line_of(p);
    const long long H = line.items;
    long long total = 0;
    bool clamped = false;
    for (int b = lane; b < p.batch; b += 32) {
      int P, n;
      clamped |= !tree_lens(line, b, &P, &n);
      total += H * tree_tiles(P, n);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (blockIdx.x == 0 && clamped) flag_status(p.status, SAGA_STATUS_LEN_CLAMPED);
    const int ctas = tree_ctas(total, p.ctas);
    const bool working = (int)blockIdx.x < ctas;
    const long long first = working ? tree_first_tile(total, ctas, blockIdx.x) : 0;
    const long long count = working ? tree_first_tile(total, ctas, blockIdx.x + 1) - first : 0;
    long long base = 0;
    if (lane == 0) share[2] = count;
    for (int b0 = 0; b0 < p.batch && count > 0; b0 += 32) {
      long long mine = 0;
      if (b0 + lane < p.batch) {
        int P, n;
        tree_lens(line, b0 + lane, &P, &n);
        mine = H * tree_tiles(P, n);
      }
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + incl > first);
      if (hit != 0u) {
        if (lane == __ffs(hit) - 1) {
          share[0] = b0 + lane;
          share[1] = first - (base + incl - mine);
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t o_tmem = tmem + 2 * cols;
  int issued = 0;  // TMA loads (warp 0, lane 0)
  TreeWalk w;
  const bool any = tree_walk_begin(line_of(p), share, w);

  if (warp == 0 && !E4M3) {
    if (lane == 0 && any) {
      Ring r;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, size_t row) {
        if (!ok) return;
        if (r.round > 0 && !mbar_wait(&bar.empty[r.st], (r.round - 1) & 1, abort_flag)) {
          ok = false;
          return;
        }
        mbar_arrive_expect_tx(&bar.full[r.st], (uint32_t)L.stage_bytes);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_load_2d(smem + r.st * L.stage_bytes + h * (kTreeTile * 128), map, &bar.full[r.st], h * 64, (int)row);
        r.step(stages);
        ++issued;
      };
      do {
        const Heads h = heads_of(p, w);
        const size_t kr = key_row(p, w, h);
        load(&kmap, kr + (size_t)w.t0 * kTreeTile);
        for (int t = w.t0; t < w.t1; ++t) {
          if (t + 1 < w.t1) load(&kmap, kr + (size_t)(t + 1) * kTreeTile);
          for (int v = 0; v < h.nv; ++v) load(&vmap, value_row(p, w, h, v) + (size_t)t * kTreeTile);
        }
      } while (ok && tree_walk_next(line_of(p), w));
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && any) {
      const uint32_t idesc_s = idesc16(E4M3, kTreeTile, cols, false);
      const uint32_t idesc_o = idesc16(E4M3, D, p.plan.nvp, true);
      const uint32_t q0 = smem_u32(smem + L.q);
      Ring r;
      uint32_t fixed = 0;  // parity of each stage's vfix barrier
      int gs = 0, gp = 0, seg = 0;  // score products, value products, segments so far
      bool ok = true;
      auto scores = [&]() {
        if (!mbar_wait(&bar.full[r.st], r.round & 1, abort_flag)) return false;
        if (gs >= 2 && !mbar_wait(&bar.s_empty[gs & 1], ((gs >> 1) - 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t a0 = smem_u32(smem + r.st * L.stage_bytes);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          // 64-column halves: K of the tile 16 KB apart, Q cols * 128 bytes
          const uint32_t a = a0 + (k >> 2) * (kTreeTile * 128) + (k & 3) * 32;
          const uint32_t b = q0 + (k >> 2) * (cols * 128) + (k & 3) * 32;
          umma_bf16(tmem + (gs & 1) * cols, umma_sdesc_sw128(a), umma_sdesc_sw128(b), idesc_s, k > 0);
        }
        umma_commit(&bar.empty[r.st]);
        umma_commit(&bar.s_full[gs & 1]);
        r.step(stages);
        ++gs;
        return true;
      };
      do {
        const Heads h = heads_of(p, w);
        ok = mbar_wait(bar.q_full, seg & 1, abort_flag);
        ++seg;
        tc_fence_after();
        ok = ok && scores();
        for (int t = w.t0; ok && t < w.t1; ++t) {
          if (t + 1 < w.t1) ok = scores();
          if (!ok || !mbar_wait(&bar.p_full[gp & 1], (gp >> 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t b0 = smem_u32(smem + L.p + (gp & 1) * L.p_bytes);
          const bool fix = !E4M3 && (t + 1) * kTreeTile > w.P;
          for (int v = 0; ok && v < h.nv; ++v) {
            ok = mbar_wait(&bar.full[r.st], r.round & 1, abort_flag);
            if (ok && fix) {
              ok = mbar_wait(&bar.vfix[r.st], fixed >> r.st & 1, abort_flag);
              fixed ^= 1u << r.st;
            }
            if (!ok) break;
            tc_fence_after();
            const uint32_t a0 = smem_u32(smem + r.st * L.stage_bytes);
#pragma unroll
            for (int k = 0; k < kTreeTile / 16; ++k)
              umma_bf16(o_tmem + v * p.plan.nvp, desc_v(a0 + k * 2048, kTreeTile * 128),
                        desc_p(b0 + v * (p.plan.nvp >> 3) * 2048 + k * 256), idesc_o, (t > w.t0 || k > 0) ? 1u : 0u);
            umma_commit(&bar.empty[r.st]);
            r.step(stages);
          }
          if (ok) umma_commit(&bar.pv_done[gp & 1]);
          ++gp;
        }
      } while (ok && tree_walk_next(line_of(p), w));
    }
    __syncwarp();
  } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + 8) {
    const int wg = (warp - kEpiWarp0) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;        // cache row of the tile
    const int et = threadIdx.x - kEpiWarp0 * 32;  // 0 .. 255
    const int gpv = (p.plan.rpc + 7) >> 3;    // column groups of a value head
    float* m = reinterpret_cast<float*>(smem + L.m);
    float* tau = reinterpret_cast<float*>(smem + L.tau);
    float* cs = reinterpret_cast<float*>(smem + L.cs);
    float* fac = reinterpret_cast<float*>(smem + L.f);
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(smem + L.mask);
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const int G = p.h_q / p.h_k;
    int gt = 0;  // tiles so far
    Ring seg_ring;  // ring position of the segment's first load
    float l[MAXG * 8];
    bool ok = true;
    if (any) do {
      const Heads h = heads_of(p, w);
      // column groups of this warpgroup
      const int live = h.nv * gpv, g0 = wg == 0 ? 0 : (live + 1) >> 1, ng = wg == 0 ? (live + 1) >> 1 : live >> 1;
      const int v_first = g0 / gpv, v_last = ng > 0 ? (g0 + ng - 1) / gpv : v_first - 1;
      const int nt = w.t1 - w.t0;
      float* scales = reinterpret_cast<float*>(smem + L.scales) + wg * (1 + p.plan.nv) * kTreeTile + r;
      const size_t kr = key_row(p, w, h);
      unsigned long long seen = 0;
      if (w.t1 * kTreeTile > w.P) seen = seen_by_any(p, w);
      auto fetch_scales = [&](int i) {  // of the segment's tile i
        if (!E4M3) return;
        float* dst = scales + (i & 1) * 2 * (1 + p.plan.nv) * kTreeTile;
        const int row = (w.t0 + i) * kTreeTile + r;
        const bool there = row_seen(w, seen, row);
        const size_t safe = there ? row : 0;
        cp_async4_zfill(dst, p.k_scale + kr + safe, there);
        for (int v = v_first; v <= v_last; ++v)
          cp_async4_zfill(dst + (1 + v - v_first) * kTreeTile, p.v_scale + value_row(p, w, h, v) + safe, there);
        cp_async_commit();
      };
      fetch_scales(0);
      // Q and the columns' words
      named_bar_sync(3, kEpiAll);  // the last segment's words and Q are no longer read
      constexpr int LPR = D / 8;
      for (int i = et; i < cols * LPR; i += kEpiAll) {  // whole warps: cols * LPR is a multiple of 128
        const int col = i / LPR, c = i % LPR;
        int jj = 0, t = 0;
        const bool there = tree_row(p.plan, p.tokens, h.chunk, col, &jj, &t) && t < w.n;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (there)
          x = *reinterpret_cast<const uint4*>(p.q + (((size_t)w.b * p.tokens + t) * p.h_q + h.kh * G + jj) * D + c * 8);
        if (E4M3) {
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
          for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // a power of two that brings the row's largest element into [1, 2); both it and its inverse are normal
          const int ex = min(max((int)(__float_as_uint(amax) >> 23) - 127, -126), 126);
          const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = pack2<true>(f[2 * k] * down, f[2 * k + 1] * down);
          x = make_uint4(y[0], y[1], y[2], y[3]);
          if (c == 0) cs[col] = __uint_as_float((uint32_t)(127 + ex) << 23) * p.scale;
        }
        *reinterpret_cast<uint4*>(smem + L.q + (c >> 3) * (cols * 128) + col * 128 + (((c & 7) ^ (col & 7)) << 4)) = x;
        if (c == 0) {
          m[col] = there ? kUnset : -kUnset;  // padding: weights of zero whatever its scores
          tau[col] = !there ? INFINITY : p.tau != nullptr ? p.tau[w.b * p.h_q + h.kh * G + jj] : -INFINITY;
          mask[col] = !there ? 0ull : p.mask != nullptr ? p.mask[(size_t)w.b * p.tokens + t] : (2ull << t) - 1ull;
        }
      }
      fence_proxy_async_shared();
      named_bar_sync(3, kEpiAll);
      if (lane == 0) mbar_arrive(bar.q_full);
#pragma unroll
      for (int i = 0; i < MAXG * 8; ++i) l[i] = 0.f;

      for (int i = 0; i < nt; ++i, ++gt) {
        const int buf = gt & 1;
        Tile<D, E4M3> t;
        t.s_tmem = tmem + buf * cols + lanes;
        t.p_buf = smem + L.p + buf * L.p_bytes;
        t.p_row = t.p_buf + r * 16;
        t.sc = scales + (i & 1) * 2 * (1 + p.plan.nv) * kTreeTile;
        t.scale = p.scale;
        const int row = (w.t0 + i) * kTreeTile + r;
        t.all = row < w.P;
        t.bit = !t.all && row < w.P + w.n ? 1ull << (row - w.P) : 0ull;
        const bool tail = (w.t0 + i + 1) * kTreeTile > w.P;
        const bool masked = tail || p.tau != nullptr;
        if (E4M3) {
          cp_async_wait_all();
          if (i + 1 < nt) fetch_scales(i + 1);
        }
        ok = mbar_wait(&bar.s_full[buf], (gt >> 1) & 1, abort_flag) &&
             (gt < 2 || mbar_wait(&bar.pv_done[buf], ((gt >> 1) - 1) & 1, abort_flag));
        // the 256 threads meet at the same barriers, so they give up together
        if (named_bar_or(3, kEpiAll, !ok || *abort_flag != 0)) {
          ok = false;
          break;
        }
        tc_fence_after();
        auto pass = [&](auto mode) {
          constexpr int kMode = decltype(mode)::value;
          return masked ? tile_pass<D, E4M3, MAXG, true, kMode>(p, t, g0, ng, gpv, m, tau, cs, mask, l)
                        : tile_pass<D, E4M3, MAXG, false, kMode>(p, t, g0, ng, gpv, m, tau, cs, mask, l);
        };
        bool redo = i == 0;
        if (!redo) {
          redo = named_bar_or(1 + wg, 128, pass(Mode<kAccumulate>()));
          if (redo) {
            pass(Mode<kUndo>());
            // the accumulators are moved below: the products so far must be in them (a wait that gives up sets
            // the abort flag, seen at the next tile)
            mbar_wait(&bar.pv_done[buf ^ 1], ((gt - 1) >> 1) & 1, abort_flag);
            tc_fence_after();
          }
        }
        if (redo) {
          pass(Mode<kMax>());
          named_bar_sync(1 + wg, 128);
          const int c = et & 127;
          if (c < ng * 8) {
            const int ag = g0 + (c >> 3), vl = ag / gpv, col = vl * p.plan.nvp + (ag - vl * gpv) * 8 + (c & 7);
            const float* words = column_words(t.p_buf, col) + (c & 7);
            const float top = fmaxf(fmaxf(words[0], words[8]), fmaxf(words[16], words[24]));
            const float old = m[col];
            const float now = top > -INFINITY ? fmaxf(old, top - (E4M3 ? 8.f : 0.f)) : old;
            m[col] = now;
            fac[col] = old == kUnset ? 0.f : ex2(old - now);
          }
          named_bar_sync(1 + wg, 128);
#pragma unroll
          for (int g = 0; g < MAXG; ++g) {
            if (g < ng) {
              const int vl = (g0 + g) / gpv, col = vl * p.plan.nvp + (g0 + g - vl * gpv) * 8;
              float f[8];
              *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(fac + col);
              *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(fac + col + 4);
#pragma unroll
              for (int k = 0; k < 8; ++k) l[g * 8 + k] *= f[k];
              if (i > 0) {
                float o[8];
                tmem_ld8(o_tmem + lanes + col, o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= f[k];
                tmem_st8(o_tmem + lanes + col, o);
              }
            }
          }
          pass(Mode<kAccumulate>());
        }
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.s_empty[buf]);
          mbar_arrive(&bar.p_full[buf]);
        }
        if (!E4M3 && tail && wg == 0) {
          // value rows that no token sees may hold anything: zero them before the product reads them
          const bool bad = !row_seen(w, seen, row);
          Ring vr = seg_ring;
          vr.jump(tree_value_place(i, nt, h.nv), stages);
          for (int v = 0; v < h.nv; ++v) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bar.full[vr.st], vr.round & 1, abort_flag))) break;
            if (bad) {
#pragma unroll
              for (int k = 0; k < D / 8; ++k)
                *reinterpret_cast<uint4*>(smem + vr.st * L.stage_bytes + (k >> 3) * (kTreeTile * 128) + r * 128 +
                                          (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async_shared();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.vfix[vr.st]);
            vr.step(stages);
          }
          __syncwarp();
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
      uint8_t* words0 = smem + L.p;
      int* out_row = reinterpret_cast<int*>(tau);
#pragma unroll
      for (int g = 0; g < MAXG; ++g) {
        if (g < ng) {
          const int vl = (g0 + g) / gpv, col = vl * p.plan.nvp + (g0 + g - vl * gpv) * 8;
          const float x = octet_sum(l + g * 8, lane);
          if ((lane & 3) == 0)
            column_words(words0, col)[quarter * 8 + (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)] = x;
        }
      }
      named_bar_sync(1 + wg, 128);
      {
        const int c = et & 127;
        if (c < ng * 8) {
          const int ag = g0 + (c >> 3), vl = ag / gpv, col = vl * p.plan.nvp + (ag - vl * gpv) * 8 + (c & 7);
          const float* words = column_words(words0, col) + (c & 7);
          const float sum = (words[0] + words[8]) + (words[16] + words[24]);
          int jj = 0, t = 0;
          const bool there = tree_row(p.plan, p.tokens, h.chunk, col, &jj, &t) && t < w.n;
          out_row[col] = there ? (w.b * p.tokens + t) * p.h_q + h.kh * G + jj : -1;
          if (whole) {
            fac[col] = sum > 0.f ? 1.f / sum : 0.f;
          } else if (there) {
            p.part_l[slot * cols + col] = sum;
            p.part_m[slot * cols + col] = m[col];
          }
        }
      }
      named_bar_sync(1 + wg, 128);
      // lane of the accumulators: d (D = 128), or 16 of each warp's 32 (M = 64)
      const bool has_d = D == 128 || lane < 16;
      const int dd = D == 128 ? r : quarter * 16 + (lane & 15);
      for (int g = 0; g < ng; ++g) {
        const int vl = (g0 + g) / gpv, col = vl * p.plan.nvp + (g0 + g - vl * gpv) * 8;
        float o[8];
        tmem_ld8(o_tmem + lanes + col, o);
        if (!has_d) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = out_row[col + k];
          if (row < 0) continue;
          if (!whole) {
            p.part_o[(slot * cols + col + k) * D + dd] = o[k];
          } else {
            const float x = fac[col + k] > 0.f ? o[k] * fac[col + k] : 0.f;
            if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[(size_t)row * D + dd] = __float2bfloat16(x);
            else static_cast<float*>(p.out)[(size_t)row * D + dd] = x;
          }
        }
      }
      tc_fence_before();
    } while (tree_walk_next(line_of(p), w));
    if (E4M3) cp_async_wait_all();
  } else if (E4M3 && warp >= kConvWarp0) {
    if (any) widen_tiles<D>(p, w, smem, bar, abort_flag);
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag != 0) {
    if (threadIdx.x == 0) {
      flag_status(p.status, SAGA_STATUS_TIMEOUT);
      // loads still in flight land before the shared memory is given up
      for (int x = issued > stages ? issued - stages : 0; x < issued; ++x)
        mbar_wait_drain(&bar.full[x % stages], (x / stages) & 1);
    }
    if (threadIdx.x == 32) {  // and so do the products
      umma_commit(bar.drain);
      mbar_wait_drain(bar.drain, 0);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// ------------------------------------------------------------------ the join
// One CTA per query row: the partials of the CTAs that shared its item, each
// relative to its own power of two.  A row whose item one CTA held is there
// already.
constexpr int kJoinThreads = 512;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) saga_tree_join_kernel(const TreeParams p) {
  constexpr int GROUPS = kJoinThreads / D;
  __shared__ float weight[kJoinThreads], acc[GROUPS][D], red[2][kJoinThreads / 32];
  __shared__ long long line[2];
  pdl_trigger();
  pdl_wait();
  const int j = blockIdx.x % p.h_q, bt = blockIdx.x / p.h_q, b = bt / p.tokens, t = bt - b * p.tokens;
  const TreeLine rows = line_of(p);
  int P, n;
  tree_lens(rows, b, &P, &n);
  if (t >= n) return;
  const int G = p.h_q / p.h_k, H = rows.items;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    long long before = 0, total = 0;
    for (int i = lane; i < p.batch; i += 32) {
      int P2, n2;
      tree_lens(rows, i, &P2, &n2);
      const long long x = (long long)H * tree_tiles(P2, n2);
      total += x;
      if (i < b) before += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (lane == 0) {
      line[0] = before;
      line[1] = total;
    }
  }
  __syncthreads();
  const int tiles = tree_tiles(P, n);
  const TreeSpot spot = tree_spot(p.plan, p.tokens, j % G, t);
  const int hc = (j / G) * p.plan.chunks + spot.chunk;
  const long long first = line[0] + (long long)hc * tiles;
  const int ctas = tree_ctas(line[1], p.ctas);
  const int c0 = tree_cta_of(line[1], ctas, first), c1 = tree_cta_of(line[1], ctas, first + tiles - 1);
  if (c0 == c1) return;
  const size_t slot0 = (size_t)c0 + b * H + hc;
  const int parts = c1 - c0 + 1;  // at most the CTAs of the attention kernel, under kJoinThreads
  float mine = kUnset, ml = 0.f;
  if (threadIdx.x < parts) {
    mine = p.part_m[(slot0 + threadIdx.x) * p.plan.cols + spot.col];
    ml = p.part_l[(slot0 + threadIdx.x) * p.plan.cols + spot.col];
  }
  float top = ml > 0.f ? mine : kUnset;
  top = warp_max(top);
  if (lane == 0) red[0][warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, red[0][i]);
  const float wt = ml > 0.f ? ex2(mine - top) : 0.f;
  weight[threadIdx.x] = wt;
  float sum = wt * ml;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[1][warp] = sum;
  __syncthreads();
  const int d = threadIdx.x % D, g = threadIdx.x / D;
  float o = 0.f;
  const float* src = p.part_o + (slot0 * p.plan.cols + spot.col) * D + d;
  const size_t step = (size_t)p.plan.cols * D;
#pragma unroll 8
  for (int i = g; i < parts; i += GROUPS) {
    const float x = src[i * step], f = weight[i];
    o += f > 0.f ? x * f : 0.f;
  }
  acc[g][d] = o;
  __syncthreads();
  if (threadIdx.x < D) {
    float total_o = 0.f, total_l = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) total_o += acc[i][d];
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) total_l += red[1][i];
    const float x = total_l > 0.f ? total_o / total_l : 0.f;
    const size_t at = (size_t)blockIdx.x * D + d;
    if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(x);
    else static_cast<float*>(p.out)[at] = x;
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
  size_t slots, part_m, part_l, total;  // byte offsets; the sums follow the status word
};

TreeSizes tree_sizes(const saga_shape* s, const TreePlan& plan, int ctas) {
  TreeSizes z;
  z.slots = (size_t)ctas + (size_t)s->batch * s->h_k * plan.chunks;
  z.part_m = kTreeStatusBytes + z.slots * plan.cols * s->d * 4;
  z.part_l = z.part_m + z.slots * plan.cols * 4;
  z.total = z.part_l + z.slots * plan.cols * 4;
  return z;
}

typedef void (*TreeKernel)(CUtensorMap, CUtensorMap, TreeParams);

template <int D, bool E4M3>
TreeKernel pick_groups(int half, int* which) {
  *which = half <= 1 ? 0 : half <= 2 ? 1 : half <= 4 ? 2 : 3;
  return half <= 1 ? saga_tree_kernel<D, E4M3, 1> : half <= 2 ? saga_tree_kernel<D, E4M3, 2>
         : half <= 4 ? saga_tree_kernel<D, E4M3, 4> : saga_tree_kernel<D, E4M3, 8>;
}

}  // namespace
}  // namespace saga

using namespace saga;

extern "C" {

size_t saga_tree_workspace_bytes(const saga_shape* s, int tokens) {
  if (validate_tree(s, tokens)) return 0;
  int sms = 0;
  if (api_device_sms(&sms)) return 0;
  return tree_sizes(s, tree_plan(s->h_q, s->h_k, s->h_v, s->d, tokens), sms).total;
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
  p.plan = tree_plan(s->h_q, s->h_k, s->h_v, s->d, tokens);
  const TreeSizes z = tree_sizes(s, p.plan, sms);
  if (ws_bytes < z.total) return api_fail(SAGA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, z.total);
  const bool e4m3 = cache->format == SAGA_CACHE_E4M3;
  p.smem = tree_smem(p.plan, s->d, e4m3);
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
  p.ctas = std::min(sms, kJoinThreads);  // the join holds one partial of each in a thread
  char* base = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(base + kTreeStatusBytes);
  p.part_m = reinterpret_cast<float*>(base + z.part_m);
  p.part_l = reinterpret_cast<float*>(base + z.part_l);
  CUtensorMap km{}, vm{};
  if (!e4m3) {
    rc = api_rows_map(&km, cache->k, (long long)s->batch * s->h_k * s->l_cap, s->d);
    if (rc) return rc;
    rc = api_rows_map(&vm, cache->v, (long long)s->batch * s->h_v * s->l_cap, s->d);
    if (rc) return rc;
  }
  const int half = (p.plan.groups + 1) / 2;
  int which = 0;
  const TreeKernel kernel = s->d == 64 ? (e4m3 ? pick_groups<64, true>(half, &which) : pick_groups<64, false>(half, &which))
                                       : (e4m3 ? pick_groups<128, true>(half, &which) : pick_groups<128, false>(half, &which));
  static std::atomic<uint64_t> done[16], done_join[2];
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), 227 * 1024,
                                 done[which + (e4m3 ? 4 : 0) + (s->d == 64 ? 0 : 8)]);
  if (e == cudaSuccess)
    e = launch_pdl(kernel, dim3(p.ctas), dim3(e4m3 ? kTreeThreads<true> : kTreeThreads<false>), p.smem.total, st, km, vm, p);
  if (e != cudaSuccess) return api_cuda_fail(e, "drafted-token attention launch");
  auto join = s->d == 64 ? saga_tree_join_kernel<64> : saga_tree_join_kernel<128>;
  e = prepare_kernel(reinterpret_cast<const void*>(join), 0, done_join[s->d == 64 ? 0 : 1]);
  if (e == cudaSuccess)
    e = launch_pdl(join, dim3((unsigned)s->batch * tokens * s->h_q), dim3(kJoinThreads), 0, st, p);
  if (e != cudaSuccess) return api_cuda_fail(e, "drafted-token join launch");
  return api_ok();
}

}  // extern "C"
