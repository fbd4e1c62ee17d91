// saga_cache.cu - rows on their way into and out of the caches: per-head norm
// and position rotation with the append (saga_norm_rope_append), the ragged
// append alone (saga_kv_store), both into bf16 or 8-bit caches, and the 8-bit
// rows read back (saga_kv_load).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <initializer_list>

#include "saga_device.cuh"
#include "saga_launch.cuh"
#include "saga_serve.h"

namespace saga {
namespace {

__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = reinterpret_cast<const uint32_t&>(h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// cos and sin of position * inv_freq.  The product and its remainder modulo
// one turn are taken in fp64 (a far position loses all of fp32's fraction),
// the sine of the remainder in fp32.
__device__ __forceinline__ float2 turn_of(int position, float inv_freq) {
  double t = (double)position * (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= rint(t);
  float s, c;
  sincospif(2.f * (float)t, &s, &c);
  return make_float2(c, s);
}

// cos and sin of a token's angles in shared memory, 16 bytes per two angles.
// Half-split pairs: a lane reads 8 angles, 64 bytes; the 16-byte pieces of
// neighbouring lanes are rotated against each other, so that four lanes' reads
// of one piece fall on different banks.
__device__ __forceinline__ int turn_slot(int f, bool interleaved) {
  if (interleaved) return f;
  const int c = f >> 3, j = f >> 1 & 3;
  return (c << 3) + ((j ^ (c & 3)) << 1) + (f & 1);
}

// 8 fp32 values as e4m3 codes of x * up.
__device__ __forceinline__ uint2 codes8(const float* x, float up) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * up, x[2 * i + 1] * up), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// A CTA's tokens of one batch row.
struct Tokens {
  int b, t0, nt, shift, start;  // shift: log2 nt where that is a power of two, else -1
  __device__ __forceinline__ void split(int item, int* head, int* t) const {
    *head = shift >= 0 ? item >> shift : item / nt;
    *t = item - *head * nt;
  }
  // The cache row of a token; false if it is none (a start that is no row may wrap: then it does not fit).
  __device__ __forceinline__ bool slot(const RowParams& p, int t, int* at) const {
    *at = (int)((unsigned)start + (unsigned)(t0 + t));
    return (unsigned)*at < (unsigned)p.l_cap;
  }
};

__device__ __forceinline__ bool tokens_of(const RowParams& p, Tokens& k) {
  k.b = blockIdx.x / p.groups;
  k.t0 = (blockIdx.x - k.b * p.groups) * p.group;
  const int count = p.counts != nullptr ? p.counts[k.b] : p.tokens;
  k.start = p.starts[k.b];
  k.nt = min(p.group, min(max(count, 0), p.tokens) - k.t0);
  k.shift = k.nt == p.group ? p.group_log2 : -1;
  return k.nt > 0;
}

// Rows of one kind in flight: a row of a head is D / 8 lanes of 16 bytes each.
enum { kQuery, kKey, kValue };
template <int D, int KIND>
struct RowFeed {
  const uint16_t* base;
  long long ts, hs;
  int items;
  __device__ __forceinline__ RowFeed(const RowParams& p, const Tokens& k) {
    const uint16_t* data = KIND == kQuery ? p.q : KIND == kKey ? p.k : p.v;
    const long long bs = KIND == kQuery ? p.q_bs : KIND == kKey ? p.k_bs : p.v_bs;
    ts = KIND == kQuery ? p.q_ts : KIND == kKey ? p.k_ts : p.v_ts;
    hs = KIND == kQuery ? p.q_hs : KIND == kKey ? p.k_hs : p.v_hs;
    base = data + k.b * bs + k.t0 * ts;
    items = (KIND == kQuery ? p.h_q : KIND == kKey ? p.h_k : p.h_v) * k.nt;
  }
  __device__ __forceinline__ const uint16_t* at(const Tokens& k, int item) const {
    int head, t;
    k.split(item < items ? item : 0, &head, &t);
    return base + t * ts + head * hs;
  }
};

template <int D, bool E4M3, int KIND>
__device__ __forceinline__ void rows_of(const RowParams& p, const Tokens& k, const RowFeed<D, KIND>& f, uint4 raw,
                                        const float2* turns) {
  constexpr int LPR = D / 8, RPP = kRowThreads / LPR;  // lanes per row, rows per pass
  const int c = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  const int half = p.rot >> 1;
  float w[8];
  if (KIND != kValue && p.norm) {
    const uint16_t* wp = KIND == kQuery ? p.q_weight : p.k_weight;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (wp != nullptr) unpack8(__ldg(reinterpret_cast<const uint4*>(wp + c * 8)), w);
  }
  for (int base = 0; base < f.items; base += RPP) {
    const int item = base + r0;
    float x[8];
    unpack8(raw, x);
    // the next row's load is in flight while this one is worked on and stored
    if (base + RPP < f.items) raw = *reinterpret_cast<const uint4*>(f.at(k, item + RPP) + c * 8);
    int head, t;
    k.split(item < f.items ? item : 0, &head, &t);
    if (KIND != kValue && p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
    }
    if (KIND != kValue && p.inv_freq != nullptr) {
      const float2* tt = turns + t * half;
      if (p.interleaved) {
        if (c * 8 < p.rot) {
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float4 cs = *reinterpret_cast<const float4*>(tt + c * 4 + i);
            float a = x[2 * i], e = x[2 * i + 1];
            x[2 * i] = a * cs.x - e * cs.y;
            x[2 * i + 1] = e * cs.x + a * cs.y;
            a = x[2 * i + 2], e = x[2 * i + 3];
            x[2 * i + 2] = a * cs.z - e * cs.w;
            x[2 * i + 3] = e * cs.z + a * cs.w;
          }
        }
      } else {
        const int rc = p.rot >> 4;  // 8-element chunks of half the rotated elements
        const int peer = c < rc ? c + rc : c < 2 * rc ? c - rc : c;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], peer, LPR);
        if (c < 2 * rc) {
          const int fc = c < rc ? c : c - rc;
          const float sign = c < rc ? -1.f : 1.f;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 cs = *reinterpret_cast<const float4*>(tt + (fc << 3) + (((i >> 1) ^ (fc & 3)) << 1));
            x[i] = fmaf(x[i], cs.x, sign * (y[i] * cs.y));
            x[i + 1] = fmaf(x[i + 1], cs.z, sign * (y[i + 1] * cs.w));
          }
        }
      }
    }
    float amax = 0.f;
    if (E4M3 && KIND != kQuery) {
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      amax = fmaxf(amax, kAmaxFloor);
    }
    if (item >= f.items) continue;
    if (KIND == kQuery) {
      const size_t row = (size_t)((size_t)k.b * p.tokens + k.t0 + t) * p.h_q + head;
      *reinterpret_cast<uint4*>(p.q_out + row * D + c * 8) = pack8(x);
      continue;
    }
    int slot;
    if (!k.slot(p, t, &slot)) {
      if (c == 0) flag_status(p.status, SAGA_STATUS_LEN_CLAMPED);
      continue;
    }
    const size_t row = ((size_t)k.b * (KIND == kKey ? p.h_k : p.h_v) + head) * p.l_cap + slot;
    void* cache = KIND == kKey ? p.k_cache : p.v_cache;
    if (E4M3) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D + c * 8) = codes8(x, kE4m3Max / amax);
      if (c == 0) (KIND == kKey ? p.k_scale : p.v_scale)[row] = amax / kE4m3Max;
    } else {
      // an untouched row round-trips through fp32 exactly
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + row * D + c * 8) = pack8(x);
    }
  }
}

// One CTA holds `group` tokens of one batch row and all their heads, queries
// first, then keys, then values, each in a loop of its own without the others'
// choices.  A row of a head (d elements) is D / 8 lanes of 16 bytes each, so
// its sum of squares, its rotation partners and its largest magnitude are
// shuffles.  The angles are the same for every head: they are computed once per
// token into shared memory, while the first rows of each kind are on their way.
// Rows are taken head by head, so neighbouring lanes write neighbouring cache
// rows and scales.  For few tokens the time is that of one chain of loads (one
// token: 3.1 us in a graph).  Calls on new rows each time: 8191 tokens of 42
// heads of 64 normed and rotated, 88 MB, 25 us, 54 % of the copy rate; two prompts
// of up to 4097 tokens of 17 heads of 128, half rotated, into an 8-bit cache,
// 56 MB, 18 us, 47 %.  The same rows again and again, of which the L2 keeps some
// or all: 22.5 and 12.5 us.  The first is bound by its instructions before HBM
// (71 % of the issue slots while a CTA runs; a warp is mostly ready or in a
// fixed-latency wait), the second waits for its loads as much (58 % of the issue
// slots; a third of a warp's time in those waits).
template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) saga_rows_kernel(const RowParams p) {
  constexpr int LPR = D / 8;
  __shared__ __align__(16) float2 turns[kMaxRowTokens * (D / 2)];
  pdl_trigger();
  pdl_wait();
  Tokens k;
  if (!tokens_of(p, k)) return;
  const int c = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  const RowFeed<D, kQuery> fq(p, k);
  const RowFeed<D, kKey> fk(p, k);
  const RowFeed<D, kValue> fv(p, k);
  const uint4 q0 = *reinterpret_cast<const uint4*>(fq.at(k, r0) + c * 8);
  const uint4 k0 = *reinterpret_cast<const uint4*>(fk.at(k, r0) + c * 8);
  const uint4 v0 = *reinterpret_cast<const uint4*>(fv.at(k, r0) + c * 8);
  if (p.inv_freq != nullptr) {
    const int half = p.rot >> 1;
    for (int i = threadIdx.x; i < k.nt * half; i += kRowThreads) {
      const int t = i / half, f = i - t * half;
      const int pos = p.positions != nullptr ? p.positions[(size_t)k.b * p.tokens + k.t0 + t]
                                             : (int)((unsigned)k.start + (unsigned)(k.t0 + t));
      turns[t * half + turn_slot(f, p.interleaved)] = turn_of(pos, p.inv_freq[f]);
    }
    __syncthreads();
  }
  rows_of<D, E4M3, kQuery>(p, k, fq, q0, turns);
  rows_of<D, E4M3, kKey>(p, k, fk, k0, turns);
  rows_of<D, E4M3, kValue>(p, k, fv, v0, turns);
}

// Keys or values as they are into the cache (saga_kv_store), 32 bytes of a row
// per thread: the quantisation is bound by its instructions, and a row's
// magnitude, scale and addresses are then shared by 16 elements (131072 tokens
// of 5 heads of 128 into an 8-bit cache, 254 MB: 49 us, 80 % of the copy rate;
// with 16 bytes per thread 74).
template <int D, bool E4M3, int KIND>
__device__ __forceinline__ void store_rows(const RowParams& p, const Tokens& k, const RowFeed<D, KIND>& f, uint4 a, uint4 b) {
  constexpr int LPR = D / 16, RPP = kRowThreads / LPR;
  const int c = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  for (int base = 0; base < f.items; base += RPP) {
    const int item = base + r0;
    const uint4 now[2] = {a, b};
    if (base + RPP < f.items) {
      const uint4* src = reinterpret_cast<const uint4*>(f.at(k, item + RPP) + c * 16);
      a = src[0];
      b = src[1];
    }
    int head, t, slot;
    k.split(item < f.items ? item : 0, &head, &t);
    float amax = 0.f;
    if (E4M3) {
      // magnitudes as bf16 pairs: the maximum of two needs no widening
      const uint32_t w[8] = {now[0].x, now[0].y, now[0].z, now[0].w, now[1].x, now[1].y, now[1].z, now[1].w};
      uint32_t most = w[0] & 0x7fff7fffu;
#pragma unroll
      for (int i = 1; i < 8; ++i) most = __vmaxu2(most, w[i] & 0x7fff7fffu);
      amax = __uint_as_float(max(most << 16, most & 0xffff0000u));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      amax = fmaxf(amax, kAmaxFloor);
    }
    if (item >= f.items) continue;
    if (!k.slot(p, t, &slot)) {
      if (c == 0) flag_status(p.status, SAGA_STATUS_LEN_CLAMPED);
      continue;
    }
    const size_t row = ((size_t)k.b * (KIND == kKey ? p.h_k : p.h_v) + head) * p.l_cap + slot;
    void* cache = KIND == kKey ? p.k_cache : p.v_cache;
    if (E4M3) {
      const float up = kE4m3Max / amax;
      float x[8];
      unpack8(now[0], x);
      const uint2 lo = codes8(x, up);
      unpack8(now[1], x);
      const uint2 hi = codes8(x, up);
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(cache) + row * D + c * 16) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      if (c == 0) (KIND == kKey ? p.k_scale : p.v_scale)[row] = amax / kE4m3Max;
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + row * D + c * 16);
      dst[0] = now[0];
      dst[1] = now[1];
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) saga_store_kernel(const RowParams p) {
  constexpr int LPR = D / 16;
  pdl_trigger();
  pdl_wait();
  Tokens k;
  if (!tokens_of(p, k)) return;
  const int c = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  const RowFeed<D, kKey> fk(p, k);
  const RowFeed<D, kValue> fv(p, k);
  const uint4* k0 = reinterpret_cast<const uint4*>(fk.at(k, r0) + c * 16);
  const uint4* v0 = reinterpret_cast<const uint4*>(fv.at(k, r0) + c * 16);
  const uint4 ka = k0[0], kb = k0[1], va = v0[0], vb = v0[1];
  store_rows<D, E4M3, kKey>(p, k, fk, ka, kb);
  store_rows<D, E4M3, kValue>(p, k, fv, va, vb);
}

// Codes of rows [start, start + rows) times their scales, rounded to bf16:
// pieces of 8 codes, so that a warp's stores are 512 bytes on end, kPieces of
// them in flight per thread.  Bound by HBM: 1.0 million rows of 64, 197 MB: 36 us,
// 83 % of the copy rate (with pieces of 16 codes 41).
constexpr int kPieces = 4;

template <int D>
__global__ void __launch_bounds__(256) saga_load_kernel(const LoadParams p) {
  constexpr int PPR = D / 8;  // pieces per row
  pdl_trigger();
  pdl_wait();
  int h = blockIdx.y;
  const int b = h / (p.h_k + p.h_v);
  h -= b * (p.h_k + p.h_v);
  const bool key = h < p.h_k;
  if (!key) h -= p.h_k;
  uint16_t* out = key ? p.k_out : p.v_out;
  if (out == nullptr) return;
  const int heads = key ? p.h_k : p.h_v;
  const int rows = p.lens != nullptr ? min(p.rows, max(p.lens[b], 0) - p.start) : p.rows;
  const size_t row0 = ((size_t)b * heads + h) * p.l_cap + p.start;
  const uint8_t* codes = (key ? p.k : p.v) + row0 * D;
  const float* scales = (key ? p.k_scale : p.v_scale) + row0;
  out += ((size_t)b * heads + h) * p.rows * D;
  const long long pieces = (long long)max(rows, 0) * PPR, first = (long long)blockIdx.x * (256 * kPieces) + threadIdx.x;
  uint2 u[kPieces];
  float s[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const long long at = first + i * 256;
    u[i] = make_uint2(0u, 0u);
    s[i] = 0.f;
    if (at < pieces) {
      u[i] = reinterpret_cast<const uint2*>(codes)[at];
      s[i] = scales[at / PPR];
    }
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const long long at = first + i * 256;
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = k < 2 ? u[i].x : u[i].y;
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (k & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(hr));
      x[2 * k] = f.x * s[i];
      x[2 * k + 1] = f.y * s[i];
    }
    if (at < pieces) *reinterpret_cast<uint4*>(out + at * 8) = pack8(x);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_rows(const saga_rows* r, const char* name) {
  if (r == nullptr || r->data == nullptr) return api_fail(SAGA_ERR_ARG, "%s rows are NULL", name);
  if (!aligned16(r->data)) return api_fail(SAGA_ERR_ARG, "%s rows must be 16-byte aligned", name);
  for (long long st : {r->batch_stride, r->token_stride, r->head_stride})
    if (st < 0 || st % 8 != 0)
      return api_fail(SAGA_ERR_ARG, "%s strides (%lld, %lld, %lld) must be non-negative multiples of 8 elements", name,
                      r->batch_stride, r->token_stride, r->head_stride);
  return SAGA_OK;
}

int check_cache(const saga_shape* s, const saga_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return api_fail(SAGA_ERR_ARG, "NULL cache");
  if (!aligned16(c->k) || !aligned16(c->v)) return api_fail(SAGA_ERR_ARG, "caches must be 16-byte aligned");
  if (c->format != SAGA_CACHE_BF16 && c->format != SAGA_CACHE_E4M3)
    return api_fail(SAGA_ERR_ARG, "unknown cache format %d", c->format);
  if (c->format == SAGA_CACHE_E4M3 &&
      (c->k_scale == nullptr || c->v_scale == nullptr || (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) != 0 ||
       (reinterpret_cast<uintptr_t>(c->v_scale) & 3u) != 0))
    return api_fail(SAGA_ERR_ARG, "an 8-bit cache needs 4-byte aligned k_scale and v_scale");
  return SAGA_OK;
}

int run_rows(const saga_shape* s, int tokens, const saga_rows* q, const saga_rows* k, const saga_rows* v,
             const saga_norm_rope* op, const int* starts, const int* positions, const int* counts, void* q_out,
             const saga_cache* cache, unsigned* status, void* stream) {
  int rc = api_validate_shape(s);
  if (rc) return rc;
  if (tokens < 1) return api_fail(SAGA_ERR_ARG, "tokens=%d must be >= 1", tokens);
  if (tokens > s->l_cap) return api_fail(SAGA_ERR_ARG, "tokens=%d exceeds l_cap=%d", tokens, s->l_cap);
  if (q != nullptr) {
    rc = check_rows(q, "q");
    if (rc) return rc;
    if (q_out == nullptr || !aligned16(q_out)) return api_fail(SAGA_ERR_ARG, "q_out must be a 16-byte aligned buffer");
    // in place, a row must be written where it was read
    if (q_out == q->data && ((s->h_q > 1 && q->head_stride != s->d) || (tokens > 1 && q->token_stride != (long long)s->h_q * s->d) ||
                             (s->batch > 1 && q->batch_stride != (long long)tokens * s->h_q * s->d)))
      return api_fail(SAGA_ERR_ARG, "q_out may be q only where q is dense");
  }
  rc = check_rows(k, "k");
  if (rc) return rc;
  rc = check_rows(v, "v");
  if (rc) return rc;
  rc = check_cache(s, cache);
  if (rc) return rc;
  if (starts == nullptr) return api_fail(SAGA_ERR_ARG, "starts is NULL");
  if ((reinterpret_cast<uintptr_t>(status) & 3u) != 0) return api_fail(SAGA_ERR_ARG, "status must be 4-byte aligned");
  RowParams p{};
  p.q = q != nullptr ? static_cast<const uint16_t*>(q->data) : nullptr;
  p.k = static_cast<const uint16_t*>(k->data);
  p.v = static_cast<const uint16_t*>(v->data);
  if (q != nullptr) {
    p.q_bs = q->batch_stride;
    p.q_ts = q->token_stride;
    p.q_hs = q->head_stride;
  }
  p.k_bs = k->batch_stride;
  p.k_ts = k->token_stride;
  p.k_hs = k->head_stride;
  p.v_bs = v->batch_stride;
  p.v_ts = v->token_stride;
  p.v_hs = v->head_stride;
  if (op != nullptr) {
    if (op->norm) {
      if (!(op->eps >= 0.f) || !(op->eps < 1e30f)) return api_fail(SAGA_ERR_ARG, "eps must be finite and >= 0");
      if (!aligned16(op->q_weight) || !aligned16(op->k_weight))
        return api_fail(SAGA_ERR_ARG, "norm weights must be 16-byte aligned");
      p.norm = 1;
      p.eps = op->eps;
      p.q_weight = static_cast<const uint16_t*>(op->q_weight);
      p.k_weight = static_cast<const uint16_t*>(op->k_weight);
    }
    if (op->inv_freq != nullptr) {
      if (op->rot_dim < 16 || op->rot_dim > s->d || op->rot_dim % 16 != 0)
        return api_fail(SAGA_ERR_ARG, "rot_dim=%d must be a multiple of 16 in [16, d=%d]", op->rot_dim, s->d);
      p.inv_freq = op->inv_freq;
      p.rot = op->rot_dim;
      p.interleaved = op->interleaved != 0;
      p.positions = positions;
    }
  }
  p.starts = starts;
  p.counts = counts;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = cache->k;
  p.v_cache = cache->v;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.status = status;
  p.batch = s->batch;
  p.tokens = tokens;
  p.h_q = s->h_q;
  p.h_k = s->h_k;
  p.h_v = s->h_v;
  p.l_cap = s->l_cap;
  int sms = 0;
  rc = api_device_sms(&sms);
  if (rc) return rc;
  // Tokens of a CTA: its start takes about as long as two tokens, and an SM
  // holds 4 CTAs at a time.  17 heads of 128, normed and rotated: 2048 tokens in
  // 2048, 1024 and 512 CTAs 14.8, 10.2 and 7.8 us; 42 heads of 64: 8191 tokens in
  // 2048, 1024 and 512 CTAs 25.5, 23.1 and 25.5 us (the same rows again and again,
  // warm in the L2 as far as they fit).  Tokens of 2200 and 2700 elements; much
  // smaller ones were not measured.
  const int most = q == nullptr ? 64 : kMaxRowTokens;
  int group = 1;
  long long least = 0;
  for (int g = 1; g <= most; g *= 2) {
    const long long ctas = (long long)s->batch * ((tokens - 1) / g + 1);
    const long long cost = std::max(ctas, 4ll * sms) * (2 + g);
    if (g == 1 || cost < least) {
      least = cost;
      group = g;
    }
  }
  p.group = group;
  for (p.group_log2 = 0; 1 << p.group_log2 < group;) ++p.group_log2;
  p.groups = (tokens - 1) / group + 1;
  const long long ctas = (long long)s->batch * p.groups;
  if (ctas >= (1ll << 31)) return api_fail(SAGA_ERR_UNSUPPORTED, "batch * tokens too large");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->format == SAGA_CACHE_E4M3;
  void (*const kernels[8])(RowParams) = {saga_rows_kernel<64, false>,  saga_store_kernel<64, false>,
                                         saga_rows_kernel<64, true>,   saga_store_kernel<64, true>,
                                         saga_rows_kernel<128, false>, saga_store_kernel<128, false>,
                                         saga_rows_kernel<128, true>,  saga_store_kernel<128, true>};
  const int which = (s->d == 64 ? 0 : 4) + (e4m3 ? 2 : 0) + (q == nullptr ? 1 : 0);
  const auto kernel = kernels[which];
  static std::atomic<uint64_t> done[8];
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), 0, done[which]);
  if (e == cudaSuccess) e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(kRowThreads), 0, st, p);
  if (e != cudaSuccess) return api_cuda_fail(e, "row kernel launch");
  return api_ok();
}

}  // namespace

int api_check_cache(const saga_shape* s, const saga_cache* c) { return check_cache(s, c); }

}  // namespace saga

using namespace saga;

extern "C" {

int saga_norm_rope_append(const saga_shape* s, int tokens, const saga_rows* q, const saga_rows* k, const saga_rows* v,
                          const saga_norm_rope* op, const int* starts, const int* positions, const int* counts,
                          void* q_out, const saga_cache* cache, unsigned* status, void* stream) {
  if (op == nullptr) return api_fail(SAGA_ERR_ARG, "the norm and rotation arguments are NULL");
  if (q == nullptr) return api_fail(SAGA_ERR_ARG, "q rows are NULL");
  return run_rows(s, tokens, q, k, v, op, starts, positions, counts, q_out, cache, status, stream);
}

int saga_kv_store(const saga_shape* s, int tokens, const saga_rows* k, const saga_rows* v, const int* starts,
                  const int* counts, const saga_cache* cache, unsigned* status, void* stream) {
  return run_rows(s, tokens, nullptr, k, v, nullptr, starts, nullptr, counts, nullptr, cache, status, stream);
}

int saga_kv_load(const saga_shape* s, const saga_cache* cache, int start, int rows, const int* lens, void* k_out,
                 void* v_out, void* stream) {
  int rc = api_validate_shape(s);
  if (rc) return rc;
  rc = api_check_cache(s, cache);
  if (rc) return rc;
  if (cache->format != SAGA_CACHE_E4M3) return api_fail(SAGA_ERR_ARG, "saga_kv_load reads 8-bit caches");
  if (k_out == nullptr && v_out == nullptr) return api_fail(SAGA_ERR_ARG, "k_out and v_out are both NULL");
  if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15u)
    return api_fail(SAGA_ERR_ARG, "k_out and v_out must be 16-byte aligned");
  if (start < 0 || rows < 1 || rows > s->l_cap - start)
    return api_fail(SAGA_ERR_ARG, "rows [%d, %d + %d) outside [0, l_cap=%d)", start, start, rows, s->l_cap);
  LoadParams p{};
  p.k = static_cast<const uint8_t*>(cache->k);
  p.v = static_cast<const uint8_t*>(cache->v);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.lens = lens;
  p.batch = s->batch;
  p.h_k = s->h_k;
  p.h_v = s->h_v;
  p.l_cap = s->l_cap;
  p.start = start;
  p.rows = rows;
  const long long pairs = (long long)s->batch * (s->h_k + s->h_v);
  if (pairs > 65535) return api_fail(SAGA_ERR_UNSUPPORTED, "batch * (h_k + h_v) = %lld exceeds 65535", pairs);
  const long long threads = (long long)rows * (s->d / 8);
  const dim3 grid((unsigned)((threads + 256 * kPieces - 1) / (256 * kPieces)), (unsigned)pairs);
  auto kernel = s->d == 64 ? saga_load_kernel<64> : saga_load_kernel<128>;
  static std::atomic<uint64_t> done[2];
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), 0, done[s->d == 64 ? 0 : 1]);
  if (e == cudaSuccess) e = launch_pdl(kernel, grid, dim3(256), 0, static_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) return api_cuda_fail(e, "load launch");
  return api_ok();
}

}  // extern "C"
