// saga_cache.cu - rows on their way into and out of the caches: per-head norm
// and position rotation with the append (saga_norm_rope_append), the ragged
// append alone (saga_kv_store), both into bf16 or 8-bit caches, and the 8-bit
// rows read back (saga_kv_load).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

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

// One CTA holds `group` tokens of one batch row and all their heads; a row of
// a head (d elements) is D / 8 lanes of 16 bytes each, so its sum of squares,
// its rotation partners and its largest magnitude are shuffles.  The angles
// are the same for every head: they are computed once per token into shared
// memory.  Rows are taken head by head, so neighbouring lanes write
// neighbouring cache rows and scales.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) saga_rows_kernel(const RowParams p) {
  constexpr int LPR = D / 8;  // lanes per row
  constexpr int RPP = kRowThreads / LPR;  // rows per pass
  __shared__ float2 turns[kMaxRowTokens * (D / 2)];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x / p.groups;
  const int t0 = (blockIdx.x - b * p.groups) * p.group;
  int count = p.counts != nullptr ? p.counts[b] : p.tokens;
  count = min(max(count, 0), p.tokens);
  const int nt = min(p.group, count - t0);
  if (nt <= 0) return;
  const int start = p.starts[b];
  const int half = p.rot >> 1;
  if (p.inv_freq != nullptr) {
    for (int i = threadIdx.x; i < nt * half; i += kRowThreads) {
      const int t = i / half, f = i - t * half;
      const int pos = p.positions != nullptr ? p.positions[(size_t)b * p.tokens + t0 + t]
                                             : (int)((unsigned)start + (unsigned)(t0 + t));
      turns[t * half + f] = turn_of(pos, p.inv_freq[f]);
    }
    __syncthreads();
  }
  const int hq = p.q != nullptr ? p.h_q : 0;
  const int items = (hq + p.h_k + p.h_v) * nt;
  const int c = threadIdx.x % LPR;
  for (int base = 0; base < items; base += RPP) {
    const int item = base + threadIdx.x / LPR;
    const bool live = item < items;
    int head = live ? item / nt : 0;
    const int t = live ? item - head * nt : 0;
    const uint16_t* src;
    int kind;  // 0: query, 1: key, 2: value
    if (head < hq) {
      kind = 0;
      src = p.q + b * p.q_bs + (t0 + t) * p.q_ts + head * p.q_hs;
    } else if (head < hq + p.h_k) {
      kind = 1;
      head -= hq;
      src = p.k + b * p.k_bs + (t0 + t) * p.k_ts + head * p.k_hs;
    } else {
      kind = 2;
      head -= hq + p.h_k;
      src = p.v + b * p.v_bs + (t0 + t) * p.v_ts + head * p.v_hs;
    }
    float x[8];
    const uint4 raw = *reinterpret_cast<const uint4*>(src + c * 8);
    unpack8(raw, x);
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (kind != 2) {
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const uint16_t* wp = kind == 0 ? p.q_weight : p.k_weight;
        float w[8];
        if (wp != nullptr) {
          unpack8(*reinterpret_cast<const uint4*>(wp + c * 8), w);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = 1.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
      }
    }
    if (p.inv_freq != nullptr) {
      const float2* tt = turns + t * half;
      if (p.interleaved) {
        if (kind != 2 && c * 8 < p.rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 cs = tt[c * 4 + i];
            const float a = x[2 * i], e = x[2 * i + 1];
            x[2 * i] = a * cs.x - e * cs.y;
            x[2 * i + 1] = e * cs.x + a * cs.y;
          }
        }
      } else {
        const int rc = p.rot >> 4;  // 8-element chunks of half the rotated elements
        const int peer = c < rc ? c + rc : c < 2 * rc ? c - rc : c;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], peer, LPR);
        if (kind != 2 && c < 2 * rc) {
          const int f0 = (c < rc ? c : c - rc) * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 cs = tt[f0 + i];
            x[i] = c < rc ? x[i] * cs.x - y[i] * cs.y : x[i] * cs.x + y[i] * cs.y;
          }
        }
      }
    }
    const int slot = (int)((unsigned)start + (unsigned)(t0 + t));  // may wrap for a start that is no row: then it does not fit
    const bool fits = (unsigned)slot < (unsigned)p.l_cap;
    float amax = 0.f;
    if (E4M3) {
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      amax = fmaxf(amax, kAmaxFloor);
    }
    if (!live) continue;
    if (kind == 0) {
      *reinterpret_cast<uint4*>(p.q_out + ((size_t)((size_t)b * p.tokens + t0 + t) * p.h_q + head) * D + c * 8) = pack8(x);
      continue;
    }
    if (!fits) {
      if (c == 0) flag_status(p.status, SAGA_STATUS_LEN_CLAMPED);
      continue;
    }
    const size_t row = ((size_t)b * (kind == 1 ? p.h_k : p.h_v) + head) * p.l_cap + slot;
    void* cache = kind == 1 ? p.k_cache : p.v_cache;
    if (E4M3) {
      const float up = kE4m3Max / amax;
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h] * up, x[4 * h + 1] * up), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h + 2] * up, x[4 * h + 3] * up), __NV_SATFINITE, __NV_E4M3);
        w[h] = lo | hi << 16;
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D + c * 8) = make_uint2(w[0], w[1]);
      if (c == 0) (kind == 1 ? p.k_scale : p.v_scale)[row] = amax / kE4m3Max;
    } else {
      // an untouched value row (or key row without norm and rotation) round-trips through fp32 exactly
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + row * D + c * 8) = pack8(x);
    }
  }
}

// Codes of rows [start, start + rows) times their scales, rounded to bf16:
// 16 codes per thread.
template <int D>
__global__ void __launch_bounds__(256) saga_load_kernel(const LoadParams p) {
  constexpr int TPR = D / 16;
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
  const int r = (int)((blockIdx.x * 256u + threadIdx.x) / TPR), c = threadIdx.x % TPR;
  if (r >= rows) return;
  const size_t row = ((size_t)b * heads + h) * p.l_cap + p.start + r;
  const uint4 u = *reinterpret_cast<const uint4*>((key ? p.k : p.v) + row * D + c * 16);
  const float s = (key ? p.k_scale : p.v_scale)[row];
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(hr));
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
  uint4* dst = reinterpret_cast<uint4*>(out + (((size_t)b * heads + h) * p.rows + r) * D + c * 16);
  dst[0] = pack8(x);
  dst[1] = pack8(x + 8);
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
  }
  rc = check_rows(k, "k");
  if (rc) return rc;
  rc = check_rows(v, "v");
  if (rc) return rc;
  rc = check_cache(s, cache);
  if (rc) return rc;
  if (starts == nullptr) return api_fail(SAGA_ERR_ARG, "starts is NULL");
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
  // Few tokens: one CTA each.  Many: up to kMaxRowTokens a CTA, as long as every SM keeps eight CTAs.
  int group = 1;
  while (group < kMaxRowTokens && (long long)s->batch * ((tokens + 2 * group - 1) / (2 * group)) >= 8ll * sms) group *= 2;
  p.group = group;
  p.groups = (tokens + group - 1) / group;
  const long long ctas = (long long)s->batch * p.groups;
  if (ctas >= (1ll << 31)) return api_fail(SAGA_ERR_UNSUPPORTED, "batch * tokens too large");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->format == SAGA_CACHE_E4M3;
  auto kernel = s->d == 64 ? (e4m3 ? saga_rows_kernel<64, true> : saga_rows_kernel<64, false>)
                           : (e4m3 ? saga_rows_kernel<128, true> : saga_rows_kernel<128, false>);
  static std::atomic<uint64_t> done[4];
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), 0, done[(s->d == 64 ? 0 : 2) + (e4m3 ? 1 : 0)]);
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
  const long long threads = (long long)rows * (s->d / 16);
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)pairs);
  auto kernel = s->d == 64 ? saga_load_kernel<64> : saga_load_kernel<128>;
  static std::atomic<uint64_t> done[2];
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), 0, done[s->d == 64 ? 0 : 1]);
  if (e == cudaSuccess) e = launch_pdl(kernel, grid, dim3(256), 0, static_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) return api_cuda_fail(e, "load launch");
  return api_ok();
}

}  // extern "C"
