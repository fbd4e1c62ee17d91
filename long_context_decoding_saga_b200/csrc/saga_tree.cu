// saga_tree.cu - attention of drafted tokens (a tree, a chain or one token)
// over a bf16 or 8-bit cache: saga_tree_attn.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "saga_device.cuh"
#include "saga_launch.cuh"
#include "saga_serve.h"

namespace saga {
namespace {

constexpr int kTreeThreads = 128;

template <bool E4M3>
__device__ __forceinline__ float cached(const void* base, const float* scale, size_t row, int D, int c) {
  if (!E4M3) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[row * D + c] << 16);
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[row * D + c], __NV_E4M3);
  return __half2float(__half(h)) * scale[row];
}

// One CTA per (batch row, token, query head): blocks of 128 rows, one score
// per thread, a running maximum and sum, and one output column per thread.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kTreeThreads) saga_tree_kernel(const TreeParams p) {
  __shared__ float qs[D], ps[kTreeThreads], red[4];
  pdl_trigger();
  pdl_wait();
  const int j = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
  int n = p.counts != nullptr ? p.counts[b] : p.tokens;
  n = min(max(n, 0), p.tokens);
  int P = p.prefix_lens[b];
  if (P < 0 || P > p.l_cap - n) {
    if (threadIdx.x == 0) flag_status(p.status, SAGA_STATUS_LEN_CLAMPED);
    P = P < 0 ? 0 : p.l_cap - n;
  }
  if (t >= n) return;
  const size_t orow = ((size_t)b * p.tokens + t) * p.h_q + j;
  if (threadIdx.x < D) qs[threadIdx.x] = __uint_as_float((uint32_t)p.q[orow * D + threadIdx.x] << 16);
  __syncthreads();
  const unsigned long long word = p.mask != nullptr ? p.mask[(size_t)b * p.tokens + t] : (2ull << t) - 1ull;
  const float tau = p.tau != nullptr ? p.tau[b * p.h_q + j] : -INFINITY;
  const size_t krow = ((size_t)b * p.h_k + (long long)j * p.h_k / p.h_q) * p.l_cap;
  const size_t vrow = ((size_t)b * p.h_v + (long long)j * p.h_v / p.h_q) * p.l_cap;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int i0 = 0; i0 < P + n; i0 += kTreeThreads) {
    const int i = i0 + threadIdx.x;
    float a = -INFINITY;
    if (i < P || (i < P + n && (word >> (i - P) & 1ull))) {
      float dot = 0.f;
      for (int c = 0; c < D; ++c) dot = fmaf(qs[c], cached<E4M3>(p.k, p.k_scale, krow + i, D, c), dot);
      dot *= p.scale;
      if (dot >= tau) a = dot;
    }
    const float wm = warp_max(a);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = wm;
    __syncthreads();
    const float bm = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    if (bm > -INFINITY) {
      const float mn = fmaxf(m, bm), f = expf(m - mn);
      ps[threadIdx.x] = expf(a - mn);
      __syncthreads();
      l *= f;
      o *= f;
      m = mn;
      const int lim = min(kTreeThreads, P + n - i0);
      for (int k = 0; k < lim; ++k) {
        const float w = ps[k];
        l += w;
        if (w != 0.f && threadIdx.x < D)
          o = fmaf(w, cached<E4M3>(p.v, p.v_scale, vrow + i0 + k, D, threadIdx.x), o);
      }
    }
    __syncthreads();
  }
  if (threadIdx.x < D) {
    const float r = l > 0.f ? o / l : 0.f;
    if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[orow * D + threadIdx.x] = __float2bfloat16(r);
    else static_cast<float*>(p.out)[orow * D + threadIdx.x] = r;
  }
}

constexpr size_t kTreeStatusBytes = 256;

int validate_tree(const saga_shape* s, int tokens) {
  int rc = api_validate_shape(s);
  if (rc) return rc;
  if (tokens < 1 || tokens > SAGA_TREE_MAX_TOKENS)
    return api_fail(SAGA_ERR_ARG, "tokens=%d outside [1, %d]", tokens, SAGA_TREE_MAX_TOKENS);
  if (tokens > s->l_cap) return api_fail(SAGA_ERR_ARG, "tokens=%d exceeds l_cap=%d", tokens, s->l_cap);
  return SAGA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace saga

using namespace saga;

extern "C" {

size_t saga_tree_workspace_bytes(const saga_shape* s, int tokens) {
  if (validate_tree(s, tokens)) return 0;
  return kTreeStatusBytes;
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
  if (ws_bytes < kTreeStatusBytes)
    return api_fail(SAGA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, kTreeStatusBytes);
  TreeParams p{};
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
  const bool e4m3 = cache->format == SAGA_CACHE_E4M3;
  auto kernel = s->d == 64 ? (e4m3 ? saga_tree_kernel<64, true> : saga_tree_kernel<64, false>)
                           : (e4m3 ? saga_tree_kernel<128, true> : saga_tree_kernel<128, false>);
  if (s->batch > 65535) return api_fail(SAGA_ERR_UNSUPPORTED, "batch=%d exceeds 65535", s->batch);
  cudaError_t e = launch_pdl(kernel, dim3(s->h_q, tokens, s->batch), dim3(kTreeThreads), 0,
                             static_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) return api_cuda_fail(e, "drafted-token attention launch");
  return api_ok();
}

}  // extern "C"
