// saga_serve.h - parameter blocks and host helpers of the serving operators:
// per-head norm and position rotation with the append, the 8-bit cache's
// store and load, and attention of drafted tokens.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "saga.h"
#include "saga_tree.h"

namespace saga {

// Defined in saga_api.cu: the error text of saga_last_error and the checks
// shared by every entry point.
int api_fail(int code, const char* fmt, ...);
int api_ok();
int api_cuda_fail(cudaError_t e, const char* what);
int api_validate_shape(const saga_shape* s);
int api_device_sms(int* sms);
unsigned api_take_test_wait();  // the limit of saga_test_expire_next_wait, once (0: none)
// Tensor map over `rows` cache rows of d elements, kTreeTile rows a box: 64
// columns of bf16 (one 128-byte swizzle row), or the whole row of e4m3 codes
// (swizzled in its own 64 or 128 bytes).
int api_rows_map(CUtensorMap* m, const void* base, long long rows, int d, bool e4m3);

// A quantised row: value = code * scale with scale = amax / kE4m3Max over the
// row's d elements.  Rows whose largest magnitude is below kAmaxFloor use it
// in amax's place, so neither the scale nor its reciprocal leaves the normal
// fp32 range.
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100

constexpr int kRowThreads = 256;
constexpr int kMaxRowTokens = 16;  // most tokens of one CTA of the row kernel

struct RowParams {
  const uint16_t* q;  // nullable: no queries
  const uint16_t* k;
  const uint16_t* v;
  long long q_bs, q_ts, q_hs;  // batch, token and head strides, in elements
  long long k_bs, k_ts, k_hs;
  long long v_bs, v_ts, v_hs;
  const uint16_t* q_weight;  // nullable: ones
  const uint16_t* k_weight;
  const float* inv_freq;  // nullable: no rotation
  const int* positions;   // nullable: the cache row
  const int* starts;
  const int* counts;  // nullable: every token is there
  uint16_t* q_out;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  unsigned* status;
  float eps;
  int norm, rot, interleaved;
  int batch, tokens, h_q, h_k, h_v, l_cap;
  int group;   // tokens of one CTA, a power of two
  int group_log2;
  int groups;  // CTAs per batch row
};

struct LoadParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  uint16_t* k_out;  // nullable
  uint16_t* v_out;
  const int* lens;  // nullable
  int batch, h_k, h_v, l_cap, start, rows;
};

struct TreeParams {
  const uint16_t* q;  // bf16 [B, T, h_q, d]
  const void* k;
  const void* v;
  const float* k_scale;  // e4m3 caches
  const float* v_scale;
  const int* prefix_lens;
  const int* counts;                // nullable
  const unsigned long long* mask;   // nullable: u <= t
  const float* tau;                 // nullable
  void* out;
  unsigned* status;
  float scale;  // fp32(1 / sqrt(d))
  int out_bf16;
  int batch, tokens, h_q, h_k, h_v, l_cap;
  TreePlan plan;
  TreeSmem smem;
  int ctas;        // of the attention kernel
  unsigned test_wait_ns;  // saga_test_expire_next_wait: a wait in vain before the products, for so long (0: none)
  float* part_o;   // [slots, cols, d]: sums of weights times values
  float* part_m;   // [slots, cols]: the power of two that the weights are relative to
  float* part_l;   // [slots, cols]: sums of weights
  int2* holders;   // [items]: first and last CTA of an item
};

int api_check_cache(const saga_shape* s, const saga_cache* c);

}  // namespace saga
