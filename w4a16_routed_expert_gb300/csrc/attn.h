// Internal launch interface of the attention operators (include/moe_attention.h):
// between their runtime (attn_api.cu) and the kernel files attn_*.cu.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.h"

namespace moe {

// codes in the handle's error word
constexpr uint32_t kAttnErrTimeout = 1;
constexpr uint32_t kAttnErrBounds = 2;

// Norm + rotation, and with slots the store into the cache.
struct RopeArgs {
  const void *q, *k, *v;  // q or k may be nullptr; v only with slots
  void *q_out, *k_out;    // k_out unused with slots
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements between tokens
  int T, Hq, Hk, D, rotary;
  int interleaved;
  const int32_t* positions;
  const uint64_t* freq;  // [rotary / 2] turns per position as fractions of 2^64
  float m;               // factor on cosine and sine
  const float *q_norm, *k_norm;  // [D] or nullptr
  float eps;
  const int32_t* slots;  // [T] or nullptr
  void *k_cache, *v_cache;
  long long page_stride, slot_stride, head_stride, num_slots;
  int page_size;
  int heads_per_warp;    // heads of the (query, key, value) list one warp takes
  uint32_t* err;
};
cudaError_t launch_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t s, bool pdl);

// One forward over the paged cache.
struct AttnArgs {
  const void* q;
  long long q_stride;
  const void *k_cache, *v_cache;
  long long page_stride, slot_stride, head_stride;
  int page_size;
  int num_pages;
  int T, B, Hq, Hk, g, D;
  const int32_t *q_offsets, *seq_lens, *block_table, *prefix_pages;
  int table_stride, prefix_len, causal, max_q_len, max_seq_len;
  float scale;           // of the logits
  void* out;
  long long out_stride;
  float* lse;            // nullable
  uint32_t* err;
};
cudaError_t launch_attn_simple(const AttnArgs& a, bool bf16, cudaStream_t s);

}  // namespace moe
