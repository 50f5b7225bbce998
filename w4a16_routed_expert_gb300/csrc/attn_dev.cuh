// Device helpers shared by the attention operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "attn.h"
#include "attn_tree.h"
#include "common.cuh"

namespace moe {

// The two 16-bit types: a pair of values in a 32-bit word, low half first.
template <typename T>
struct Half16;
template <>
struct Half16<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Half16<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// A sequence of the batch: its query tokens [t0, t0 + n) and its own keys,
// clamped to the batch and to the bounds the caller gave. All three words are
// asked for before any is looked at.
struct Seq {
  int t0, n, keys;
};
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  const int lo = __ldg(a.q_offsets + b), hi = __ldg(a.q_offsets + b + 1), keys = __ldg(a.seq_lens + b);
  Seq s;
  s.t0 = min(max(lo, 0), a.T);
  s.n = min(min(max(hi - lo, 0), a.max_q_len), a.T - s.t0);
  s.keys = min(max(keys, 0), a.max_seq_len);
  if (s.t0 != lo || s.n != hi - lo || s.keys != keys) record_error(a.err, kAttnErrBounds);
  return s;
}
// A page of the cache, clamped to it.
__device__ __forceinline__ int page_in_cache(const AttnArgs& a, int page) {
  if ((unsigned)page >= (unsigned)a.num_pages) {
    record_error(a.err, kAttnErrBounds);
    return 0;
  }
  return page;
}
// Own keys that query token i of n sees when its sequence holds `keys`.
__device__ __forceinline__ int keys_seen(const AttnArgs& a, int keys, int n, int i) {
  return a.causal ? min(keys, max(0, keys - n + i + 1)) : keys;
}

// A drafted token's row of AttnArgs::tree (tree_window).
struct TreeRow {
  const uint32_t* at;
  __device__ __forceinline__ uint32_t operator[](int w) const { return __ldg(at + w); }
};

}  // namespace moe
