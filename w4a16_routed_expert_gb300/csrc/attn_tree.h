// Bits of a drafted token's row (AttnArgs::tree), in plain C++ so that which
// words are read can be checked without a GPU.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MOE_TREE_FN __host__ __device__ __forceinline__
#else
#define MOE_TREE_FN inline
#endif

namespace moe {

// Words of a row that are read where sequences have at most max_q_len tokens:
// not those up to the next row, which behind the last one need not be there.
MOE_TREE_FN int tree_row_words(int max_q_len) { return (max_q_len + 31) / 32; }

// 32 bits of a row from bit `off` on, which may lie before its first: those are
// keys of the context, all seen. row[w] is its word w < words.
template <typename Row>
MOE_TREE_FN uint32_t tree_window(const Row& row, int words, int off) {
  if (off <= -32) return 0xffffffffu;
  const int w = off >> 5;  // -1 or more
  const uint32_t lo = w < 0 ? 0xffffffffu : w < words ? row[w] : 0u;
  const uint32_t hi = (off & 31) && w + 1 < words ? row[w + 1] : 0u;
#ifdef __CUDA_ARCH__
  return __funnelshift_r(lo, hi, off & 31);
#else
  return (uint32_t)((((uint64_t)hi << 32) | lo) >> (off & 31));
#endif
}
// The first n bits (all for 32 and more, none for 0 and less).
MOE_TREE_FN uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

}  // namespace moe
