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
  int32_t* seq_of;       // workspace [T]: each token's sequence
  void* out;
  long long out_stride;
  float* lse;            // nullable
  uint32_t* err;
};

// How one kernel's share of a forward is cut up. The keys that a block of
// `row_block` query rows reads (a row is a query token and one of the g query
// heads of a key head) form a group of key tiles: per key head and row block
// of all tokens the prefix's tiles, then per sequence, key head and row block
// the own keys'. All groups' tiles stand in one line, and each of n_cta
// blocks takes an equal run of it, so the work is even whatever the lengths.
// A block's run within one group gives one partial result (running maximum,
// sum, unnormalised output rows); the rows' partials are joined by
// launch_attn_join.
struct LineArgs {
  int row_block;         // rows of a group at most
  int key_tile;          // keys of a tile
  int has_prefix, has_own;
  int n_cta;
  int part_rows;         // rows a partial takes at most: min(row_block, most rows of a group)
  // device workspace, written by the kernel's first block for the join
  long long* share;      // tiles per block
  int32_t* own_off;      // [B + 1] own tiles of one key head before each sequence
  float* part_o;         // [rows][DP]: a group's rows at its first row + block * part_rows
  float2* part_ml;       // [rows] maximum (log2 units), sum
};
// Rows of partial results one kernel can write.
inline long long line_part_rows(const LineArgs& ln, long long T, long long Hq) {
  return (ln.has_prefix + ln.has_own) * T * Hq + (long long)ln.n_cta * ln.part_rows;
}

// Tensor maps of one cache tensor: boxes of `slots` slots x 64 elements, or of
// a whole head where head_dim is a multiple of 64 (dimensions d, slot, 64-wide
// half, head, page).
bool encode_cache_map(CUtensorMap* tm, const void* cache, bool bf16, int D, int page_size, int Hk, long long num_pages,
                      long long page_stride, long long slot_stride, long long head_stride, int slots, bool whole_head);

// Few rows to a key (at most 32): legacy tensor-core tiles of 16 rows.
constexpr int kRowsMax = 32;       // rows of a group it takes
constexpr int kRowsKeyTile = 64;
struct AttnRowsPlan {
  int n_cta, stages;
  size_t smem;
};
AttnRowsPlan plan_attn_rows(int D, int rows, int B, int num_sms);
cudaError_t launch_attn_rows(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln,
                             const AttnRowsPlan& plan, int box_slots, bool bf16, bool late_wait, cudaStream_t s, bool pdl);

// Many rows to a key: 128-row tcgen05 tiles, two to a block, one block per SM.
constexpr int kTileRows = 256;
constexpr int kTileKeyTile = 128;
cudaError_t launch_attn_tile(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln,
                             int box_slots, bool bf16, cudaStream_t s, bool pdl);

// Joins the partials of up to two kernels (n_cta = 0: not run) into out and lse.
struct JoinArgs {
  AttnArgs a;
  LineArgs line[2];
  int DP;
};
cudaError_t launch_attn_join(const JoinArgs& j, bool bf16, cudaStream_t s, bool pdl);

}  // namespace moe
