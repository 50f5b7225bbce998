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
  const uint32_t* tree;  // nullable: a row of bits a token, bit j: it sees its sequence's token j (causal is 0)
  int tree_words, tree_stride;  // words of a row that are read; from one row to the next
  float scale;           // of the logits
  void* out;
  long long out_stride;
  float* lse;            // nullable
  uint32_t* err;
};

// How one kernel's share of a forward is cut up. The keys that a block of
// `row_block` query rows reads (a row is a query token and one of the g query
// heads of a key head) form a group of key tiles: per key head and row block
// of all tokens the prefix's tiles, then per sequence, key head and row block
// the own keys'. (Where sequences have row blocks of their own anyway, the
// prefix's tiles stand at the front of every sequence's groups instead.) All groups stand in one line, each as its tiles after
// `weight` empty places (what starting on a group costs, in tiles), and each
// of n_cta blocks takes an equal run of it, so the work is even whatever the
// lengths. A block's run within one group gives one partial result (running
// maximum, sum, unnormalised output rows); launch_attn_join joins the rows'
// partials. Places are counted in 32 bits; the host checks that they fit.
struct LineArgs {
  int row_block;         // rows of a group at most
  int key_tile;          // keys of a tile
  int weight;
  int has_prefix, has_own;
  int joined;            // the prefix's tiles stand at the front of every own group (has_prefix is 0)
  int own_most;          // most places that one key head's own groups can have (line_own_places)
  int n_cta;
  int part_rows;         // rows a partial takes at most: min(row_block, most rows of a group)
  int part_row0;         // this kernel's first row of partials
  float* part_o;         // [rows][DP]: block c's partial of a group stands at the group's first row + c * part_rows
  float2* part_ml;       // [rows] reference maximum (a logit before the scale), sum
  int2 *info_prefix, *info_own;  // [T][Hq] first partial row and number of partials, 0 between forwards
  int whole;             // not 0: no line; a block takes whole groups (own keys, `joined` the prefix's before them),
                         // this many blocks of row_block rows a sequence, and stores their results: nothing is left to
                         // join
  int final_prefix, final_own;   // 1: these groups' rows have no other partials, one part alone is the result
};
// Rows of partial results one kernel can write.
inline long long line_part_rows(const LineArgs& ln, long long T, long long Hq) {
  return (ln.has_prefix + ln.has_own) * T * Hq + (long long)ln.n_cta * ln.part_rows;
}
// Most places that one key head's own groups can have on the line; most places
// of the line.
inline long long line_own_places(const AttnArgs& a, const LineArgs& ln) {
  const long long rows = (long long)a.T * a.g, kt = ln.key_tile, rb = ln.row_block;
  return ln.has_own ? (rows / rb + a.B) * ((a.max_seq_len + kt - 1) / kt + ln.weight +
                                           (ln.joined ? (a.prefix_len + kt - 1) / kt : 0))
                    : 0;
}
inline long long line_places(const AttnArgs& a, const LineArgs& ln) {
  const long long rows = (long long)a.T * a.g, kt = ln.key_tile, rb = ln.row_block;
  const long long prefix = ln.has_prefix ? (rows + rb - 1) / rb * ((a.prefix_len + kt - 1) / kt + ln.weight) : 0;
  return (prefix + line_own_places(a, ln)) * a.Hk;
}

// Tensor maps of one cache tensor: boxes of `slots` slots x 64 elements, or of
// a whole head where head_dim is a multiple of 64 (dimensions d, slot, 64-wide
// half, head, page).
bool encode_cache_map(CUtensorMap* tm, const void* cache, bool bf16, int D, int page_size, int Hk, long long num_pages,
                      long long page_stride, long long slot_stride, long long head_stride, int slots, bool whole_head);

// Few rows to a key: tiles of 16 rows on mma.sync. Up to 32 rows at head sizes
// to 64, up to 16 above: there two row tiles' outputs do not fit the registers
// beside a second block (20 rows of 128 over 16 sequences of 8000 keys: 173 us,
// 138 with one block an SM, 95 on the tcgen05 tiles; at 64, 20 rows behind 8192
// keys: 23 us, 29 on the tcgen05 tiles).
// Over trees up to 64, the warps as 1 by 4, 2 by 2 or 4 by 1 groups of 16 rows
// and of keys, at head sizes above 64 up to 32 where contexts may be long: 16
// trees of 64 rows of 128 to a key after 100, 500, 2000 keys 18, 32, 62 us (24,
// 35, 59 on the tcgen05 tiles in a line; in whole groups, which 33 rows and more
// may take, see whole_rows in attn_api.cu), 64 trees after 100 keys 52 (70), but 8 after
// 15000 keys 107 (86): there the products bind. 128 rows after 500 keys 57 (39).
constexpr int kRowsMax = 64;
constexpr int kRowsLong = 4096;  // own keys
constexpr int rows_most(int D, bool tree, int max_keys) {
  return tree ? (D <= 64 || max_keys <= kRowsLong ? 64 : 32) : D <= 64 ? 32 : 16;
}
// (query token, query head, prefix key) triples up to which it takes the
// prefix's rows beside few own rows, however many. In its launch / in one of
// the tcgen05 kernel before it, own keys to 200: 24 rows of 128 over 300, 4000,
// 16000 prefix keys of 16 heads (0.1, 1.5, 6.1 million) 15 / 23, 24 / 31, 44 /
// 48 us; 96 rows over 4000, 16000 of 8 heads (3.1, 12) 23 / 27, 54 / 38; 256
// rows of 64 over 1000, 4000 (2.0, 8.2) 21 / 24, 33 / 27.
// Over trees, whose row groups read a key once for 32 rows and more: 128
// tokens of up to 64 rows of 64 over 4000 keys (8.8 million) 37 / 33 us, over
// 2000 of 128-wide heads (4.4) 36 / 41; 300 tokens of 128-wide heads over 1000
// (9.6) 77 / 75.
constexpr long long few_triples(bool tree) { return tree ? 1LL << 23 : 1LL << 22; }
constexpr int kRowsKeyTile = 64;
// Over trees without a prefix, own keys up to which a block takes whole groups
// (LineArgs::whole): the scan over the sequences, parts and the join's launch go,
// for the time that a group's tiles take one block instead of several. 16 heads
// of 128, trees of 16 tokens after up to 100, 250, 490 keys, whole / in a line:
// one 7.6 / 8.5, 9.7 / 9.5, 12.0 / 10.4 us, 16 8.3 / 12.9, 10.6 / 15.4, 16.7 /
// 19.6, 64 25.4 / 30.1, 32.4 / 35.8, 44.8 / 47.2; and the call's second launch.
// (One bound for all: a lone sequence in a captured step, which pays for no
// launch, would be better off in a line from about 240 keys on, many from 500.)
constexpr int kWholeKeys = 320;
struct AttnRowsPlan {
  int n_cta, stages, row_groups;
  size_t smem;
};
AttnRowsPlan plan_attn_rows(int D, int rows, int B, int num_sms, bool tree);
// LineArgs::weight (0, 1, 2, 3, 5 for 16 sequences behind 4099 keys: 36.4, 26.1,
// 26.0, 26.1, 26.9 us; for 48 sequences of drafts: 59.5, 50.5, 47.7, 48.1, 48.5)
constexpr int kRowsWeight = 2;
cudaError_t launch_attn_rows(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln,
                             const AttnRowsPlan& plan, int box_slots, bool bf16, bool late_wait, cudaStream_t s, bool pdl);

// Many rows to a key: 128-row tcgen05 tiles, two to a block, one block per SM.
constexpr int kTileRows = 256;
constexpr int kTileKeyTile = 128;
// LineArgs::weight (0, 2, 3, 5, 8 for 48 sequences of drafts: 50.9, 48.5, 47.7,
// 49.6, 49.3 us; for 64 behind 32768 keys: 88.1, 84.0, 83.6, 83.3, 83.5)
constexpr int kTileWeight = 3;
cudaError_t launch_attn_tile(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln,
                             int box_slots, bool bf16, cudaStream_t s, bool pdl);

// Joins the partials of a forward into out and lse.
struct JoinArgs {
  AttnArgs a;
  const float* part_o;
  const float2* part_ml;
  int2 *info_prefix, *info_own;
  int prefix_step, own_step;  // rows between the partials of one row (0: that kind was not computed)
  int DP;
};
cudaError_t launch_attn_join(const JoinArgs& j, bool bf16, cudaStream_t s, bool pdl);

// A step's tables (moe_attn_plan_t).
struct PlanArgs {
  int B, T, max_nodes, words, prefix_len;
  const int32_t *context_lens, *new_lens, *parents;
  int32_t* block_table;
  int table_stride, ring_size, page_size, num_pages;
  int32_t* free_pages;
  const int32_t* state;
  int32_t* state_out;
  int32_t *q_offsets, *seq_lens, *positions, *slots;
  uint32_t* tree;
  uint32_t* ticket;  // blocks that are done, 0 between plans
  uint32_t* err;
};
cudaError_t launch_attn_plan(const PlanArgs& a, int num_sms, cudaStream_t s, bool pdl);

// The confirmed branch of each tree (moe_attn_accept_t).
struct AcceptArgs {
  int B, T, P;
  const int32_t *q_offsets, *parents, *tokens, *targets, *seq_lens, *context_lens;
  int32_t *path, *counts, *next_tokens, *context_out;
  uint32_t* err;
};
cudaError_t launch_attn_accept(const AcceptArgs& a, cudaStream_t s, bool pdl);

// Accepted nodes' keys and values in up to kKeepCaches cache tensors to their
// places.
constexpr int kKeepCaches = 64;
struct KeepArgs {
  void* caches[kKeepCaches];
  int count, B, Hk, D, page_size, num_pages, max_seq_len, table_stride;
  int path_stride, path_len;  // from one sequence's path to the next, its words
  long long page_stride, slot_stride, head_stride;
  const int32_t *q_offsets, *seq_lens, *block_table, *path, *counts;
  uint32_t* err;
};
cudaError_t launch_attn_keep(const KeepArgs& a, int num_sms, cudaStream_t s, bool pdl);

}  // namespace moe
