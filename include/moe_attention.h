/*
 * moe_attention.h — C ABI of the attention operators that stand beside the
 * routed-expert layer in a decoder block (GB300, sm_103a).
 *
 * Operators over one handle. Three in the order a decoder block runs them:
 *
 *   rotate   RMS norm of every query and key head, then the rotary rotation
 *              y[d]  = x[d] * rsqrt(mean_d x^2 + eps) * w[d]     (w given)
 *              (a, b) -> m * (a cos(p f_i) - b sin(p f_i),
 *                             b cos(p f_i) + a sin(p f_i))
 *            for the pairs i = 0 .. rotary_dim/2 - 1 of a head at position p:
 *            (a, b) = (y[i], y[i + rotary_dim/2]), or (y[2i], y[2i+1]) when
 *            interleaved; elements from rotary_dim on are only normed
 *   append   the same pass; the keys and the values go to slots of a paged
 *            cache
 *   forward  attention of a ragged batch over that cache: the keys of one
 *            prefix shared by every sequence, then each sequence's own keys
 *              o = sum_j e^(s_j) v_j / sum_j e^(s_j),  s_j = scale * q . k_j
 *              lse = ln sum_j e^(s_j)
 *            A row is a query token and one of the query heads of a key head.
 *            The prefix's keys of a key head are read once for every block of
 *            rows of all tokens: 256 of them, or 16 (32 at head sizes to 64)
 *            where few rows read a key; where the batch has as many tokens as
 *            fill a block of 256 rows for each sequence on average, once for
 *            every block of each sequence's rows, together with its own keys.
 *            (Over trees the few rows' blocks are of 16, 32 or 64, and where
 *            lengths are short the prefix may be read for every 128 or 256 rows
 *            of each sequence, however few tokens there are)
 *
 * and, around a step that checks trees of drafted tokens (the lengths then
 * stand on the GPU, where it is first known how many were right):
 *
 *   plan     offsets, positions, cache slots, block table entries and the
 *            trees' masks, from lengths, parents and a ring of free pages
 *   forward_tree  forward where a token sees, behind its sequence's context,
 *            the tokens of its own branch
 *   accept   the branch that the model's choices confirm
 *   keep     that branch's keys and values moved behind the context
 *
 * Frequencies: f_i = theta^(-2i/rotary_dim), scaled for long contexts by
 * moe_rope_scaling_t. An angle p * f_i is reduced to a fraction of a turn in
 * 64-bit fixed point, so it keeps its accuracy at any 32-bit position.
 *
 * Types: queries, keys, values, outputs and the cache are all FP16 or all
 * BF16; norms, angles, logits, softmax statistics and sums are FP32. Results
 * are rounded once when they are stored. (The probabilities that multiply
 * the values go to the tensor cores in the 16-bit type: in two parts, which
 * lose nothing beside the result's own rounding, where few rows read a key,
 * in one otherwise, and over trees from 17 rows on: a line of 17 to 32 rows of
 * at most 64 elements is then a little less exact as a tree than as causal.)
 *
 * Conventions are those of moe_layer.h: every call returns a moe_status_t
 * (moe_layer_last_error(NULL) describes the calling thread's last failure),
 * device pointers are borrowed, calls are asynchronous on the given CUDA
 * stream and allocate nothing, so they can be captured in a CUDA graph. One
 * forward and one plan at a time per handle (two that overlap share its
 * workspace); the others use none of it. Kernels never trap and every device-side
 * wait is bounded; moe_attn_sync reports what they recorded.
 */
#ifndef MOE_ATTENTION_H
#define MOE_ATTENTION_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_DTYPE_F16 = 0, MOE_DTYPE_BF16 = 1 } moe_dtype_t;

typedef enum {
  MOE_ROPE_NONE = 0,   /* f_i as they are */
  MOE_ROPE_LINEAR = 1, /* f_i / factor */
  MOE_ROPE_NTK = 2,    /* theta * factor^(rotary_dim / (rotary_dim - 2)): the slowest pair slows by factor */
  MOE_ROPE_YARN = 3    /* pairs that turn at least beta_fast times within original_max_position keep f_i, those
                          that turn at most beta_slow times take f_i / factor, a linear ramp over i between;
                          m = 0.1 ln(factor) + 1 where factor > 1 (m = 1 everywhere else) */
} moe_rope_scaling_t;

typedef struct {
  int32_t dtype;        /* moe_dtype_t */
  int32_t num_q_heads;  /* Hq, a multiple of Hk; query head h reads key head h / (Hq / Hk) */
  int32_t num_kv_heads; /* Hk, 1..1024 */
  int32_t head_dim;     /* D, a multiple of 8, 8..128 */
  int32_t max_tokens;   /* most query tokens of one forward, 1..2^20 (sizes the workspace) */
  int32_t max_seqs;     /* most sequences of one forward, 1..4096 */
  /* rotation */
  int32_t rotary_dim;       /* a multiple of 8, 0..D; 0: no rotation */
  int32_t rope_interleaved; /* 0: pairs (i, i + rotary_dim/2); 1: pairs (2i, 2i + 1) */
  int32_t rope_scaling;     /* moe_rope_scaling_t */
  int32_t rope_original_max_position; /* MOE_ROPE_YARN only */
  double rope_theta;
  double rope_factor;    /* > 0; ignored by MOE_ROPE_NONE */
  double rope_beta_fast; /* MOE_ROPE_YARN only (0: 32) */
  double rope_beta_slow; /* MOE_ROPE_YARN only (0: 1) */
  double norm_eps;       /* >= 0 */
  double scale;          /* of the logits, 1e-44 to 2e38; 0: 1 / sqrt(D) */
  /* cache: element (page, slot, head, d) of k_cache and of v_cache is at
   * page * page_stride + slot * slot_stride + head * head_stride + d
   * (elements; each stride a positive multiple of 8). */
  int32_t page_size; /* slots of a page, a multiple of 16, 16..1024 */
  int32_t reserved;  /* 0 */
  int64_t num_pages; /* num_pages * page_size <= 2^31 - 1 */
  int64_t page_stride, slot_stride, head_stride;
} moe_attn_config_t;

typedef struct {
  void* k_cache;       /* device, 16-byte aligned; both NULL: a handle for moe_attn_rotate only */
  void* v_cache;
  const float* q_norm; /* device FP32 [D] weights of the query heads' norm, 16-byte aligned, or NULL: no norm */
  const float* k_norm; /* the same of the key heads' norm */
} moe_attn_buffers_t;

typedef struct moe_attn moe_attn_t;

/* Frequencies in radians per position (inv_freq [rotary_dim / 2]) and the
 * factor m on cosine and sine of a configuration. Host only. Either output
 * may be NULL. */
moe_status_t moe_attn_frequencies(const moe_attn_config_t* config, double* inv_freq, double* m);

/* Validates the configuration, records the borrowed pointers and allocates
 * the workspace on the current CUDA device. Fails with INVALID_ARG /
 * UNSUPPORTED / OOM / CUDA; *out is NULL on failure. */
moe_status_t moe_attn_create(const moe_attn_config_t* config, const moe_attn_buffers_t* buffers, moe_attn_t** out);

/* Norm and rotation of T tokens' query and key heads.
 *   q, q_out   device [T][Hq][D], heads contiguous, tokens q_stride /
 *              q_out_stride elements apart (multiples of 8, at least Hq * D),
 *              16-byte aligned; both NULL: keys only
 *   k, k_out   the same with Hk; both NULL: queries only
 *   positions  device int32 [T] (any sign)
 * An output may be its own input (same pointer and stride); otherwise they
 * must not overlap. T = 0 returns MOE_OK without launching; T <= 2^22. */
moe_status_t moe_attn_rotate(moe_attn_t* attn, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const int32_t* positions, int32_t T, void* q_out, int64_t q_out_stride, void* k_out,
                             int64_t k_out_stride, void* stream);

/* moe_attn_rotate with the rotated keys, and the values as they are, stored
 * in the cache: token t's go to slot slots[t] % page_size of page
 * slots[t] / page_size. A token with a negative slot is stored nowhere (its
 * query is still written). A slot beyond the cache is skipped and recorded
 * (moe_attn_sync: MOE_ERR_INVALID_ARG). Tokens of one call must have
 * different slots. q and q_out as above (both NULL: no queries). */
moe_status_t moe_attn_append(moe_attn_t* attn, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const int32_t* positions, const int32_t* slots,
                             int32_t T, void* q_out, int64_t q_out_stride, void* stream);

/* A ragged batch of queries. Device arrays are read when the kernels run;
 * what the host passes are bounds that size the launch. */
typedef struct {
  int32_t num_tokens;          /* T: all sequences' query tokens, back to back */
  int32_t num_seqs;            /* B */
  const int32_t* q_offsets;    /* device [B + 1], ascending from 0 to T: sequence b's tokens */
  int32_t max_q_len;           /* at least every sequence's number of query tokens */
  const int32_t* seq_lens;     /* device [B]: sequence b's own keys (its query tokens' among them), 0 or more */
  int32_t max_seq_len;         /* at least every seq_lens[b], at most table_stride * page_size; 0: there are no own
                                  keys, and seq_lens and q_offsets are not looked at */
  const int32_t* block_table;  /* device [B][table_stride]: own key j is in slot j % page_size of page
                                  block_table[b][j / page_size]; NULL when max_seq_len is 0 */
  int32_t table_stride;
  int32_t prefix_len;          /* keys that every sequence sees before its own, 0 or more */
  const int32_t* prefix_pages; /* device [ceil(prefix_len / page_size)], laid out the same; NULL when 0 */
  int32_t causal;              /* 1: of its n own keys, query token i of m sees the first n - m + i + 1 (none
                                  when that is not positive); 0: all n */
} moe_attn_batch_t;

/* Attention of a batch.
 *   q    device [T][Hq][D], tokens q_stride elements apart, as above
 *   out  device [T][Hq][D], tokens out_stride elements apart; must not
 *        overlap q or the cache
 *   lse  device FP32 [T][Hq] or NULL
 * A query that sees no key gets zeros and lse = -infinity. Slots beyond a
 * sequence's (or the prefix's) length may hold anything, NaN included; a
 * value that is not finite at a key some query of a sequence sees may reach
 * every query of that sequence in the call. A length beyond its bound, an
 * offset out of order or a page beyond the cache is clamped and recorded
 * (moe_attn_sync: MOE_ERR_INVALID_ARG); the results of that call are
 * undefined, memory outside the cache is not touched. */
moe_status_t moe_attn_forward(moe_attn_t* attn, const void* q, int64_t q_stride, const moe_attn_batch_t* batch,
                              void* out, int64_t out_stride, float* lse, void* stream);

/* moe_attn_forward where the new tokens of each sequence are the nodes of a
 * tree (or any set of which each sees some): of its sequence's n keys, the last
 * m of which are its m query tokens', token i sees the first n - m and key
 * n - m + j where bit j % 32 of tree[token * tree_stride + j / 32] is set; a
 * row with no bit sees not even itself. Bits from m on are ignored. The prefix
 * is seen by all; batch->causal is not looked at. A step may be padded (up to
 * max_q_len * num_seqs tokens): tokens behind the last sequence's change nothing
 * in the others' rows; their own get zeros, or behind a prefix nothing of use.
 *   tree         device [T], rows of W = max_q_len / 32 rounded up words; none
 *                behind a row's first W is read
 *   tree_stride  words from one token's row to the next, at least W;
 *                T * tree_stride below 2^31
 * NULL with max_seq_len 0 (there are no own keys). */
moe_status_t moe_attn_forward_tree(moe_attn_t* attn, const void* q, int64_t q_stride, const moe_attn_batch_t* batch,
                                   const uint32_t* tree, int32_t tree_stride, void* out, int64_t out_stride, float* lse,
                                   void* stream);

/* The tables of one step. Sequence b holds context_lens[b] own keys in
 * state[2 + b] pages and adds new_lens[b] tokens; the pages that they need
 * beyond those are taken from the free ones in order of sequences, and a
 * sequence that ends gives all of its pages back (free from the next step on).
 * Where the free pages do not reach for a sequence that needs some, neither it
 * nor any later one that needs some is served: it gets no pages, no slots and
 * seq_lens 0, and its tokens see the prefix alone.
 * All arrays are on the device. */
typedef struct {
  int32_t num_seqs;            /* B, 0..4096 */
  int32_t num_tokens;          /* T, 0..2^22: room of the tokens' outputs, at least the sum of new_lens */
  int32_t max_nodes;           /* most new tokens of a tree, 0..1024; 0: no trees */
  int32_t prefix_len;          /* position of the first own key, 0..2^30 */
  const int32_t* context_lens; /* [B] */
  const int32_t* new_lens;     /* [B], 0 or more; -1: the sequence ends */
  const int32_t* parents;      /* [T] with max_nodes: the new token, counted within the sequence and before this
                                  one, that each continues; -1: the context */
  int32_t* block_table;        /* [B][table_stride]: new entries are written */
  int32_t table_stride;        /* at least 1 */
  int32_t free_capacity;       /* F: places of the ring, at least as many as there are pages in use */
  int32_t* free_pages;         /* [F]: the free pages are those at (first + i) % F, i < count */
  const int32_t* state;        /* [2 + B]: first, count, then the pages that each sequence holds */
  int32_t* state_out;          /* [2 + B]: after the step; may be state */
  int32_t* q_offsets;          /* out [B + 1]: each sequence's first token */
  int32_t* seq_lens;           /* out [B]: context_lens + new_lens; 0 for one that ends or is not served */
  int32_t* positions;          /* out [T]: prefix_len + context + place in the line, or depth in the tree */
  int32_t* slots;              /* out [T]: of key context + place; -1: not served */
  uint32_t* tree;              /* out [T][ceil(max_nodes / 32)]: a token's branch (moe_attn_forward_tree); NULL without */
} moe_attn_plan_t;

/* Fills a step's tables. Tokens behind the last sequence get position 0, slot
 * -1 and no bits; ring places and table entries that the step does not give out
 * or take back stay as they were. One plan at a time per handle. Lengths that
 * stand in an output (the last step's seq_lens as context_lens, in the same
 * tables) are refused: MOE_ERR_INVALID_ARG. A length,
 * parent, page or count out of range (a context that is negative, a sequence
 * longer than its row of the table or 2^30, more tokens than T or max_nodes, a parent
 * not before its child, a free page beyond the cache) is recorded (moe_attn_sync:
 * MOE_ERR_INVALID_ARG); such a sequence is not served, such a token has slot -1
 * or no parent. */
moe_status_t moe_attn_plan(moe_attn_t* attn, const moe_attn_plan_t* plan, void* stream);

/* The confirmed branch of each sequence's tree. Node 0 is the token that was
 * decided before; from an accepted node i the branch goes on to the first later
 * node whose parent is i and whose token is targets[i]. */
typedef struct {
  int32_t num_seqs;            /* B, 0..2^20 */
  int32_t num_tokens;          /* T, 0..2^22 */
  int32_t max_path;            /* P, 1..2^20: longest branch taken */
  int32_t reserved;            /* 0 */
  const int32_t* q_offsets;    /* device [B + 1] */
  const int32_t* parents;      /* device [T], counted within the sequence */
  const int32_t* tokens;       /* device [T]: what was drafted */
  const int32_t* targets;      /* device [T]: the model's choice after each token */
  const int32_t* seq_lens;     /* device [B] or NULL: a sequence with fewer keys than tokens (it was not served)
                                  accepts nothing */
  const int32_t* context_lens; /* device [B] */
  int32_t* path;               /* out [B][P]: the branch's nodes, then -1 */
  int32_t* counts;             /* out [B]: nodes of the branch */
  int32_t* next_tokens;        /* out [B]: targets of its last node; -1 where there is none */
  int32_t* context_out;        /* out [B]: context_lens + counts; may be context_lens */
} moe_attn_accept_t;

/* Uses no cache: a handle without one will do. An offset out of order or
 * beyond T is recorded (MOE_ERR_INVALID_ARG) and clamped. */
moe_status_t moe_attn_accept(moe_attn_t* attn, const moe_attn_accept_t* accept, void* stream);

/* Moves the keys and values of each sequence's accepted nodes: those of node
 * path[b][i] to key seq_lens[b] - m + i for i < counts[b], m the sequence's
 * tokens; in the caches of all n handles, which must be of one shape, type and
 * strides and no cache twice (one handle's keys and values may be one cache).
 *   path    device [num_seqs][path_stride], ascending from i or more;
 *           moe_attn_keep_strided: rows of path_len nodes, path_stride (at least
 *           that) words apart; none behind a row's path_len is read
 *   counts  device [num_seqs]
 * Errors are recorded in attns[0]: a path or count out of order or range, a
 * page beyond the cache; what stands before it in the path is moved. */
moe_status_t moe_attn_keep(moe_attn_t* const* attns, int32_t n, int32_t num_seqs, const int32_t* q_offsets,
                           const int32_t* seq_lens, int32_t max_seq_len, const int32_t* block_table,
                           int32_t table_stride, const int32_t* path, int32_t path_stride, const int32_t* counts,
                           void* stream);
moe_status_t moe_attn_keep_strided(moe_attn_t* const* attns, int32_t n, int32_t num_seqs, const int32_t* q_offsets,
                                   const int32_t* seq_lens, int32_t max_seq_len, const int32_t* block_table,
                                   int32_t table_stride, const int32_t* path, int32_t path_stride, int32_t path_len,
                                   const int32_t* counts, void* stream);

/* Synchronises `stream` and reports (then clears) the first of what the
 * handle's kernels recorded, on this stream or on others, since the last report:
 * MOE_ERR_INVALID_ARG for a slot, page, length or offset out of range,
 * MOE_ERR_TIMEOUT if a bounded wait gave up, MOE_ERR_CUDA on a CUDA error. */
moe_status_t moe_attn_sync(moe_attn_t* attn, void* stream);

/* Frees the workspace. NULL is accepted. Call after the last call on the
 * handle has completed. */
moe_status_t moe_attn_destroy(moe_attn_t* attn);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTENTION_H */
