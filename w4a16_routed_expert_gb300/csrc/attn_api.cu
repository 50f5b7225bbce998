// Runtime of the attention operators (include/moe_attention.h): validates the
// configuration and every call's arguments, owns the workspace, and enqueues
// the kernels on the caller's stream.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <new>

#include "attn.h"
#include "layer_internal.h"
#include "moe_attention.h"

using moe::set_error;

struct moe_attn {
  moe_attn_config_t cfg;
  moe_attn_buffers_t buf;
  int device = 0;
  int num_sms = 0;
  bool pdl = true;
  float scale = 0.f;
  float rope_m = 1.f;
  void* ws = nullptr;
  uint32_t* err = nullptr;
  uint64_t* freq = nullptr;
  // forward's workspace
  int2* info[2] = {};            // [max_tokens][Hq] of the prefix, of own keys: where a row's partials are
  float* part_o = nullptr;       // [part_rows][DP]
  float2* part_ml = nullptr;     // [part_rows]
  size_t part_rows = 0;
  int DP = 0;
  int box_rows = 0, box_tile = 0;  // slots of one copy of the few-row and of the tile kernel
  CUtensorMap rows_k, rows_v, tile_k, tile_v;
};

namespace {

constexpr double kPi = 3.14159265358979323846;

moe_status_t cuda_error(cudaError_t e, const char* what) {
  cudaGetLastError();
  return set_error(MOE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

moe_status_t validate_rope(const moe_attn_config_t* c) {
  if (c->head_dim < 8 || c->head_dim > 128 || c->head_dim % 8)
    return set_error(MOE_ERR_UNSUPPORTED, "head_dim=%d: supported 8..128, multiple of 8", c->head_dim);
  if (c->rotary_dim < 0 || c->rotary_dim > c->head_dim)
    return set_error(MOE_ERR_INVALID_ARG, "rotary_dim=%d out of 0..head_dim", c->rotary_dim);
  if (c->rotary_dim % 8)
    return set_error(MOE_ERR_UNSUPPORTED, "rotary_dim=%d: supported multiples of 8", c->rotary_dim);
  if (c->rope_interleaved != 0 && c->rope_interleaved != 1)
    return set_error(MOE_ERR_INVALID_ARG, "rope_interleaved must be 0 or 1");
  if (c->rope_scaling < MOE_ROPE_NONE || c->rope_scaling > MOE_ROPE_YARN)
    return set_error(MOE_ERR_INVALID_ARG, "rope_scaling=%d unknown", c->rope_scaling);
  if (c->rotary_dim > 0) {
    if (!(c->rope_theta > 1.0) || !std::isfinite(c->rope_theta))
      return set_error(MOE_ERR_INVALID_ARG, "rope_theta=%g must be above 1", c->rope_theta);
    if (c->rope_scaling != MOE_ROPE_NONE && (!(c->rope_factor > 0.0) || !std::isfinite(c->rope_factor)))
      return set_error(MOE_ERR_INVALID_ARG, "rope_factor=%g must be positive", c->rope_factor);
    if (c->rope_scaling == MOE_ROPE_YARN) {
      if (c->rope_original_max_position < 1)
        return set_error(MOE_ERR_INVALID_ARG, "rope_original_max_position=%d must be positive",
                         c->rope_original_max_position);
      if (!(c->rope_beta_fast >= 0.0) || !(c->rope_beta_slow >= 0.0) || !std::isfinite(c->rope_beta_fast) ||
          !std::isfinite(c->rope_beta_slow))
        return set_error(MOE_ERR_INVALID_ARG, "rope_beta_fast and rope_beta_slow must not be negative");
    }
  }
  return MOE_OK;
}

// f_i and m; c has passed validate_rope.
void frequencies(const moe_attn_config_t* c, double* inv, double* m) {
  const int rd = c->rotary_dim;
  double base = c->rope_theta;
  const double f = c->rope_factor;
  *m = 1.0;
  if (c->rope_scaling == MOE_ROPE_NTK && rd > 2) base *= std::pow(f, (double)rd / (rd - 2));
  for (int i = 0; i < rd / 2; ++i) inv[i] = std::pow(base, -2.0 * i / rd);
  if (c->rope_scaling == MOE_ROPE_LINEAR)
    for (int i = 0; i < rd / 2; ++i) inv[i] /= f;
  if (c->rope_scaling == MOE_ROPE_YARN) {
    const double fast = c->rope_beta_fast > 0.0 ? c->rope_beta_fast : 32.0;
    const double slow = c->rope_beta_slow > 0.0 ? c->rope_beta_slow : 1.0;
    // the pair that turns `turns` times within the original context
    auto dim_of = [&](double turns) {
      return rd * std::log(c->rope_original_max_position / (turns * 2.0 * kPi)) / (2.0 * std::log(base));
    };
    const double lo = std::max(std::floor(dim_of(fast)), 0.0);
    const double hi = std::min(std::ceil(dim_of(slow)), (double)rd - 1);
    const double width = std::max(hi - lo, 0.001);
    for (int i = 0; i < rd / 2; ++i) {
      const double ramp = std::min(std::max((i - lo) / width, 0.0), 1.0);
      inv[i] = inv[i] / f * ramp + inv[i] * (1.0 - ramp);
    }
    *m = f > 1.0 ? 0.1 * std::log(f) + 1.0 : 1.0;
  }
}

moe_status_t validate(const moe_attn_config_t* c, const moe_attn_buffers_t* b) {
  if (!c || !b) return set_error(MOE_ERR_INVALID_ARG, "config and buffers must not be NULL");
  if (c->dtype != MOE_DTYPE_F16 && c->dtype != MOE_DTYPE_BF16)
    return set_error(MOE_ERR_INVALID_ARG, "dtype=%d unknown", c->dtype);
  if (c->num_kv_heads < 1 || c->num_kv_heads > 1024)
    return set_error(MOE_ERR_INVALID_ARG, "num_kv_heads=%d out of 1..1024", c->num_kv_heads);
  if (c->num_q_heads < 1 || c->num_q_heads > 1024 || c->num_q_heads % c->num_kv_heads)
    return set_error(MOE_ERR_INVALID_ARG, "num_q_heads=%d: a multiple of num_kv_heads=%d, at most 1024",
                     c->num_q_heads, c->num_kv_heads);
  const moe_status_t st = validate_rope(c);
  if (st != MOE_OK) return st;
  if (!(c->norm_eps >= 0.0) || !std::isfinite(c->norm_eps))
    return set_error(MOE_ERR_INVALID_ARG, "norm_eps=%g must not be negative", c->norm_eps);
  if (!std::isfinite(c->scale) || c->scale < 0.0)
    return set_error(MOE_ERR_INVALID_ARG, "scale=%g must not be negative", c->scale);
  // zero or infinite in FP32, it would make NaN of masked logits or of the largest
  if (c->scale > 0.0 && (c->scale < 1e-44 || c->scale > 2e38))
    return set_error(MOE_ERR_INVALID_ARG, "scale=%g must be 0 or from 1e-44 to 2e38", c->scale);
  if ((reinterpret_cast<uintptr_t>(b->q_norm) | reinterpret_cast<uintptr_t>(b->k_norm)) % 16)
    return set_error(MOE_ERR_INVALID_ARG, "q_norm and k_norm must be 16-byte aligned");
  if (c->reserved != 0) return set_error(MOE_ERR_INVALID_ARG, "reserved must be 0");
  if ((b->k_cache == nullptr) != (b->v_cache == nullptr))
    return set_error(MOE_ERR_INVALID_ARG, "k_cache and v_cache go together");
  if (b->k_cache) {
    if (c->max_tokens < 1 || c->max_tokens > (1 << 20))
      return set_error(MOE_ERR_INVALID_ARG, "max_tokens=%d out of 1..2^20", c->max_tokens);
    if ((long long)c->max_tokens * c->num_q_heads > (1LL << 27))
      return set_error(MOE_ERR_INVALID_ARG, "max_tokens * num_q_heads too large (at most 2^27)");
    if (c->max_seqs < 1 || c->max_seqs > 4096)
      return set_error(MOE_ERR_INVALID_ARG, "max_seqs=%d out of 1..4096", c->max_seqs);
    if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16)
      return set_error(MOE_ERR_UNSUPPORTED, "page_size=%d: supported 16..1024, multiple of 16", c->page_size);
    if (c->num_pages < 1 || c->num_pages > INT_MAX / c->page_size)
      return set_error(MOE_ERR_INVALID_ARG, "num_pages=%lld: num_pages * page_size out of 1..2^31 - 1",
                       (long long)c->num_pages);
    const int64_t strides[3] = {c->page_stride, c->slot_stride, c->head_stride};
    for (int64_t s : strides)
      if (s <= 0 || s % 8 || s >= (1LL << 38))
        return set_error(MOE_ERR_INVALID_ARG, "cache strides must be positive multiples of 8 elements");
    if (c->head_stride < c->head_dim || c->slot_stride < c->head_dim || c->page_stride < c->head_dim)
      return set_error(MOE_ERR_INVALID_ARG, "cache strides must be at least head_dim");
    if ((reinterpret_cast<uintptr_t>(b->k_cache) | reinterpret_cast<uintptr_t>(b->v_cache)) % 16)
      return set_error(MOE_ERR_INVALID_ARG, "k_cache and v_cache must be 16-byte aligned");
  }
  return MOE_OK;
}

// A [T][heads][D] operand with `stride` elements between tokens.
moe_status_t check_rows(const moe_attn* h, const char* fn, const char* name, const void* p, int64_t stride,
                        int heads) {
  if (reinterpret_cast<uintptr_t>(p) % 16)
    return set_error(MOE_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", fn, name);
  if (stride % 8 || stride < (int64_t)heads * h->cfg.head_dim || stride >= (1LL << 38))
    return set_error(MOE_ERR_INVALID_ARG, "%s: %s: token stride %lld must be a multiple of 8, at least heads * head_dim",
                     fn, name, (long long)stride);
  return MOE_OK;
}

moe_status_t check_handle(const moe_attn* h, const char* fn) {
  if (!h) return set_error(MOE_ERR_INVALID_ARG, "%s: handle must not be NULL", fn);
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_error(e, fn);
  if (dev != h->device)
    return set_error(MOE_ERR_INVALID_ARG, "%s: the handle was created on device %d, device %d is current", fn,
                     h->device, dev);
  return MOE_OK;
}

void fill_rope(const moe_attn* h, moe::RopeArgs* a) {
  const moe_attn_config_t& c = h->cfg;
  a->Hq = c.num_q_heads;
  a->Hk = c.num_kv_heads;
  a->D = c.head_dim;
  a->rotary = c.rotary_dim;
  a->interleaved = c.rope_interleaved;
  a->freq = h->freq;
  a->m = h->rope_m;
  a->q_norm = h->buf.q_norm;
  a->k_norm = h->buf.k_norm;
  a->eps = (float)c.norm_eps;
  a->err = h->err;
}

// Enqueue a forward whose arguments have been checked.
moe_status_t forward(moe_attn* h, const moe::AttnArgs& a, cudaStream_t s) {
  const char* fn = "moe_attn_forward";
  const bool bf16 = h->cfg.dtype == MOE_DTYPE_BF16;
  const int own_rows = a.max_seq_len > 0 ? a.max_q_len * a.g : 0;
  const int prefix_rows = a.prefix_len > 0 ? (int)std::min<long long>((long long)a.T * a.g, INT_MAX / 2) : 0;
  // Few rows to a key go to the few-row kernel (16-row tiles, hardly any
  // padding, two blocks an SM), more to the 128-row tiles of the tcgen05
  // kernel, of which a block takes two. Beside few own rows a prefix of many
  // stays in the few-row kernel's launch while there is little to compute, in
  // row blocks that read its keys once each.
  const int most = moe::rows_most(a.D);
  const bool little = own_rows && (long long)a.T * a.Hq * a.prefix_len <= moe::kFewTriples;
  const bool tile_own = own_rows > most;
  const bool tile_prefix = prefix_rows && (tile_own || (prefix_rows > most && !little));
  const bool few_own = own_rows && !tile_own, few_prefix = prefix_rows && !tile_prefix;
  // Sequences of a row block and more on average: no block would serve two of
  // them, so the prefix is read in one go with the own keys (one partial
  // instead of two; four chunks of 770 tokens behind 8200 keys: 370 us so, 417
  // apart). The average is what the host knows: a batch of one long chunk and
  // many short ones may pass too, and then reads the prefix for each.
  const bool joined = tile_own && tile_prefix && (long long)a.T * a.g >= (long long)a.B * moe::kTileRows;
  moe::JoinArgs j = {};
  j.a = a;
  j.DP = h->DP;
  j.part_o = h->part_o;
  j.part_ml = h->part_ml;
  j.info_prefix = h->info[0];
  j.info_own = h->info[1];
  long long used = 0;
  auto line = [&](moe::LineArgs* ln, int row_block, int key_tile, int weight, int n_cta, bool prefix, bool own) {
    ln->row_block = row_block;
    ln->key_tile = key_tile;
    ln->weight = weight;
    ln->has_prefix = prefix && !joined;
    ln->has_own = own;
    ln->joined = joined;
    ln->n_cta = n_cta;
    ln->part_rows = std::min(std::max(prefix ? prefix_rows : 0, own ? own_rows : 0), row_block);
    ln->part_row0 = (int)used;
    ln->part_o = h->part_o;
    ln->part_ml = h->part_ml;
    ln->info_prefix = h->info[0];
    ln->info_own = h->info[1];
    ln->final_own = joined || !prefix_rows;
    ln->final_prefix = !own_rows;
    used += moe::line_part_rows(*ln, a.T, a.Hq);
    if (ln->has_prefix) j.prefix_step = ln->part_rows;
    if (own) j.own_step = ln->part_rows;
    ln->own_most = (int)std::min<long long>(moe::line_own_places(a, *ln), INT_MAX - 1);
    return moe::line_places(a, *ln) < INT_MAX;
  };
  moe::LineArgs tile = {}, few = {};
  moe::AttnRowsPlan plan = {};
  bool fits = true;
  if (tile_own || tile_prefix)
    fits = line(&tile, moe::kTileRows, moe::kTileKeyTile, moe::kTileWeight, h->num_sms, tile_prefix, tile_own);
  if (few_own || few_prefix) {
    const int rows = std::max(few_own ? own_rows : 0, few_prefix ? prefix_rows : 0);
    const int block = rows <= 16 ? 16 : most;
    plan = moe::plan_attn_rows(a.D, std::min(rows, block), a.B, h->num_sms);
    fits = line(&few, block, moe::kRowsKeyTile, moe::kRowsWeight, plan.n_cta, few_prefix,
                few_own) && fits;
  }
  if (!fits) return set_error(MOE_ERR_INVALID_ARG, "%s: tokens and lengths beyond what one call takes", fn);
  // The join sets the words that it reads back to zero. Without it what the
  // kernels before it left is cleared behind them, on their own stream.
  auto failed = [&](cudaError_t e) {
    const size_t words = (size_t)h->cfg.max_tokens * h->cfg.num_q_heads * sizeof(int2);
    for (int2* info : h->info) cudaMemsetAsync(info, 0, words, s);
    return cuda_error(e, fn);
  };
  if (tile.n_cta) {
    const cudaError_t e = moe::launch_attn_tile(h->tile_k, h->tile_v, a, tile, h->box_tile, bf16, s, h->pdl);
    if (e != cudaSuccess) return failed(e);
  }
  if (few.n_cta) {
    // behind the tile kernel it need not wait for its results, only not end before it
    const cudaError_t e = moe::launch_attn_rows(h->rows_k, h->rows_v, a, few, plan, h->box_rows, bf16,
                                                tile.n_cta && h->pdl, s, h->pdl);
    if (e != cudaSuccess) return failed(e);
  }
  const cudaError_t e = moe::launch_attn_join(j, bf16, s, h->pdl);
  return e == cudaSuccess ? MOE_OK : failed(e);
}

}  // namespace

extern "C" {

moe_status_t moe_attn_frequencies(const moe_attn_config_t* config, double* inv_freq, double* m) {
  if (!config) return set_error(MOE_ERR_INVALID_ARG, "config must not be NULL");
  const moe_status_t st = validate_rope(config);
  if (st != MOE_OK) return st;
  double f[64], mm;
  frequencies(config, f, &mm);
  if (inv_freq) memcpy(inv_freq, f, sizeof(double) * (config->rotary_dim / 2));
  if (m) *m = mm;
  return MOE_OK;
}

moe_status_t moe_attn_create(const moe_attn_config_t* config, const moe_attn_buffers_t* buffers, moe_attn_t** out) {
  if (!out) return set_error(MOE_ERR_INVALID_ARG, "out must not be NULL");
  *out = nullptr;
  const moe_status_t st = validate(config, buffers);
  if (st != MOE_OK) return st;
  moe_attn* h = new (std::nothrow) moe_attn();
  if (!h) return set_error(MOE_ERR_OOM, "host allocation failed");
  h->cfg = *config;
  h->buf = *buffers;
  const char* pdl_env = getenv("MOE_PDL");
  h->pdl = !(pdl_env && pdl_env[0] == '0');
  h->scale = (float)(config->scale > 0.0 ? config->scale : 1.0 / std::sqrt((double)config->head_dim));
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) {
    delete h;
    return cuda_error(e, "device query");
  }
  // workspace: error word, frequencies; with a cache the forward's tables and
  // the blocks' partial rows
  size_t bytes = align256(4) + align256(64 * 8);
  const size_t NR = (size_t)config->max_tokens * config->num_q_heads;
  if (buffers->k_cache) {
    h->DP = config->head_dim <= 64 ? 64 : 128;
    h->part_rows = 2 * NR + (size_t)h->num_sms * (2 * moe::kRowsMax + moe::kTileRows);
    bytes += 2 * align256(NR * 8) + align256(h->part_rows * h->DP * 4) + align256(h->part_rows * 8);
    h->box_rows = 16;  // the largest box that pages divide into
    while (h->box_rows < moe::kRowsKeyTile && config->page_size % (2 * h->box_rows) == 0) h->box_rows *= 2;
    h->box_tile = h->box_rows;
    while (h->box_tile < moe::kTileKeyTile && config->page_size % (2 * h->box_tile) == 0) h->box_tile *= 2;
    const bool bf16 = config->dtype == MOE_DTYPE_BF16;
    auto map = [&](CUtensorMap* tm, const void* cache, int slots, bool whole) {
      return moe::encode_cache_map(tm, cache, bf16, config->head_dim, config->page_size, config->num_kv_heads,
                                   config->num_pages, config->page_stride, config->slot_stride, config->head_stride,
                                   slots, whole);
    };
    if (!map(&h->rows_k, buffers->k_cache, h->box_rows, true) || !map(&h->rows_v, buffers->v_cache, h->box_rows, true) ||
        !map(&h->tile_k, buffers->k_cache, h->box_tile, false) || !map(&h->tile_v, buffers->v_cache, h->box_tile, false)) {
      delete h;
      return set_error(MOE_ERR_UNSUPPORTED, "the cache's shape and strides make no tensor map");
    }
  }
  e = cudaMalloc(&h->ws, bytes);
  if (e != cudaSuccess) {
    delete h;
    cudaGetLastError();
    return set_error(MOE_ERR_OOM, "workspace allocation of %zu bytes failed: %s", bytes, cudaGetErrorString(e));
  }
  char* p = static_cast<char*>(h->ws);
  h->err = reinterpret_cast<uint32_t*>(p);
  p += align256(4);
  h->freq = reinterpret_cast<uint64_t*>(p);
  p += align256(64 * 8);
  if (buffers->k_cache) {
    auto carve = [&](size_t b) {
      char* at = p;
      p += align256(b);
      return at;
    };
    for (int i = 0; i < 2; ++i) h->info[i] = reinterpret_cast<int2*>(carve(NR * 8));
    h->part_o = reinterpret_cast<float*>(carve(h->part_rows * h->DP * 4));
    h->part_ml = reinterpret_cast<float2*>(carve(h->part_rows * 8));
  }
  uint64_t turns[64] = {};
  if (config->rotary_dim > 0) {
    double f[64], m;
    frequencies(config, f, &m);
    h->rope_m = (float)m;
    for (int i = 0; i < config->rotary_dim / 2; ++i) {
      // positions are whole numbers, so whole turns per position change nothing
      const double t = std::fmod(f[i] / (2.0 * kPi), 1.0) * 18446744073709551616.0;
      turns[i] = t < 18446744073709551615.0 ? (uint64_t)t : 0;
    }
  }
  // the small words and tables; partial rows are written before they are read
  e = cudaMemset(h->ws, 0, h->part_o ? (size_t)((char*)h->part_o - (char*)h->ws) : bytes);
  if (e == cudaSuccess) e = cudaMemcpy(h->freq, turns, sizeof(turns), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaFree(h->ws);
    delete h;
    return cuda_error(e, "workspace init");
  }
  *out = h;
  return MOE_OK;
}

moe_status_t moe_attn_rotate(moe_attn_t* h, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const int32_t* positions, int32_t T, void* q_out, int64_t q_out_stride, void* k_out,
                             int64_t k_out_stride, void* stream) {
  const char* fn = "moe_attn_rotate";
  moe_status_t st = check_handle(h, fn);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (T < 0 || T > (1 << 22)) return set_error(MOE_ERR_INVALID_ARG, "%s: T=%d out of 0..2^22", fn, T);
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (!q && !k))
    return set_error(MOE_ERR_INVALID_ARG, "%s: q with q_out, k with k_out, at least one pair", fn);
  if (!positions) return set_error(MOE_ERR_INVALID_ARG, "%s: positions must not be NULL", fn);
  if (q) {
    st = check_rows(h, fn, "q", q, q_stride, h->cfg.num_q_heads);
    if (st == MOE_OK) st = check_rows(h, fn, "q_out", q_out, q_out_stride, h->cfg.num_q_heads);
  }
  if (st == MOE_OK && k) {
    st = check_rows(h, fn, "k", k, k_stride, h->cfg.num_kv_heads);
    if (st == MOE_OK) st = check_rows(h, fn, "k_out", k_out, k_out_stride, h->cfg.num_kv_heads);
  }
  if (st != MOE_OK) return st;
  moe::RopeArgs a = {};
  fill_rope(h, &a);
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.T = T;
  a.positions = positions;
  const cudaError_t e =
      moe::launch_rope(a, h->cfg.dtype == MOE_DTYPE_BF16, h->num_sms, static_cast<cudaStream_t>(stream), h->pdl);
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

moe_status_t moe_attn_append(moe_attn_t* h, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const int32_t* positions, const int32_t* slots,
                             int32_t T, void* q_out, int64_t q_out_stride, void* stream) {
  const char* fn = "moe_attn_append";
  moe_status_t st = check_handle(h, fn);
  if (st != MOE_OK) return st;
  if (!h->buf.k_cache) return set_error(MOE_ERR_INVALID_ARG, "%s: the handle has no cache", fn);
  if (T == 0) return MOE_OK;
  if (T < 0 || T > (1 << 22)) return set_error(MOE_ERR_INVALID_ARG, "%s: T=%d out of 0..2^22", fn, T);
  if (!k || !v || !positions || !slots)
    return set_error(MOE_ERR_INVALID_ARG, "%s: k, v, positions and slots must not be NULL", fn);
  if ((q == nullptr) != (q_out == nullptr)) return set_error(MOE_ERR_INVALID_ARG, "%s: q goes with q_out", fn);
  if (q) {
    st = check_rows(h, fn, "q", q, q_stride, h->cfg.num_q_heads);
    if (st == MOE_OK) st = check_rows(h, fn, "q_out", q_out, q_out_stride, h->cfg.num_q_heads);
  }
  if (st == MOE_OK) st = check_rows(h, fn, "k", k, k_stride, h->cfg.num_kv_heads);
  if (st == MOE_OK) st = check_rows(h, fn, "v", v, v_stride, h->cfg.num_kv_heads);
  if (st != MOE_OK) return st;
  moe::RopeArgs a = {};
  fill_rope(h, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.T = T;
  a.positions = positions;
  a.slots = slots;
  a.k_cache = h->buf.k_cache;
  a.v_cache = h->buf.v_cache;
  a.page_stride = h->cfg.page_stride;
  a.slot_stride = h->cfg.slot_stride;
  a.head_stride = h->cfg.head_stride;
  a.num_slots = h->cfg.num_pages * h->cfg.page_size;
  a.page_size = h->cfg.page_size;
  const cudaError_t e =
      moe::launch_rope(a, h->cfg.dtype == MOE_DTYPE_BF16, h->num_sms, static_cast<cudaStream_t>(stream), h->pdl);
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

moe_status_t moe_attn_forward(moe_attn_t* h, const void* q, int64_t q_stride, const moe_attn_batch_t* b, void* out,
                              int64_t out_stride, float* lse, void* stream) {
  const char* fn = "moe_attn_forward";
  moe_status_t st = check_handle(h, fn);
  if (st != MOE_OK) return st;
  const moe_attn_config_t& c = h->cfg;
  if (!h->buf.k_cache) return set_error(MOE_ERR_INVALID_ARG, "%s: the handle has no cache", fn);
  if (!b) return set_error(MOE_ERR_INVALID_ARG, "%s: batch must not be NULL", fn);
  if (b->num_tokens < 0 || b->num_tokens > c.max_tokens)
    return set_error(MOE_ERR_INVALID_ARG, "%s: num_tokens=%d out of 0..max_tokens=%d", fn, b->num_tokens,
                     c.max_tokens);
  if (b->num_seqs < 0 || b->num_seqs > c.max_seqs)
    return set_error(MOE_ERR_INVALID_ARG, "%s: num_seqs=%d out of 0..max_seqs=%d", fn, b->num_seqs, c.max_seqs);
  if (b->num_tokens == 0) return MOE_OK;
  if (b->num_seqs == 0) return set_error(MOE_ERR_INVALID_ARG, "%s: tokens without sequences", fn);
  if (!q || !out || !b->q_offsets || !b->seq_lens)
    return set_error(MOE_ERR_INVALID_ARG, "%s: q, out, q_offsets and seq_lens must not be NULL", fn);
  if (b->max_q_len < 1 || b->max_q_len > b->num_tokens)
    return set_error(MOE_ERR_INVALID_ARG, "%s: max_q_len=%d out of 1..num_tokens", fn, b->max_q_len);
  if ((long long)b->max_q_len * b->num_seqs < b->num_tokens)
    return set_error(MOE_ERR_INVALID_ARG, "%s: max_q_len * num_seqs is less than num_tokens", fn);
  if (b->max_seq_len < 0 || b->prefix_len < 0 || b->table_stride < 0)
    return set_error(MOE_ERR_INVALID_ARG, "%s: max_seq_len, prefix_len and table_stride must not be negative", fn);
  if ((long long)b->max_seq_len > (long long)b->table_stride * c.page_size)
    return set_error(MOE_ERR_INVALID_ARG, "%s: max_seq_len=%d beyond table_stride * page_size", fn, b->max_seq_len);
  if ((long long)b->max_seq_len + b->prefix_len > (1LL << 30))
    return set_error(MOE_ERR_INVALID_ARG, "%s: more than 2^30 keys", fn);
  if (b->max_seq_len > 0 && !b->block_table)
    return set_error(MOE_ERR_INVALID_ARG, "%s: block_table must not be NULL", fn);
  if (b->prefix_len > 0 && !b->prefix_pages)
    return set_error(MOE_ERR_INVALID_ARG, "%s: prefix_pages must not be NULL", fn);
  if (b->causal != 0 && b->causal != 1) return set_error(MOE_ERR_INVALID_ARG, "%s: causal must be 0 or 1", fn);
  st = check_rows(h, fn, "q", q, q_stride, c.num_q_heads);
  if (st == MOE_OK) st = check_rows(h, fn, "out", out, out_stride, c.num_q_heads);
  if (st != MOE_OK) return st;
  moe::AttnArgs a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = h->buf.k_cache;
  a.v_cache = h->buf.v_cache;
  a.page_stride = c.page_stride;
  a.slot_stride = c.slot_stride;
  a.head_stride = c.head_stride;
  a.page_size = c.page_size;
  a.num_pages = (int)c.num_pages;
  a.T = b->num_tokens;
  a.B = b->num_seqs;
  a.Hq = c.num_q_heads;
  a.Hk = c.num_kv_heads;
  a.g = c.num_q_heads / c.num_kv_heads;
  a.D = c.head_dim;
  a.q_offsets = b->q_offsets;
  a.seq_lens = b->seq_lens;
  a.block_table = b->block_table;
  a.prefix_pages = b->prefix_pages;
  a.table_stride = b->table_stride;
  a.prefix_len = b->prefix_len;
  a.causal = b->causal;
  a.max_q_len = b->max_q_len;
  a.max_seq_len = b->max_seq_len;
  a.scale = h->scale;
  a.out = out;
  a.out_stride = out_stride;
  a.lse = lse;
  a.err = h->err;
  return forward(h, a, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_attn_sync(moe_attn_t* h, void* stream) {
  const char* fn = "moe_attn_sync";
  const moe_status_t st = check_handle(h, fn);
  if (st != MOE_OK) return st;
  // Only this stream is waited for and nothing but the error word is touched:
  // a forward may be under way on another.
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  uint32_t err = 0;
  if (e == cudaSuccess) e = cudaMemcpyAsync(&err, h->err, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && err) {
    e = cudaMemsetAsync(h->err, 0, 4, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return cuda_error(e, fn);
  if (err == moe::kAttnErrTimeout) return set_error(MOE_ERR_TIMEOUT, "%s: a device-side wait gave up", fn);
  if (err) return set_error(MOE_ERR_INVALID_ARG, "%s: a slot, page, length or offset was out of range", fn);
  return MOE_OK;
}

moe_status_t moe_attn_destroy(moe_attn_t* h) {
  if (!h) return MOE_OK;
  if (h->ws) cudaFree(h->ws);
  delete h;
  return MOE_OK;
}

}  // extern "C"
