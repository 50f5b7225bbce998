// Attention for many query rows to a key, on the 5th-generation tensor cores:
// a prefix shared by a batch, chunks of prompt.
//
// A block takes up to 256 rows of a group as two tiles of 128 (a row is a
// query token and one of the g query heads of a key head) over a run of its
// keys, 128 at a time: S = Q K^T into tensor memory, running softmax in
// registers (a thread a row), the probabilities back to tensor memory as the
// A operand of O += P V, whose accumulator stays in tensor memory. Per SM a
// key tile costs 4 products of 128 x 128 x 128 (~2100 cycles at the measured
// peak for two row tiles) and 64 KB of keys and values (~2800 cycles at the
// measured copy rate): up to ~190 rows the keys' bytes bound it, above that
// the products.
// Measured: four chunks of 301 to 1024 tokens behind 8200 keys, 32 query and 8
// key heads of 128, 370 us = 1.30 PFLOP/s, 0.67 of the measured bf16 rate; a
// key tile took 2700 to 2950 cycles when that was 361 us. P V runs at the tensor cores' rate
// (64 cycles an MMA), Q K^T, which reads both operands from shared memory, at
// ~95; the softmax of a row tile takes 1000 to 1300 and hides.
//
// Warp roles (one block per SM):
//   warps 0-3, 4-7  softmax of row tile 0, 1 (a warp reaches the 32 lanes of
//                   tensor memory of its number mod 4); queries in, output out
//   warp 8          TMA: pages to shared memory, 128-byte swizzle, keys and
//                   values in turn through one ring
//   warp 9          tensor memory and the MMAs, issued by one elected lane:
//                   P V of a key tile, then the next Q K^T of the same rows,
//                   row tiles in turn, so that one's products run under the
//                   other's softmax (with a warp for each row tile the two
//                   fell into step, both in softmax, then both waiting for
//                   products: 3900 cycles a key tile instead of 3000)
//   warp 10         waits for the copies in the MMA warp's place and joins the
//                   probabilities' barrier: a wait costs ~170 cycles even when
//                   it is complete, and the tensor cores hold only a few MMAs
//                   in advance, so the MMA warp waits once a row tile
// Tensor memory: two S tiles (three at head sizes to 64; P takes the first half
// of S's columns) and two output tiles, 512 columns.
//
// MMAs of one lane run in order, so a Q K^T may overwrite the columns that the
// P V issued before it reads. At head sizes above 64 a completed Q K^T means
// that the P V before it has completed, so the softmax warps may rescale the
// output without another barrier; below, with three S tiles, they wait for it.
#include "attn_line.cuh"
#include "attn_tc.cuh"

namespace moe {
namespace {

constexpr int kKT = kTileKeyTile;
constexpr int kThreads = 11 * 32;
constexpr int kWarpCopy = 8, kWarpMma = 9, kWarpLanded = 10;
constexpr int kMaxStages = 8;
// A row's weights of one tile: a reference at the maximum gives at most 128 *
// 2^7 (FP16, ProbBias), and below 2^15 no FP16 weight overflows.
constexpr float kSumMost = 32768.f;

struct SmemPlan {
  uint32_t ring, bars, seg, misc, off, bytes;
};
__host__ __device__ inline SmemPlan smem_plan(int DP, int stages, int B) {
  SmemPlan p;
  p.ring = 2u * 128 * DP * 2;  // after the queries
  p.bars = p.ring + (uint32_t)stages * kKT * DP * 2;
  p.seg = p.bars + (2 * (kMaxStages + kSegSlots) + 16) * 8;
  p.misc = p.seg + kSegSlots * sizeof(Segment);
  p.off = p.misc + 80;
  p.bytes = p.off + (uint32_t)(B + 1) * 4;
  return p;
}

struct Misc {
  uint32_t tmem;
  int abort_flag;
  int issued;  // stages handed to TMA
  int mma_issued;
  int32_t scratch[12];
};
static_assert(sizeof(Misc) <= 80, "SmemPlan's room for Misc");

// RSUM: the quotient takes the sum of the weights as they were rounded for the
// products (few rows, see launch_attn_tile).
template <typename T, int DP, bool RSUM>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tile(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const AttnArgs a,
                const LineArgs ln, int stages, int box_log2) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int NH = DP / 64;
  constexpr bool kBf16 = sizeof(T) == 2 && ProbBias<T>::value == 0.f;
  // Head sizes to 64 leave room for a third S tile: the next key tile's Q K^T is
  // issued before a row tile's probabilities are in, S_t(j) in place (2 j + t)
  // mod 3, which the P V two before it has left (four chunks of 770 tokens, 32
  // query heads of 64: 280 us, 313 with two S tiles).
  constexpr bool kAhead = DP == 64;
  constexpr uint32_t kOut = kAhead ? 384 : 256;     // columns of the output tiles
  constexpr uint32_t kHalf = 128 * 128;             // bytes of 64 elements of 128 rows
  constexpr uint32_t kTileBytes = NH * kHalf;       // a query, key or value tile
  const SmemPlan sp = smem_plan(DP, stages, a.B);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + sp.bars);
  uint64_t* empty = full + kMaxStages;
  uint64_t* q_full = empty + kMaxStages;  // [2] queries in shared memory and the output tile drained
  // [2][2] by row tile and, with kAhead, by the key tile's parity: those of two
  // tiles in a row may be complete before the other side has looked, and a
  // phase two ahead would look like the one before it
  uint64_t* s_full = q_full + 2;          // logits in tensor memory
  uint64_t* p_full = s_full + 4;          // probabilities in tensor memory
  uint64_t* o_full = p_full + 4;          // output complete (kAhead: with each key tile)
  uint64_t* seg_full = o_full + 4;
  uint64_t* seg_empty = seg_full + kSegSlots;
  uint64_t* drain = seg_empty + kSegSlots;
  Segment* segs = reinterpret_cast<Segment*>(smem + sp.seg);
  Misc* misc = reinterpret_cast<Misc*>(smem + sp.misc);
  int32_t* own_off = reinterpret_cast<int32_t*>(smem + sp.off);
  volatile int* abort_flag = &misc->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 4);
      for (int par = 0; par < 2; ++par) {
        mbar_init(&s_full[2 * t + par], 1);
        mbar_init(&p_full[2 * t + par], 5);  // four softmax warps, kWarpLanded
        mbar_init(&o_full[2 * t + par], 1);
      }
    }
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 10);  // eight softmax warps, kWarpMma, kWarpLanded
    }
    mbar_init(drain, 1);
    misc->abort_flag = 0;
    misc->issued = 0;
    misc->mma_issued = 0;
    fence_mbar_init();
  }
  if (warp == kWarpCopy && lane == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == kWarpMma) tmem_alloc(&misc->tmem, 512);
  pdl_wait();
  // only now: a kernel that starts on this trigger and does not wait itself
  // may rely on everything before this launch
  pdl_trigger();
  const int own_total = scan_own<kThreads, kKT, kTileRows>(a, ln, own_off, misc->scratch);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;

  if (warp >= kWarpCopy) {
  if (warp == kWarpCopy) {
    // ------------------------------------------------ the walk and its copies
    // lane (box, half of the head): one box of every key and value tile
    const int c = lane / NH, hf = lane % NH;
    const int box = 1 << box_log2;
    const bool mine = c < (kKT >> box_log2);
    const bool split = (a.D & 63) != 0;
    const int cx = split ? hf * 64 : 0, ch = split ? 0 : hf;
    const uint32_t dst0 = smem_u32(smem) + sp.ring + (uint32_t)hf * kHalf + (uint32_t)c * box * 128;
    int st = 0, issued = 0, slot_i = 0;
    uint32_t ph = 0, sph = 0;
    bool ok = true;
    Walk<kKT, kTileRows> w;
    w.init(a, ln, own_off, own_total);
    while (ok) {
      Segment s;
      const bool some = w.next(a, ln, own_off, &s);
      if (!some) {
        s.tiles = 0;
        s.tile = s.b = s.nkeys = s.front = 0;  // no page to ask for
      }
      const int32_t* own = s.b < 0 ? a.prefix_pages : a.block_table + (long long)s.b * a.table_stride;
      int slot = 0;  // of the page, of the lane's box of the current tile
      int here = 0;  // keys of the tile that exist
      bool have = false;  // the lane's box has any
      auto page_of = [&](int tile) {
        const bool pre = tile < s.front;
        const int k0 = (pre ? tile : tile - s.front) * kKT, key = k0 + (c << box_log2);
        const int nk = pre ? a.prefix_len : s.nkeys;
        here = min(kKT, max(0, nk - k0));
        have = mine && key < nk;
        if (!have) return 0;
        const int pg = key / a.page_size;
        slot = key - pg * a.page_size;
        return __ldg((pre ? a.prefix_pages : own) + pg);  // looked at (page_in_cache) when it is used, not before
      };
      auto issue = [&](const CUtensorMap* tm, bool some_keys, int page, int at, int boxes) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1u, abort_flag, a.err));
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)boxes * box * 128 * NH);
        __syncwarp();
        if (some_keys)
          tma_load_5d(dst0 + (uint32_t)st * kTileBytes, tm, cx, at, ch, s.h, page_in_cache(a, page), &full[st]);
        ++issued;
        if (++st == stages) {
          st = 0;
          ph ^= 1u;
        }
      };
      // keys and values in turn, with kAhead the next tile's keys before a
      // tile's values: the order in which the MMA warp comes to them
      int page = page_of(s.tile);
      // (the first page's number is on its way meanwhile)
      ok = __all_sync(0xffffffffu, mbar_wait(&seg_empty[slot_i], sph ^ 1u, abort_flag, a.err));
      if (!ok) break;
      if (lane == 0) {
        segs[slot_i] = s;
        mbar_arrive(&seg_full[slot_i]);
      }
      if (++slot_i == kSegSlots) {
        slot_i = 0;
        sph ^= 1u;
      }
      if (!some) break;
      int vpage = 0, vat = 0, vboxes = 0;
      bool vhave = false;
#pragma unroll 1
      for (int i = 0; i < s.tiles + (kAhead ? 1 : 0) && ok; ++i) {
        const int at = slot, boxes = (here + box - 1) >> box_log2;
        const bool has = have;
        const int next = i + 1 < s.tiles ? page_of(s.tile + i + 1) : 0;
        if (i < s.tiles) issue(&tk, has, page, at, boxes);
        if (!kAhead) {
          if (ok) issue(&tv, has, page, at, boxes);
        } else {
          if (ok && i > 0) issue(&tv, vhave, vpage, vat, vboxes);
          vhave = has;
          vpage = page;
          vat = at;
          vboxes = boxes;
        }
        page = next;
      }
    }
    if (lane == 0) misc->issued = issued;
  } else if (warp == kWarpMma) {
    // ----------------------------------------------------------------- MMA
    {
      constexpr uint32_t id_s = attn_idesc(128, kKT, kBf16, false);
      constexpr uint32_t id_o = attn_idesc(128, DP, kBf16, true);
      // descriptors: addresses count 16 bytes in the low bits and stay inside
      // them, so a tile's are its stage's plus a constant
      const uint64_t dq = smem_desc_sw128(smem_u32(smem));
      const uint64_t dk = smem_desc_sw128(smem_u32(smem) + sp.ring);
      const uint64_t dv = smem_desc_rows_k(smem_u32(smem) + sp.ring, kHalf);
      int st = 0, slot_i = 0;
      uint32_t ph = 0, qph[2] = {0, 0}, pph[4] = {0, 0, 0, 0}, sph = 0;
      const uint32_t elect = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err)) != 0;
      };
      auto step = [&]() {
        if (++st == stages) {
          st = 0;
          ph ^= 1u;
        }
      };
      auto place = [&](int t, int j) { return (uint32_t)(kAhead ? (2 * j + t) % 3 : t) * 128; };
      auto bar = [&](int t, int j) { return 2 * t + (kAhead ? j & 1 : 0); };
      auto qk = [&](int t, int j, int stage) {
        const uint64_t q = dq + (uint64_t)(t * (kTileBytes >> 4)), k0 = dk + (uint64_t)(stage * (kTileBytes >> 4));
        const uint32_t d = tm + place(t, j);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint64_t off = (uint64_t)(((k >> 2) * kHalf + (k & 3) * 32) >> 4);
          mma_ss(elect, d, q + off, k0 + off, id_s, k > 0);
        }
        commit_elect(elect, &s_full[bar(t, j)]);
      };
      // waits for the probabilities of (t, j) in tensor memory, and with them
      // (kWarpLanded) for what the products up to the next wait read
      auto pv = [&](int t, int j, int stage) {
        const int i = bar(t, j);
        if (!wait(&p_full[i], pph[i])) return false;
        pph[i] ^= 1u;
        tc_fence_after();
        const uint64_t v0 = dv + (uint64_t)(stage * (kTileBytes >> 4));
        const uint32_t d = tm + kOut + t * DP, p = tm + place(t, j);
#pragma unroll
        for (int k = 0; k < kKT / 16; ++k)
          mma_ts(elect, d, p + k * 8, v0 + (uint64_t)(k * (2048 >> 4)), id_o, (j > 0 || k > 0) ? 1u : 0u);
        return true;
      };
      bool ok = true;
      while (ok) {
        ok = wait(&seg_full[slot_i], sph);
        if (!ok) break;
        const int tiles = __shfl_sync(0xffffffffu, segs[slot_i].tiles, 0);
        const int nt = __shfl_sync(0xffffffffu, segs[slot_i].rows, 0) > 128 ? 2 : 1;
        __syncwarp();
        if (elect) mbar_arrive(&seg_empty[slot_i]);
        if (++slot_i == kSegSlots) {
          slot_i = 0;
          sph ^= 1u;
        }
        if (tiles == 0) break;
        if (elect) misc->mma_issued = 1;
        ok = wait(&full[st], ph);
        for (int t = 0; t < nt && ok; ++t) {
          ok = wait(&q_full[t], qph[t]);
          qph[t] ^= 1u;
          if (!ok) break;
          tc_fence_after();
          qk(t, 0, st);
        }
        if (!ok) break;
        commit_elect(elect, &empty[st]);
        step();
        if (!kAhead) {
#pragma unroll 1
          for (int i = 0; i < tiles && ok; ++i) {
            const int vst = st;
            const bool more = i + 1 < tiles;
            step();
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
              ok = pv(t, i, vst);
              if (!ok) break;
              if (t == nt - 1) commit_elect(elect, &empty[vst]);
              if (more)
                qk(t, i + 1, st);
              else
                commit_elect(elect, &o_full[2 * t]);
            }
            if (ok && more) {
              commit_elect(elect, &empty[st]);
              step();
            }
          }
        } else {
          int k1 = st;  // stage of the next key tile
          if (tiles > 1) {
            ok = wait(&full[st], ph);
            if (!ok) break;
            tc_fence_after();
            qk(0, 1, k1);
            if (nt == 1) commit_elect(elect, &empty[k1]);
            step();
          }
#pragma unroll 1
          for (int i = 0; i < tiles; ++i) {
            const int vst = st;
            step();
            const int k2 = st;  // of the one after it
            if (i + 2 < tiles) step();
            ok = pv(0, i, vst);
            if (!ok) break;
            commit_elect(elect, &o_full[bar(0, i)]);
            if (nt == 2) {
              if (i + 1 < tiles) {
                qk(1, i + 1, k1);
                commit_elect(elect, &empty[k1]);
              }
              ok = pv(1, i, vst);
              if (!ok) break;
              commit_elect(elect, &o_full[bar(1, i)]);
            }
            commit_elect(elect, &empty[vst]);
            if (i + 2 < tiles) {
              qk(0, i + 2, k2);
              if (nt == 1) commit_elect(elect, &empty[k2]);
            }
            k1 = k2;
          }
        }
      }
    }
  } else if (warp == kWarpLanded) {
    // -------------------------------------------------------------- landed
    int st = 0, slot_i = 0;
    uint32_t ph = 0, sph = 0, pph[4] = {1, 1, 1, 1};  // p_full: parity of the phase before the one to join
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err)) != 0;
    };
    auto landed = [&]() {
      if (!wait(&full[st], ph)) return false;
      if (++st == stages) {
        st = 0;
        ph ^= 1u;
      }
      return true;
    };
    bool ok = true;
    while (ok) {
      ok = wait(&seg_full[slot_i], sph);
      if (!ok) break;
      const int tiles = segs[slot_i].tiles, nt = segs[slot_i].rows > 128 ? 2 : 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[slot_i]);
      if (++slot_i == kSegSlots) {
        slot_i = 0;
        sph ^= 1u;
      }
      if (tiles == 0) break;
      auto join = [&](int t, int j) {
        const int i = 2 * t + (kAhead ? j & 1 : 0);
        if (!wait(&p_full[i], pph[i])) return false;  // the phase before is over: this arrival counts for the next
        pph[i] ^= 1u;
        if (lane == 0) mbar_arrive(&p_full[i]);
        return true;
      };
      // behind P V of (t, i) the MMA warp goes on to the Q K^T of (t, i + 1), or
      // with kAhead of the other row tile's next key tile
      ok = landed() && (!kAhead || tiles == 1 || landed());
#pragma unroll 1
      for (int i = 0; i < tiles && ok; ++i) {
        if (!kAhead) {
          ok = landed() && (i + 1 == tiles || landed());
          for (int t = 0; t < nt && ok; ++t) ok = join(t, i);
        } else {
          ok = landed();
          if (ok && nt == 2) ok = join(0, i);
          if (ok && i + 2 < tiles) ok = landed();
          if (ok) ok = join(nt - 1, i);
        }
      }
    }
  }
  } else {
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2;                       // row tile
    const int r = t * 128 + (warp & 3) * 32 + lane;  // row of the group
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + kOut + t * DP;
    const float sc = a.scale * kLog2e;
    const float2 sc2 = make_float2(sc, sc), bias2 = make_float2(ProbBias<T>::value, ProbBias<T>::value);
    // queries of this row tile, 16 bytes a thread, consecutive threads along a
    // row: asynchronous copies, complete after cp_async_wait_all; zeros beyond
    // the group's rows and the head's elements
    auto load_q = [&](const Segment* s) {
      constexpr int kStep = 128 / (DP / 8);  // rows the 128 threads cover
      const int z = tid & 127, c8 = z & (DP / 8 - 1);
      const int step_tok = kStep / a.g, step_head = kStep - step_tok * a.g;
      int rl = z / (DP / 8);
      const int row = s->row0 + t * 128 + rl, rows = s->rows - t * 128;
      int tok = row / a.g, hd = row - tok * a.g;
      const T* src = static_cast<const T*>(a.q) + (long long)(s->t0 + tok) * a.q_stride +
                     (long long)(s->h * a.g + hd) * a.D + c8 * 8;
      const uint32_t dst = smem_u32(smem) + (uint32_t)t * kTileBytes + (uint32_t)(c8 >> 3) * kHalf;
#pragma unroll 4
      for (int i = 0; i < DP / 8; ++i, rl += kStep) {
        const bool valid = rl < rows && c8 * 8 < a.D;
        cp_async16(dst + (uint32_t)rl * 128 + (uint32_t)(((c8 & 7) ^ (rl & 7)) << 4), valid ? (const void*)src : a.q,
                   valid);
        src += (long long)step_tok * a.q_stride + (long long)step_head * a.D;
        hd += step_head;
        if (hd >= a.g) {  // the next token's first heads
          hd -= a.g;
          src += a.q_stride - (long long)a.g * a.D;
        }
      }
    };
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    uint32_t sph[2] = {0, 0}, outs[2] = {0, 0}, gph = 0;  // outs: phases of o_full before this part
    int slot_i = 0;
    int vst = 0;  // ring stage of the next key tile, and its phase
    uint32_t vph = 0;
    // A part's description stays in its slot until the part is done: `cur` is
    // read where it is needed, and gives no registers to what the tiles' loop
    // does not use.
    auto peek_segment = [&]() {
      const bool got = __all_sync(0xffffffffu, mbar_wait(&seg_full[slot_i], gph, abort_flag, a.err));
      return got && segs[slot_i].tiles > 0;
    };
    auto next_slot = [&]() {
      if (++slot_i == kSegSlots) {
        slot_i = 0;
        gph ^= 1u;
      }
    };
    auto uses = [&](const Segment* s) { return t == 0 || s->rows > 128; };
    auto q_arrive = [&]() {
      cp_async_wait_all();
      fence_async_smem();
      arrive(&q_full[t]);
    };
    bool ok = true, some = peek_segment();
    const Segment* cur = &segs[slot_i];
    if (some) {
      if (uses(cur)) {
        load_q(cur);
        q_arrive();
      }
      next_slot();
    }
    while (some) {
      const bool used = uses(cur);
      bool more = false, more_used = false;  // there is another part, and this row tile has rows in it
      const bool any_row = t * 128 + (warp & 3) * 32 < cur->rows;
      const int tiles = cur->tiles;  // this warp has a row
      float mref = -INFINITY;
      // sums of the weights, and (RSUM) of the weights as rounded: the quotient
      // takes the latter, so that a key that stands alone gives its value
      // exactly, the logarithm the former
      float2 l2 = make_float2(0.f, 0.f), lr2 = l2;
      if (used) {
        const int row = cur->row0 + min(r, cur->rows - 1);
        const int lim = cur->b < 0 ? cur->klen : keys_seen(a, cur->klen, cur->n, row / a.g);
        const int all_see = cur->b < 0 ? cur->klen : keys_seen(a, cur->klen, cur->n, cur->row0 / a.g);
        const int tile0 = cur->tile, front = cur->front, nkeys = cur->nkeys;
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          const bool pre = tile0 + i < front;  // a tile of the prefix before own keys
          const int k0 = (tile0 + i - (pre ? 0 : front)) * kKT;
          const int nk = pre ? a.prefix_len : nkeys;
          const int par = kAhead ? i & 1 : 0;
          const uint32_t ts = tmem + lanes + (uint32_t)(kAhead ? (2 * i + t) % 3 : t) * 128;
          const bool got = mbar_wait(&s_full[2 * t + par], sph[par], abort_flag, a.err);
          sph[par] ^= 1u;
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (i + 1 == tiles) {
            // this part's last Q K^T has completed: the next one's queries may
            // come in under its softmax
            more = peek_segment();
            more_used = more && uses(&segs[slot_i]);
            if (more_used) load_q(&segs[slot_i]);
          }
          if (any_row) {
            const bool edge = k0 + kKT > (pre ? a.prefix_len : all_see);
            const int seen = pre ? a.prefix_len : lim;
            uint32_t p[64];
            float2 lt, lrt;
            // The weights are taken against the reference maximum as it stands;
            // a tile's own maximum is not looked for. Only when a row's weights
            // add up to more than kSumMost (none can pass it then, so none
            // overflows), or a row that has no reference yet sees keys, is the
            // reference moved to the maximum and the tile, still in tensor
            // memory, done again: once, after which no weight passes 2^bias.
            // The first tile sets it beforehand.
            auto mask = [&](uint32_t(&v)[32], int c) {
              if (edge) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (k0 + c * 32 + e >= seen) v[e] = 0xff800000u;
              }
            };
            bool move = i == 0;
#pragma unroll 1
            while (true) {  // a pass that moves the reference is the last
              if (move) {
                float m = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                  uint32_t v[32];
                  tmem_ld32(ts + c * 32, v);
                  tmem_ld_wait_for(v);
                  mask(v, c);
                  float mx[2] = {m, -INFINITY};
#pragma unroll
                  for (int e = 0; e < 32; ++e) mx[e & 1] = fmaxf(mx[e & 1], __uint_as_float(v[e]));
                  m = fmaxf(mx[0], mx[1]);
                }
                const float mn = fmaxf(mref, m);
                const float f = mref == mn ? 1.f : exp2_fast((mref - mn) * sc);
                mref = mn;
                l2.x *= f;
                l2.y *= f;
                lr2.x *= f;
                lr2.y *= f;
                if (i > 0) {
                  if (kAhead) {  // the P V before has been issued, but need not be over
                    const int j = i - 1;
                    mbar_wait(&o_full[2 * t + (j & 1)], (outs[j & 1] + (uint32_t)(j >> 1)) & 1u, abort_flag, a.err);
                    __syncwarp();
                    tc_fence_after();
                  }
#pragma unroll 1
                  for (int c = 0; c < DP / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(to + c * 32, v);
                    tmem_ld_wait_for(v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                    tmem_st32(to + c * 32, v);
                  }
                  tmem_st_wait();
                }
              }
              const float ref = mref == -INFINITY ? 0.f : mref;
              const float2 nref = make_float2(-ref, -ref);
              lt = lrt = make_float2(0.f, 0.f);
              uint32_t sr[2][32];
              tmem_ld32(ts, sr[0]);
              tmem_ld_wait_for(sr[0]);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t(&v)[32] = sr[c & 1];
                if (c < 3) tmem_ld32(ts + (c + 1) * 32, sr[(c + 1) & 1]);
                mask(v, c);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  float2 w = fadd2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), nref);
                  w = ffma2(w, sc2, bias2);
                  w.x = exp2_fast(w.x);
                  w.y = exp2_fast(w.y);
                  lt = fadd2(lt, w);
                  p[c * 16 + e] = Half16<T>::pack(w.x, w.y);
                  if (RSUM) lrt = fadd2(lrt, Half16<T>::unpack(p[c * 16 + e]));
                }
                if (c < 3) tmem_ld_wait_for(sr[(c + 1) & 1]);
              }
              if (move) break;
              move = __any_sync(0xffffffffu, lt.x + lt.y > kSumMost || (mref == -INFINITY && k0 < seen));
              if (!move) break;
            }
            l2 = fadd2(l2, lt);
            lr2 = fadd2(lr2, lrt);
            tmem_st32(ts, *reinterpret_cast<uint32_t(*)[32]>(&p[0]));
            tmem_st32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(&p[32]));
            tmem_st_wait();
          }
          if (nk - k0 < kKT) {
            // slots past the end may hold anything: their values become zeros
            // (a zero weight would not stop a NaN)
            // the tile's values' place in the ring
            int z = 2 * i + (kAhead && i + 1 < tiles ? 2 : 1) + vst;
            const uint32_t zph = vph ^ ((uint32_t)(z / stages) & 1u);
            z %= stages;
            const bool there = mbar_wait(&full[z], zph, abort_flag, a.err);
            if (!__all_sync(0xffffffffu, there)) {
              ok = false;
              break;
            }
            const int here = max(0, nk - k0);
            unsigned char* vt = smem + sp.ring + (uint32_t)z * kTileBytes;
            for (int y = tid & 127; y < (kKT - here) * (DP / 8); y += 128) {
              const int zr = here + y / (DP / 8), c8 = y % (DP / 8);
              *reinterpret_cast<uint4*>(vt + (uint32_t)(c8 >> 3) * kHalf + (uint32_t)zr * 128 +
                                        (uint32_t)((c8 & 7) << 4)) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
          }
          tc_fence_before();
          arrive(&p_full[2 * t + par]);
        }
      }
      if (!ok) break;
      {
        const int z = vst + 2 * tiles;
        vph ^= (uint32_t)(z / stages) & 1u;
        vst = z % stages;
      }
      if (!used) {
        more = peek_segment();
        more_used = more && uses(&segs[slot_i]);
        if (more_used) load_q(&segs[slot_i]);
      }
      if (used) {
        const int j = kAhead ? tiles - 1 : 0;
        const bool got = mbar_wait(&o_full[2 * t + (j & 1)], (outs[j & 1] + (uint32_t)(j >> 1)) & 1u, abort_flag, a.err);
        outs[0] += (uint32_t)(j >> 1) + 1u;  // tiles 0, 2, ... and 1, 3, ...
        outs[1] += (uint32_t)(j + 1) >> 1;
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (any_row) {
          const bool done = whole(ln, *cur);
          const int2 at = cur->parts ? row_place(a, *cur, r) : make_int2(0, 0);
          const float l = l2.x + l2.y, lr = RSUM ? lr2.x + lr2.y : l, inv = inverse_sum(lr);
          const float own = l == lr ? 1.f : l / lr;  // a partial stands against the sum l
          float* dst = ln.part_o + (long long)(cur->prow + r) * DP;
          T* out = static_cast<T*>(a.out) + (long long)at.x * a.out_stride + (long long)at.y * a.D;
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(to + c * 32, o);
            tmem_ld_wait_for(o);
            if (r < cur->rows) {
              if (!done) {
                if (RSUM) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * own);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) st_global_32(dst + c * 32 + e * 8, o + e * 8);
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint4 v;
                  v.x = Half16<T>::pack(__uint_as_float(o[8 * e]) * inv, __uint_as_float(o[8 * e + 1]) * inv);
                  v.y = Half16<T>::pack(__uint_as_float(o[8 * e + 2]) * inv, __uint_as_float(o[8 * e + 3]) * inv);
                  v.z = Half16<T>::pack(__uint_as_float(o[8 * e + 4]) * inv, __uint_as_float(o[8 * e + 5]) * inv);
                  v.w = Half16<T>::pack(__uint_as_float(o[8 * e + 6]) * inv, __uint_as_float(o[8 * e + 7]) * inv);
                  if (c * 32 + e * 8 < a.D) *reinterpret_cast<uint4*>(out + c * 32 + e * 8) = v;
                }
              }
            }
          }
          if (r < cur->rows) {
            if (!done)
              ln.part_ml[cur->prow + r] = make_float2(mref, l);
            else if (a.lse)
              a.lse[(long long)at.x * a.Hq + at.y] = log_sum<T>(mref, l, a.scale);
            if (cur->parts) write_info(a, ln, *cur, r, at);
          }
        }
        tc_fence_before();
      }
      if (more_used) q_arrive();
      arrive(&seg_empty[cur - segs]);
      some = more;
      cur = &segs[slot_i];
      if (some) next_slot();
    }
    cp_async_wait_all();  // (none are left unless a wait gave up)
  }

  // ------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (misc->abort_flag) {
    // a block that gave up lets its copies and MMAs end before it leaves
    if (warp == kWarpCopy && lane == 0) {
      const int n = misc->issued;
      for (int i = 0; i < stages && i < n; ++i)
        mbar_wait(&full[i], (uint32_t)((n - 1 - i) / stages) & 1u, nullptr, nullptr);
    }
    if (warp == kWarpMma && misc->mma_issued) {
      commit_elect(elect_one(), drain);  // the lane that issued the MMAs
      mbar_wait(drain, 0, nullptr, nullptr);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <typename T, int DP, bool RSUM>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln, int box_log2,
                   cudaStream_t s, bool pdl) {
  int stages = kMaxStages;  // as many as fit
  while (stages > 2 && smem_plan(DP, stages, a.B).bytes + 1024 > 227 * 1024) --stages;
  const size_t smem = smem_plan(DP, stages, a.B).bytes + 1024;
  const cudaError_t e = ensure_smem(k_attn_tile<T, DP, RSUM>, smem);
  if (e != cudaSuccess) return e;
  return launch_ex(k_attn_tile<T, DP, RSUM>, dim3(ln.n_cta), dim3(kThreads), smem, s, pdl, tk, tv, a, ln, stages,
                   box_log2);
}

// A weight's rounding to 16 bits is as large as the output's own. Against
// 64-bit results the outputs of many rows together are 1.35 times as far off
// as rounding alone would leave them; a few rows by themselves, with a few
// hundred keys, up to 1.8 times, or 1.4 with the quotient by the rounded sum,
// which costs about 10% (four chunks of 770 tokens 406 us against 370, 64
// sequences behind 32768 keys 92 against 83). Below 4096 rows it is taken.
template <typename T>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln, int bl,
                     cudaStream_t s, bool pdl) {
  const bool few = (long long)a.T * a.Hq < 4096;
  if (a.D <= 64)
    return few ? launch<T, 64, true>(tk, tv, a, ln, bl, s, pdl) : launch<T, 64, false>(tk, tv, a, ln, bl, s, pdl);
  return few ? launch<T, 128, true>(tk, tv, a, ln, bl, s, pdl) : launch<T, 128, false>(tk, tv, a, ln, bl, s, pdl);
}

}  // namespace

cudaError_t launch_attn_tile(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln,
                             int box_slots, bool bf16, cudaStream_t s, bool pdl) {
  int bl = 4;
  while ((1 << bl) < box_slots) ++bl;
  return bf16 ? launch_t<__nv_bfloat16>(tk, tv, a, ln, bl, s, pdl) : launch_t<__half>(tk, tv, a, ln, bl, s, pdl);
}

}  // namespace moe
