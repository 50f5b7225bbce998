// Attention for few query rows to a key: a decode step over each sequence's
// own pages, drafted tokens, or a prefix shared by a handful of rows.
//
// A group's rows (at most 16, or 32 in two tiles at head sizes to 64; over trees
// 16, 32 or 64) meet a run of its keys: S = Q K^T, running softmax, O += P V, one
// pass over the keys. Every key and value is read once by one block, so up to 16
// rows the bound is memory; what has to hold is that the SM's copies never wait.
// Per SM at the measured copy rate a 16-key step (8 KB at head size 128) takes
// ~350 cycles; a 16-row tile costs ~150 issue slots, spread over the SM's eight
// computing warps. That leaves room to multiply the probabilities in two 16-bit
// parts; over trees of 17 rows and more it does not, there is one part, and the
// products bind.
// Measured: 32 sequences of up to 24000 own keys, 8 key heads of 128 (1.53
// GB), 228 us = 6.7 TB/s, 0.99 of the measured copy rate; 16 behind 4099
// shared keys with up to 1000 own (92 MB) 25 us: 4 us until the first copy
// (two dependent loads, then the page's number), 12 us of copies at full rate,
// 1.5 us to end each part, 4 us for the join. Trees of drafted tokens: 16 of up
// to 31 rows of 128 to a key over up to 2600 own keys (175 MB) 40 us, with a
// prefix of 1000 in the same launch 49; 50 of up to 52 rows of 64 over up to 713
// (39 MB) 24 us, where the products of mma.sync bind (1019 multiply-adds a cycle
// and SM, an eighth of tcgen05's).
//
// A block is four computing warps and one that copies. Keys and values come
// page by page as TMA boxes (16 to 64 slots of one head, 128-byte swizzle)
// into a ring of 64-key stages. Where a group is one block of rows (WR 1) warp w
// takes keys 16w .. 16w+15 of each with its own running maximum, sum and output
// tile in registers, and the four are joined at the end of the block's part of a
// group. Over trees of 17 to 32 rows two warps share each half of the rows, 32
// keys of a stage each, and are joined in pairs; with 33 to 64 rows every warp
// has 16 rows and all keys, and nothing is joined. Two blocks per SM.
#include <cudaTypedefs.h>

#include <algorithm>

#include "attn_line.cuh"
#include "attn_tc.cuh"

namespace moe {
namespace {

constexpr int kKT = kRowsKeyTile;
constexpr int kWarps = 4;  // computing warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kMaxStages = 4;

struct SmemPlan {
  uint32_t q, merge, ml, bars, seg, misc, off, bytes;
};
__host__ __device__ inline SmemPlan smem_plan(int DP, int MT, int WR, int rows, int stages, int B) {
  SmemPlan p;
  p.q = (uint32_t)stages * 2 * kKT * DP * 2;
  p.merge = p.q + (uint32_t)WR * MT * 16 * DP * 2;
  p.ml = p.merge + (WR == 4 ? 0u : 2u * MT * (rows > 8 ? 16 : 8) * DP * 4);
  p.bars = p.ml + (uint32_t)kWarps * MT * 16 * (WR > 1 ? 16 : 8);
  p.seg = p.bars + 2 * (kMaxStages + kSegSlots) * 8;
  p.misc = p.seg + kSegSlots * sizeof(Segment);
  p.off = p.misc + 64;
  p.bytes = p.off + (uint32_t)(B + 1) * 4;
  return p;
}

// The computing warps. These barriers have no limit of their own: every
// computing warp comes to each of them, whatever its bounded waits returned.
__device__ __forceinline__ void bar_compute() { asm volatile("bar.sync 1, %0;" ::"r"(kWarps * 32) : "memory"); }
// The same, and whether v holds for any of them.
__device__ __forceinline__ bool bar_any(bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)v), "r"(kWarps * 32)
      : "memory");
  return any != 0;
}

// WR: the computing warps are WR row groups of 16 MT rows by 4 / WR key groups;
// a row group's warps share the 64 keys of a stage. TREE: a token sees of its
// sequence's new tokens those that its bits name (AttnArgs::tree); a tile that
// reaches behind the context takes a word of them a row.
template <typename T, int DP, int MT, int WR, bool TREE>
__global__ void __launch_bounds__(kThreads, 2)
    k_attn_rows(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const AttnArgs a,
                const LineArgs ln, int stages, int box_log2, int late_wait) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int WK = kWarps / WR;      // key groups
  constexpr int RB = WR * MT * 16;     // rows of a group at most
  // Sixteens of keys that a warp takes in one step: more of them share a step's
  // chain of waits (products, maximum, exponentials, products). (50
  // trees of up to 52 rows of 64: 26.7 us, 29.6 with one sixteen a step; 64 rows
  // of 128 over 8 sequences of 15000 keys 135 and 156.)
  constexpr int KS = WR == 1 ? 1 : DP == 64 ? WR : 2;
  // The weights as two 16-bit numbers, the rounded one and what it leaves: with
  // few rows their rounding would not average out, and the second product hides
  // under the copies. With several row groups it does not (16 trees of up to 31
  // rows of 128 behind 1000 keys 53 us, 48 with one): there one, and the quotient
  // by the sum of the rounded weights (as in the tcgen05 kernel).
  constexpr bool kTwoParts = WR == 1;
  const SmemPlan sp = smem_plan(DP, MT, WR, ln.part_rows, stages, a.B);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + sp.bars);
  uint64_t* empty = full + kMaxStages;
  uint64_t* seg_full = empty + kMaxStages;
  uint64_t* seg_empty = seg_full + kSegSlots;
  Segment* segs = reinterpret_cast<Segment*>(smem + sp.seg);
  volatile int* abort_flag = reinterpret_cast<int*>(smem + sp.misc);
  int32_t* scratch = reinterpret_cast<int32_t*>(smem + sp.misc) + 4;
  int32_t* own_off = reinterpret_cast<int32_t*>(smem + sp.off);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr uint32_t kTileBytes = kKT * DP * 2;  // keys or values of a stage
  constexpr int NH = DP / 64;
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], kWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (tid == kWarps * 32) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  pdl_trigger();
  if (!late_wait) pdl_wait();
  const bool whole_groups = TREE && ln.whole;
  const int own_total = whole_groups ? 0 : scan_own<kThreads, kKT, RB>(a, ln, own_off, scratch);
  if (whole_groups || !ln.has_own) __syncthreads();
  const int box = 1 << box_log2;

  if (warp == kWarps) {
    // ---------------------------------------------- the walk and its copies
    // lane c < kKT / box copies the tile's box c of keys, lane 16 + c of values
    const int c = lane & 15;
    const bool mine = c < (kKT >> box_log2);
    const CUtensorMap* tm = lane < 16 ? &tk : &tv;
    const bool split = (a.D & 63) != 0;  // one box per 64 elements of the head
    int st = 0, slot_i = 0;
    uint32_t ph = 0, sph = 0;
    int issued = 0;
    bool ok = true;
    Walk<kKT, RB> w;
    int group = (int)blockIdx.x;
    if (!whole_groups) w.init(a, ln, own_off, own_total);
    if (whole_groups) clear_behind<T>(a, lane);
    while (ok) {
      Segment s;
      const bool some = whole_groups ? next_whole<T, kKT>(a, ln, &group, RB, lane, &s) : w.next(a, ln, own_off, &s);
      if (!some) {
        s.tiles = 0;
        s.tile = s.b = s.nkeys = s.front = 0;  // no page to ask for
      }
      const int32_t* tab = s.b < 0 ? a.prefix_pages : a.block_table + (long long)s.b * a.table_stride;
      int slot = 0;  // of the page, of the lane's box of the current tile
      bool have = false;  // that box has keys
      auto page_of = [&](int tile) {
        const int key = tile * kKT + (c << box_log2);
        have = mine && key < s.nkeys;
        if (!have) return 0;
        const int pg = key / a.page_size;
        slot = key - pg * a.page_size;
        return __ldg(tab + pg);  // looked at (page_in_cache) when it is used, not before
      };
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
#pragma unroll 1
      for (int i = 0; i < s.tiles; ++i) {
        const int tile = s.tile + i, at = slot;
        const bool has = have;
        const int next = i + 1 < s.tiles ? page_of(tile + 1) : 0;
        const int boxes = (min(kKT, max(0, s.nkeys - tile * kKT)) + box - 1) >> box_log2;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1u, abort_flag, a.err));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)boxes * 2 * box * DP * 2);
        __syncwarp();
        if (has) {
          page = page_in_cache(a, page);
          const uint32_t dst = smem_u32(smem) + (uint32_t)st * 2 * kTileBytes + (lane < 16 ? 0u : kTileBytes) +
                               (uint32_t)c * box * DP * 2;
          if (split) {
#pragma unroll
            for (int hf = 0; hf < NH; ++hf)
              tma_load_5d(dst + (uint32_t)hf * box * 128, tm, hf * 64, at, 0, s.h, page, &full[st]);
          } else {
            tma_load_5d(dst, tm, 0, at, 0, s.h, page, &full[st]);
          }
        }
        ++issued;
        page = next;
        if (++st == stages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    // a block that gave up lets its copies land before its memory is released
    if (!ok && lane == 0)
      for (int i = 0; i < stages && i < issued; ++i)
        mbar_wait(&full[i], (uint32_t)((issued - 1 - i) / stages) & 1u, nullptr, nullptr);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ compute
    const int g8 = lane >> 2, t4 = lane & 3;
    const float sc = a.scale * kLog2e;
    const int wr = warp / WK, wk = warp % WK;  // row group, key group
    // shared-memory address of 16 of the stage's keys (all in one box)
    auto keys_off = [&](int key) {
      return (uint32_t)(key >> box_log2) * box * DP * 2 + (uint32_t)(key & (box - 1)) * 128;
    };
    const uint32_t half_step = (uint32_t)box * 128;
    const uint32_t warp_off = keys_off(warp * 16);  // WR 1: a warp's keys stand in one place of every stage
    const int krow = (lane & 7) + ((lane >> 4) << 3), ksel = (lane >> 3) & 1;
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vsel = lane >> 4;
    const uint32_t qs = smem_u32(smem + sp.q);
    const int qrow = (lane & 7) + (((lane >> 3) & 1) << 3), qsel = lane >> 4;
    float2* ml = reinterpret_cast<float2*>(smem + sp.ml);
    float* mlr = reinterpret_cast<float*>(ml + kWarps * MT * 16);
    float* merge = reinterpret_cast<float*>(smem + sp.merge);
    int st = 0, slot_i = 0;
    uint32_t ph = 0, sph = 0;
    bool ok = true;
    auto next_segment = [&](Segment* s) {
      ok = __all_sync(0xffffffffu, mbar_wait(&seg_full[slot_i], sph, abort_flag, a.err));
      if (!ok) return false;
      *s = segs[slot_i];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[slot_i]);
      if (++slot_i == kSegSlots) {
        slot_i = 0;
        sph ^= 1u;
      }
      return s->tiles > 0;
    };
    // queries: rows of 128-byte halves, swizzled as the boxes are; zeros
    // beyond the group's rows and the head's elements
    constexpr int kQ = RB * DP / 8 / (kWarps * 32);  // 16-byte words of a thread
    constexpr bool kAsyncQ = WR > 1;  // by asynchronous copies, once no warp reads the last ones (in registers they spill)
    uint4 qv[kAsyncQ ? 1 : kQ] = {};
    auto q_place = [&](int r, int c8) {
      return sp.q + (uint32_t)(c8 >> 3) * RB * 128 + (uint32_t)r * 128 + (uint32_t)(((c8 & 7) ^ (r & 7)) << 4);
    };
    auto load_q = [&](const Segment& s) {
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const int z = tid + i * kWarps * 32, r = z / (DP / 8), c8 = z % (DP / 8);
        const bool valid = r < s.rows && c8 * 8 < a.D;
        auto word = [&]() {  // (its divisions are for words that there are: a group of one to three rows has few)
          const int row = s.row0 + r, tok = row / a.g, hq = s.h * a.g + row - tok * a.g;
          return static_cast<const T*>(a.q) + (long long)(s.t0 + tok) * a.q_stride + (long long)hq * a.D + c8 * 8;
        };
        if (kAsyncQ) {
          const T* src = word();
          cp_async16(smem_u32(smem) + q_place(r, c8), valid ? (const void*)src : a.q, valid);
        } else {
          qv[kAsyncQ ? 0 : i] = make_uint4(0, 0, 0, 0);
          if (valid) qv[kAsyncQ ? 0 : i] = *reinterpret_cast<const uint4*>(word());
        }
      }
    };
    Segment s;
    bool some = next_segment(&s);
    if (some) load_q(s);
    // A warp whose wait gave up (ok is false; the timeout is recorded, the
    // results are not looked at) goes through its part's barriers with the
    // others, and all of them end at the next part's first one. (After the
    // last part the words stored before it are nobody's.)
    while (true) {
      if (kAsyncQ) {
        cp_async_wait_all();
      } else {
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const int z = tid + i * kWarps * 32, r = z / (DP / 8), c8 = z % (DP / 8);
          *reinterpret_cast<uint4*>(smem + q_place(r, c8)) = qv[kAsyncQ ? 0 : i];
        }
      }
      if (bar_any(!ok) || !some) break;
      float o[MT][DP / 8][4];
      float mref[MT][2], l[MT][2], lr[MT][2];  // reference, sum of the weights, of the rounded ones
      int lim[MT][2];  // keys each of the lane's rows sees; TREE: where its token's bits are
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[m][n][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mref[m][e] = -INFINITY;
          l[m][e] = lr[m][e] = 0.f;
          const int row = s.row0 + min((wr * MT + m) * 16 + g8 + 8 * e, s.rows - 1);
          if (TREE)
            lim[m][e] = (s.t0 + row / a.g) * a.tree_stride;
          else
            lim[m][e] = s.b < 0 ? s.klen : keys_seen(a, s.klen, s.n, row / a.g);
        }
      }
      // keys that every row sees: no masking needed below it
      const int all_see = s.b < 0 ? s.klen : TREE ? s.klen - s.n : keys_seen(a, s.klen, s.n, s.row0 / a.g);

#pragma unroll 1
      for (int i = 0; i < s.tiles; ++i) {
        // TREE: the bits of this warp's keys, asked for before the wait
        constexpr int NV = (WR + 1) / 2;
        uint32_t vis[MT][2][NV];
        if (TREE) {
          const int k0 = (s.tile + i) * kKT + wk * WR * 16;
          if (k0 + WR * 16 > all_see) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int w = 0; w < NV; ++w) {
                  vis[m][e][w] = low_bits(s.klen - k0 - w * 32);
                  if (s.b >= 0)
                    vis[m][e][w] &= tree_window(TreeRow{a.tree + lim[m][e]}, a.tree_words, k0 + w * 32 - all_see);
                }
          }
        }
        const bool got = mbar_wait(&full[st], ph, abort_flag, a.err);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int sub = 0; sub < WR / KS && (WR == 1 || wr * MT * 16 < s.rows); ++sub) {
          const int key = (wk * WR + sub * KS) * 16, k0 = (s.tile + i) * kKT + key;
          const int here = s.nkeys - k0;  // keys of this step's that exist
          if (here <= 0) break;
          const uint32_t stage = smem_u32(smem) + (uint32_t)st * 2 * kTileBytes;
          uint32_t kb[KS];  // each sixteen keys (all in one box); the values kTileBytes behind them
#pragma unroll
          for (int j = 0; j < KS; ++j) kb[j] = stage + (WR == 1 ? warp_off : keys_off(key + 16 * j));
          if (here < 16 * KS) {
            // slots past the end may hold anything: their values become zeros
            // (a zero weight would not stop a NaN); their logits are masked
            for (int z = lane; z < (16 * KS - here) * (DP / 8); z += 32) {
              const int r = here + z / (DP / 8), c8 = z % (DP / 8);
              *reinterpret_cast<uint4*>(smem + (stage + kTileBytes - smem_u32(smem)) +
                                        (WR == 1 ? warp_off + (uint32_t)r * 128 : keys_off(key + r)) +
                                        (uint32_t)(c8 >> 3) * half_step + (uint32_t)((c8 & 7) << 4)) =
                  make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
          }
          float sv[MT][2 * KS][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) sv[m][n][e] = 0.f;
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            const int c16 = (kk & 3) * 2;
            uint32_t qf[MT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
              ldsm4(qs + (uint32_t)(kk >> 2) * RB * 128 + (uint32_t)((wr * MT + m) * 16 + qrow) * 128 +
                        (uint32_t)(((c16 + qsel) ^ (qrow & 7)) << 4),
                    qf[m]);
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              uint32_t kf[4];
              ldsm4(kb[j] + (uint32_t)(kk >> 2) * half_step + (uint32_t)krow * 128 +
                        (uint32_t)(((c16 + ksel) ^ (krow & 7)) << 4),
                    kf);
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma16816<T>(sv[m][2 * j], qf[m], kf[0], kf[1]);
                mma16816<T>(sv[m][2 * j + 1], qf[m], kf[2], kf[3]);
              }
            }
          }
          uint32_t pf[MT][KS][4], pl[kTwoParts ? MT : 1][KS][4];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (TREE && k0 + 16 * KS > all_see) {
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int n = 0; n < 2 * KS; ++n) {
                  const uint32_t word = WR > KS ? (sub ? vis[m][e][NV - 1] : vis[m][e][0]) : vis[m][e][n / 4];
                  const uint32_t bits = word >> ((n & 3) * 8 + t4 * 2);
                  if (!(bits & 1u)) sv[m][n][2 * e] = -INFINITY;
                  if (!(bits & 2u)) sv[m][n][2 * e + 1] = -INFINITY;
                }
            }
            if (!TREE && k0 + 16 * KS > all_see) {
#pragma unroll
              for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (k0 + n * 8 + t4 * 2 + (e & 1) >= lim[m][e >> 1]) sv[m][n][e] = -INFINITY;
            }
            float mx[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mx[e] = fmaxf(fmaxf(sv[m][0][2 * e], sv[m][0][2 * e + 1]), fmaxf(sv[m][1][2 * e], sv[m][1][2 * e + 1]));
#pragma unroll
              for (int n = 2; n < 2 * KS; ++n) mx[e] = fmaxf(mx[e], fmaxf(sv[m][n][2 * e], sv[m][n][2 * e + 1]));
              mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
              mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
            }
            if (__any_sync(0xffffffffu, (mx[0] - mref[m][0]) * sc > kLazy || (mx[1] - mref[m][1]) * sc > kLazy)) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float mn = fmaxf(mref[m][e], mx[e]);
                const float f = mref[m][e] == mn ? 1.f : exp2_fast((mref[m][e] - mn) * sc);
                mref[m][e] = mn;
                l[m][e] *= f;
                if (!kTwoParts) lr[m][e] *= f;
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                  o[m][n][2 * e] *= f;
                  o[m][n][2 * e + 1] *= f;
                }
              }
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              float p[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float ref = mref[m][e] == -INFINITY ? 0.f : mref[m][e];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  const float(&v)[4] = sv[m][2 * j + n];
                  float2 w = fadd2(make_float2(v[2 * e], v[2 * e + 1]), make_float2(-ref, -ref));
                  w = ffma2(w, make_float2(sc, sc), make_float2(ProbBias<T>::value, ProbBias<T>::value));
                  p[n][2 * e] = exp2_fast(w.x);
                  p[n][2 * e + 1] = exp2_fast(w.y);
                  l[m][e] += p[n][2 * e];
                  l[m][e] += p[n][2 * e + 1];
                }
              }
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const float w0 = p[f >> 1][2 * (f & 1)], w1 = p[f >> 1][2 * (f & 1) + 1];
                pf[m][j][f] = Half16<T>::pack(w0, w1);
                const float2 r = Half16<T>::unpack(pf[m][j][f]);
                if (kTwoParts)
                  pl[kTwoParts ? m : 0][j][f] = Half16<T>::pack(w0 - r.x, w1 - r.y);
                else
                  lr[m][f & 1] += r.x + r.y;  // (row g8 + 8 (f & 1))
              }
            }
          }
#pragma unroll
          for (int nn = 0; nn < DP / 16; ++nn) {
            const int c16 = (nn & 3) * 2;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              uint32_t vf[4];
              ldsm4t(kb[j] + kTileBytes + (uint32_t)(nn >> 2) * half_step + (uint32_t)vrow * 128 +
                         (uint32_t)(((c16 + vsel) ^ (vrow & 7)) << 4),
                     vf);
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma16816<T>(o[m][2 * nn], pf[m][j], vf[0], vf[1]);
                mma16816<T>(o[m][2 * nn + 1], pf[m][j], vf[2], vf[3]);
                if (kTwoParts) {
                  mma16816<T>(o[m][2 * nn], pl[m][j], vf[0], vf[1]);
                  mma16816<T>(o[m][2 * nn + 1], pl[m][j], vf[2], vf[3]);
                }
              }
            }
          }
          if (here < 16 * KS) fence_async_smem();  // the zeros before the stage's next copies
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (++st == stages) {
          st = 0;
          ph ^= 1u;
        }
      }
      // the next part's queries are on their way while this one is joined
      const Segment cur = s;
      some = ok && next_segment(&s);
      if (!kAsyncQ && some) load_q(s);

      // ---- the four warps' results become one: a common maximum, then the
      // rescaled sums and output tiles added in a fixed order (key groups 3 into
      // 1, 2 into 0, 1 into 0)
      const int r0 = wk * RB + wr * MT * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[m][e] += __shfl_xor_sync(0xffffffffu, l[m][e], 1);
          l[m][e] += __shfl_xor_sync(0xffffffffu, l[m][e], 2);
          if (t4 == 0) ml[r0 + m * 16 + g8 + 8 * e] = make_float2(mref[m][e], l[m][e]);
          if (!kTwoParts) {
            lr[m][e] += __shfl_xor_sync(0xffffffffu, lr[m][e], 1);
            lr[m][e] += __shfl_xor_sync(0xffffffffu, lr[m][e], 2);
            if (t4 == 0) mlr[r0 + m * 16 + g8 + 8 * e] = lr[m][e];
          }
        }
      bar_compute();
      if (kAsyncQ && some) load_q(s);
      float mt[MT][2], lt[MT][2], lrt[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = (wr * MT + m) * 16 + g8 + 8 * e;
          float mm = -INFINITY, ll = 0.f, lq = 0.f;
#pragma unroll
          for (int w = 0; w < WK; ++w) mm = fmaxf(mm, ml[w * RB + r].x);
#pragma unroll
          for (int w = 0; w < WK; ++w) {
            const float2 v = ml[w * RB + r];
            const float x = v.x == mm ? 1.f : exp2_fast((v.x - mm) * sc);
            ll += v.y * x;
            if (!kTwoParts) lq += mlr[w * RB + r] * x;
          }
          mt[m][e] = mm;
          lt[m][e] = ll;
          lrt[m][e] = kTwoParts ? ll : lq;
          const float f = mref[m][e] == mm ? 1.f : exp2_fast((mref[m][e] - mm) * sc);
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            o[m][n][2 * e] *= f;
            o[m][n][2 * e + 1] *= f;
          }
        }
      // [slot][row half of 8][tile, column block][lane]
      const int halves = ln.part_rows > 8 ? 2 : 1;
      float2* buf = reinterpret_cast<float2*>(merge) + (WK == 4 ? wk & 1 : wr) * (halves * MT * (DP / 8) * 32) + lane;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (wk >= 2 && e < halves) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
              buf[((e * MT + m) * (DP / 8) + n) * 32] = make_float2(o[m][n][2 * e], o[m][n][2 * e + 1]);
        }
      bar_compute();
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (WK > 1 && (WK == 4 ? wk < 2 : wk == 1) && e < halves) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
              float2* at = buf + ((e * MT + m) * (DP / 8) + n) * 32;
              const float2 v = WK == 4 ? *at : make_float2(0.f, 0.f);
              o[m][n][2 * e] += v.x;
              o[m][n][2 * e + 1] += v.y;
              if (wk == 1) *at = make_float2(o[m][n][2 * e], o[m][n][2 * e + 1]);
            }
        }
      bar_compute();
      if (wk == 0) {
        const float2* src = reinterpret_cast<const float2*>(merge) + (WK == 4 ? 1 : wr) * halves * MT * (DP / 8) * 32 + lane;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = (wr * MT + m) * 16 + g8 + 8 * e;
            if (r < cur.rows) {
              const bool done = whole(ln, cur);
              const int2 at = cur.parts ? row_place(a, cur, r) : make_int2(0, 0);
              const float inv = inverse_sum(lrt[m][e]);
              // a partial stands against the exact sum
              const float own = kTwoParts || lt[m][e] == lrt[m][e] ? 1.f : lt[m][e] / lrt[m][e];
              float* dst = ln.part_o + (long long)(cur.prow + r) * DP + t4 * 2;
              T* out = static_cast<T*>(a.out) + (long long)at.x * a.out_stride + (long long)at.y * a.D + t4 * 2;
#pragma unroll
              for (int n = 0; n < DP / 8; ++n) {
                const float2 v = WK > 1 ? src[((e * MT + m) * (DP / 8) + n) * 32] : make_float2(0.f, 0.f);
                const float2 w = make_float2(o[m][n][2 * e] + v.x, o[m][n][2 * e + 1] + v.y);
                if (!done)
                  *reinterpret_cast<float2*>(dst + n * 8) = kTwoParts ? w : make_float2(w.x * own, w.y * own);
                else if (n * 8 < a.D)
                  *reinterpret_cast<uint32_t*>(out + n * 8) = Half16<T>::pack(w.x * inv, w.y * inv);
              }
              if (t4 == 0) {
                if (!done)
                  ln.part_ml[cur.prow + r] = make_float2(mt[m][e], lt[m][e]);
                else if (a.lse)
                  a.lse[(long long)at.x * a.Hq + at.y] = log_sum<T>(mt[m][e], lt[m][e], a.scale);
                if (cur.parts && !whole_groups) write_info(a, ln, cur, r, at);
              }
            }
          }
      }
      // the buffers are free again once the next part's queries are in
      // (its first barrier comes after these reads)
    }
  }
  if (late_wait) pdl_wait();  // ends after the kernel before it, so what waits for this one waits for both
}

template <typename T, int DP, bool TREE>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln,
                   const AttnRowsPlan& p, int box_log2, bool late_wait, cudaStream_t s, bool pdl) {
  auto run = [&](auto kern) {
    const cudaError_t e = ensure_smem(kern, p.smem);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3(p.n_cta), dim3(kThreads), p.smem, s, pdl, tk, tv, a, ln, p.stages, box_log2,
                     (int)late_wait);
  };
  if constexpr (TREE) {
    if (p.row_groups == 4) return run(k_attn_rows<T, DP, 1, 4, true>);
    if (p.row_groups == 2) return run(k_attn_rows<T, DP, 1, 2, true>);
  } else if constexpr (rows_most(DP, false, 0) > 16) {
    if (ln.part_rows > 16) return run(k_attn_rows<T, DP, 2, 1, false>);
  }
  return run(k_attn_rows<T, DP, 1, 1, TREE>);
}

template <typename T>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln,
                     const AttnRowsPlan& p, int bl, bool late_wait, cudaStream_t s, bool pdl) {
  if (a.D <= 64)
    return a.tree ? launch<T, 64, true>(tk, tv, a, ln, p, bl, late_wait, s, pdl)
                  : launch<T, 64, false>(tk, tv, a, ln, p, bl, late_wait, s, pdl);
  return a.tree ? launch<T, 128, true>(tk, tv, a, ln, p, bl, late_wait, s, pdl)
                : launch<T, 128, false>(tk, tv, a, ln, p, bl, late_wait, s, pdl);
}

}  // namespace

AttnRowsPlan plan_attn_rows(int D, int rows, int B, int num_sms, bool tree) {
  const int DP = D <= 64 ? 64 : 128, MT = tree || rows <= 16 ? 1 : 2;
  AttnRowsPlan p;
  const int WR = p.row_groups = !tree || rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  // as many stages as let two blocks share an SM (228 KB, 1 KB of it kept per
  // block, and up to 1 KB to align the ring)
  for (p.stages = kMaxStages; p.stages > 2; --p.stages)
    if (smem_plan(DP, MT, WR, rows, p.stages, B).bytes + 2048 <= 114 * 1024) break;
  p.smem = smem_plan(DP, MT, WR, rows, p.stages, B).bytes + 1024;
  p.n_cta = num_sms * (p.smem + 1024 <= 114 * 1024 ? 2 : 1);
  return p;
}

cudaError_t launch_attn_rows(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, const LineArgs& ln,
                             const AttnRowsPlan& p, int box_slots, bool bf16, bool late_wait, cudaStream_t s,
                             bool pdl) {
  int bl = 4;
  while ((1 << bl) < box_slots) ++bl;
  return bf16 ? launch_t<__nv_bfloat16>(tk, tv, a, ln, p, bl, late_wait, s, pdl)
              : launch_t<__half>(tk, tv, a, ln, p, bl, late_wait, s, pdl);
}

bool encode_cache_map(CUtensorMap* tm, const void* cache, bool bf16, int D, int page_size, int Hk, long long num_pages,
                      long long page_stride, long long slot_stride, long long head_stride, int slots, bool whole_head) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!fn) return false;
  // heads of a multiple of 64 elements are rows of 64-wide halves; in other
  // heads a box past the end is filled with zeros
  const bool halves = D % 64 == 0;
  const cuuint64_t dims[5] = {(cuuint64_t)(halves ? 64 : D), (cuuint64_t)page_size, (cuuint64_t)(halves ? D / 64 : 1),
                              (cuuint64_t)Hk, (cuuint64_t)num_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)slot_stride * 2, 128, (cuuint64_t)head_stride * 2,
                                 (cuuint64_t)page_stride * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)slots, (cuuint32_t)(halves && whole_head ? D / 64 : 1), 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(cache),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
