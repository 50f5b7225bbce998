// The line of key tiles that a forward's blocks share (LineArgs), and the
// walk of one block over its run of it.
#pragma once

#include "attn_dev.cuh"

namespace moe {

// KT keys of a tile, RB rows of a group at most: LineArgs' key_tile and
// row_block as the kernel was built for (powers of two, so that no division
// stands before its first copy).

// Keys that row block rb of a sequence's n * g rows reads: as many as its
// last token sees.
template <int RB>
__device__ __forceinline__ int block_keys(const AttnArgs& a, int keys, int n, int rb) {
  const int last = min(n * a.g, (rb + 1) * RB) - 1;
  return a.causal ? keys_seen(a, keys, n, last / a.g) : keys;
}
// Tiles of `keys` keys; tiles of the prefix at the front of each own group.
template <int KT>
__device__ __forceinline__ int tiles_of(int keys) {
  return (int)((unsigned)(keys + KT - 1) / KT);
}
template <int KT>
__device__ __forceinline__ int front_tiles(const AttnArgs& a, const LineArgs& ln) {
  return ln.joined ? tiles_of<KT>(a.prefix_len) : 0;
}
// Row blocks of n query tokens.
template <int RB>
__device__ __forceinline__ int row_blocks(const AttnArgs& a, int n) {
  return (int)((unsigned)(n * a.g + RB - 1) / RB);
}
// Places on the line of a group of `tiles` tiles.
__device__ __forceinline__ int group_span(const LineArgs& ln, int tiles) { return tiles > 0 ? tiles + ln.weight : 0; }

// Whole block (NT threads): own_off[b] = places of one key head's groups
// before sequence b, in shared memory; returns their total. scratch: NT / 32
// ints. Sequences that overlap (offsets out of order) can come to more than
// the host counted on and than 32 bits hold: sums stop one place above
// own_most, and then there is no work.
template <int NT, int KT, int RB>
__device__ int scan_own(const AttnArgs& a, const LineArgs& ln, int32_t* own_off, int32_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!ln.has_own) return 0;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  const unsigned most = (unsigned)ln.own_most + 1u;
  auto add = [&](unsigned x, unsigned y) { return min(x + y, most); };  // (both below 2^31)
  unsigned sum = 0;
  const int front = front_tiles<KT>(a, ln);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Seq q = load_seq(a, b);
    const int blocks = row_blocks<RB>(a, q.n);
    int span = 0;
#pragma unroll 1
    for (int rb = 0; rb < blocks; ++rb) span += group_span(ln, front + tiles_of<KT>(block_keys<RB>(a, q.keys, q.n, rb)));
    own_off[b + 1] = span;
    sum = add(sum, (unsigned)span);
  }
  unsigned incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl = add(incl, y);
  }
  if (lane == 31) scratch[warp] = (int)incl;
  __syncthreads();
  unsigned base = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base = add(base, (unsigned)scratch[w]);
    total = add(total, (unsigned)scratch[w]);
  }
  if (tid == 0) own_off[0] = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    base = add(base, (unsigned)own_off[b + 1]);
    own_off[b + 1] = (int)base;
  }
  __syncthreads();
  if (total < most) return (int)total;
  if (tid == 0) record_error(a.err, kAttnErrBounds);
  return 0;
}

// One block's part of one group, handed through shared memory from the
// copying warp to the others.
struct Segment {
  int b;            // sequence, or -1: the prefix
  int h;            // key head
  int tile, tiles;  // first tile of the group and number of tiles in this part (0: no more parts)
  int row0, rows;   // first row of the group among its sequence's (all tokens') rows, rows
  int t0, n;        // the sequence's (batch's) first token and tokens
  int klen;         // its keys
  int nkeys;        // keys the group reads (its last row's), those of the tiles before `front` aside
  int front;        // tiles of the prefix at the front of a sequence's group (LineArgs::joined)
  int prow;         // first row of the partial
  int parts;        // the part with the group's first tile: parts of the group (else 0)
};
constexpr int kSegSlots = 4;  // parts handed ahead

// The walk: every lane of a warp runs it with the same values.
template <int KT, int RB>
struct Walk {
  int x, end, share;   // place, end of this block's run, places per block
  int start, nt;       // the group's first place, its tiles
  int blocks;          // row blocks of the sequence (the batch)
  int rb;
  Segment s;           // b, h, t0, n, klen, nkeys of the group

  __device__ __forceinline__ void set_seq(const AttnArgs& a, int b) {
    const Seq q = load_seq(a, b);
    s.b = b;
    s.t0 = q.t0;
    s.n = q.n;
    s.klen = q.keys;
    blocks = row_blocks<RB>(a, s.n);
  }
  __device__ __forceinline__ void set_group(const AttnArgs& a, const LineArgs& ln) {
    s.nkeys = s.b < 0 ? s.klen : block_keys<RB>(a, s.klen, s.n, rb);
    s.front = s.b < 0 ? 0 : front_tiles<KT>(a, ln);
    nt = s.front + tiles_of<KT>(s.nkeys);
  }
  // The first group of own keys that has any, from sequence b on.
  __device__ __forceinline__ void first_own(const AttnArgs& a, const LineArgs& ln, const int32_t* own_off, int b) {
    while (b < a.B - 1 && own_off[b + 1] == own_off[b]) ++b;
    set_seq(a, b);
    s.h = 0;
    rb = 0;
    set_group(a, ln);
  }
  // To the group after this one (its start is where this one ended); false
  // after the last.
  __device__ __forceinline__ bool next_group(const AttnArgs& a, const LineArgs& ln, const int32_t* own_off) {
    start += group_span(ln, nt);
    if (++rb >= blocks) {
      rb = 0;
      if (++s.h >= a.Hk) {
        if (!ln.has_own || s.b + 1 >= a.B) return false;
        first_own(a, ln, own_off, s.b + 1);
        return true;
      }
    }
    set_group(a, ln);
    return true;
  }
  // own_total: places of one key head's own groups (scan_own).
  __device__ __forceinline__ void init(const AttnArgs& a, const LineArgs& ln, const int32_t* own_off, int own_total) {
    const int pblocks = ln.has_prefix ? row_blocks<RB>(a, a.T) : 0;
    const int pspan = ln.has_prefix ? group_span(ln, tiles_of<KT>(a.prefix_len)) : 0;
    const int total_prefix = a.Hk * pblocks * pspan;
    const int total = total_prefix + own_total * a.Hk;
    share = max(1, (int)(((unsigned)total + ln.n_cta - 1) / (unsigned)ln.n_cta));
    x = (int)min((long long)share * blockIdx.x, (long long)total);
    end = (int)min((long long)x + share, (long long)total);
    if (x >= end) return;
    if (x < total_prefix) {
      const int grp = x / pspan;
      start = grp * pspan;
      s.b = -1;
      s.h = grp / pblocks;
      rb = grp - s.h * pblocks;
      blocks = pblocks;
      s.t0 = 0;
      s.n = a.T;
      s.klen = a.prefix_len;
      set_group(a, ln);
      return;
    }
    const unsigned y = (unsigned)(x - total_prefix);
    int lo = 0, hi = a.B - 1;  // last sequence that starts at or before y
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((unsigned)own_off[mid] * a.Hk <= y)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int per_head = max(1, own_off[lo + 1] - own_off[lo]);
    set_seq(a, lo);
    s.h = min((int)((y - (unsigned)own_off[lo] * a.Hk) / (unsigned)per_head), a.Hk - 1);
    start = total_prefix + own_off[lo] * a.Hk + s.h * per_head;
    rb = 0;
    set_group(a, ln);
    while (start + group_span(ln, nt) <= x && rb + 1 < blocks) {
      start += group_span(ln, nt);
      ++rb;
      set_group(a, ln);
    }
  }
  // The next part of this block's run; false when there is none.
  __device__ __forceinline__ bool next(const AttnArgs& a, const LineArgs& ln, const int32_t* own_off, Segment* out) {
    while (x < end) {
      const int first = start + ln.weight;  // the group's first tile
      const int lo = max(x, first), hi = min(end, first + nt);
      const bool some = hi > lo;
      if (some) {
        *out = s;
        out->tile = lo - first;
        out->tiles = hi - lo;
        out->row0 = rb * RB;
        out->rows = min(RB, s.n * a.g - out->row0);
        out->prow = ln.part_row0 + (int)blockIdx.x * ln.part_rows + out->row0 + s.h * s.n * a.g +
                    (s.b < 0 ? 0 : (ln.has_prefix * a.T + s.t0) * a.Hq);
        // (never more than there are blocks, whatever the lengths do meanwhile)
        out->parts = lo == first ? min((first + nt - 1) / share, ln.n_cta - 1) - (int)blockIdx.x + 1 : 0;
      }
      // (lengths that change under the kernel move groups, but every step
      // still goes on along the line or to a later group)
      if (nt > 0) x = max(x + 1, first + nt);
      if (x < end && !next_group(a, ln, own_off)) x = end;
      if (some) return true;
    }
    return false;
  }
};

// Whether the part is its rows' whole result, to be stored as it is.
__device__ __forceinline__ bool whole(const LineArgs& ln, const Segment& s) {
  return s.parts == 1 && (s.b < 0 ? ln.final_prefix : ln.final_own);
}
// The token and query head of row r of a group.
__device__ __forceinline__ int2 row_place(const AttnArgs& a, const Segment& s, int r) {
  const int row = s.row0 + r, tok = row / a.g;
  return make_int2(s.t0 + tok, s.h * a.g + row - tok * a.g);
}
// Leaves, for each row of a group, where its partials start and how many
// there are (the part with the group's first tile does), or -1 where the
// result is stored already.
__device__ __forceinline__ void write_info(const AttnArgs& a, const LineArgs& ln, const Segment& s, int r, int2 at) {
  int2* info = s.b < 0 ? ln.info_prefix : ln.info_own;
  info[(long long)at.x * a.Hq + at.y] = whole(ln, s) ? make_int2(0, -1) : make_int2(s.prow + r, s.parts);
}

}  // namespace moe
