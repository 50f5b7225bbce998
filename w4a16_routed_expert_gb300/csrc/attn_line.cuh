// The line of key tiles that a forward's blocks share (LineArgs), and the
// walk of one block over its run of it.
#pragma once

#include "attn_dev.cuh"

namespace moe {

// Keys the row block starting at row r0 of a sequence's n * g rows reads: as
// many as its last token sees.
__device__ __forceinline__ int block_keys(const AttnArgs& a, const LineArgs& ln, int keys, int n, int rb) {
  const int last = min(n * a.g, (rb + 1) * ln.row_block) - 1;
  return keys_seen(a, keys, n, last / a.g);
}
// Tiles of a sequence for one key head.
__device__ __forceinline__ int seq_tiles(const AttnArgs& a, const LineArgs& ln, int keys, int n) {
  const int blocks = (n * a.g + ln.row_block - 1) / ln.row_block;
  int tiles = 0;
  for (int rb = 0; rb < blocks; ++rb)
    tiles += (block_keys(a, ln, keys, n, rb) + ln.key_tile - 1) / ln.key_tile;
  return tiles;
}
// (key heads, row blocks, tiles each) of the prefix.
__device__ __forceinline__ int prefix_blocks(const AttnArgs& a, const LineArgs& ln) {
  return (int)(((long long)a.T * a.g + ln.row_block - 1) / ln.row_block);
}
__device__ __forceinline__ int prefix_tiles(const AttnArgs& a, const LineArgs& ln) {
  return ln.has_prefix ? (a.prefix_len + ln.key_tile - 1) / ln.key_tile : 0;
}
__device__ __forceinline__ long long prefix_line(const AttnArgs& a, const LineArgs& ln) {
  return (long long)a.Hk * prefix_blocks(a, ln) * prefix_tiles(a, ln);
}

// Whole block (NT threads): own_off[b] = own tiles of one key head before
// sequence b, in shared memory; returns their total. scratch: NT / 32 ints.
template <int NT>
__device__ int scan_own(const AttnArgs& a, const LineArgs& ln, int32_t* own_off, int32_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!ln.has_own) {
    if (tid == 0) own_off[0] = 0;
    __syncthreads();
    return 0;
  }
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    int t0;
    const int n = seq_tokens(a, b, &t0);
    const int tiles = seq_tiles(a, ln, seq_keys(a, b), n);
    own_off[b + 1] = tiles;
    sum += tiles;
    if (blockIdx.x == b % gridDim.x)
      for (int i = 0; i < n; ++i) a.seq_of[t0 + i] = b;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int base = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += scratch[w];
    total += scratch[w];
  }
  if (tid == 0) own_off[0] = 0;
  for (int b = b0; b < b1; ++b) {
    base += own_off[b + 1];
    own_off[b + 1] = base;
  }
  __syncthreads();
  return total;
}

// One block's part of one group.
struct Segment {
  int b;            // sequence, or -1: the prefix
  int h;            // key head
  int tile, tiles;  // first tile of the group and number of tiles in this part
  int row0, rows;   // first row of the group among its sequence's (all tokens') rows, rows
  int t0, n;        // the sequence's (batch's) first token and tokens
  int klen;         // its keys
  int nkeys;        // keys the group reads (its last row's)
  long long prow;   // first row of the partial
};

// The part of the line from tile x (x < end), this block's run.
__device__ __forceinline__ Segment segment_at(const AttnArgs& a, const LineArgs& ln, const int32_t* own_off,
                                              long long x, long long end) {
  Segment s;
  const long long wp = prefix_line(a, ln);
  int left;  // tiles of the group from s.tile on
  long long base;
  if (x < wp) {
    const int nt = prefix_tiles(a, ln), nb = prefix_blocks(a, ln);
    const int grp = (int)(x / nt);
    s.b = -1;
    s.tile = (int)(x - (long long)grp * nt);
    left = nt - s.tile;
    s.h = grp / nb;
    const int rb = grp - s.h * nb;
    s.t0 = 0;
    s.n = a.T;
    s.row0 = rb * ln.row_block;
    s.rows = min(ln.row_block, a.T * a.g - s.row0);
    s.klen = s.nkeys = a.prefix_len;
    base = (long long)s.h * a.T * a.g + s.row0;
  } else {
    const long long y = x - wp;
    int lo = 0, hi = a.B - 1;  // last b with own_off[b] * Hk <= y
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)own_off[mid] * a.Hk <= y)
        lo = mid;
      else
        hi = mid - 1;
    }
    s.b = lo;
    const int per_head = own_off[lo + 1] - own_off[lo];
    const long long r = y - (long long)own_off[lo] * a.Hk;
    s.h = (int)(r / per_head);
    int in = (int)(r - (long long)s.h * per_head);
    s.n = seq_tokens(a, lo, &s.t0);
    s.klen = seq_keys(a, lo);
    const int blocks = (s.n * a.g + ln.row_block - 1) / ln.row_block;
    int rb = 0;
    left = 0;
    for (; rb < blocks; ++rb) {
      s.nkeys = block_keys(a, ln, s.klen, s.n, rb);
      const int nt = (s.nkeys + ln.key_tile - 1) / ln.key_tile;
      if (in < nt) {
        left = nt - in;
        break;
      }
      in -= nt;
    }
    if (left == 0) {  // the lengths changed under the kernel: nothing to read, one tile on
      record_error(a.err, kAttnErrBounds);
      rb = in = s.nkeys = 0;
      left = 1;
    }
    s.tile = in;
    s.row0 = rb * ln.row_block;
    s.rows = min(ln.row_block, s.n * a.g - s.row0);
    base = ((long long)ln.has_prefix * a.T + s.t0) * a.g * a.Hk + (long long)s.h * s.n * a.g + s.row0;
  }
  s.tiles = (int)min((long long)left, end - x);
  s.prow = base + (long long)blockIdx.x * ln.part_rows;
  return s;
}

// Tile line of the launch: tiles per block, with the first block leaving what
// the join needs in the workspace. All threads call it after scan_own.
__device__ __forceinline__ long long line_share(const AttnArgs& a, const LineArgs& ln, const int32_t* own_off,
                                                int own_total, long long* total) {
  *total = prefix_line(a, ln) + (long long)own_total * a.Hk;
  const long long share = max(1LL, (*total + ln.n_cta - 1) / ln.n_cta);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) *ln.share = share;
    if (ln.has_own)
      for (int b = threadIdx.x; b <= a.B; b += blockDim.x) ln.own_off[b] = own_off[b];
  }
  return share;
}

}  // namespace moe
