// A step's tables (moe_attn_plan): from each sequence's context, new tokens and
// pages held, three running sums over the sequences (tokens, pages taken, pages
// given back) say where everything goes:
//   q_offsets[b] = sum_{b' < b} m_b',   need_b = max(0, ceil((c_b + m_b) / p) - held_b)
//   table[b][held_b + i] = ring[first + sum_{b' < b} need_b' + i]
// and a tree's masks are the closure of its parents:
//   row(i) = bit i | row(parent(i)),   depth(i) = popcount(row(i)) - 1
// taken by doubling (row |= row(jump), jump = jump(jump)): log2(depth) rounds.
//
// A decode step reads and writes a few kilobytes, so launch and the chain of
// dependent loads bound it (lengths, then parents or ring, then the stores); a
// step of prompts stores 8 bytes a token beside them (4 MB for half a million
// tokens, 0.6 us at the copy rate), which hides under that chain. One launch:
// every block takes the sums over all sequences for itself (at most 4096, a few
// words a thread) instead of waiting for another, and then its share of the
// sequences, pages and tokens. The pool's state may be updated in place: the
// last block to have read it writes it (which costs each block a turn at one
// counter: 512 prompts of up to 1999 tokens, half a million in all, take 7.9 us
// with 304 blocks; where each block read the state twice 8.3, and then 11.3 with
// 500, 10.3 with 152). Four trees of up to 8 tokens take 4.3 us, 50 of up to 63
// 7.4.
#include <algorithm>

#include "attn_dev.cuh"
#include "attn_plan.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct SmemPlan {
  uint32_t off, take, back, held, served, rows, jump, bytes;
};
__host__ __device__ inline SmemPlan smem_plan(int B, int max_nodes, int words) {
  SmemPlan p;
  p.off = 0;
  p.take = p.off + (uint32_t)(B + 1) * 4;
  p.back = p.take + (uint32_t)(B + 1) * 4;
  p.held = p.back + (uint32_t)(B + 1) * 4;
  p.served = p.held + (uint32_t)B * 4;
  p.rows = (p.served + (uint32_t)B + 3) & ~3u;
  const uint32_t nodes = max_nodes > 32 ? (uint32_t)max_nodes : 0u;
  p.jump = p.rows + nodes * (uint32_t)words * 4;
  p.bytes = p.jump + 2 * nodes * 4;
  return p;
}

__device__ __forceinline__ PlanAsk ask_of(const PlanArgs& a, int ctx, int fresh, int held) {
  return plan_ask(a.T, a.max_nodes, a.table_stride, a.page_size, ctx, fresh, held);
}

// The last b with at[b] <= x; at ascends, at[0] = 0.
__device__ __forceinline__ int find(const int* at, int B, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) k_attn_plan(const PlanArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int part[3][kThreads / 32];
  __shared__ int most_taken, is_last;
  const SmemPlan sp = smem_plan(a.B, a.max_nodes, a.words);
  int* off = reinterpret_cast<int*>(smem + sp.off);
  int* take = reinterpret_cast<int*>(smem + sp.take);
  int* back = reinterpret_cast<int*>(smem + sp.back);
  int* hold = reinterpret_cast<int*>(smem + sp.held);  // pages held before the step
  unsigned char* served = smem + sp.served;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.B, F = a.ring_size;
  pdl_trigger();
  pdl_wait();

  // ---- the three running sums
  int first = a.state[0], count = a.state[1];
  bool bad = first < 0 || first >= F || count < 0 || count > F;
  first = first < 0 || first >= F ? 0 : first;
  count = min(max(count, 0), F);
  const int per = (B + kThreads - 1) / kThreads, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  auto ask = [&](int b) { return ask_of(a, a.context_lens[b], a.new_lens[b], a.state[2 + b]); };
  int sum[3] = {0, 0, 0};
  if (tid == 0) most_taken = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const PlanAsk k = ask(b);
    sum[0] = plan_add(sum[0], k.m);
    sum[1] = plan_add(sum[1], k.need);
    sum[2] = plan_add(sum[2], k.back);
    bad |= !k.valid;
  }
  int incl[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    incl[i] = sum[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl[i], o);
      if (lane >= o) incl[i] = plan_add(incl[i], y);
    }
    if (lane == 31) part[i][warp] = incl[i];
  }
  __syncthreads();
  int base[3], total[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int y = __shfl_up_sync(0xffffffffu, incl[i], 1);
    base[i] = lane ? y : 0;
    total[i] = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base[i] = plan_add(base[i], part[i][w]);
      total[i] = plan_add(total[i], part[i][w]);
    }
  }
  int mine = 0;  // pages taken up to this thread's last sequence that is served
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const PlanAsk k = ask(b);
    hold[b] = a.state[2 + b];
    off[b] = base[0];
    take[b] = base[1];
    back[b] = base[2];
    const bool room = base[0] + k.m <= a.T;
#pragma unroll
    for (int i = 0; i < 3; ++i) base[i] = plan_add(base[i], i == 0 ? k.m : i == 1 ? k.need : k.back);
    const bool ok = k.valid && a.new_lens[b] >= 0 && room && (k.need == 0 || base[1] <= count);
    served[b] = ok;
    if (ok && k.need) mine = base[1];
    bad |= !room;
  }
  if (tid == 0) {
    off[B] = total[0];
    take[B] = total[1];
    back[B] = total[2];
  }
  if (mine) atomicMax(&most_taken, mine);
  if (bad && blockIdx.x == 0) record_error(a.err, kAttnErrBounds);
  __syncthreads();
  // The old state has been read: this block's turn at the counter, whose answer
  // is on its way under the rest.
  unsigned turn = 0;
  if (tid == 0 && gridDim.x > 1) turn = atom_acq_rel_add(a.ticket, 1u);
  const int taken = most_taken;
  const int given = min(back[B], F - count);
  if (given < back[B] && blockIdx.x == 0 && tid == 0) record_error(a.err, kAttnErrBounds);

  const int grid_threads = gridDim.x * kThreads, gtid = blockIdx.x * kThreads + tid;
  auto ring_at = [&](int i) {  // i < 2 F
    const int x = first + (i >= F ? i - F : i);
    return x >= F ? x - F : x;
  };
  // ---- per sequence, per page
  for (int b = gtid; b <= B; b += grid_threads) {
    a.q_offsets[b] = min(off[b], a.T);
    if (b < B) a.seq_lens[b] = served[b] ? a.context_lens[b] + a.new_lens[b] : 0;
  }
  for (int i = gtid; i < taken; i += grid_threads) {
    const int b = find(take, B, i);
    a.block_table[(long long)b * a.table_stride + hold[b] + i - take[b]] = a.free_pages[ring_at(i)];
  }
  for (int i = gtid; i < given; i += grid_threads) {
    const int b = find(back, B, i);
    a.free_pages[ring_at(count + i)] = a.block_table[(long long)b * a.table_stride + i - back[b]];
  }

  // ---- per token
  // The slot of a sequence's key: its page stands in the table, or is being
  // taken from the ring by this step.
  auto page_of = [&](int b, int held, int pg) {
    return pg < held ? a.block_table[(long long)b * a.table_stride + pg] : a.free_pages[ring_at(take[b] + pg - held)];
  };
  auto slot_in = [&](int page, int at) {
    if ((unsigned)page >= (unsigned)a.num_pages) {
      record_error(a.err, kAttnErrBounds);
      return -1;
    }
    return page * a.page_size + at;
  };
  auto slot = [&](int b, int key) {
    const int pg = key / a.page_size;
    return slot_in(page_of(b, hold[b], pg), key - pg * a.page_size);
  };
  const int tokens = min(off[B], a.T);
  if (a.max_nodes == 0) {
    // lines: four tokens a thread, mostly of one sequence and one page (512
    // prompts of up to 1999 tokens: 7.9 us, 11.0 with one)
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.slots)) & 15) == 0;
    for (int t = gtid * 4; t < tokens; t += grid_threads * 4) {
      const int n = min(4, tokens - t);
      int b = find(off, B, t), ctx = 0, next = off[b], held = 0, pg = -1, page = 0;
      bool ok = false;
      int pos[4], slots[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pos[i] = 0;
        slots[i] = -1;
        if (i < n) {
          if (i == 0 || t + i >= next) {  // a sequence (the next that has tokens)
            if (i)
              do ++b;
              while (off[b + 1] <= t + i);
            next = off[b + 1];
            ctx = a.context_lens[b];
            held = hold[b];
            ok = served[b];
            pg = -1;
          }
          const int key = ctx + t + i - off[b];
          pos[i] = a.prefix_len + key;
          if (ok) {
            if (pg < 0 || key >= (pg + 1) * a.page_size) {
              pg = key / a.page_size;
              page = page_of(b, held, pg);
            }
            slots[i] = slot_in(page, key - pg * a.page_size);
          }
        }
      }
      if (aligned && n == 4) {
        *reinterpret_cast<int4*>(a.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(a.slots + t) = make_int4(slots[0], slots[1], slots[2], slots[3]);
      } else {
        for (int i = 0; i < n; ++i) {
          a.positions[t + i] = pos[i];
          a.slots[t + i] = slots[i];
        }
      }
    }
  } else {
    auto parent_of = [&](int t, int i) {
      int p = a.parents[t];
      if (p < -1 || p >= i) {
        record_error(a.err, kAttnErrBounds);
        p = -1;
      }
      return p;
    };
    // slots come before the branches: their loads run under these
    auto place = [&](int b, int t, int i) { a.slots[t] = served[b] ? slot(b, a.context_lens[b] + i) : -1; };
    // trees of up to 32 tokens: a warp each, a lane a token
    for (int b = blockIdx.x + gridDim.x * warp; b < B; b += gridDim.x * (kThreads / 32)) {
      const int t0 = min(off[b], a.T), m = min(off[b + 1], a.T) - t0;
      if (m <= 0 || m > 32) continue;
      int jump = lane < m ? parent_of(t0 + lane, lane) : -1;
      if (lane < m) place(b, t0 + lane, lane);
      uint32_t row = 1u << lane;
      while (__any_sync(0xffffffffu, jump >= 0)) {
        const uint32_t r = __shfl_sync(0xffffffffu, row, jump & 31);
        const int j = __shfl_sync(0xffffffffu, jump, jump & 31);
        if (jump >= 0) {
          row |= r;
          jump = j;
        }
      }
      if (lane < m) {
        a.positions[t0 + lane] = a.prefix_len + a.context_lens[b] + __popc(row) - 1;
        uint32_t* out = a.tree + (long long)(t0 + lane) * a.words;
        out[0] = row;
        for (int w = 1; w < a.words; ++w) out[w] = 0;
      }
    }
    // larger ones: a block each
    uint32_t* rows = reinterpret_cast<uint32_t*>(smem + sp.rows);
    const int W = a.words;
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
      const int t0 = min(off[b], a.T), m = min(off[b + 1], a.T) - t0;
      if (m <= 32) continue;
      if (m > a.max_nodes) {  // (recorded above)
        for (int i = tid; i < m * W; i += kThreads) a.tree[(long long)t0 * W + i] = 0;
        for (int i = tid; i < m; i += kThreads) {
          a.slots[t0 + i] = -1;
          a.positions[t0 + i] = a.prefix_len + a.context_lens[b];
        }
        continue;
      }
      int* jump = reinterpret_cast<int*>(smem + sp.jump);
      int* next = jump + a.max_nodes;
      __syncthreads();  // the tree before has been read
      for (int i = tid; i < m; i += kThreads) jump[i] = parent_of(t0 + i, i);
      for (int i = tid; i < m; i += kThreads) place(b, t0 + i, i);
      for (int i = tid; i < m * W; i += kThreads) rows[i] = i % W == (i / W) >> 5 ? 1u << ((i / W) & 31) : 0u;
      __syncthreads();
      // A row may be read while its own thread adds to it: whatever is read holds
      // at least the branch up to where `jump` stood before the round.
      while (true) {
        bool more = false;
        for (int i = tid; i < m * W; i += kThreads) {
          const int n = i / W, w = i - n * W, j = jump[n];
          if (j >= 0) {
            more = true;
            const uint32_t r = *(volatile uint32_t*)(rows + j * W + w);
            *(volatile uint32_t*)(rows + i) |= r;
          }
          if (w == 0) next[n] = j >= 0 ? jump[j] : -1;
        }
        int* x = jump;
        jump = next;
        next = x;
        if (!__syncthreads_or(more)) break;
      }
      for (int i = tid; i < m * W; i += kThreads) a.tree[(long long)t0 * W + i] = rows[i];
      for (int i = tid; i < m; i += kThreads) {
        int depth = -1;
        for (int w = 0; w < W; ++w) depth += __popc(rows[i * W + w]);
        a.positions[t0 + i] = a.prefix_len + a.context_lens[b] + depth;
      }
    }
    for (long long i = (long long)tokens * a.words + gtid; i < (long long)a.T * a.words; i += grid_threads) a.tree[i] = 0;
  }
  for (int t = tokens + gtid; t < a.T; t += grid_threads) {
    a.positions[t] = 0;
    a.slots[t] = -1;
  }

  // ---- the pool's state: no block reads the old one any more when the last has
  // had its turn
  if (tid == 0) is_last = turn == gridDim.x - 1;
  __syncthreads();
  if (!is_last) return;
  for (int b = tid; b < B; b += kThreads) {
    const int held = hold[b];
    a.state_out[2 + b] = served[b] ? held + take[b + 1] - take[b] : back[b + 1] > back[b] ? 0 : held;
  }
  if (tid == 0) {
    a.state_out[0] = ring_at(taken);
    a.state_out[1] = count - taken + given;
    *a.ticket = 0;
  }
}

}  // namespace

cudaError_t launch_attn_plan(const PlanArgs& a, int num_sms, cudaStream_t s, bool pdl) {
  const size_t smem = smem_plan(a.B, a.max_nodes, a.words).bytes;
  const cudaError_t e = ensure_smem(k_attn_plan, smem);
  if (e != cudaSuccess) return e;
  const int by_tokens = (a.T + 4 * kThreads - 1) / (4 * kThreads), by_trees = a.max_nodes ? a.B : 0;
  const int grid = std::max(1, std::min(2 * num_sms, std::max(by_tokens, by_trees)));
  return launch_ex(k_attn_plan, dim3(grid), dim3(kThreads), smem, s, pdl, a);
}

}  // namespace moe
