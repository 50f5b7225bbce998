// After a step over drafted trees: the branch that the model's choices confirm
// (moe_attn_accept), and its keys and values moved behind the context
// (moe_attn_keep).
#include <algorithm>

#include "attn_dev.cuh"

namespace moe {
namespace {

// -------------------------------------------------------------------- accept
// A warp a sequence. A node's children stand behind it, so the walk
//   next(i) = first j > i with parent_j = i and token_j = target_i
// goes once over the sequence's words, 32 nodes a ballot, kChunks ballots'
// words asked for together and the next ones while these are looked at. What
// bounds it is launch and two dependent loads (the offsets, then the words): 4
// trees of up to 8 nodes 1.7 us, 500 of up to 200 3.2 us.
constexpr int kAcceptThreads = 128;
constexpr int kChunks = 4;

__global__ void __launch_bounds__(kAcceptThreads) k_attn_accept(const AcceptArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, b = blockIdx.x * (kAcceptThreads / 32) + (threadIdx.x >> 5);
  if (b >= a.B) return;
  const int lo = __ldg(a.q_offsets + b), hi = __ldg(a.q_offsets + b + 1);
  const int held = a.seq_lens ? __ldg(a.seq_lens + b) : 0, ctx = a.context_lens[b];
  const int t0 = min(max(lo, 0), a.T), m = min(max(hi, t0), a.T) - t0;
  if (lane == 0 && (t0 != lo || m != hi - lo)) record_error(a.err, kAttnErrBounds);
  const bool alive = m > 0 && !(a.seq_lens && held < m);
  int32_t* path = a.path + (long long)b * a.P;
  int n = 0, want = -1, cur = 0, slot = 0;  // slot: lane l holds node l of the last 32
  if (alive) {
    int par[kChunks], tok[kChunks], tgt[kChunks];
    auto load = [&](int base) {
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const int i = base + u * 32 + lane;
        par[u] = -2;
        tok[u] = tgt[u] = 0;
        if (i < m) {
          par[u] = __ldg(a.parents + t0 + i);
          tok[u] = __ldg(a.tokens + t0 + i);
          tgt[u] = __ldg(a.targets + t0 + i);
        }
      }
    };
    load(0);
    want = __shfl_sync(0xffffffffu, tgt[0], 0);
    n = 1;
#pragma unroll 1
    for (int base = 0; base < m && n < a.P; base += kChunks * 32) {
      int p[kChunks], k[kChunks], g[kChunks];
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        p[u] = par[u];
        k[u] = tok[u];
        g[u] = tgt[u];
      }
      if (base + kChunks * 32 < m) load(base + kChunks * 32);
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const int i = base + u * 32 + lane;
        while (n < a.P) {
          const uint32_t hit = __ballot_sync(0xffffffffu, i > cur && p[u] == cur && k[u] == want);
          if (!hit) break;
          const int at = __ffs(hit) - 1;
          cur = base + u * 32 + at;
          want = __shfl_sync(0xffffffffu, g[u], at);
          if (lane == (n & 31)) slot = cur;
          if ((++n & 31) == 0) path[n - 32 + lane] = slot;
        }
      }
    }
  }
  const int rest = n & ~31;
  if (rest + lane < n) path[rest + lane] = slot;
  for (int i = n + lane; i < a.P; i += 32) path[i] = -1;
  if (lane == 0) {
    a.counts[b] = n;
    a.next_tokens[b] = want;
    a.context_out[b] = ctx + n;
  }
}

// ---------------------------------------------------------------------- keep
// A block takes some 16-byte columns (cache tensor, head, 8 elements)
// of one sequence's tokens, a thread a column: the words of kMoves nodes are
// asked for together, then stored. The path ascends and stands at or behind its
// places, so nothing is overwritten before it is read. Bound: memory where
// there is much to move, else launch and three dependent loads before the data
// (offsets and counts, path and table). 16 layers of 16 heads of 128, 64
// sequences of up to 9 nodes (66 MB read and written): 13.4 us, 0.73 of the copy
// rate; one layer of 4 sequences 2.2 us.
constexpr int kKeepThreads = 256;
constexpr int kKeepPath = 64;  // nodes at a time
constexpr int kMoves = 8;

__global__ void __launch_bounds__(kKeepThreads) k_attn_keep(const __grid_constant__ KeepArgs a) {
  __shared__ long long src[kKeepPath], dst[kKeepPath];  // elements
  __shared__ int stop;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, b = blockIdx.y;
  const int lo = __ldg(a.q_offsets + b), hi = __ldg(a.q_offsets + b + 1), len = __ldg(a.seq_lens + b);
  const int count = __ldg(a.counts + b);
  // the path's first words come with the lengths
  const int32_t* path = a.path + (long long)b * a.path_stride;
  int p = -1, before = -1;
  auto ask = [&](int j) {
    if (tid < kKeepPath && j < a.path_len) {
      p = __ldg(path + j);
      before = j ? __ldg(path + j - 1) : -1;
    }
  };
  ask(tid);
  const int m = max(hi - lo, 0), start = len - m;
  const bool bad = hi < lo || len < 0 || len > a.max_seq_len || count < 0 || count > min(m, a.path_len) ||
                   (count > 0 && start < 0);
  if (bad) {
    if (tid == 0) record_error(a.err, kAttnErrBounds);
    return;
  }
  const int32_t* table = a.block_table + (long long)b * a.table_stride;
  const int d8 = a.D / 8, per = a.Hk * d8, items = a.count * per;
#pragma unroll 1
  for (int base = 0; base < count; base += kKeepPath) {
    const int here = min(kKeepPath, count - base);
    if (base) ask(base + tid);
    if (tid == 0) stop = here;
    __syncthreads();
    if (tid < here) {
      const int j = base + tid;
      bool ok = p >= j && p < m && p > before;
      if (ok) {
        auto place = [&](int node, long long* at) {
          const int key = start + node, pg = key / a.page_size, page = __ldg(table + pg);
          *at = (long long)page * a.page_stride + (long long)(key - pg * a.page_size) * a.slot_stride;
          return (unsigned)page < (unsigned)a.num_pages;
        };
        ok = place(p, &src[tid]);
        if (ok) ok = place(j, &dst[tid]);
      }
      if (!ok) {
        record_error(a.err, kAttnErrBounds);
        atomicMin(&stop, tid);
      }
    }
    __syncthreads();
    const int n = stop;
    int from = 0;  // the first nodes mostly stand where they are kept
    while (from < n && src[from] == dst[from]) ++from;
    if (from < n)
      for (int it = blockIdx.x * kKeepThreads + tid; it < items; it += gridDim.x * kKeepThreads) {
        const int cache = it / per, c = it - cache * per, head = c / d8;
        uint16_t* at = static_cast<uint16_t*>(a.caches[cache]) + head * a.head_stride + (c - head * d8) * 8;
#pragma unroll 1
        for (int i = from; i < n; i += kMoves) {
          uint4 v[kMoves];
#pragma unroll
          for (int u = 0; u < kMoves; ++u)
            if (i + u < n) v[u] = *reinterpret_cast<const uint4*>(at + src[i + u]);
#pragma unroll
          for (int u = 0; u < kMoves; ++u)
            if (i + u < n) *reinterpret_cast<uint4*>(at + dst[i + u]) = v[u];
        }
      }
    if (n < here) return;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_attn_accept(const AcceptArgs& a, cudaStream_t s, bool pdl) {
  const int per = kAcceptThreads / 32;
  return launch_ex(k_attn_accept, dim3((a.B + per - 1) / per), dim3(kAcceptThreads), 0, s, pdl, a);
}

cudaError_t launch_attn_keep(const KeepArgs& a, int num_sms, cudaStream_t s, bool pdl) {
  // columns over as many blocks as stay resident together (8 an SM)
  const int items = a.count * a.Hk * (a.D / 8), most = (items + kKeepThreads - 1) / kKeepThreads;
  const int slices = std::max(1, std::min(most, (8 * num_sms + a.B - 1) / a.B));
  return launch_ex(k_attn_keep, dim3(slices, a.B), dim3(kKeepThreads), 0, s, pdl, a);
}

}  // namespace moe
