// Joins the partial results of one forward: for each (query token, query
// head) the rows that the blocks left in the workspace (maximum m_i in powers
// of two, sum l_i, output o_i relative to 2^m_i) become
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i,
//   lse = ln 2 (m + log2 sum_i 2^(m_i - m) l_i) - ln 2 * bias
// in a fixed order. One warp a row; the partials were just written, so the
// reads mostly hit L2.
#include "attn_line.cuh"
#include "attn_tc.cuh"

namespace moe {
namespace {

constexpr int kJoinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const JoinArgs j) {
  pdl_trigger();
  pdl_wait();
  const AttnArgs& a = j.a;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  if (row >= (long long)a.T * a.Hq) return;
  const int t = (int)(row / a.Hq), hq = (int)(row - (long long)t * a.Hq), h = hq / a.g, hg = hq - h * a.g;

  // up to four runs of partials: of each kernel, the prefix's and the own keys'
  const float2* ml[4];
  const float* po[4];
  long long step[4];
  int count[4];
  int runs = 0, all = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const LineArgs& ln = j.line[k];
    if (ln.n_cta == 0) continue;
    const long long share = *ln.share;
    auto add = [&](long long x0, long long x1, long long base) {  // the group's tiles on the line, its first row
      if (x1 <= x0) return;
      const long long c0 = x0 / share, c1 = (x1 - 1) / share;
      const long long at = base + c0 * ln.part_rows;
      ml[runs] = ln.part_ml + at;
      po[runs] = ln.part_o + at * j.DP;
      step[runs] = ln.part_rows;
      count[runs] = (int)(c1 - c0 + 1);
      all += count[runs++];
    };
    if (ln.has_prefix) {
      const int r = t * a.g + hg, rb = r / ln.row_block;
      const long long x = ((long long)h * prefix_blocks(a, ln) + rb) * prefix_tiles(a, ln);
      add(x, x + prefix_tiles(a, ln), (long long)h * a.T * a.g + r);
    }
    if (ln.has_own) {
      const int b = min(max(a.seq_of[t], 0), a.B - 1);
      int t0;
      const int n = seq_tokens(a, b, &t0), keys = seq_keys(a, b);
      const int i = t - t0;
      if (i >= 0 && i < n) {
        const int r = i * a.g + hg, rb = r / ln.row_block;
        const int per_head = ln.own_off[b + 1] - ln.own_off[b];
        long long x = prefix_line(a, ln) + (long long)ln.own_off[b] * a.Hk + (long long)h * per_head;
        for (int q = 0; q < rb; ++q) x += (block_keys(a, ln, keys, n, q) + ln.key_tile - 1) / ln.key_tile;
        const int nt = (block_keys(a, ln, keys, n, rb) + ln.key_tile - 1) / ln.key_tile;
        add(x, x + nt, ((long long)ln.has_prefix * a.T + t0) * a.g * a.Hk + (long long)h * n * a.g + r);
      }
    }
  }

  float m = -INFINITY;
  for (int k = 0; k < runs; ++k)
    for (int i = lane; i < count[k]; i += 32) m = fmaxf(m, ml[k][i * step[k]].x);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool act = lane * 4 < a.D;
  for (int k = 0; k < runs; ++k) {
#pragma unroll 4
    for (int i = 0; i < count[k]; ++i) {
      const float2 v = ml[k][i * step[k]];
      float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
      if (act) p = *reinterpret_cast<const float4*>(po[k] + i * step[k] * j.DP + lane * 4);
      const float w = exp2_fast(v.x - ref);
      l = fmaf(w, v.y, l);
      o.x = fmaf(w, p.x, o.x);
      o.y = fmaf(w, p.y, o.y);
      o.z = fmaf(w, p.z, o.z);
      o.w = fmaf(w, p.w, o.w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees no key: zeros
  if (act) {
    uint2 r;
    r.x = Half16<T>::pack(o.x * inv, o.y * inv);
    r.y = Half16<T>::pack(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (long long)t * a.out_stride + (long long)hq * a.D + lane * 4) = r;
  }
  if (a.lse && lane == 0)
    a.lse[row] = l == 0.f ? -INFINITY : 0.693147180559945309f * (m - ProbBias<T>::value + log2f(l));
}

}  // namespace

cudaError_t launch_attn_join(const JoinArgs& j, bool bf16, cudaStream_t s, bool pdl) {
  const long long rows = (long long)j.a.T * j.a.Hq;
  const dim3 grid((unsigned)((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
  return bf16 ? launch_ex(k_attn_join<__nv_bfloat16>, grid, dim3(kJoinThreads), 0, s, pdl, j)
              : launch_ex(k_attn_join<__half>, grid, dim3(kJoinThreads), 0, s, pdl, j);
}

}  // namespace moe
