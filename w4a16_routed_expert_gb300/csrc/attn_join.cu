// Joins the partial results of one forward: for each (query token, query
// head) the rows that the blocks left in the workspace (maximum m_i in powers
// of two, sum l_i, output o_i relative to 2^m_i) become
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i,
//   lse = ln 2 (m + log2 sum_i 2^(m_i - m) l_i) - ln 2 * bias
// in a fixed order. One warp a row; the partials were just written, so the
// reads mostly hit L2.
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
  const int t = (int)(row / a.Hq), hq = (int)(row - (long long)t * a.Hq);

  // the row's partials of the prefix and of its own keys; the words go back to
  // zero for the next forward
  int2 ip = make_int2(0, 0), io = make_int2(0, 0);
  if (j.prefix_step) ip = j.info_prefix[row];
  if (j.own_step) io = j.info_own[row];
  __syncwarp();
  if (lane == 0) {
    if (j.prefix_step) j.info_prefix[row] = make_int2(0, 0);
    if (j.own_step) j.info_own[row] = make_int2(0, 0);
  }
  const int n = ip.y + io.y;
  auto part = [&](int i) {
    return i < ip.y ? (long long)ip.x + (long long)i * j.prefix_step
                    : (long long)io.x + (long long)(i - ip.y) * j.own_step;
  };

  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, j.part_ml[part(i)].x);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool act = lane * 4 < a.D;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const long long at = part(i);
    const float2 v = j.part_ml[at];
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
    if (act) p = *reinterpret_cast<const float4*>(j.part_o + at * j.DP + lane * 4);
    const float w = exp2_fast(v.x - ref);
    l = fmaf(w, v.y, l);
    o.x = fmaf(w, p.x, o.x);
    o.y = fmaf(w, p.y, o.y);
    o.z = fmaf(w, p.z, o.z);
    o.w = fmaf(w, p.w, o.w);
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
