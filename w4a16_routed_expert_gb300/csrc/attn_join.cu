// Joins the partial results of one forward: for each (query token, query
// head) the rows that the blocks left in the workspace (reference logit m_i,
// sum l_i and output o_i of weights taken against it) become
//   out = sum_i w_i o_i / sum_i w_i l_i,  w_i = e^(scale (m_i - m)),  m = max_i m_i,
//   lse = scale m + ln sum_i w_i l_i - ln 2 * bias
// in a fixed order. The partials were just written, so the reads mostly hit
// L2; what bounds it is the chain of two loads (where the partials are, then
// they) of the rows in flight.
#include "attn_tc.cuh"

namespace moe {
namespace {

constexpr int kJoinThreads = 256;

// A warp a row, DP / 8 lanes to a partial and 8 values a lane, so 2 (4 at
// DP 64) partials side by side; a partial's maximum, sum and row are loaded
// together and taken into a running result, which the lane groups then join.
template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const JoinArgs j) {
  constexpr int W = DP / 8, G = 32 / W;
  constexpr int U = 2;  // partials in flight per lane group
  pdl_trigger();
  pdl_wait();
  const AttnArgs& a = j.a;
  const int lane = threadIdx.x & 31, gl = lane & (W - 1), grp = lane / W;
  const long long row = (long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  if (row >= (long long)a.T * a.Hq) return;

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
  if (ip.y < 0 || io.y < 0) return;  // stored by the one block that had all its keys
  const int n = ip.y + io.y;
  const bool act = gl * 8 < a.D;
  float m = -INFINITY, l = 0.f;
  float o[8] = {};
  const float sc = a.scale * kLog2e;
  // m and the running sums move to max(m, mi); -inf stays -inf
  auto scale_to = [&](float mn, float mi) { return mi == mn ? 1.f : exp2_fast((mi - mn) * sc); };
#pragma unroll 1
  for (int i = grp; i < n; i += G * U) {
    float2 v[U];
    float4 p[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = i + u * G;
      p[u] = q[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      v[u] = make_float2(-INFINITY, 0.f);
      if (k < n) {
        const long long at = k < ip.y ? (long long)ip.x + (long long)k * j.prefix_step
                                      : (long long)io.x + (long long)(k - ip.y) * j.own_step;
        v[u] = j.part_ml[at];
        if (act) {
          p[u] = *reinterpret_cast<const float4*>(j.part_o + at * DP + gl * 8);
          q[u] = *reinterpret_cast<const float4*>(j.part_o + at * DP + gl * 8 + 4);
        }
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mn = fmaxf(mn, v[u].x);
    const float f = scale_to(mn, m);
    m = mn;
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = scale_to(mn, v[u].x);
      l = fmaf(w, v[u].y, l);
      o[0] = fmaf(w, p[u].x, o[0]);
      o[1] = fmaf(w, p[u].y, o[1]);
      o[2] = fmaf(w, p[u].z, o[2]);
      o[3] = fmaf(w, p[u].w, o[3]);
      o[4] = fmaf(w, q[u].x, o[4]);
      o[5] = fmaf(w, q[u].y, o[5]);
      o[6] = fmaf(w, q[u].z, o[6]);
      o[7] = fmaf(w, q[u].w, o[7]);
    }
  }
#pragma unroll
  for (int s = W; s < 32; s <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, s), l2 = __shfl_xor_sync(0xffffffffu, l, s);
    const float mn = fmaxf(m, m2), f = scale_to(mn, m), f2 = scale_to(mn, m2);
    // the lower group's share first, on both sides
    const bool lower = (lane & s) == 0;
    l = lower ? fmaf(l2, f2, l * f) : fmaf(l, f, l2 * f2);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o2 = __shfl_xor_sync(0xffffffffu, o[e], s);
      o[e] = lower ? fmaf(o2, f2, o[e] * f) : fmaf(o[e], f, o2 * f2);
    }
    m = mn;
  }
  const float inv = inverse_sum(l);  // a row that sees no key: zeros
  const int t = (int)(row / a.Hq), hq = (int)(row - (long long)t * a.Hq);
  if (act && grp == 0) {
    uint4 r;
    r.x = Half16<T>::pack(o[0] * inv, o[1] * inv);
    r.y = Half16<T>::pack(o[2] * inv, o[3] * inv);
    r.z = Half16<T>::pack(o[4] * inv, o[5] * inv);
    r.w = Half16<T>::pack(o[6] * inv, o[7] * inv);
    *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (long long)t * a.out_stride + (long long)hq * a.D + gl * 8) = r;
  }
  if (a.lse && lane == 0) a.lse[row] = log_sum<T>(m, l, a.scale);
}

template <typename T>
cudaError_t launch(const JoinArgs& j, cudaStream_t s, bool pdl) {
  const long long rows = (long long)j.a.T * j.a.Hq;
  const dim3 grid((unsigned)((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
  return j.DP == 128 ? launch_ex(k_attn_join<T, 128>, grid, dim3(kJoinThreads), 0, s, pdl, j)
                     : launch_ex(k_attn_join<T, 64>, grid, dim3(kJoinThreads), 0, s, pdl, j);
}

}  // namespace

cudaError_t launch_attn_join(const JoinArgs& j, bool bf16, cudaStream_t s, bool pdl) {
  return bf16 ? launch<__nv_bfloat16>(j, s, pdl) : launch<__half>(j, s, pdl);
}

}  // namespace moe
