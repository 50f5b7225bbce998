// Joins the partial results of one forward: for each (query token, query
// head) the rows that the blocks left in the workspace (maximum m_i in powers
// of two, sum l_i, output o_i relative to 2^m_i) become
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i,
//   lse = ln 2 (m + log2 sum_i 2^(m_i - m) l_i) - ln 2 * bias
// in a fixed order. The partials were just written, so the reads mostly hit
// L2; what bounds it is the chain of two loads (where the partials are, then
// they) of the rows in flight.
#include "attn_tc.cuh"

namespace moe {
namespace {

constexpr int kJoinThreads = 256;

// DP / 8 lanes to a row, 8 values each
template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const JoinArgs j) {
  constexpr int W = DP / 8;
  pdl_trigger();
  pdl_wait();
  const AttnArgs& a = j.a;
  const int gl = threadIdx.x & (W - 1);
  const long long row = ((long long)blockIdx.x * kJoinThreads + threadIdx.x) / W;
  const bool in = row < (long long)a.T * a.Hq;

  // the row's partials of the prefix and of its own keys; the words go back to
  // zero for the next forward
  int2 ip = make_int2(0, 0), io = make_int2(0, 0);
  if (in && j.prefix_step) ip = j.info_prefix[row];
  if (in && j.own_step) io = j.info_own[row];
  __syncwarp();
  if (in && gl == 0) {
    if (j.prefix_step) j.info_prefix[row] = make_int2(0, 0);
    if (j.own_step) j.info_own[row] = make_int2(0, 0);
  }
  if (!in || ip.y < 0 || io.y < 0) return;  // stored by the one block that had all its keys
  const int n = ip.y + io.y;
  auto part = [&](int i) {
    return i < ip.y ? (long long)ip.x + (long long)i * j.prefix_step
                    : (long long)io.x + (long long)(i - ip.y) * j.own_step;
  };
  const unsigned lanes = (W == 16 ? 0xffffu : 0xffu) << (threadIdx.x & 31 & ~(W - 1));
  float m = -INFINITY;
  for (int i = gl; i < n; i += W) m = fmaxf(m, j.part_ml[part(i)].x);
#pragma unroll
  for (int o = W >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float o[8] = {};
  const bool act = gl * 8 < a.D;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const long long at = part(i);
    const float2 v = j.part_ml[at];
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f), q = p;
    if (act) {
      p = *reinterpret_cast<const float4*>(j.part_o + at * DP + gl * 8);
      q = *reinterpret_cast<const float4*>(j.part_o + at * DP + gl * 8 + 4);
    }
    const float w = exp2_fast(v.x - ref);
    l = fmaf(w, v.y, l);
    o[0] = fmaf(w, p.x, o[0]);
    o[1] = fmaf(w, p.y, o[1]);
    o[2] = fmaf(w, p.z, o[2]);
    o[3] = fmaf(w, p.w, o[3]);
    o[4] = fmaf(w, q.x, o[4]);
    o[5] = fmaf(w, q.y, o[5]);
    o[6] = fmaf(w, q.z, o[6]);
    o[7] = fmaf(w, q.w, o[7]);
  }
  const float inv = inverse_sum(l);  // a row that sees no key: zeros
  const int t = (int)(row / a.Hq), hq = (int)(row - (long long)t * a.Hq);
  if (act) {
    uint4 r;
    r.x = Half16<T>::pack(o[0] * inv, o[1] * inv);
    r.y = Half16<T>::pack(o[2] * inv, o[3] * inv);
    r.z = Half16<T>::pack(o[4] * inv, o[5] * inv);
    r.w = Half16<T>::pack(o[6] * inv, o[7] * inv);
    *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (long long)t * a.out_stride + (long long)hq * a.D + gl * 8) = r;
  }
  if (a.lse && gl == 0) a.lse[row] = log_sum<T>(m, l);
}

template <typename T>
cudaError_t launch(const JoinArgs& j, cudaStream_t s, bool pdl) {
  const long long threads = (long long)j.a.T * j.a.Hq * (j.DP / 8);
  const dim3 grid((unsigned)((threads + kJoinThreads - 1) / kJoinThreads));
  return j.DP == 128 ? launch_ex(k_attn_join<T, 128>, grid, dim3(kJoinThreads), 0, s, pdl, j)
                     : launch_ex(k_attn_join<T, 64>, grid, dim3(kJoinThreads), 0, s, pdl, j);
}

}  // namespace

cudaError_t launch_attn_join(const JoinArgs& j, bool bf16, cudaStream_t s, bool pdl) {
  return bf16 ? launch<__nv_bfloat16>(j, s, pdl) : launch<__half>(j, s, pdl);
}

}  // namespace moe
