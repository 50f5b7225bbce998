// Attention over the paged cache, the plain way: one warp for each (query
// token, query head), one key at a time, everything in FP32. Every row reads
// every key it sees by itself.
#include "attn_dev.cuh"

namespace moe {
namespace {

template <typename T>
__global__ void __launch_bounds__(128) k_attn_simple(AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)a.T * a.Hq) return;
  const int t = (int)(row / a.Hq), hq = (int)(row % a.Hq), hk = hq / a.g;
  int b = 0, t0 = 0, n = 0;
  for (; b < a.B; ++b) {
    n = seq_tokens(a, b, &t0);
    if (t >= t0 && t < t0 + n) break;
  }
  const int seen = b < a.B ? keys_seen(a, seq_keys(a, b), n, t - t0) : 0;
  const T* qp = static_cast<const T*>(a.q) + (long long)t * a.q_stride + (long long)hq * a.D;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < 4; ++i) q[i] = lane + 32 * i < a.D ? Half16<T>::to_float(qp[lane + 32 * i]) * a.scale : 0.f;
  float m = -INFINITY, l = 0.f;
  const int total = b < a.B ? a.prefix_len + seen : 0;
  for (int j = 0; j < total; ++j) {
    const bool own = j >= a.prefix_len;
    const int jj = own ? j - a.prefix_len : j;
    const int32_t* tab = own ? a.block_table + (long long)b * a.table_stride : a.prefix_pages;
    const int page = page_in_cache(a, __ldg(tab + jj / a.page_size));
    const long long at = (long long)page * a.page_stride + (jj % a.page_size) * a.slot_stride + hk * a.head_stride;
    const T* kp = static_cast<const T*>(a.k_cache) + at;
    const T* vp = static_cast<const T*>(a.v_cache) + at;
    float s = 0.f;
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.D) s = fmaf(q[i], Half16<T>::to_float(kp[lane + 32 * i]), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float c = expf(m - ref), p = expf(s - ref);
    l = l * c + p;
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.D) o[i] = fmaf(p, Half16<T>::to_float(vp[lane + 32 * i]), o[i] * c);
    m = mn;
  }
  T* op = static_cast<T*>(a.out) + (long long)t * a.out_stride + (long long)hq * a.D;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.D) op[lane + 32 * i] = T(o[i] * inv);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attn_simple(const AttnArgs& a, bool bf16, cudaStream_t s) {
  const long long rows = (long long)a.T * a.Hq;
  const dim3 grid((unsigned)((rows + 3) / 4));
  return bf16 ? launch_ex(k_attn_simple<__nv_bfloat16>, grid, dim3(128), 0, s, false, a)
              : launch_ex(k_attn_simple<__half>, grid, dim3(128), 0, s, false, a);
}

}  // namespace moe
