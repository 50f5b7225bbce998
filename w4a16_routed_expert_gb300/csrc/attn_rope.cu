// RMS norm of query and key heads and the rotary rotation, optionally storing
// keys and values into the pages of a cache (include/moe_attention.h).
//
// Every value is read once and written once, so the bound is memory: 4 bytes
// a value. A group of 8 or 16 lanes (32 where only 8-byte accesses fit) holds
// one head, VEC elements a lane; the sum of squares is a shuffle reduction in
// the group. For
// the half layout the other element of a pair is VEC elements of another
// lane, fetched by shuffles of the packed words.
//
// out[d] = r * (x[d] * C[d] + x[pair(d)] * S[d]) with r = rsqrt(mean x^2 +
// eps) (1 without a norm), C = m cos * w[d], S = -+ m sin * w[pair(d)]: the
// norm's weights and the sign go into C and S, which a lane computes once per
// token and keeps in registers over all the heads it takes.
//
// Angles: freq is the turns per position as a 64-bit fraction, so position *
// freq modulo 2^64 is the angle's fraction of a turn, exact at any position;
// its top 32 bits as a signed number give an angle in [-pi, pi), where the
// hardware sine and cosine are within 2^-21.4 absolute, far inside the 16-bit
// rounding of the result (2^-12 relative).
#include "attn_dev.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;

template <int VEC>
struct Words;
template <>
struct Words<8> {
  using type = uint4;
};
template <>
struct Words<4> {
  using type = uint2;
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kRopeThreads) k_rope(RopeArgs a, int W, int n_chunks) {
  using Vec = typename Words<VEC>::type;
  constexpr int NW = VEC / 2;
  constexpr int U = 4;  // heads in flight per group
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long task = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(task / n_chunks);
  if (t >= a.T) return;
  const int chunk = (int)(task - (long long)t * n_chunks);
  const int gl = lane & (W - 1), grp = lane / W, ngrp = 32 / W;
  const int d0 = gl * VEC;
  const bool act = d0 < a.D;

  // this token's cosines and sines for the lane's elements
  const int half = a.rotary >> 1;
  float C0[VEC], S0[VEC];
  {
    const uint64_t pos = (uint64_t)(int64_t)__ldg(a.positions + t);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int d = d0 + e;
      C0[e] = 1.f;
      S0[e] = 0.f;
      if (d < a.rotary) {
        const bool second = a.interleaved ? (d & 1) : d >= half;
        const int i = a.interleaved ? d >> 1 : (second ? d - half : d);
        const int32_t turn = (int32_t)(uint32_t)((pos * __ldg(a.freq + i)) >> 32);
        float sn, cs;
        __sincosf((float)turn * 1.46291807926715968e-9f, &sn, &cs);  // 2 pi / 2^32
        C0[e] = cs * a.m;
        S0[e] = (second ? sn : -sn) * a.m;
      }
    }
  }
  const bool split = !a.interleaved && a.rotary > 0;  // pairs in two lanes
  int partner = lane;
  if (split && d0 < a.rotary) partner = d0 < half ? lane + half / VEC : lane - half / VEC;

  // the destination slot in the cache
  long long slot_base = -1;
  if (a.slots) {
    const long long slot = __ldg(a.slots + t);
    if (slot >= a.num_slots) {
      record_error(a.err, kAttnErrBounds);
    } else if (slot >= 0) {
      const long long page = slot / a.page_size;
      slot_base = page * a.page_stride + (slot - page * a.page_size) * a.slot_stride;
    }
  }

  const int nq = a.q ? a.Hq : 0, nk = a.k ? a.Hk : 0, nv = a.slots ? a.Hk : 0;
  const int h_begin = chunk * a.heads_per_warp, h_end = min(h_begin + a.heads_per_warp, nq + nk + nv);
  for (int sec = 0; sec < 2; ++sec) {
    const int lo = max(h_begin, sec ? nq : 0), hi = min(h_end, sec ? nq + nk : nq);
    if (lo >= hi) continue;
    const float* w = sec ? a.k_norm : a.q_norm;
    const T* src = sec ? static_cast<const T*>(a.k) + (long long)t * a.k_stride
                       : static_cast<const T*>(a.q) + (long long)t * a.q_stride;
    T* dst;
    long long hstep = a.D;
    bool store = act;
    if (!sec) {
      dst = static_cast<T*>(a.q_out) + (long long)t * a.q_out_stride;
    } else if (a.slots) {
      dst = static_cast<T*>(a.k_cache) + slot_base;
      hstep = a.head_stride;
      store = store && slot_base >= 0;
    } else {
      dst = static_cast<T*>(a.k_out) + (long long)t * a.k_out_stride;
    }
    const int h0 = sec ? nq : 0;
    float C[VEC], S[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      C[e] = C0[e];
      S[e] = S0[e];
      if (w && act) {
        const int d = d0 + e;
        int pd = d;
        if (d < a.rotary) pd = a.interleaved ? d ^ 1 : (d < half ? d + half : d - half);
        C[e] *= __ldg(w + d);
        S[e] *= __ldg(w + pd);
      }
    }
    for (int h = lo; h < hi; h += ngrp * U) {
      Vec raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = h + u * ngrp + grp;
        raw[u] = Vec{};
        if (act && hh < hi) raw[u] = *reinterpret_cast<const Vec*>(src + (long long)(hh - h0) * a.D + d0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = h + u * ngrp + grp;
        const uint32_t* rw = reinterpret_cast<const uint32_t*>(&raw[u]);
        float x[VEC], y[VEC];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const float2 f = Half16<T>::unpack(rw[i]);
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
          ss = fmaf(f.x, f.x, fmaf(f.y, f.y, ss));
          if (split) {
            const float2 p = Half16<T>::unpack(__shfl_sync(0xffffffffu, rw[i], partner));
            y[2 * i] = p.x;
            y[2 * i + 1] = p.y;
          } else {
            y[2 * i] = f.y;
            y[2 * i + 1] = f.x;
          }
        }
        float r = 1.f;
        if (w) {
          for (int o = W >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          r = rsqrtf(ss / (float)a.D + a.eps);
        }
        Vec res;
        uint32_t* ow = reinterpret_cast<uint32_t*>(&res);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          // an element that is not rotated keeps its value whatever stands beside it
          const float s0 = d0 + 2 * i < a.rotary ? y[2 * i] * S[2 * i] : 0.f;
          const float s1 = d0 + 2 * i + 1 < a.rotary ? y[2 * i + 1] * S[2 * i + 1] : 0.f;
          ow[i] = Half16<T>::pack(r * fmaf(x[2 * i], C[2 * i], s0), r * fmaf(x[2 * i + 1], C[2 * i + 1], s1));
        }
        if (store && hh < hi) *reinterpret_cast<Vec*>(dst + (long long)(hh - h0) * hstep + d0) = res;
      }
    }
  }
  // values: copied to the cache as they are
  if (nv && slot_base >= 0) {
    const int h0 = nq + nk;
    const int lo = max(h_begin, h0);
    const T* src = static_cast<const T*>(a.v) + (long long)t * a.v_stride;
    T* dst = static_cast<T*>(a.v_cache) + slot_base;
    for (int h = lo; h < h_end; h += ngrp * U) {
      Vec raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = h + u * ngrp + grp;
        if (act && hh < h_end) raw[u] = *reinterpret_cast<const Vec*>(src + (long long)(hh - h0) * a.D + d0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = h + u * ngrp + grp;
        if (act && hh < h_end) *reinterpret_cast<Vec*>(dst + (long long)(hh - h0) * a.head_stride + d0) = raw[u];
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RopeArgs& in, int num_sms, cudaStream_t s, bool pdl) {
  RopeArgs a = in;
  // 16 bytes a lane; 8 where the half layout's pairs are not a whole number of 16-byte words apart
  const int vec = (!a.interleaved && a.rotary % 16 != 0) ? 4 : 8;
  int W = 1;
  while (W * vec < a.D) W <<= 1;
  const int heads = (a.q ? a.Hq : 0) + (a.k ? a.Hk : 0) + (a.slots ? a.Hk : 0);
  // One warp takes one token's heads (its sines and cosines are computed
  // once); with few tokens the heads are spread over more warps until the
  // card has about 32 warps per SM.
  const int step = 32 / W;
  int per = heads;
  while (per > step && (long long)a.T * ((heads + per - 1) / per) < 32LL * num_sms) per = (per + 1) / 2;
  per = (per + step - 1) / step * step;
  a.heads_per_warp = per;
  const int n_chunks = (heads + per - 1) / per;
  const long long warps = (long long)a.T * n_chunks;
  const dim3 grid((unsigned)((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32)));
  if (vec == 8) return launch_ex(k_rope<T, 8>, grid, dim3(kRopeThreads), 0, s, pdl, a, W, n_chunks);
  return launch_ex(k_rope<T, 4>, grid, dim3(kRopeThreads), 0, s, pdl, a, W, n_chunks);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t s, bool pdl) {
  return bf16 ? launch<__nv_bfloat16>(a, num_sms, s, pdl) : launch<__half>(a, num_sms, s, pdl);
}

}  // namespace moe
