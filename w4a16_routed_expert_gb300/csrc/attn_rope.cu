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
// freq modulo 2^64 is the angle's fraction of a turn, off by the frequency's
// own rounding alone (2^-56 of a turn a position at most); its top 32 bits as a signed number give an angle in [-pi, pi), where the
// hardware sine and cosine are within 2^-21.4 absolute, far inside the 16-bit
// rounding of the result (2^-12 relative).
//
// Measured (FP16, 16 query and 16 key heads of 128, norm, 8192 tokens): rotate
// 28 us = 4.8 TB/s, append with the values 37 us = 5.4 TB/s (0.70 and 0.80 of
// the measured copy rate); one token 2.7 us. At 8192 tokens half of the issue
// slots are used; the warps wait for loads and for shuffles. 32 warps of two
// 512-byte loads are 32 KB in flight an SM, short of what the copy rate takes:
// but more heads in flight (U = 4: 32 us) or more warps (48 registers, spills:
// 34 us) are slower.
#include <algorithm>

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

// (x, y) products in pairs
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return ffma2(a, b, make_float2(0.f, 0.f)); }

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kRopeThreads, 4) k_rope(const RopeArgs a, int cq, int ck, int n_chunks) {
  using Vec = typename Words<VEC>::type;
  constexpr int NW = VEC / 2;
  constexpr int U = 2;  // heads in flight per group of lanes (4: 10% slower, fewer warps fit)
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int task = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)((unsigned)task / (unsigned)n_chunks);
  if (t >= a.T) return;
  int c = task - t * n_chunks;
  const int sec = c < cq ? 0 : c < cq + ck ? 1 : 2;  // queries, keys, values
  c -= sec == 0 ? 0 : sec == 1 ? cq : cq + ck;
  const int h0 = c * a.heads_per_warp, n = min(a.heads_per_warp, (sec == 0 ? a.Hq : a.Hk) - h0);
  constexpr int ngrp = 32 / W;
  const int gl = lane & (W - 1), grp = lane / W;
  const int d0 = gl * VEC;
  const bool act = d0 < a.D, rot = d0 < a.rotary;

  // the first heads are on their way while the angles are worked out
  const T* src = sec == 0 ? static_cast<const T*>(a.q) + (long long)t * a.q_stride
                          : sec == 1 ? static_cast<const T*>(a.k) + (long long)t * a.k_stride
                                     : static_cast<const T*>(a.v) + (long long)t * a.v_stride;
  const int sstep = ngrp * a.D;
  src += (h0 + grp) * a.D + d0;
  Vec raw[U];
  auto load = [&](int i) {  // heads i, i + ngrp, ...
#pragma unroll
    for (int u = 0; u < U; ++u) {
      raw[u] = Vec{};
      if (act && i + u * ngrp + grp < n) raw[u] = *reinterpret_cast<const Vec*>(src + u * sstep);
    }
    src += U * sstep;
  };
  load(0);

  // where they go
  T* dst;
  long long hstep = a.D;
  bool store = act;
  if (sec == 0) {
    dst = static_cast<T*>(a.q_out) + (long long)t * a.q_out_stride;
  } else if (a.slots) {
    const long long slot = __ldg(a.slots + t);
    if (slot >= a.num_slots) record_error(a.err, kAttnErrBounds);
    store = store && slot >= 0 && slot < a.num_slots;
    const int page = store ? (int)slot / a.page_size : 0, at = store ? (int)slot - page * a.page_size : 0;
    dst = static_cast<T*>(sec == 1 ? a.k_cache : a.v_cache) + page * a.page_stride + at * a.slot_stride;
    hstep = a.head_stride;
  } else {
    dst = static_cast<T*>(a.k_out) + (long long)t * a.k_out_stride;
  }
  dst += (h0 + grp) * hstep + d0;
  hstep *= ngrp;

  if (sec == 2) {  // values go as they are
#pragma unroll 1
    for (int i = 0; i < n; i += U * ngrp) {
      Vec cur[U];
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = raw[u];
      load(i + U * ngrp);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (store && i + u * ngrp + grp < n) *reinterpret_cast<Vec*>(dst) = cur[u];
        dst += hstep;
      }
    }
    return;
  }

  // this token's cosines and sines for the lane's elements, with the norm's
  // weights of the elements and of their pairs' other elements
  const int half = a.rotary >> 1;
  const bool split = !a.interleaved && a.rotary > 0;  // pairs in two lanes
  const bool second = d0 >= half;                     // then: the lane holds second elements
  const int partner = split && rot ? (second ? lane - half / VEC : lane + half / VEC) : lane;
  // the other elements of the pairs, from the partner's words: as they are,
  // swapped, or zeros where nothing is rotated (an element that is not keeps
  // its value whatever stands beside it)
  const uint32_t pick = !rot ? 0x4444u : split ? 0x3210u : 0x1032u;
  float2 C[NW], S[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    C[i] = make_float2(1.f, 1.f);
    S[i] = make_float2(0.f, 0.f);
  }
  if (rot) {
    const uint64_t pos = (uint64_t)(int64_t)__ldg(a.positions + t);
    auto angle = [&](uint64_t f, float* sn, float* cs) {
      __sincosf((float)(int32_t)(uint32_t)((pos * f) >> 32) * 1.46291807926715968e-9f, sn, cs);  // 2 pi / 2^32
    };
    if (a.interleaved) {
      const uint64_t* f = a.freq + (d0 >> 1);
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        float sn, cs;
        angle(__ldg(f + i), &sn, &cs);
        C[i] = make_float2(cs * a.m, cs * a.m);
        S[i] = make_float2(-sn * a.m, sn * a.m);
      }
    } else {
      const ulonglong2* f = reinterpret_cast<const ulonglong2*>(a.freq + (second ? d0 - half : d0));
      const float sm = second ? a.m : -a.m;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const ulonglong2 ff = __ldg(f + i);
        float2 sn, cs;
        angle(ff.x, &sn.x, &cs.x);
        angle(ff.y, &sn.y, &cs.y);
        C[i] = make_float2(cs.x * a.m, cs.y * a.m);
        S[i] = make_float2(sn.x * sm, sn.y * sm);
      }
    }
  }
  const float* w = sec == 0 ? a.q_norm : a.k_norm;
  if (w && act) {
    const float* wp = w + (!split || !rot ? d0 : second ? d0 - half : d0 + half);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const float2 wd = __ldg(reinterpret_cast<const float2*>(w + d0) + i);
      float2 wo = __ldg(reinterpret_cast<const float2*>(wp) + i);
      if (a.interleaved) wo = make_float2(wd.y, wd.x);
      C[i] = mul2(C[i], wd);
      S[i] = mul2(S[i], wo);
    }
  }
  const float inv_d = 1.f / (float)a.D;

#pragma unroll 1
  for (int i = 0; i < n; i += U * ngrp) {
    Vec cur[U];
#pragma unroll
    for (int u = 0; u < U; ++u) cur[u] = raw[u];
    load(i + U * ngrp);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t* rw = reinterpret_cast<const uint32_t*>(&cur[u]);
      float2 x[NW];
      float r = 1.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) x[k] = Half16<T>::unpack(rw[k]);
      if (w) {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NW; ++k) s2 = ffma2(x[k], x[k], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = W >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = rsqrtf(fmaf(ss, inv_d, a.eps));
      }
      const float2 r2 = make_float2(r, r);
      Vec res;
      uint32_t* ow = reinterpret_cast<uint32_t*>(&res);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float2 y = Half16<T>::unpack(__byte_perm(__shfl_sync(0xffffffffu, rw[k], partner), 0u, pick));
        const float2 v = mul2(r2, ffma2(x[k], C[k], mul2(y, S[k])));
        ow[k] = Half16<T>::pack(v.x, v.y);
      }
      if (store && i + u * ngrp + grp < n) *reinterpret_cast<Vec*>(dst) = res;
      dst += hstep;
    }
  }
}

template <typename T>
cudaError_t launch(const RopeArgs& in, int num_sms, cudaStream_t s, bool pdl) {
  RopeArgs a = in;
  // 16 bytes a lane; 8 where the half layout's pairs are not a whole number of 16-byte words apart
  const int vec = (!a.interleaved && a.rotary % 16 != 0) ? 4 : 8;
  const int W = (a.D <= 64 ? 64 : 128) / vec;  // lanes of a head
  const int nq = a.q ? a.Hq : 0, nk = a.k ? a.Hk : 0, nv = a.slots ? a.Hk : 0;
  // One warp takes a token's query, key or value heads, whose sines and
  // cosines it computes once; with few tokens the heads are spread over more
  // warps until the card has about 24 warps per SM.
  const int step = 32 / W;
  auto chunks = [](int n, int per) { return (n + per - 1) / per; };
  int per = std::max(nq, nk);
  while (per > step &&
         (long long)a.T * (chunks(nq, per) + chunks(nk, per) + chunks(nv, per)) < 24LL * num_sms)
    per = (per + 1) / 2;
  per = (per + step - 1) / step * step;
  a.heads_per_warp = per;
  const int cq = chunks(nq, per), ck = chunks(nk, per), n_chunks = cq + ck + chunks(nv, per);
  const long long warps = (long long)a.T * n_chunks;
  const dim3 grid((unsigned)((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32)));
  auto run = [&](auto kern) {
    return launch_ex(kern, grid, dim3(kRopeThreads), 0, s, pdl, a, cq, ck, n_chunks);
  };
  if (vec == 8) return W == 8 ? run(k_rope<T, 8, 8>) : run(k_rope<T, 8, 16>);
  return W == 16 ? run(k_rope<T, 4, 16>) : run(k_rope<T, 4, 32>);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t s, bool pdl) {
  return bf16 ? launch<__nv_bfloat16>(a, num_sms, s, pdl) : launch<__half>(a, num_sms, s, pdl);
}

}  // namespace moe
