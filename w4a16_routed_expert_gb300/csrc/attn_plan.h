// The arithmetic of a step's running sums (attn_plan.cu) and a check of its
// arguments, in plain C++ so that they can be run without a GPU.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MOE_PLAN_FN __host__ __device__ __forceinline__
#else
#define MOE_PLAN_FN inline
#endif

namespace moe {

constexpr int kPlanMost = 1 << 30;  // sums stop here

MOE_PLAN_FN int plan_least(int x, int y) { return x < y ? x : y; }
// x and y from 0 to 2^31 - 1: their sum fits 32 bits without a sign, and 32 with
// one again once it is cut. (A sum of two at the bound has no room in a signed
// one: places reckoned from it would lie before the outputs.)
MOE_PLAN_FN int plan_add(int x, int y) {
  const unsigned sum = (unsigned)x + (unsigned)y;
  return (int)(sum < (unsigned)kPlanMost ? sum : (unsigned)kPlanMost);
}

// What a sequence asks for.
struct PlanAsk {
  int m;     // tokens
  int need;  // pages beyond those it holds
  int back;  // pages it gives back
  bool valid;
};
MOE_PLAN_FN PlanAsk plan_ask(int T, int max_nodes, int table_stride, int page_size, int ctx, int fresh, int held) {
  PlanAsk k;
  const int some = fresh > 0 ? fresh : 0;
  const long long keys = (long long)ctx + some, room = (long long)table_stride * page_size;
  k.valid = fresh >= -1 && held >= 0 && held <= table_stride &&
            (fresh < 0 || (ctx >= 0 && keys <= (room < (1LL << 30) ? room : 1LL << 30))) &&
            (max_nodes == 0 || fresh <= max_nodes);
  k.m = plan_least(some, T + 1);
  k.need = 0;
  if (k.valid && fresh >= 0) {
    const int more = (int)((keys + page_size - 1) / page_size) - held;
    k.need = more > 0 ? more : 0;
  }
  k.back = k.valid && fresh < 0 ? held : 0;
  return k;
}

// Whether the lengths stand in an output: every block reads them more than once,
// when others have stored theirs already. Plan: moe_attn_plan_t.
template <typename Plan>
inline bool plan_overlaps_lengths(const Plan& p) {
  const long long B = p.num_seqs, T = p.num_tokens, words = (p.max_nodes + 31) / 32;
  const struct {
    const void* at;
    long long n;
  } out[] = {{p.q_offsets, B + 1}, {p.seq_lens, B}, {p.positions, T}, {p.slots, T}, {p.tree, T * words}, {p.state_out, B + 2}};
  const int32_t* const in[] = {p.context_lens, p.new_lens};
  for (const int32_t* lengths : in)
    for (const auto& o : out) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(lengths), y = reinterpret_cast<uintptr_t>(o.at);
      if (lengths && B > 0 && o.at && o.n > 0 && x < y + (uintptr_t)o.n * 4 && y < x + (uintptr_t)B * 4) return true;
    }
  return false;
}

}  // namespace moe
