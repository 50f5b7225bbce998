// The arithmetic of a step's running sums (attn_plan.cu), in plain C++ so that
// it can be checked without a GPU.
#pragma once

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

}  // namespace moe
