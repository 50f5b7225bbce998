"""The running sums of a step's plan, by the kernel's own arithmetic compiled for
the CPU and in the kernel's order: a thread's sequences, a warp's threads, the
block's warps. Lengths out of range at the sizes that the header allows stop at
the sums' bound and never pass below zero (as 32 bits do where a sum wraps),
because places in the outputs are reckoned from them. (On a GPU a wrapped sum
would store before the outputs.)"""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from w4a16_routed_expert_gb300 import build as B

HARNESS = r"""
#include "attn_plan.h"
extern "C" void sums(int T, int max_nodes, int table_stride, int page_size, int B, const int* ctx, const int* fresh, const int* held,
                     int* at /* [3][B + 1] */) {
  constexpr int kThreads = 256, kWarps = kThreads / 32;
  const int per = (B + kThreads - 1) / kThreads;
  for (int i = 0; i < 3; ++i) {
    auto asked = [&](int b) {
      const moe::PlanAsk k = moe::plan_ask(T, max_nodes, table_stride, page_size, ctx[b], fresh[b], held[b]);
      return i == 0 ? k.m : i == 1 ? k.need : k.back;
    };
    int incl[kThreads], part[kWarps];
    for (int t = 0; t < kThreads; ++t) {
      incl[t] = 0;
      for (int b = t * per; b < B && b < (t + 1) * per; ++b) incl[t] = moe::plan_add(incl[t], asked(b));
    }
    for (int o = 1; o < 32; o <<= 1)
      for (int t = kThreads - 1; t >= 0; --t)
        if ((t & 31) >= o) incl[t] = moe::plan_add(incl[t], incl[t - o]);
    for (int w = 0; w < kWarps; ++w) part[w] = incl[w * 32 + 31];
    int total = 0;
    for (int w = 0; w < kWarps; ++w) total = moe::plan_add(total, part[w]);
    for (int t = 0; t < kThreads; ++t) {
      int base = t & 31 ? incl[t - 1] : 0;
      for (int w = 0; w < t / 32; ++w) base = moe::plan_add(base, part[w]);
      for (int b = t * per; b < B && b < (t + 1) * per; ++b) {
        at[i * (B + 1) + b] = base;
        base = moe::plan_add(base, asked(b));
      }
    }
    at[i * (B + 1) + B] = total;
  }
}
extern "C" int most() { return moe::kPlanMost; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("plan_sums")
    src, so = str(d / "sums.cpp"), str(d / "sums.so")
    with open(src, "w") as f:
        f.write(HARNESS)
    # (-fwrapv: what the GPU's 32-bit adds do)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", B.CSRC, "-o", so, src], check=True)
    return ctypes.CDLL(so)


def run(lib, T, max_nodes, stride, page, ctx, fresh, held):
    n = len(ctx)
    at = np.zeros((3, n + 1), dtype=np.int32)
    arrays = [np.asarray(x, dtype=np.int32) for x in (ctx, fresh, held)]
    lib.sums(T, max_nodes, stride, page, n, *[x.ctypes.data_as(ctypes.c_void_p) for x in arrays], at.ctypes.data_as(ctypes.c_void_p))
    # the same in 64 bits: sums of what is not negative, cut where they stop
    ctx, fresh, held = (np.asarray(x, dtype=np.int64) for x in (ctx, fresh, held))
    keys = ctx + np.maximum(fresh, 0)
    valid = (fresh >= -1) & (held >= 0) & (held <= stride) & ((fresh < 0) | ((ctx >= 0) & (keys <= min(stride * page, 1 << 30))))
    if max_nodes:
        valid &= fresh <= max_nodes
    asked = [np.minimum(np.maximum(fresh, 0), T + 1), np.where(valid & (fresh >= 0), np.maximum(-(-keys // page) - held, 0), 0),
             np.where(valid & (fresh < 0), held, 0)]
    want = np.stack([np.minimum(np.concatenate([[0], np.cumsum(a)]), lib.most()) for a in asked])
    np.testing.assert_array_equal(at, want)
    return at


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("n", [1, 255, 256, 257, 1000, 1793, 2048, 3850, 4096])
@pytest.mark.parametrize("T", [0, 5, 1 << 20, 1 << 21, (1 << 22) - 1, 1 << 22])
def test_lengths_out_of_range(lib, T, n):
    run(lib, T, 0, 64, 16, [0] * n, [BIG] * n, [0] * n)
    at = run(lib, T, 1024, 64, 16, [5] * n, [T + 7 + i % 3 for i in range(n)], [0] * n)
    assert (np.diff(at) >= 0).all() and at.min() == 0  # so that no place is before an output


@pytest.mark.parametrize("n", [2, 300, 2048, 4096])
def test_pages_out_of_range(lib, n):
    run(lib, 1 << 22, 0, BIG, 16, [0] * n, [-1] * n, [BIG - i for i in range(n)])  # given back
    run(lib, 1 << 22, 0, BIG, 16, [1 << 30 if i % 2 else (1 << 30) - 40 for i in range(n)], [i % 41 for i in range(n)], [0] * n)  # needed


def test_lengths_in_range(lib):
    rng = np.random.default_rng(1)
    for n in (1, 31, 513, 4096):
        ctx, fresh = rng.integers(0, 900, n), rng.integers(-1, 60, n)
        run(lib, 1 << 18, 64, 64, 16, ctx, fresh, -(-ctx // 16) + rng.integers(0, 2, n))
        run(lib, 1000, 0, 64, 16, ctx - 3, fresh - 2, rng.integers(-2, 70, n))  # some of each kind out of range
