"""Which words of a drafted token's row the attention kernels read, by their own
arithmetic compiled for the CPU. A row may be a part of a wider one (a slice of
an array's columns), and the last row's words then end where the array does."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from w4a16_routed_expert_gb300 import build as B

HARNESS = r"""
#include "attn_tree.h"
namespace {
struct Row {  // notes the furthest word that is read
  const uint32_t* at;
  int* most;
  uint32_t operator[](int w) const {
    if (w > *most) *most = w;
    return w < 0 ? 0 : at[w];
  }
};
}
// the windows of 32 keys from key k0 on that a row of a sequence of n keys, m of them new, takes
extern "C" int windows(const uint32_t* row, int max_q_len, int n, int m, int k0, int count, uint32_t* out) {
  int most = -1;
  const int words = moe::tree_row_words(max_q_len);
  for (int i = 0; i < count; ++i)
    out[i] = moe::low_bits(n - k0 - 32 * i) & moe::tree_window(Row{row, &most}, words, k0 + 32 * i - (n - m));
  return most;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("tree_rows")
    src, so = str(d / "rows.cpp"), str(d / "rows.so")
    with open(src, "w") as f:
        f.write(HARNESS)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", B.CSRC, "-o", so, src], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("wider", [0, 1, 5])
@pytest.mark.parametrize("max_q_len", [1, 8, 31, 32, 33, 64, 100, 1024])
def test_no_word_behind_the_widest_tree_is_read(lib, max_q_len, wider):
    rng = np.random.default_rng(max_q_len)
    words = -(-max_q_len // 32)
    for m in sorted({1, max_q_len // 2 + 1, max_q_len}):
        for context in (-m, -1, 0, 1, 31, 33, 63, 127, 200):
            n = max(context + m, 0)
            row = rng.integers(0, 1 << 32, words + wider + 8, dtype=np.uint64).astype(np.uint32)  # (as much as any window asks for)
            bits = (row[:, None] >> np.arange(32, dtype=np.uint32) & 1).astype(bool).ravel()
            sees = np.zeros(n + 160, dtype=bool)
            sees[:n] = [True if j < n - m else bits[j - (n - m)] for j in range(n)]
            for k0 in range(0, max(n, 1), 64):  # tiles of 64 keys, and of 128
                out = np.zeros(4, dtype=np.uint32)
                most = lib.windows(row.ctypes.data_as(ctypes.c_void_p), max_q_len, n, m, k0, 4,
                                   out.ctypes.data_as(ctypes.c_void_p))
                assert most < words, (m, n, k0)
                got = (out[:, None] >> np.arange(32, dtype=np.uint32) & 1).astype(bool).ravel()
                np.testing.assert_array_equal(got, sees[k0:k0 + 128])
