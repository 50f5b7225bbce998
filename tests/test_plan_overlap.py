"""plan refuses lengths that stand in its own outputs (a decode loop that passes
the last step's seq_lens as context_lens, into the same tables): other blocks
read them again after they have been written, and pages would be looked up for
lengths that the step never had. The check, compiled for the CPU."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from w4a16_routed_expert_gb300 import build as B
from w4a16_routed_expert_gb300 import capi

HARNESS = """
#include "attn_plan.h"
#include "moe_attention.h"
extern "C" int overlap(const moe_attn_plan_t* p) { return moe::plan_overlaps_lengths(*p); }
"""


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("plan_overlap")
    src, so = str(d / "overlap.cpp"), str(d / "overlap.so")
    with open(src, "w") as f:
        f.write(HARNESS)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", B.INCLUDE, "-I", B.CSRC, "-o", so, src], check=True)
    lib = ctypes.CDLL(so)
    return lambda **kw: bool(lib.overlap(ctypes.byref(capi.moe_attn_plan_t(**{**OK, **kw}))))


SEQS, T = 6, 40
OK = dict(num_seqs=SEQS, num_tokens=T, max_nodes=33, context_lens=0x1000, new_lens=0x1018, parents=0x2000, state=0x3000, state_out=0x3000,
          q_offsets=0x4000, seq_lens=0x5000, positions=0x6000, slots=0x7000, tree=0x8000)
SIZE = dict(q_offsets=SEQS + 1, seq_lens=SEQS, positions=T, slots=T, tree=2 * T, state_out=SEQS + 2)


def test_apart(overlap):
    assert not overlap()
    assert not overlap(context_lens=OK["new_lens"])  # inputs may be one
    assert not overlap(num_tokens=0, max_nodes=0, positions=None, slots=None, tree=None, parents=None)
    assert not overlap(num_seqs=0, context_lens=None, new_lens=None, seq_lens=None)
    assert not overlap(max_nodes=0, tree=OK["context_lens"] + 4)  # not written
    assert not overlap(num_seqs=0, context_lens=OK["slots"] + 4, new_lens=OK["slots"] + 4)  # not read


@pytest.mark.parametrize("out", SIZE)
@pytest.mark.parametrize("lengths", ["context_lens", "new_lens"])
def test_lengths_in_an_output(overlap, lengths, out):
    at, n = OK[out], SIZE[out]
    for first, inside in ((at, True), (at + 4 * (n - 1), True), (at - 4 * (SEQS - 1), True), (at + 4 * n, False), (at - 4 * SEQS, False)):
        assert overlap(**{lengths: first}) == inside, hex(first)


def test_plan_asks_for_it():
    src = open(os.path.join(B.CSRC, "attn_api.cu")).read()
    body = src[src.index("moe_status_t moe_attn_plan("):]
    body = body[:body.index("\n}\n")]
    assert re.search(r"plan_overlaps_lengths\(\*p\)\)\s*return set_error\(MOE_ERR_INVALID_ARG", body)
    assert body.index("plan_overlaps_lengths") < body.index("launch_attn_plan")
