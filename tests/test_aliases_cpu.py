"""Outputs that share memory with an input, another output or the workspace are refused: all pairs of an entry
point, through the C ABI with made-up addresses (refused calls read nothing), and the test of two layouts against
counting their bytes."""
import os
import shutil
import subprocess

import pytest

from async_rl_b200 import _lib
from async_rl_b200.build import build
from tests.test_layer_refusals_cpu import ARG, BWD, FWD, QK, QKB, _call

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def pairs(outs, ins):
    return [(o, x) for i, o in enumerate(outs) for x in outs[:i] + ins]


SAME = dict(Hq=4, Hkv=4, q_ld=1024, k_ld=1024, v_ld=1024)  # query and key rows of one shape
BWD_SAME = dict(SAME, do_ld=1024, dq_ld=1024, dk_ld=1024, dv_ld=1024)


@pytest.mark.parametrize("out,other", pairs(["out", "lse", "st", "ws"], ["q", "k", "v", "qo", "ko", "kl"]))
def test_attn_fwd(lib, out, other):
    base = {**FWD, **SAME, "kl": 200 << 20}
    assert _call(lib.bi_attn_fwd, base, **{out: base[other]}) == ARG


@pytest.mark.parametrize("out,other", pairs(["dq", "dk", "dv", "st", "ws"],
                                            ["do", "q", "k", "v", "out", "lse", "qo", "ko", "kl"]))
def test_attn_bwd(lib, out, other):
    base = {**BWD, **BWD_SAME, "kl": 200 << 20}
    assert _call(lib.bi_attn_bwd, base, **{out: base[other]}) == ARG


QK_SAME = dict(Hq=4, Hkv=4, q_ld=1024, k_ld=1024)


@pytest.mark.parametrize("out,other", pairs(["qo", "ko", "st"], ["q", "k", "gq", "gk", "pos", "inv"]))
def test_qk_norm_rope(lib, out, other):
    base = {**QK, **QK_SAME, "qo_ld": 1024, "ko_ld": 1024}
    assert _call(lib.bi_qk_norm_rope, base, **{out: base[other]}) == ARG


@pytest.mark.parametrize("out,other", pairs(["dq", "dk", "dgq", "dgk", "st", "ws"],
                                            ["dqo", "dko", "q", "k", "gq", "gk", "pos", "inv"]))
def test_qk_norm_rope_bwd(lib, out, other):
    base = {**QKB, **QK_SAME, "dqo_ld": 1024, "dko_ld": 1024, "dq_ld": 1024, "dk_ld": 1024}
    assert _call(lib.bi_qk_norm_rope_bwd, base, **{out: base[other]}) == ARG


@pytest.mark.parametrize("shift", [512, 1024 + 16, 62 * 2048 + 1024 + 16, -512, -(63 * 2048 + 1024) + 16])
def test_partial_overlaps(lib, shift):
    """64 rows of 1024 bytes, 2048 apart, against rows of the same shape: half of a row shared, 16 bytes more than
    the gap behind a row (the first, the last but one), and 16 bytes of the last row alone."""
    base = {**BWD, **BWD_SAME}
    assert _call(lib.bi_attn_bwd, base, dk=base["q"] + shift) == ARG


PROGRAM = r"""
#include "host.h"
#include <cstdio>
#include <random>
#include <set>
using namespace bi::host;
int main() {
  std::mt19937 r(1);
  auto pick = [&](int lo, int hi) { return lo + static_cast<int>(r() % (hi - lo + 1)); };
  int hits = 0, misses = 0;
  for (int i = 0; i < 300000; ++i) {
    Span s[2];
    for (Span& x : s) {
      x.row = pick(1, 6);
      x.rows = pick(0, 7);
      x.ld = x.row + pick(0, 12);
      x.at = 1000 + pick(0, 60);
    }
    if (i % 2) s[1].ld = s[0].ld >= s[1].row ? s[0].ld : s[1].ld;  // slices of one buffer
    std::set<uintptr_t> bytes;
    bool want = false;
    for (uint64_t j = 0; j < s[0].rows; ++j)
      for (uint64_t e = 0; e < s[0].row; ++e) bytes.insert(s[0].at + j * s[0].ld + e);
    for (uint64_t j = 0; j < s[1].rows; ++j)
      for (uint64_t e = 0; e < s[1].row; ++e) want |= bytes.count(s[1].at + j * s[1].ld + e) != 0;
    if (overlap(s[0], s[1]) != want || overlap(s[1], s[0]) != want) {
      std::printf("wrong: %d\n", i);
      return 1;
    }
    ++(want ? hits : misses);
  }
  std::printf("%d %d\n", hits, misses);
  return hits > 50000 && misses > 50000 ? 0 : 2;
}
"""


def test_overlap_against_counting_bytes(tmp_path):
    gxx = shutil.which("g++")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    if gxx is None or not os.path.exists(os.path.join(cuda, "include", "cuda.h")):
        pytest.skip("no host compiler or CUDA headers")
    src = tmp_path / "overlap.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "overlap"
    # optimised, so that the header's CUDA calls, which nothing here uses, are not linked
    subprocess.run([gxx, "-O2", "-std=c++17", "-I", os.path.join(ROOT, "async_rl_b200", "csrc"), "-I",
                    os.path.join(cuda, "include"), "-o", str(exe), str(src)], check=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True)
    assert p.returncode == 0, p.stdout
