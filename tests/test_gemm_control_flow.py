"""Host checks of the control flow of the BF16 products' kernels: the plain C++
headers that the kernels include, compiled for the CPU."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a16_mixture_experts_moe_b200", "csrc")


def _compile(tmp, source):
    cxx = shutil.which("g++")
    assert cxx, "g++ is part of the toolchain"
    src, lib = os.path.join(tmp, "t.cpp"), os.path.join(tmp, "t.so")
    with open(src, "w") as f:
        f.write(source)
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-fwrapv", "-shared", "-fPIC", "-pthread", "-I", CSRC, src,
                    "-o", lib], check=True)
    return C.CDLL(lib)


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    return _compile(str(tmp_path_factory.mktemp("parts")), """
#include "gemm_parts.h"
extern "C" int parts(int steps) { return moe::reduction_parts<true>(steps); }
extern "C" int whole(int steps) { return moe::reduction_parts<false>(steps); }
extern "C" int start(int steps, int parts, int p) { return moe::part_start(steps, parts, p); }
// 0: parts begin at 0, end at `steps`, rise, and hold 1 to `most` k-steps each
extern "C" int check(int steps, int most) {
  const int n = moe::reduction_parts<true>(steps);
  if (moe::part_start(steps, n, 0) != 0) return 1;
  if (moe::part_start(steps, n, n) != steps) return 2;
  for (int p = 0; p < n; ++p) {
    const int len = moe::part_start(steps, n, p + 1) - moe::part_start(steps, n, p);
    if (len < 1 || len > most) return 3;
  }
  return 0;
}
""")


# up to 2^24 k-steps of 64: 2^30 rows in one group
@pytest.mark.parametrize("steps", [17, 18, 28, 29, 224, 1025, 16384, 173_399, 173_400, 175_000, 1 << 20, (1 << 24) - 1, 1 << 24])
def test_parts_cover_long_reductions(parts, steps):
    assert parts.check(steps, 14) == 0


@pytest.mark.parametrize("steps", [1, 2, 15, 16])
def test_short_reductions_are_one_part(parts, steps):
    assert parts.parts(steps) == 1 and parts.start(steps, 1, 0) == 0 and parts.start(steps, 1, 1) == steps


@pytest.mark.parametrize("steps", [1, 17, 1 << 24])
def test_16_bit_outputs_are_one_part(parts, steps):
    assert parts.whole(steps) == 1
