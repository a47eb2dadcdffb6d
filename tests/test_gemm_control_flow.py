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
extern "C" int parts(int steps, int f32) { return f32 ? moe::reduction_parts<true>(steps) : moe::reduction_parts<false>(steps); }
extern "C" int start(int steps, int parts, int p) { return moe::part_start(steps, parts, p); }
// 0: parts begin at 0, end at `steps`, rise, and hold 1 to `most` k-steps each
extern "C" int check(int steps, int most, int f32) {
  const int n = parts(steps, f32);
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
@pytest.mark.parametrize("steps", [17, 18, 28, 29, 224, 257, 512, 513, 1025, 16384, 173_399, 173_400, 175_000, 1 << 20, (1 << 24) - 1, 1 << 24])
def test_parts_cover_long_reductions(parts, steps):
    assert parts.check(steps, 14, 1) == 0
    assert parts.check(steps, 256, 0) == 0


@pytest.mark.parametrize("f32,most", [(1, 16), (0, 256)])
def test_short_reductions_are_one_part(parts, f32, most):
    for steps in (1, 2, most - 1, most):
        assert parts.parts(steps, f32) == 1 and parts.start(steps, 1, 0) == 0 and parts.start(steps, 1, 1) == steps
    assert parts.parts(most + 1, f32) > 1


@pytest.fixture(scope="module")
def flow(tmp_path_factory):
    return _compile(str(tmp_path_factory.mktemp("flow")), """
#include <atomic>
#include <chrono>
#include <condition_variable>
#include <mutex>
#include <thread>
#include <vector>
#include "ring_flow.h"

// A meeting of n threads that gives up after a while (a thread that never comes).
struct Meeting {
  std::mutex m;
  std::condition_variable cv;
  int n, in = 0, turn = 0, kind = 0;
  bool all = true, last = true, stuck = false, mixed = false;
  bool meet(int kind_, bool ok) {
    std::unique_lock<std::mutex> l(m);
    const int mine = turn;
    if (in && kind != kind_) mixed = true;  // a vote and a plain meeting at once
    kind = kind_;
    all = all && ok;
    if (++in == n) {
      last = all; all = true; in = 0; ++turn;
      cv.notify_all();
    } else if (!cv.wait_for(l, std::chrono::seconds(5), [&] { return turn != mine || stuck; }) || stuck) {
      stuck = true;
      cv.notify_all();
      return false;
    }
    return last;
  }
};

// n consumers go through groups of stages[g] stages of 10, 11, ... rows; consumer
// c's wait number fail_at[c] (and all behind it) gives up. Sums pass on behind
// `most` additions: odd consumers put theirs, even ones add theirs. Returns 0: all
// of them left alike, 1: some did not, 2: a meeting that not all came to, or that
// some came to for a vote and some not, 3: group sums that are not the group's.
extern "C" int run(int n, int groups, const int *stages, const int *fail_at, int most) {
  Meeting meeting;
  meeting.n = n;
  std::vector<int> left(n, -1);
  std::vector<std::atomic<int>> sum(groups);
  for (auto &v : sum) v = -1000000;
  std::atomic<int> wrong{0};
  std::vector<std::thread> t;
  for (int c = 0; c < n; ++c)
    t.emplace_back([&, c] {
      int waits = 0;
      for (int g = 0; g < groups; ++g) {
        int i = 0, mine = 0, adds = 0;
        const int r = moe::sum_group<true>(
            most, [&] { return waits++ >= fail_at[c] ? -1 : i < stages[g] ? 10 + i++ : 0; }, [&] { mine = adds = 0; },
            [&](int rows) { mine += rows; adds += (rows + 15) / 16; },
            [&](bool first) {
              if (adds > most + 3) wrong = 1;
              if (c == 1 && first) sum[g] = mine;
              else if (c == 1) sum[g] += mine;
            },
            [&](bool ok) { return meeting.meet(1, ok); }, [&] { if (c == 0) sum[g] += mine; }, [&] { meeting.meet(2, true); });
        if (r < 0) { left[c] = g; return; }
        if (r != (stages[g] > 0)) wrong = 1;
        if (r) {
          if (sum[g] != 2 * (10 * stages[g] + stages[g] * (stages[g] - 1) / 2)) wrong = 1;
          meeting.meet(2, true);
        }
      }
      left[c] = meeting.meet(1, true) ? 1000 : 2000;
    });
  for (auto &x : t) x.join();
  if (meeting.stuck || meeting.mixed) return 2;
  bool some = false, every = true;
  for (int c = 0; c < n; ++c) { some |= left[c] != 1000; every &= left[c] != 1000; }
  if (some != every) return 1;
  return wrong ? 3 : 0;
}

// The waits of a producer's end after `issued` uses of a ring: parity[q], or -1 for a slot that is not waited for.
extern "C" void ends(int stages, int issued, int *parity) {
  for (int q = 0; q < stages; ++q) parity[q] = -1;
  moe::last_uses(stages, issued % stages, issued / stages, [&](int q, int p) { parity[q] = parity[q] < 0 ? p : 9; });
}
""")


def _run_flow(flow, stages, fail_at, most):
    a, b = (C.c_int * len(stages))(*stages), (C.c_int * len(fail_at))(*fail_at)
    return flow.run(len(fail_at), len(stages), a, b, most)


NEVER = 1 << 30


@pytest.mark.parametrize("most", [1, 2, 3, 100])
@pytest.mark.parametrize("stages", [[1], [0], [3, 0, 2], [0, 0, 0], [5, 1, 0, 7], [40, 2]])
def test_groups_without_failures(flow, stages, most):
    assert _run_flow(flow, stages, [NEVER] * 8, most) == 0


@pytest.mark.parametrize("most", [1, 2, 100])
@pytest.mark.parametrize("stages", [[1], [3, 0, 2], [0, 4, 0], [2, 2]])
@pytest.mark.parametrize("late", [[0], [3], [0, 7], [1, 2, 3, 4, 5, 6, 7], list(range(8))])
def test_a_wait_that_gives_up_takes_every_consumer_out(flow, stages, late, most):
    """Some consumers' waits give up, at every place where they can, the others' do not (a stage that lands just at
    the limit): all leave, and none stays at a meeting."""
    for at in range(sum(stages) + len(stages)):
        assert _run_flow(flow, stages, [at if c in late else NEVER for c in range(8)], most) == 0, at
        # ... and the others one wait later
        assert _run_flow(flow, stages, [at if c in late else at + 1 for c in range(8)], most) == 0, at


@pytest.mark.parametrize("stages", [2, 3, 7, 12])
def test_a_producer_ends_behind_its_last_loads(flow, stages):
    for issued in range(4 * stages):
        got = (C.c_int * stages)()
        flow.ends(stages, issued, got)
        want = [-1] * stages
        for use in range(issued):           # phase `use // stages` of the slot's barrier
            want[use % stages] = use // stages & 1
        assert list(got) == want, issued
