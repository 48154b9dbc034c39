"""A warp that gives up a wait in the ring of streamed weights does not leave its block's other warps at a barrier: the walk through
the stages that the kernel uses (csrc/stages.h), compiled for the host with threads as warps (no GPU needed)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_histogram_gb300", "csrc")

# Stage i has come for all warps but `who`, which gives up at stage `at` and raises the flag; `depth` stages had been asked for by
# then, later ones never come, and a wait for one of those gives up once the flag is up. A barrier gives up after two seconds.
PROGRAM = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <thread>
#include <vector>
#include "stages.h"

constexpr int WARPS = 8;
struct Barrier {
  std::mutex m;
  std::condition_variable cv;
  int here = 0, turn = 0;
  bool stuck = false;
  void meet() {
    std::unique_lock<std::mutex> l(m);
    if (stuck) return;
    const int mine = turn;
    if (++here == WARPS) {
      here = 0;
      ++turn;
      cv.notify_all();
    } else if (!cv.wait_for(l, std::chrono::seconds(2), [&] { return turn != mine || stuck; })) {
      stuck = true;
      cv.notify_all();
    }
  }
};

// What the walk replaces: a warp that gives up leaves
template <typename Wait, typename Use, typename Meet>
bool leaving(int total, int per_group, const Wait &wait, const Use &use, const Meet &meet) {
  for (int i = 0, k = 0; i < total; ++i) {
    if (!wait(i)) return false;
    use(i);
    if (++k < per_group) continue;
    k = 0;
    meet(true);
  }
  return true;
}

int main(int, char **a) {
  const int total = atoi(a[1]), per = atoi(a[2]), who = atoi(a[3]), at = atoi(a[4]), depth = atoi(a[5]);
  const bool leave = atoi(a[6]);
  Barrier bar;
  std::mutex m;
  bool flag = false;
  std::vector<int> used(WARPS), met(WARPS), oks(WARPS), good(WARPS);
  std::vector<std::thread> warps;
  for (int w = 0; w < WARPS; ++w)
    warps.emplace_back([&, w] {
      auto wait = [&](int i) {
        if (w == who && i == at) {
          std::lock_guard<std::mutex> l(m);
          return !(flag = true);
        }
        if (at < 0 || i < at + depth) return true;
        for (;;) {
          std::lock_guard<std::mutex> l(m);
          if (flag) return false;
        }
      };
      auto use = [&](int) { ++used[w]; };
      auto meet = [&](bool ok) { bar.meet(); ++met[w]; good[w] += ok; };
      oks[w] = leave ? leaving(total, per, wait, use, meet) : moe::through_stages(total, per, wait, use, meet);
    });
  for (auto &t : warps) t.join();
  if (bar.stuck) {
    puts("stuck");
    return 0;
  }
  for (int w = 0; w < WARPS; ++w) printf("%d %d %d %d\n", used[w], met[w], good[w], oks[w]);
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    at = tmp_path_factory.mktemp("stages")
    (at / "main.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{CSRC}", str(at / "main.cpp"), "-o", str(at / "main")], check=True)

    def call(total, per, who, stage, depth, leave=False):
        out = subprocess.run([str(at / "main"), *map(str, (total, per, who, stage, depth, int(leave)))], capture_output=True, text=True,
                             check=True, timeout=60).stdout
        return "stuck" if out.startswith("stuck") else [tuple(map(int, line.split())) for line in out.splitlines()]
    return call


@pytest.mark.parametrize("total,per", [(0, 3), (1, 1), (6, 2), (12, 4), (30, 1)])
def test_nobody_gives_up(run, total, per):
    assert run(total, per, -1, -1, 0) == [(total, total // per, total // per, 1)] * 8


@pytest.mark.parametrize("total,per,who,stage,depth", [(1, 1, 0, 0, 1), (6, 2, 3, 2, 1), (6, 2, 7, 5, 4), (12, 4, 0, 0, 3), (12, 4, 5, 11, 1),
                                                       (30, 1, 2, 9, 2), (8, 8, 1, 3, 5)])
def test_one_gives_up(run, total, per, who, stage, depth):
    """It meets the others as often as they meet; groups that it did not finish are not good to it, and what never came is not used."""
    got = run(total, per, who, stage, depth)
    for w, (used, met, good, ok) in enumerate(got):
        mine = stage if w == who else min(total, stage + depth)
        assert (used, met, good, ok) == (mine, total // per, mine // per, int(mine == total)), (w, got)


def test_leaving_would_keep_the_others(run):
    """Warp 3 gives up at stage 2, and stage 3, which ends the group, has come for the others."""
    assert run(6, 2, 3, 2, 2, leave=True) == "stuck"
    assert run(6, 2, 3, 2, 2) == [(2 if w == 3 else 4, 3, 1 if w == 3 else 2, 0) for w in range(8)]
