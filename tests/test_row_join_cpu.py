"""The join of a row's values over the threads that share it (csrc/row_join.h),
run by host threads in the order that is worst for it: after each join's
barrier one of the threads stands still until all the others wait at the next
one.  A buffer that is written again too early then hands it a wrong value."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mla_chunked_context_gb300", "csrc")

# A piece of work is some tiles, a maximum joined for each, and at its end the
# sum of what they left.  BY_TILE: buffers chosen by the tile's number instead,
# a sum taking that of the tile to come.
HARNESS = r"""
#include <atomic>
#include <cstdio>
#include <pthread.h>
#include <sched.h>
#include <thread>
#include <vector>
#include "row_join.h"

constexpr int THREADS = 256, ROW = 5;
constexpr int TIDS[4] = {ROW, ROW ^ 64, ROW ^ 128, ROW ^ 192};

int main() {
  const std::vector<int> pieces = {1, 2, 1, 1, 3, 4, 2, 2, 5, 1};
  int joins = 0;
  for (int n : pieces) joins += n + 1;
  int wrong = 0;
  for (int slow = 0; slow < 4; ++slow) {
    std::vector<float> buffers(2 * THREADS, -1.f);
    std::atomic<int> arrived{0}, bad{0};
    pthread_barrier_t meet;
    pthread_barrier_init(&meet, nullptr, 4);
    auto run = [&](int who) {
      mla::RowJoin<THREADS> join(buffers.data(), TIDS[who]);
      int done = 0;
      auto barrier = [&] {
        ++arrived;
        pthread_barrier_wait(&meet);
        ++done;
        if (who == slow && done < joins)  // until the other three are at the next barrier
          while (arrived.load() < 4 * done + 3) sched_yield();
      };
      auto value = [](int j, int w) { return float(100 * j + w * 7 % 4); };
      int j = 0, g = 0;
      for (int n : pieces) {
        for (int t = 0; t <= n; ++t, ++j) {
          const bool sum = t == n;
#ifdef BY_TILE
          join.at = (g & 1) * THREADS;
#endif
          const float got = join(value(j, who), barrier, [&](float x, float y) {
            return sum ? x + y : x > y ? x : y;
          });
          float want = value(j, 0);
          for (int w = 1; w < 4; ++w)
            want = sum ? want + value(j, w) : want > value(j, w) ? want : value(j, w);
          if (got != want) ++bad;
          if (!sum) ++g;
        }
      }
    };
    std::vector<std::thread> threads;
    for (int w = 0; w < 4; ++w) threads.emplace_back(run, w);
    for (auto &t : threads) t.join();
    pthread_barrier_destroy(&meet);
    wrong += bad;
  }
  std::printf("%d\n", wrong);
}
"""


def wrong_joins(tmp_path, *flags):
    src, exe = tmp_path / "join.cpp", tmp_path / "join"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", "-I", CSRC, *flags, str(src), "-o", str(exe)],
                   check=True)
    return int(subprocess.run([str(exe)], check=True, capture_output=True, timeout=120).stdout)


def test_every_join_sees_its_own_values(tmp_path):
    assert wrong_joins(tmp_path) == 0


def test_buffers_by_tile_would_not_do(tmp_path):
    """A sum and the next tile's maximum in one buffer: the harness sees it."""
    assert wrong_joins(tmp_path, "-DBY_TILE") > 0


def test_the_kernel_joins_through_it_alone():
    """All of the kernel's accesses to the buffers are RowJoin's."""
    text = open(os.path.join(CSRC, "sm103_latent.cu")).read()
    uses = [line.strip() for line in text.splitlines() if "xmax" in line]
    assert len(uses) == 3, uses   # where they lie, where they end, the object
    assert "RowJoin<STHREADS> row_join(xmax, tid);" in uses
