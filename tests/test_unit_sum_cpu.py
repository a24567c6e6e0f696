"""Units and positions of the latent attention in one integer (csrc/unit_sum.h),
up to the most that a call can have."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mla_chunked_context_gb300", "csrc")

HARNESS = r"""
#include <cstdio>
#include "unit_sum.h"
using mla::UnitSum;
int main() {
  long n, units, length;  // n sequences of `units` units of `length` positions
  while (std::scanf("%ld %ld %ld", &n, &units, &length) == 3) {
    uint64_t sum = 0, last = 0;
    for (long i = 0; i < n; ++i) sum += last = UnitSum::of(int(units), int(length));
    std::printf("%d %lld %d %lld\n", UnitSum::units(sum), UnitSum::positions(sum),
                UnitSum::units(sum - last), UnitSum::positions(sum - last));
  }
}
"""


def test_units_and_positions_up_to_the_most(tmp_path):
    src, exe = tmp_path / "sum.cpp", tmp_path / "sum"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    most = 2 ** 24 + 2 ** 22
    cases = [(0, 1, 1), (1, 1, 5), (5, 3, 2052), (1, 2 ** 23 - 1, 5), (1, 2 ** 23, 5), (1, 2 ** 24, 6),
             (1, most, 20), (2 ** 22, 5, 20), (65536, 256, 2052), (1, 1, 2 ** 25 - 1024 + 4)]
    got = subprocess.run([str(exe)], input="\n".join(f"{a} {b} {c}" for a, b, c in cases), text=True,
                         check=True, capture_output=True).stdout.split("\n")
    for (n, units, length), line in zip(cases, got):
        assert n * units * length < 2 ** 39
        before = max(0, n - 1)
        assert list(map(int, line.split())) == [n * units, n * units * length, before * units,
                                                before * units * length], (n, units, length)
