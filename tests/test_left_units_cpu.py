"""The numbers that verification sums with draft rows (csrc/left_units.h), compiled
for the host: the threshold t in two floats, and values max(p - t q, 0) in units of
2^-45, against exact fractions."""

import math
import os
import random
import struct
import subprocess
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mla_chunked_context_gb300", "csrc")
UNIT = 45               # bits behind the point

HARNESS = r"""
#include <cstdio>
#include "left_units.h"
using namespace mla;
int main() {
  unsigned long long t;
  float p, q;
  while (std::scanf("%llu %a %a", &t, &p, &q) == 3) {
    const Two w = number(t);
    std::printf("%a %a %lld %lld\n", w.hi, w.lo, (long long)left_of<true>(w, p, q),
                (long long)left_of<false>(w, p, q));
  }
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    folder = tmp_path_factory.mktemp("left")
    src, exe = folder / "left.cpp", folder / "left"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def call(cases):
        """(t in units, p, q) -> (hi, lo, units of max(p - t q, 0), units of p)"""
        text = "\n".join(f"{t} {p.hex()} {q.hex()}" for t, p, q in cases)
        out = subprocess.run([str(exe)], input=text, text=True, check=True, capture_output=True).stdout.split("\n")
        return [(float.fromhex(a), float.fromhex(b), int(c), int(d)) for a, b, c, d in map(str.split, out[:-1])]
    return call


def f32(x):
    return struct.unpack("f", struct.pack("f", x))[0]


def half_step(x):
    """Of a float32: half the distance to its neighbours."""
    return Fraction(2) ** (math.frexp(x)[1] - 25)


def thresholds(rng, n):
    """1, a little more, a few, and up to the most: 1023 siblings, sums below 512."""
    most = (1 + 1022 * 512) << UNIT
    out = [1 << UNIT, (1 << UNIT) + 1, (3 << UNIT) - 1, 1024 << UNIT, 1201 << UNIT, most]
    while len(out) < n:
        k = rng.random()
        x = 1.0 if k < 0.2 else 1 + rng.random() * rng.choice([1e-6, 1, 4]) if k < 0.8 else 2 ** rng.uniform(0, 18.99)
        out.append(min(most, (1 << UNIT) if k < 0.2 else int(x * 2.0 ** UNIT) + rng.randrange(1 << 20)))
    return out


def test_threshold_in_two_floats(run):
    """hi is the nearest float32 (lo at most half a step of it), and what lo leaves
    out is half a step of lo: 2^-49 of t; nothing below 2^48 units (t < 8)."""
    ts = thresholds(random.Random(1), 20000)
    for t, (hi, lo, _, _) in zip(ts, run([(t, 0.0, 0.0) for t in ts])):
        exact = Fraction(t, 1 << UNIT)
        assert abs(lo) <= half_step(hi), t
        off = abs(Fraction(hi) + Fraction(lo) - exact)
        assert off <= exact / 2 ** 49 and (off == 0 or t >= 1 << 48), t
