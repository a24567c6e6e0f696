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


def values(rng, most, n):
    """(t, p, q): p up to `most`; q at random, near p / t, and where p - t q is near
    the middle between two steps of the first grid, 2^-22."""
    out = []
    for t in thresholds(rng, n):
        x = t / 2.0 ** UNIT
        p = min(f32(most * rng.choice([rng.random(), 2 ** rng.uniform(-40, 0)])), 2 - 2.0 ** -23)
        k = rng.random()
        if k < 0.25:
            q = rng.random()
        elif k < 0.5:
            q = p / x * (1 + rng.choice([-1, 1]) * 2 ** rng.uniform(-26, 0))
        elif k < 0.75:
            q = p / x * rng.random()
        else:
            q = max(0.0, (p - (2 * rng.randrange(1 << 21) + 1) * 2.0 ** -23) / x)
        out.append((t, p, f32(q)))
    return out


@pytest.mark.parametrize("most,bound", [(1.0, Fraction(17, 16)), (2.0, Fraction(22, 16))])
def test_values_in_units(run, most, bound):
    """In units of 2^-45.  What the grid's step i leaves of p - t.hi q is at most
    2^-23 (half a step) and the difference's two roundings (2^-25 each for p up to 1,
    2^-24 up to 2) and t.lo q (2^-24, 2^-23): 2^-22 for p up to 1 and less than 2^-21
    up to 2, so its rounding is off by a quarter of a unit (a half); then without t.lo
    q, at most 2^-22, a quarter; the reading of the rest a half; t's two floats 2^-49
    t q, a sixteenth (an eighth).  Values of p alone: the reading."""
    cases = values(random.Random(int(most)), most, 40000)
    for (t, p, q), (_, _, got, plain) in zip(cases, run(cases)):
        v = max(Fraction(p) - Fraction(t, 1 << UNIT) * Fraction(q), Fraction(0)) * 2 ** UNIT
        assert abs(v - got) <= bound, (t, p, q, float(v), got)
        assert abs(Fraction(p) * 2 ** UNIT - plain) <= Fraction(1, 2), p


def test_values_at_the_middles_of_the_grid(run):
    """t = 1 and p - q in the middle between two steps, or beside it by less than the
    difference's own rounding."""
    rng = random.Random(7)
    cases = []
    for _ in range(30000):
        q = f32(2 ** rng.uniform(-12, -1))
        p = f32(q + (2 * rng.randrange(1 << 21) + 1) * 2.0 ** -23)
        if p <= 1:
            cases.append((1 << UNIT, p, q))
    assert len(cases) > 5000
    for (_, p, q), (_, _, got, _) in zip(cases, run(cases)):
        assert abs((Fraction(p) - Fraction(q)) * 2 ** UNIT - got) <= 1, (p, q)
