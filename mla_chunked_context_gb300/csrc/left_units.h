// What verification sums of a row, p or max(p - t q, 0), in units of 2^-45, and
// the threshold t (host code compiles it too, without contraction of products and
// sums, for its test).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MLA_LEFT_FN __device__ __forceinline__
#else
#include <cmath>
#include <cstring>
#define MLA_LEFT_FN inline
#endif

namespace mla {

#ifdef __CUDACC__
MLA_LEFT_FN float add_once(float a, float b) { return __fadd_rn(a, b); }
MLA_LEFT_FN float fma_once(float a, float b, float c) { return __fmaf_rn(a, b, c); }
MLA_LEFT_FN uint32_t bits_of(float x) { return __float_as_uint(x); }
MLA_LEFT_FN float to_float(uint64_t x) { return __ull2float_rn(x); }
MLA_LEFT_FN float to_float(int64_t x) { return __ll2float_rn(x); }
#else
MLA_LEFT_FN float add_once(float a, float b) { return a + b; }
MLA_LEFT_FN float fma_once(float a, float b, float c) { return std::fma(a, b, c); }
MLA_LEFT_FN uint32_t bits_of(float x) {
  uint32_t u;
  std::memcpy(&u, &x, 4);
  return u;
}
MLA_LEFT_FN float to_float(uint64_t x) { return float(x); }
MLA_LEFT_FN float to_float(int64_t x) { return float(x); }
#endif

// A number in two floats: |lo| is at most half a step of hi.
struct Two {
  float hi, lo;
};

// Values in units of 2^-45 (0 <= w < 2): w = hi * 2^-22 + lo * 2^-45.
constexpr float GRID = 2.f, CARRY = 3.f, FINE = 1.5f / 4194304.f;
constexpr uint32_t GRID_BITS = 0x40000000u, CARRY_BITS = 0x40400000u, FINE_BITS = 0x34C00000u;
constexpr uint64_t ONE = uint64_t(1) << 45;
MLA_LEFT_FN int64_t units(uint32_t hi, uint32_t lo) {
  return (int64_t(int32_t(hi)) << 23) + int32_t(lo);
}
// A sum of units as a number, to 2^-49 of it (exactly below 2^48).
MLA_LEFT_FN Two number(uint64_t v) {
  const float hi = to_float(v);
  const float lo = to_float(int64_t(v - uint64_t(hi)));
  constexpr float UNIT = 1.f / 35184372088832.f;
  return {hi * UNIT, lo * UNIT};
}

// Adds one value, max(p - t q, 0) or (without Q) p, to hi and lo.  With Q the grid's
// step i comes from a difference that was rounded twice, so what it leaves, p - i -
// t q, may be twice half a step: a second step carries that over before the rest is
// read off.  That rest has two roundings, of 2^-47 each for p up to 1.
template <bool Q>
MLA_LEFT_FN void add_left(Two t, float p, float q, uint32_t &hi, uint32_t &lo) {
  if (!Q) {
    const float g = add_once(p, GRID);
    hi += bits_of(g) - GRID_BITS;
    lo += bits_of(add_once(add_once(p, -add_once(g, -GRID)), FINE)) - FINE_BITS;
    return;
  }
  const float d = fma_once(-t.lo, q, fma_once(-t.hi, q, p));
  const float g = add_once(d, GRID);
  const float rest = fma_once(-t.lo, q, fma_once(-t.hi, q, add_once(p, -add_once(g, -GRID))));
  const float c = add_once(rest, CARRY);
  const float f = add_once(add_once(rest, -add_once(c, -CARRY)), FINE);
  if (d > 0.f) {
    hi += bits_of(g) - GRID_BITS;
    hi += bits_of(c) - CARRY_BITS;
    lo += bits_of(f) - FINE_BITS;
  }
}
template <bool Q>
MLA_LEFT_FN int64_t left_of(Two t, float p, float q) {
  uint32_t hi = 0, lo = 0;
  add_left<Q>(t, p, q, hi, lo);
  return units(hi, lo);
}

}  // namespace mla
