// Units of the latent attention and the positions of them, summed together in
// one 64-bit integer, so that one scan over the sequences adds up both (host
// code compiles it too, for its test).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MLA_SUM_FN __host__ __device__ __forceinline__
#else
#define MLA_SUM_FN inline
#endif

namespace mla {

// Units are rows / 64 rounded up for each sequence with new tokens: a call's
// 2^30 rows and 65535 * 64 tokens make at most 2^24 + 2^22, which 25 bits hold.
// Positions (of 64 keys of a unit) have the other 39: at 2000 clocks each on 76
// clusters 2^39 are two hours of work.
struct UnitSum {
  static constexpr int POSITION_BITS = 39;
  static constexpr uint64_t MASK = (uint64_t(1) << POSITION_BITS) - 1;
  MLA_SUM_FN static uint64_t of(int units, int length) {  // units of `length` positions each
    return (uint64_t(units) << POSITION_BITS) | (uint64_t(units) * uint64_t(length));
  }
  MLA_SUM_FN static int units(uint64_t sum) { return int(sum >> POSITION_BITS); }
  MLA_SUM_FN static long long positions(uint64_t sum) { return (long long)(sum & MASK); }
};

}  // namespace mla
