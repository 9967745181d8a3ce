// The range length of the 4-bit attention's work plan (kv4.cu), in plain C++:
// of the lengths m whose ranges (at most m tiles of one head each) fit the
// CTAs, about the least.  A warp tries 32 candidates at once, a lane each.
#pragma once

#ifdef __CUDACC__
#define HY_PLAN __host__ __device__ __forceinline__
#else
#define HY_PLAN inline
#endif

namespace hy {
namespace kv4 {

HY_PLAN unsigned ceil_div(unsigned a, unsigned b) { return (a + b - 1) / b; }

// Bounds of m for `total` tiles in `items` <= grid heads: an equal share (at
// least `least` tiles), and the length that always suffices, since each head
// adds at most one range to total / m.
HY_PLAN unsigned shortest_range(unsigned total, unsigned grid, unsigned least) {
  const unsigned share = ceil_div(total, grid);
  return share > least ? share : least;
}
HY_PLAN unsigned longest_range(unsigned total, unsigned grid, unsigned items, unsigned lo) {
  const unsigned m = grid > items ? ceil_div(total, grid - items) : total;
  return m > lo ? m : lo;
}

// Candidate i of 0..31: lo + floor((hi - lo) i / 31).  Every length from lo to
// hi where they are at most 31 apart, else evenly spread with both ends.
HY_PLAN unsigned range_length(unsigned lo, unsigned hi, unsigned i) {
  const unsigned d = hi - lo;
  return lo + d / 31u * i + d % 31u * i / 31u;
}

// ceil(x / m) with inv = 1 / m in FP32: the product is off by less than 1 while
// the quotient is below 2^21; larger quotients fit nowhere all the same.
HY_PLAN unsigned ranges_of(unsigned x, unsigned m, float inv) {
  unsigned r = (unsigned)((float)x * inv);
  r += r * m < x;
  r += r * m < x;
  return r;
}

}  // namespace kv4
}  // namespace hy
