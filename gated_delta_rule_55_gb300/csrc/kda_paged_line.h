// The line of key tiles that attention over a paged cache cuts among its CTAs
// (kda_paged_attn.cu).  Plain integer arithmetic, so that the host can compile it too.
#pragma once

#ifdef __CUDACC__
#define KDA_LINE_FN __host__ __device__ __forceinline__
#else
#define KDA_LINE_FN inline
#endif

namespace kda {

constexpr int kCtas = 152;  // one per SM

// Sums of the line's units, none of them negative, stop here.  A line this long is not worked
// on: offsets in order are never this long (paged_tc_index_ok), overlapping ones can be, and a
// sum that wrapped would put an item's parts behind the last CTA's.
constexpr int kLineTooLong = 0x7fffffff;

KDA_LINE_FN int line_add(int a, int b) {
  const unsigned s = (unsigned)a + (unsigned)b;
  return s < (unsigned)kLineTooLong ? (int)s : kLineTooLong;
}

// The first unit of CTA c's stretch of a line of `total` units.
KDA_LINE_FN int stretch(int total, int c) {
  const int q = (int)((unsigned)total / kCtas), more = total - q * kCtas;
  return q * c + (c < more ? c : more);
}

// The CTA whose stretch holds a unit.
KDA_LINE_FN int stretch_of(int total, int unit) {
  const int q = (int)((unsigned)total / kCtas), more = total - q * kCtas;  // q + 1 units each
  return unit < more * (q + 1) ? unit / (q + 1)
                               : more + (unit - more * (q + 1)) / (q > 1 ? q : 1);
}

}  // namespace kda
