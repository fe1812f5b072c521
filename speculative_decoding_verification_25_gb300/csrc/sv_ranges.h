// Arithmetic of the attention's ranges, for the kernel and for host tests:
// the work is `total` keys, cut into equal ranges of `quota` keys, a CTA each.
// Divisions are 32 bits wide where their operands are: a 64-bit one is a
// hundred instructions at a CTA's start.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SV_HOST_DEVICE inline
#endif

namespace sv {

// Keys of a range: total / ctas rounded up, at least `least`.
SV_HOST_DEVICE long long range_quota(long long total, unsigned ctas, int least) {
  const long long top = total - 1;   // rounding up by adding could pass 32 bits
  const long long q = total <= 0 ? 0 : (top >> 32 == 0 ? (unsigned)top / ctas : top / ctas) + 1ll;
  return q > least ? q : least;
}

// How many ranges before this one a unit begins, `pos` of whose keys lie before it.
SV_HOST_DEVICE int ranges_back(int pos, long long quota) {
  return pos == 0 ? 0 : quota >= pos ? 1 : (pos - 1) / (int)quota + 1;
}

// How many ranges after this one has the key `ahead` keys past this one's start.
SV_HOST_DEVICE int ranges_ahead(long long ahead, long long quota) {
  return (int)((ahead | quota) >> 32 == 0 ? (unsigned)ahead / (unsigned)quota : ahead / quota);
}

}  // namespace sv
