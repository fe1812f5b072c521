// What the paged cache kernels share: device flags, the clamped view of a
// request's lengths, and the cache's geometry.
//
// The cache is [n_pages, Hk, page_size, D]: one head's part of a page is
// page_size * D consecutive elements, so an attention CTA, which reads one
// head, reads whole blocks of 1 KB (page 8, D 64) to 64 KB.
#pragma once

#include <stdint.h>

#include "sv_common.cuh"

namespace sv {

constexpr unsigned kDevLength = 32u;       // SV_DEV_BAD_LENGTH
constexpr unsigned kDevBadPage = 512u;
constexpr unsigned kDevNoPages = 1024u;
constexpr unsigned kDevTokensClipped = 2048u;
constexpr unsigned kDevTimeout = 4096u;

__device__ __forceinline__ void set_flag(unsigned* flags, unsigned bits) {
  if (flags) atomicOr(flags, bits);
}

// The checked build's test before an access of element i of n; the plain build
// takes every index for good.
__device__ __forceinline__ bool in_array(unsigned* flags, long long i, long long n) {
  if (!kChecked || (i >= 0 && i < n)) return true;
  set_flag(flags, kDevOutOfBounds);
  return false;
}

}  // namespace sv
