// Host helpers that the paged cache operators share: sizes, the device's
// properties and the driver's tensor map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_host.h"

namespace sv {

constexpr int kMaxDevices = 64;
constexpr long long k2_31 = 1ll << 31;
// Most keys of a request: the attention's walk looks up to two key tiles (of
// 128 at most) past the last key, and a unit's cost past its keys, in 32 bits.
constexpr long long kMostKeys = k2_31 - 512;

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

inline int done(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

// log2 of a page size, -1 if it is none
inline int page_shift_of(int page_size) {
  for (int s = 3; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

inline cudaError_t find_encoder(EncodeTiled* encode) {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
  cudaError_t e =
      cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
  if (e == cudaSuccess && found != cudaDriverEntryPointSuccess) e = cudaErrorSymbolNotFound;
  *encode = (EncodeTiled)fn;
  return e;
}

}  // namespace sv
