// Host helpers that the paged cache operators share: sizes, the device's
// properties and the driver's tensor map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "spec_verify.h"
#include "sv_host.h"

namespace sv {

constexpr int kMaxDevices = 64;
constexpr long long k2_31 = 1ll << 31;
// Most keys of a request over 16 bits: the attention's walk looks up to two key tiles
// (of 128 at most) past the last key, and a unit's cost past its keys, in 32 bits.
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

// What a host side keeps of each device.
struct PagedDevice {
  std::once_flag once;
  int sm_count = 0;
  EncodeTiled encode = nullptr;   // the driver's tensor map encoder
  cudaError_t error = cudaSuccess;
};
// The current device's of `devices`; nullptr if it cannot be used.  Once per device, `limits`
// sets what the kernels need.
template <typename Limits>
inline PagedDevice* current_device(PagedDevice (&devices)[kMaxDevices], Limits limits) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  PagedDevice& d = devices[dev];
  std::call_once(d.once, [&d, dev, &limits]() {
    d.error = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (d.error == cudaSuccess) d.error = limits();
    if (d.error == cudaSuccess) d.error = find_encoder(&d.encode);
  });
  return d.error == cudaSuccess ? &d : nullptr;
}

// A map of 16-bit elements for boxes of 64 columns (128 bytes, swizzled) by
// box1 (by box2): dims and boxes innermost first, pitches in bytes.
inline bool encode_map(EncodeTiled encode, CUtensorMap* map, int dtype, const void* base, int rank,
                const cuuint64_t* dims, const cuuint64_t* pitches, const cuuint32_t* box) {
  const cuuint32_t ones[3] = {1, 1, 1};
  return encode(map, dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  (cuuint32_t)rank, const_cast<void*>(base), dims, pitches, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sv
