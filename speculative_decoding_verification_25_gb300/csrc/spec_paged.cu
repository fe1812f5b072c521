// Host side of the paged cache operators declared in include/spec_verify.h:
// argument checks, launch geometry and the C entry points.  Each is one
// launch on the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "spec_verify.h"
#include "sv_host.h"
#include "sv_paged_append.cuh"
#include "sv_paged_attention.cuh"
#include "sv_paged_plan.cuh"

namespace {

using sv::aligned_to;
using sv::launch_early;

constexpr int kMaxDevices = 64;
constexpr int kMaxCluster = 8;   // portable cluster size

struct PagedDevice {
  std::once_flag once;
  int sm_count = 0;
  cudaError_t error = cudaSuccess;
};
PagedDevice g_paged[kMaxDevices];

// SM count and the kernels' shared memory limits; once per device.
PagedDevice* paged_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  PagedDevice& d = g_paged[dev];
  std::call_once(d.once, [&d, dev]() {
    d.error = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (d.error == cudaSuccess)
      d.error = cudaFuncSetAttribute((const void*)sv::sv_paged_plan_kernel,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     SV_MAX_PLAN_ROWS * sv::kPlanRowBytes);
  });
  return d.error == cudaSuccess ? &d : nullptr;
}

// log2 of a page size, -1 if it is none
int page_shift_of(int page_size) {
  for (int s = 3; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

constexpr long long k2_31 = 1ll << 31;

int done(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

template <typename E>
const void* attention_fn(int D) {
  return D == 128 ? (const void*)sv::sv_paged_attention_kernel<E, 128>
                  : (const void*)sv::sv_paged_attention_kernel<E, 64>;
}

}  // namespace

extern "C" {

int spec_paged_plan(const int32_t* seq_len, const int32_t* num_new, const int32_t* page_count,
                    int32_t* block_table, int32_t* free_pages, const int32_t* free_count, int B,
                    int page_size, int max_pages, int n_pages, int max_tokens, int32_t* cu_new,
                    int32_t* kv_len, int32_t* slot_map, int32_t* positions,
                    int32_t* page_count_out, int32_t* free_count_out, uint32_t* flags,
                    void* stream) {
  const int shift = page_shift_of(page_size);
  if (shift < 0 || B < 0 || B > SV_MAX_PLAN_ROWS || max_pages < 1 || n_pages < 1 ||
      max_tokens < 0 || (long long)B * max_pages >= k2_31 ||
      (long long)max_pages * page_size >= k2_31 || (long long)n_pages * page_size >= k2_31)
    return SV_ERR_SHAPE;
  if ((B > 0 && (!seq_len || !num_new || !page_count || !block_table || !kv_len ||
                 !page_count_out)) ||
      !free_pages || !free_count || !cu_new || !free_count_out ||
      (max_tokens > 0 && (!slot_map || !positions)))
    return SV_ERR_NULL;
  for (const void* p : {(const void*)seq_len, (const void*)num_new, (const void*)page_count,
                        (const void*)block_table, (const void*)free_pages,
                        (const void*)free_count, (const void*)cu_new, (const void*)kv_len,
                        (const void*)slot_map, (const void*)positions,
                        (const void*)page_count_out, (const void*)free_count_out,
                        (const void*)flags})
    if (!aligned_to(p, 4)) return SV_ERR_ALIGN;
  if (!paged_device()) return SV_ERR_CUDA;
  sv::PlanArgs a;
  a.seq_len = seq_len;
  a.num_new = num_new;
  a.page_count = page_count;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.B = B;
  a.page_shift = shift;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.max_tokens = max_tokens;
  a.cu_new = cu_new;
  a.kv_len = kv_len;
  a.slot_map = slot_map;
  a.positions = positions;
  a.page_count_out = page_count_out;
  a.free_count_out = free_count_out;
  a.flags = flags;
  // one CTA up to four tokens per thread, then as many as the cluster holds
  int ctas = 1;
  while (ctas < kMaxCluster && (long long)ctas * 4 * sv::kPlanThreads < max_tokens) ctas *= 2;
  void* args[] = {&a};
  return done(launch_early((const void*)sv::sv_paged_plan_kernel, dim3((unsigned)ctas),
                           dim3(sv::kPlanThreads), args, (cudaStream_t)stream,
                           (size_t)B * sv::kPlanRowBytes, (unsigned)ctas));
}

int spec_paged_append(const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                      const int32_t* slot_map, int dtype, int T, int Hk, int D, int page_size,
                      int n_pages, void* k_cache, void* v_cache, uint32_t* flags, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || T < 0 || Hk < 1 || Hk > 4096 || (D != 64 && D != 128) || n_pages < 1 ||
      (long long)n_pages * page_size >= k2_31 || k_stride < (int64_t)Hk * D ||
      v_stride < (int64_t)Hk * D)
    return SV_ERR_SHAPE;
  if (T == 0) return SV_OK;
  if (!k_new || !v_new || !slot_map || !k_cache || !v_cache) return SV_ERR_NULL;
  if (!aligned_to(k_new, 16) || !aligned_to(v_new, 16) || !aligned_to(k_cache, 16) ||
      !aligned_to(v_cache, 16) || k_stride % 8 || v_stride % 8 || !aligned_to(slot_map, 4) ||
      !aligned_to(flags, 4))
    return SV_ERR_ALIGN;
  PagedDevice* dev = paged_device();
  if (!dev) return SV_ERR_CUDA;
  sv::AppendArgs a;
  a.k_new = (const char*)k_new;
  a.v_new = (const char*)v_new;
  a.k_pitch = (long long)k_stride * 2;
  a.v_pitch = (long long)v_stride * 2;
  a.slot_map = slot_map;
  a.T = T;
  a.Hk = Hk;
  a.page_shift = shift;
  a.head_shift = D == 128 ? 4 : 3;
  a.pieces = Hk << a.head_shift;
  a.n_slots = (long long)n_pages * page_size;
  a.k_cache = (char*)k_cache;
  a.v_cache = (char*)v_cache;
  a.flags = flags;
  // a thread per piece while that leaves SMs idle, then 8 resident CTAs per SM
  const long long all = (long long)T * a.pieces;
  long long ctas = (all + sv::kAppendThreads - 1) / sv::kAppendThreads;
  if (ctas > dev->sm_count * 8ll) ctas = dev->sm_count * 8ll;
  const long long step = ctas * sv::kAppendThreads;
  a.step_tokens = (int)(step / a.pieces);
  a.step_pieces = (int)(step % a.pieces);
  void* args[] = {&a};
  return done(launch_early((const void*)sv::sv_paged_append_kernel, dim3((unsigned)ctas),
                           dim3(sv::kAppendThreads), args, (cudaStream_t)stream));
}

size_t spec_paged_attention_workspace_bytes(int D) {
  if (D != 64 && D != 128) return 0;
  return SV_ATTENTION_COUNTER_BYTES;
}

int spec_paged_attention(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                         int dtype, const int32_t* block_table, const int32_t* cu_new,
                         const int32_t* kv_len, int B, int T, int Hq, int Hk, int D, int page_size,
                         int max_pages, int n_pages, float scale, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, uint32_t* flags, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || B < 0 || T < 0 || Hk < 1 || Hq < Hk || Hq % Hk || Hq / Hk > 128 || Hq > 4096 ||
      (D != 64 && D != 128) || max_pages < 1 || n_pages < 1 ||
      (long long)max_pages * page_size >= k2_31 || (long long)n_pages * page_size >= k2_31 ||
      q_stride < (int64_t)Hq * D || !(scale > 0.f && scale <= 3.4e38f))
    return SV_ERR_SHAPE;
  if (T == 0) return SV_OK;
  if (!q || !k_cache || !v_cache || (B > 0 && (!block_table || !kv_len)) || !cu_new || !out ||
      !workspace)
    return SV_ERR_NULL;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(out, 16) || !aligned_to(workspace, 16) || q_stride % 8 ||
      !aligned_to(block_table, 4) || !aligned_to(cu_new, 4) || !aligned_to(kv_len, 4) ||
      !aligned_to(lse, 4) || !aligned_to(flags, 4))
    return SV_ERR_ALIGN;
  if (workspace_bytes < spec_paged_attention_workspace_bytes(D)) return SV_ERR_WORKSPACE;
  sv::AttnArgs a;
  a.q = (const char*)q;
  a.q_pitch = (long long)q_stride * 2;
  a.k_cache = (const char*)k_cache;
  a.v_cache = (const char*)v_cache;
  a.block_table = block_table;
  a.cu_new = cu_new;
  a.kv_len = kv_len;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  a.page_shift = shift;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.scale = scale;
  a.out = (char*)out;
  a.lse = lse;
  a.flags = flags;
  const long long warps = (long long)T * Hq;
  void* args[] = {&a};
  return done(launch_early(
      dtype == SV_BF16 ? attention_fn<__nv_bfloat16>(D) : attention_fn<__half>(D),
      dim3((unsigned)((warps * 32 + sv::kAttnThreads - 1) / sv::kAttnThreads)),
      dim3(sv::kAttnThreads), args, (cudaStream_t)stream));
}

}  // extern "C"
