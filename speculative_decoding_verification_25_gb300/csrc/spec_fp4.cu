// Host side of the attention over the 4-bit paged cache, declared in
// include/spec_verify.h: argument checks, launch geometry and the C entry point.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_fp4_attention.cuh"
#include "sv_paged_host.h"

namespace {

using sv::aligned_to;
using sv::done;
using sv::k2_31;
using sv::launch_early;
using sv::page_shift_of;

constexpr float kLog2e = 1.44269504f;
constexpr long long kMostKeys = k2_31 - 512;

}  // namespace

extern "C" {

int spec_paged_attention_fp4(const void* q, int64_t q_stride, const void* k_codes, const void* k_scales,
                             const void* v_codes, const void* v_scales, int dtype,
                             const int32_t* block_table, const int32_t* cu_new,
                             const int32_t* kv_len, int B, int T, int Hq, int Hk, int D,
                             int page_size, int max_pages, int n_pages, float scale, float k_gain,
                             float v_gain, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, uint32_t* flags, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || B < 0 || T < 0 || Hk < 1 || Hq < Hk || Hq % Hk || Hq / Hk > 128 || Hq > 4096 ||
      (D != 64 && D != 128) || max_pages < 1 || n_pages < 1 ||
      (long long)max_pages * page_size > kMostKeys ||
      (long long)n_pages * page_size * Hk >= k2_31 || q_stride < (int64_t)Hq * D ||
      !(k_gain >= 1e-30f && k_gain <= 1e30f) || !(v_gain >= 1e-30f && v_gain <= 1e30f) ||
      !(scale > 0.f && (double)scale * kLog2e * k_gain <= 3.4e38 &&
        (double)scale * kLog2e * k_gain >= 1.2e-38))
    return SV_ERR_SHAPE;
  if (T == 0) return SV_OK;
  if (!q || !k_codes || !k_scales || !v_codes || !v_scales || (B > 0 && (!block_table || !kv_len)) ||
      !cu_new || !out || !workspace)
    return SV_ERR_NULL;
  if (!aligned_to(q, 16) || !aligned_to(k_codes, 16) || !aligned_to(k_scales, 16) ||
      !aligned_to(v_codes, 16) || !aligned_to(v_scales, 16) || !aligned_to(out, 16) ||
      !aligned_to(workspace, 16) || q_stride % 8 || !aligned_to(block_table, 4) ||
      !aligned_to(cu_new, 4) || !aligned_to(kv_len, 4) || !aligned_to(lse, 4) || !aligned_to(flags, 4))
    return SV_ERR_ALIGN;
  if (workspace_bytes < spec_paged_attention_workspace_bytes(D)) return SV_ERR_WORKSPACE;
  sv::Fp4Args a;
  a.q = (const char*)q;
  a.q_pitch = (long long)q_stride * 2;
  a.k_codes = (const char*)k_codes;
  a.k_scales = (const uint8_t*)k_scales;
  a.v_codes = (const char*)v_codes;
  a.v_scales = (const uint8_t*)v_scales;
  a.block_table = block_table;
  a.cu_new = cu_new;
  a.kv_len = kv_len;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  a.G = Hq / Hk;
  a.page_shift = shift;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.scale_log2 = scale * kLog2e * k_gain;
  a.v_gain = v_gain;
  a.out = (char*)out;
  a.lse = lse;
  a.flags = flags;
  const void* fn = dtype == SV_BF16
                       ? (D == 128 ? (const void*)sv::sv_fp4_attention_kernel<__nv_bfloat16, 128>
                                   : (const void*)sv::sv_fp4_attention_kernel<__nv_bfloat16, 64>)
                       : (D == 128 ? (const void*)sv::sv_fp4_attention_kernel<__half, 128>
                                   : (const void*)sv::sv_fp4_attention_kernel<__half, 64>);
  void* args[] = {&a};
  return done(launch_early(fn, dim3((unsigned)T, (unsigned)((Hq + sv::kFp4Warps - 1) / sv::kFp4Warps)),
                           dim3(32 * sv::kFp4Warps), args, (cudaStream_t)stream));
}

}  // extern "C"
