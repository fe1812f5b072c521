// Host side of the attention over the 4-bit paged cache, declared in
// include/spec_verify.h: argument checks, launch geometry and the C entry point.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_fp4_attention.cuh"
#include "sv_fp4_rows.cuh"
#include "sv_paged_host.h"

namespace {

using sv::aligned_to;
using sv::done;
using sv::k2_31;
using sv::kMaxDevices;
using sv::launch_early;
using sv::page_shift_of;
using sv::PagedDevice;

// Most keys of a request: the walk looks up to two key tiles past the last key, and a
// unit's cost, which is higher here than over 16 bits, past its keys, in 32 bits.
constexpr long long kMostFp4Keys = k2_31 - 1024;
template <typename S>
constexpr bool fits = S::kUnitCost + 2 * S::kKeys <= k2_31 - kMostFp4Keys && kMostFp4Keys % S::kKeys == 0;
static_assert(fits<sv::Fp4Shape<64, 16>> && fits<sv::Fp4Shape<64, 32>> && fits<sv::Fp4Shape<128, 16>> &&
                  fits<sv::Fp4Shape<128, 32>>, "fits");
static_assert(fits<sv::Fp4RowsShape<64, false>> && fits<sv::Fp4RowsShape<64, true>> &&
                  fits<sv::Fp4RowsShape<128, false>> && fits<sv::Fp4RowsShape<128, true>>, "fits");

PagedDevice g_fp4[kMaxDevices];

struct Variant {
  const void* fn;
  int threads, smem_bytes, ctas_per_sm, unit_rows, rows;   // rows: of a query tile
};
template <typename E, int kD, int kRows>
Variant variant() {
  using S = sv::Fp4Shape<kD, kRows>;
  return {(const void*)sv::sv_fp4_attention_kernel<E, kD, kRows>, S::kThreads, S::kSmemBytes, S::kCtasPerSm, S::kRows, kRows};
}
template <typename E, int kD, bool kWide>
Variant rows_variant() {
  using S = sv::Fp4RowsShape<kD, kWide>;
  return {(const void*)sv::sv_fp4_rows_attention_kernel<E, kD, kWide>, S::kThreads, S::kSmemBytes, S::kCtasPerSm, S::kRows, 128};
}
enum Form { kFew16, kFew32, kNarrow, kWide, kForms };
template <typename E, int kD>
Variant variant_of(Form form) {
  return form == kFew16    ? variant<E, kD, 16>()
         : form == kFew32  ? variant<E, kD, 32>()
         : form == kNarrow ? rows_variant<E, kD, false>()
                           : rows_variant<E, kD, true>();
}
Variant variant_of(int dtype, int D, Form form) {
  if (dtype == SV_BF16)
    return D == 128 ? variant_of<__nv_bfloat16, 128>(form) : variant_of<__nv_bfloat16, 64>(form);
  return D == 128 ? variant_of<__half, 128>(form) : variant_of<__half, 64>(form);
}

PagedDevice* fp4_device() {
  return sv::current_device(g_fp4, []() {
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 4 * kForms && e == cudaSuccess; ++i) {
      const Variant v = variant_of(i & 1 ? SV_BF16 : SV_F16, i & 2 ? 128 : 64, (Form)(i / 4));
      e = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem_bytes);
    }
    return e;
  });
}

// A map of the codes' rows, one for a token and key head, in boxes of `box` rows.
bool encode_codes(const PagedDevice& d, CUtensorMap* map, const void* base, int D, long long rows, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)D / 2, (cuuint64_t)rows};
  const cuuint64_t pitches[1] = {(cuuint64_t)D / 2};
  const cuuint32_t boxes[2] = {(cuuint32_t)D / 2, (cuuint32_t)box}, ones[2] = {1, 1};
  return d.encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, pitches, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

#ifdef SV_CHECKED
int g_naps = sv::kNaps;   // tests shorten it
#else
constexpr int g_naps = sv::kNaps;
#endif

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
      (long long)max_pages * page_size > kMostFp4Keys ||
      (long long)n_pages * page_size * Hk >= k2_31 || q_stride < (int64_t)Hq * D ||
      !(k_gain >= 1e-30f && k_gain <= 1e30f) || !(v_gain >= 1e-30f && v_gain <= 1e30f) ||
      !(scale > 0.f && (double)scale * sv::kLog2e * k_gain <= 3.4e38 &&
        (double)scale * sv::kLog2e * k_gain >= 1.2e-38))
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
  PagedDevice* dev = fp4_device();
  if (!dev) return SV_ERR_CUDA;
  const int G = Hq / Hk;
  // The host knows the mean of a request's rows (the G heads of its tokens on one key
  // head) alone; every form takes requests of any length.  Measured, 64 requests
  // over contexts of 203 to 4099, microseconds:
  //            4 rows  16 rows  20 rows  32 rows  48 rows  128 rows  160 rows  256 rows
  //   16 rows      73       74      123      125      174
  //   32 rows      80       82       90       91      185
  //   narrow       98      100      102      102      106       116       195       202
  //   wide                                                      149       177       231
  // and one token of 8 rows over contexts of 60 k to 131 k: 120, 124, 175, 241.
  const long long rows = (long long)T * G, requests = B > 0 ? B : 1;
  const Form form = rows > 128 * requests               ? kWide
                    : G > 32 || rows > 32 * requests    ? kNarrow
                    : G > 16 || rows > 16 * requests    ? kFew32
                                                        : kFew16;
  const Variant v = variant_of(dtype, D, form);
  const int ctas = sv::range_ctas(dev->sm_count * v.ctas_per_sm, v.unit_rows);

  sv::Fp4Args a;
  a.block_table = block_table;
  a.cu_new = cu_new;
  a.kv_len = kv_len;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  a.G = G;
  a.page_shift = shift;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.tile_tokens = v.rows / G;
  a.scale_log2 = (float)((double)scale * sv::kLog2e * k_gain);
  a.out = (char*)out;
  a.lse = lse;
  a.tickets = (int*)workspace;
  a.status = (unsigned*)((char*)workspace + SV_ATTENTION_COUNTER_BYTES) - 1;
  a.partial = (float*)((char*)workspace + SV_ATTENTION_COUNTER_BYTES);
  a.flags = flags;
  a.naps = g_naps;
  a.v_gain = v_gain;
  a.q = (const char*)q;
  a.q_pitch = (long long)q_stride * 2;
  a.k_scales = (const char*)k_scales;
  a.v_scales = (const char*)v_scales;
  const long long cache_rows = (long long)n_pages * Hk * page_size;
  const int box = page_size < 128 ? page_size : 128;
  CUtensorMap q_map, k_map, v_map;
  if (!encode_codes(*dev, &k_map, k_codes, D, cache_rows, box) || !encode_codes(*dev, &v_map, v_codes, D, cache_rows, box))
    return SV_ERR_CUDA;
  if (form <= kFew32) {
    void* args[] = {&a, &k_map, &v_map};
    return done(launch_early(v.fn, dim3((unsigned)ctas), dim3((unsigned)v.threads), args, (cudaStream_t)stream,
                             (size_t)v.smem_bytes));
  }
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T};
  const cuuint64_t pitches[2] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)G, (cuuint32_t)a.tile_tokens};
  if (!sv::encode_map(dev->encode, &q_map, dtype, q, 3, dims, pitches, q_box)) return SV_ERR_CUDA;
  void* args[] = {&a, &q_map, &k_map, &v_map};
  return done(launch_early(v.fn, dim3((unsigned)ctas), dim3((unsigned)v.threads), args, (cudaStream_t)stream,
                           (size_t)v.smem_bytes));
}

#ifdef SV_CHECKED
void spec_checked_wait_polls_fp4(int polls) { g_naps = polls < 0 ? sv::kNaps : polls; }
#endif

}  // extern "C"
