// Host side of the paged cache operators declared in include/spec_verify.h:
// argument checks, launch geometry and the C entry points.  Each is one
// launch on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_paged_append.cuh"
#include "sv_paged_attention.cuh"
#include "sv_paged_host.h"
#include "sv_paged_plan.cuh"

namespace {

using sv::aligned_to;
using sv::done;
using sv::encode_map;
using sv::k2_31;
using sv::kMaxDevices;
using sv::kMostKeys;
using sv::launch_early;
using sv::page_shift_of;
using sv::PagedDevice;

constexpr int kMaxCluster = 8;   // portable cluster size

PagedDevice g_paged[kMaxDevices];

// The attention kernel's variants.
struct AttentionVariant {
  const void* fn;
  int threads, smem_bytes, ctas_per_sm, keys, unit_rows;
};
template <typename E, int kD, bool kWide>
AttentionVariant variant() {
  using S = sv::AttnShape<kD, kWide>;
  return {(const void*)sv::sv_paged_attention_kernel<E, kD, kWide>, S::kThreads, S::kSmemBytes,
          S::kCtasPerSm, S::kKeys, S::kRows};
}
AttentionVariant attention_variant(int dtype, int D, bool wide) {
  if (dtype == SV_BF16) {
    if (D == 128) return wide ? variant<__nv_bfloat16, 128, true>() : variant<__nv_bfloat16, 128, false>();
    return wide ? variant<__nv_bfloat16, 64, true>() : variant<__nv_bfloat16, 64, false>();
  }
  if (D == 128) return wide ? variant<__half, 128, true>() : variant<__half, 128, false>();
  return wide ? variant<__half, 64, true>() : variant<__half, 64, false>();
}

PagedDevice* paged_device() {
  return sv::current_device(g_paged, []() {
    cudaError_t e = cudaFuncSetAttribute((const void*)sv::sv_paged_plan_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SV_MAX_PLAN_ROWS * sv::kPlanRowBytes);
    for (int i = 0; i < 8 && e == cudaSuccess; ++i) {
      const AttentionVariant v = attention_variant(i & 1 ? SV_BF16 : SV_F16, i & 2 ? 128 : 64, i & 4);
      e = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem_bytes);
    }
    return e;
  });
}

static_assert(sv::kAttnMaxCtas * sizeof(int) <= SV_ATTENTION_COUNTER_BYTES - sizeof(uint32_t),
              "the status word lies behind the tickets");

static_assert(sv::AttnShape<128, true>::kUnitCost + 2 * sv::AttnShape<128, true>::kKeys <= 512, "fits");

#ifdef SV_CHECKED
int g_naps = sv::kNaps;   // tests shorten it
#else
constexpr int g_naps = sv::kNaps;
#endif

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
  a.in_place = page_count_out == page_count || free_count_out == free_count;
  // Small plans are a chain of latencies: one CTA, a lane per token.  Large
  // ones store 8 bytes per token: up to kPlanChunk of them in a row per warp,
  // which then bisects the rows once, and CTAs until the GPU is full.
  PagedDevice* dev = paged_device();
  if (!dev) return SV_ERR_CUDA;
  int threads = 256;
  while (threads < sv::kPlanThreads && (threads < B || threads < max_tokens)) threads *= 2;
  const long long most = a.in_place ? kMaxCluster : dev->sm_count;
  const long long lanes = most * threads;
  a.chunk = 32 * (int)((max_tokens + lanes - 1) / lanes);
  if (a.chunk > sv::kPlanChunk) a.chunk = sv::kPlanChunk;
  if (a.chunk < 32) a.chunk = 32;
  const long long per_cta = (long long)(threads / 32) * a.chunk;
  long long ctas = (max_tokens + per_cta - 1) / per_cta;
  if (ctas > most) ctas = most;
  if (a.in_place)
    while (ctas & (ctas - 1)) ctas &= ctas - 1;   // cluster sizes are powers of two
  if (ctas < 1) ctas = 1;
  void* args[] = {&a};
  return done(launch_early((const void*)sv::sv_paged_plan_kernel, dim3((unsigned)ctas),
                           dim3((unsigned)threads), args, (cudaStream_t)stream,
                           (size_t)B * sv::kPlanRowBytes, a.in_place ? (unsigned)ctas : 1u));
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
  return SV_ATTENTION_COUNTER_BYTES +
         (size_t)sv::kAttnRows * (D + 2) * sizeof(float);
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
      (long long)max_pages * page_size > kMostKeys ||
      (long long)n_pages * page_size * Hk >= k2_31 ||
      q_stride < (int64_t)Hq * D || !(scale > 0.f && scale * sv::kLog2e <= 3.4e38f))
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
  PagedDevice* dev = paged_device();
  if (!dev) return SV_ERR_CUDA;
  const int G = Hq / Hk;
  // The narrow form holds 128 query rows (the G heads of a request's tokens
  // on one key head) and streams the cache with two CTAs per SM; the wide
  // form holds 256 and keeps the tensor core busier.  The host knows the
  // mean of the rows alone; both forms take requests of any length.
  // Measured (in a graph), narrow and wide: 20 rows per request (64 requests) 98 and 114 us,
  // 72 rows (256 long contexts) 964 and 1008; 64 requests of 96 rows 111 and
  // 121, 128 rows 116 and 122, 160 rows 200 and 134, 256 rows 208 and 146; 580
  // rows (37 ragged requests, D = 64) 70 and 54, 8192 rows 449 and 308.
  const bool wide = (long long)T * G > 128ll * (B > 0 ? B : 1);
  const AttentionVariant v = attention_variant(dtype, D, wide);
  const int ctas = sv::range_ctas(dev->sm_count * v.ctas_per_sm, v.unit_rows);

  sv::AttnArgs a;
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
  a.tile_tokens = 128 / G;
  a.scale_log2 = scale * sv::kLog2e;
  a.out = (char*)out;
  a.lse = lse;
  a.tickets = (int*)workspace;
  a.status = (unsigned*)((char*)workspace + SV_ATTENTION_COUNTER_BYTES) - 1;
  a.partial = (float*)((char*)workspace + SV_ATTENTION_COUNTER_BYTES);
  a.flags = flags;
  a.naps = g_naps;
  CUtensorMap q_map, k_map, v_map;
  const cuuint64_t q_dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T};
  const cuuint64_t q_pitches[2] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)G, (cuuint32_t)a.tile_tokens};
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)n_pages * Hk * page_size};
  const cuuint64_t pitches[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)(page_size < v.keys ? page_size : v.keys)};
  if (!encode_map(dev->encode, &q_map, dtype, q, 3, q_dims, q_pitches, q_box) ||
      !encode_map(dev->encode, &k_map, dtype, k_cache, 2, dims, pitches, box) ||
      !encode_map(dev->encode, &v_map, dtype, v_cache, 2, dims, pitches, box))
    return SV_ERR_CUDA;
  void* args[] = {&a, &q_map, &k_map, &v_map};
  return done(launch_early(v.fn, dim3((unsigned)ctas), dim3((unsigned)v.threads), args,
                           (cudaStream_t)stream, (size_t)v.smem_bytes));
}

int spec_paged_attention_device_errors(void* workspace, void* stream, uint32_t* flags) {
  if (!workspace || !flags) return SV_ERR_NULL;
  if (!aligned_to(workspace, 16)) return SV_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  const char* status = (const char*)workspace + SV_ATTENTION_COUNTER_BYTES - sizeof(uint32_t);
  cudaError_t e = cudaMemcpyAsync(flags, status, sizeof(uint32_t), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *flags) e = cudaMemsetAsync(workspace, 0, SV_ATTENTION_COUNTER_BYTES, st);
  return done(e);
}

#ifdef SV_CHECKED
// Tests of the checked build: after how many polls a wait inside a kernel is
// given up (0: at once); a negative number restores the limit.
void spec_checked_wait_polls(int polls) { g_naps = polls < 0 ? sv::kNaps : polls; }
#endif

int spec_stream_capture_id(void* stream, uint64_t* id) {
  if (!id) return SV_ERR_NULL;
  cudaStreamCaptureStatus state = cudaStreamCaptureStatusNone;
  unsigned long long capture = 0;
  const cudaError_t e = cudaStreamGetCaptureInfo((cudaStream_t)stream, &state, &capture);
  if (e != cudaSuccess) (void)cudaGetLastError();
  *id = e == cudaSuccess && state == cudaStreamCaptureStatusActive ? capture : 0;
  return done(e);
}

}  // extern "C"
