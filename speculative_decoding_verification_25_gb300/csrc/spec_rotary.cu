// Host side of the rotated appends and of the 4-bit cache's append and read,
// declared in include/spec_verify.h: argument checks, launch geometry and the C
// entry points.  Each is one launch on the caller's stream.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_paged_host.h"
#include "sv_rotary.cuh"

namespace {

using sv::aligned_to;
using sv::done;
using sv::k2_31;
using sv::launch_early;
using sv::page_shift_of;

// Gains keep scales times gains, and six times them, far inside float32.
bool gain_ok(float g) { return g >= 1e-30f && g <= 1e30f; }
bool power_of_two(float g) {
  int e;
  return frexpf(g, &e) == 0.5f;
}

const void* rotary_kernel(int dtype, int D, bool fp4) {
  if (dtype == SV_BF16) {
    if (D == 128)
      return fp4 ? (const void*)sv::sv_rotary_kernel<__nv_bfloat16, 128, true>
                 : (const void*)sv::sv_rotary_kernel<__nv_bfloat16, 128, false>;
    return fp4 ? (const void*)sv::sv_rotary_kernel<__nv_bfloat16, 64, true>
               : (const void*)sv::sv_rotary_kernel<__nv_bfloat16, 64, false>;
  }
  if (D == 128)
    return fp4 ? (const void*)sv::sv_rotary_kernel<__half, 128, true>
               : (const void*)sv::sv_rotary_kernel<__half, 128, false>;
  return fp4 ? (const void*)sv::sv_rotary_kernel<__half, 64, true>
             : (const void*)sv::sv_rotary_kernel<__half, 64, false>;
}

// What both appends take, as it comes.
sv::RotaryArgs rotary_args(const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                           const float* cos_sin, int max_positions, int rotary_dim, int interleaved,
                           const int32_t* slot_map, int T, int Hq, int Hk, void* q_out, uint32_t* flags) {
  sv::RotaryArgs a = {};
  a.q = (const char*)q;
  a.k_new = (const char*)k_new;
  a.v_new = (const char*)v_new;
  a.positions = positions;
  a.table = cos_sin;
  a.slot_map = slot_map;
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  a.max_positions = max_positions;
  a.rot = rotary_dim;
  a.neighbours = interleaved != 0;
  a.q_out = (char*)q_out;
  a.flags = flags;
  return a;
}

int launch_rotary(sv::RotaryArgs& a, int dtype, int D, bool fp4, int64_t q_stride, int64_t k_stride,
                  int64_t v_stride, int64_t out_stride, int page_size, int n_pages, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  a.page_shift = page_shift_of(page_size);
  const bool turns = a.positions || a.table;
  if (a.page_shift < 0 || a.T < 0 || a.Hk < 1 || a.Hk > 4096 || a.Hq < 0 || a.Hq > 4096 ||
      (D != 64 && D != 128) || n_pages < 1 || (long long)n_pages * page_size >= k2_31 ||
      k_stride < (int64_t)a.Hk * D || v_stride < (int64_t)a.Hk * D ||
      (a.Hq > 0 && (q_stride < (int64_t)a.Hq * D || out_stride < (int64_t)a.Hq * D)) ||
      (turns && (a.max_positions < 1 || a.rot < 32 || a.rot > D || a.rot % 32)) ||
      (!turns && a.Hq > 0))
    return SV_ERR_SHAPE;
  if (a.T == 0) return SV_OK;
  if (!a.k_new || !a.v_new || !a.slot_map || !a.k_cache || !a.v_cache ||
      (turns && (!a.positions || !a.table)) || (a.Hq > 0 && (!a.q || !a.q_out)) ||
      (fp4 && (!a.k_scale || !a.v_scale)))
    return SV_ERR_NULL;
  if (!aligned_to(a.k_new, 16) || !aligned_to(a.v_new, 16) || !aligned_to(a.k_cache, 16) ||
      !aligned_to(a.v_cache, 16) || k_stride % 8 || v_stride % 8 || !aligned_to(a.slot_map, 4) ||
      !aligned_to(a.positions, 4) || !aligned_to(a.table, 16) || !aligned_to(a.flags, 4) ||
      (a.Hq > 0 && (!aligned_to(a.q, 16) || !aligned_to(a.q_out, 16) || q_stride % 8 || out_stride % 8)))
    return SV_ERR_ALIGN;
  if (!turns) a.rot = 0;
  a.q_pitch = (long long)q_stride * 2;
  a.k_pitch = (long long)k_stride * 2;
  a.v_pitch = (long long)v_stride * 2;
  a.out_pitch = (long long)out_stride * 2;
  a.n_slots = (long long)n_pages * page_size;
  const int warps = sv::kRotaryThreads / 32, heads = sv::kRotaryHeads * 32 / (D / 16);
  const unsigned x = (unsigned)((a.T + (long long)warps - 1) / warps);
  const unsigned y = (unsigned)((a.Hq + 2 * a.Hk + heads - 1) / heads);
  void* args[] = {&a};
  return done(launch_early(rotary_kernel(dtype, D, fp4), dim3(x, y), dim3(sv::kRotaryThreads), args,
                           (cudaStream_t)stream));
}

}  // namespace

extern "C" {

int spec_paged_append_rotary(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                             const void* v_new, int64_t v_stride, const int32_t* positions,
                             const float* cos_sin, int max_positions, int rotary_dim, int interleaved,
                             const int32_t* slot_map, int dtype, int T, int Hq, int Hk, int D,
                             int page_size, int n_pages, void* q_out, int64_t q_out_stride,
                             void* k_cache, void* v_cache, uint32_t* flags, void* stream) {
  if (T > 0 && (!positions || !cos_sin)) return SV_ERR_NULL;
  sv::RotaryArgs a = rotary_args(q, k_new, v_new, positions, cos_sin, max_positions, rotary_dim, interleaved, slot_map, T,
                                 Hq, Hk, q_out, flags);
  a.k_cache = (char*)k_cache;
  a.v_cache = (char*)v_cache;
  return launch_rotary(a, dtype, D, false, q_stride, k_stride, v_stride, q_out_stride, page_size,
                       n_pages, stream);
}

int spec_paged_append_fp4(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                          const void* v_new, int64_t v_stride, const int32_t* positions,
                          const float* cos_sin, int max_positions, int rotary_dim, int interleaved,
                          const int32_t* slot_map, int dtype, int T, int Hq, int Hk, int D,
                          int page_size, int n_pages, float k_gain, float v_gain, void* q_out,
                          int64_t q_out_stride, void* k_codes, void* k_scales, void* v_codes,
                          void* v_scales, uint32_t* flags, void* stream) {
  if (!gain_ok(k_gain) || !gain_ok(v_gain)) return SV_ERR_SHAPE;
  sv::RotaryArgs a = rotary_args(q, k_new, v_new, positions, cos_sin, max_positions, rotary_dim, interleaved, slot_map, T,
                                 Hq, Hk, q_out, flags);
  a.k_cache = (char*)k_codes;
  a.v_cache = (char*)v_codes;
  a.k_scale = (uint8_t*)k_scales;
  a.v_scale = (uint8_t*)v_scales;
  a.k_gain = k_gain;
  a.v_gain = v_gain;
  a.k_plain = power_of_two(k_gain);
  a.v_plain = power_of_two(v_gain);
  return launch_rotary(a, dtype, D, true, q_stride, k_stride, v_stride, q_out_stride, page_size,
                       n_pages, stream);
}

int spec_paged_read_fp4(const void* k_codes, const void* k_scales, const void* v_codes,
                        const void* v_scales, const int32_t* slot_map, int dtype, int T, int Hk, int D,
                        int page_size, int n_pages, float k_gain, float v_gain, void* k_out,
                        void* v_out, uint32_t* flags, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || T < 0 || Hk < 1 || Hk > 4096 || (D != 64 && D != 128) || n_pages < 1 ||
      (long long)n_pages * page_size >= k2_31 || !gain_ok(k_gain) || !gain_ok(v_gain))
    return SV_ERR_SHAPE;
  if (T == 0) return SV_OK;
  if (!k_codes || !k_scales || !v_codes || !v_scales || !slot_map || !k_out || !v_out)
    return SV_ERR_NULL;
  if (!aligned_to(k_codes, 16) || !aligned_to(v_codes, 16) || !aligned_to(k_out, 16) ||
      !aligned_to(v_out, 16) || !aligned_to(slot_map, 4) || !aligned_to(flags, 4))
    return SV_ERR_ALIGN;
  sv::ReadFp4Args a;
  a.codes[0] = (const char*)k_codes;
  a.codes[1] = (const char*)v_codes;
  a.scales[0] = (const uint8_t*)k_scales;
  a.scales[1] = (const uint8_t*)v_scales;
  a.slot_map = slot_map;
  a.T = T;
  a.Hk = Hk;
  a.page_shift = shift;
  a.n_slots = (long long)n_pages * page_size;
  a.gain[0] = k_gain;
  a.gain[1] = v_gain;
  a.out[0] = (char*)k_out;
  a.out[1] = (char*)v_out;
  a.flags = flags;
  const long long groups = (long long)T * Hk * (D / sv::kFp4Group);
  const long long ctas = (groups + sv::kReadThreads - 1) / sv::kReadThreads;
  if (ctas >= k2_31) return SV_ERR_SHAPE;
  const void* fn =
      dtype == SV_BF16
          ? (D == 128 ? (const void*)sv::sv_read_fp4_kernel<__nv_bfloat16, 128>
                      : (const void*)sv::sv_read_fp4_kernel<__nv_bfloat16, 64>)
          : (D == 128 ? (const void*)sv::sv_read_fp4_kernel<__half, 128>
                      : (const void*)sv::sv_read_fp4_kernel<__half, 64>);
  void* args[] = {&a};
  return done(launch_early(fn, dim3((unsigned)ctas), dim3(sv::kReadThreads), args, (cudaStream_t)stream));
}

}  // extern "C"
