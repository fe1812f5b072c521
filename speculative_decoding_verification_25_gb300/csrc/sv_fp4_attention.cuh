// Attention over a paged cache of 4-bit keys and values: one warp per new token
// and query head, a key per lane for the scores and kD / 32 columns per lane for
// the values, with the running maximum and sum of a softmax in float32.
#pragma once

#include "sv_fp4.cuh"
#include "sv_paged.cuh"
#include "sv_rotary.cuh"

namespace sv {

struct Fp4Args {
  const char* q;
  long long q_pitch;
  const char* k_codes;
  const uint8_t* k_scales;
  const char* v_codes;
  const uint8_t* v_scales;
  const int32_t* block_table;
  const int32_t* cu_new;
  const int32_t* kv_len;
  int B, T, Hq, Hk, G, page_shift, max_pages, n_pages;
  float scale_log2, v_gain;
  char* out;
  float* lse;
  unsigned* flags;
};
constexpr int kFp4Warps = 4;

template <typename E, int kD>
__global__ void __launch_bounds__(32 * kFp4Warps) sv_fp4_attention_kernel(const __grid_constant__ Fp4Args a) {
  wait_for_preceding_grid();
  allow_dependent_launch();
  __shared__ float q_row[kFp4Warps][kD];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int token = blockIdx.x, h = blockIdx.y * kFp4Warps + warp;
  if (h >= a.Hq) return;
  // the request that has the token, of those whose offsets are sound
  int b = -1, begin = 0, n = 0;
  bool bad = false;
  for (int i = lane; i < a.B; i += 32) {
    const int lo = a.cu_new[i], hi = a.cu_new[i + 1], len = a.kv_len[i];
    const bool sound = lo >= 0 && hi >= lo && hi <= a.T;
    bad |= !sound || len < 0 || len > (a.max_pages << a.page_shift);
    if (sound && token >= lo && token < hi) b = i, begin = lo, n = hi - lo;
  }
  if (bad && token == 0 && h == 0) set_flag(a.flags, kDevLength);
  const unsigned who = __ballot_sync(0xffffffffu, b >= 0);
  int seen = 0;
  if (who) {
    const int from = __ffs(who) - 1;
    b = __shfl_sync(0xffffffffu, b, from);
    begin = __shfl_sync(0xffffffffu, begin, from);
    n = __shfl_sync(0xffffffffu, n, from);
    const int L = min(max(a.kv_len[b], 0), a.max_pages << a.page_shift);
    seen = max(0, L - n + (token - begin) + 1);
  }
  const char* q = a.q + token * a.q_pitch + (long long)h * kD * 2;
  for (int i = lane; i < kD / 2; i += 32) Element<E>::unpack(((const uint32_t*)q)[i], &q_row[warp][2 * i]);
  __syncwarp();
  const int hk = h / a.G;
  float m = SV_NEG_INF, l = 0.f, o[kD / 32] = {};
  for (int key0 = 0; key0 < seen; key0 += 32) {
    const int key = key0 + lane;
    long long row = -1;
    float s = SV_NEG_INF;
    if (key < seen) {
      const int id = a.block_table[(long long)b * a.max_pages + (key >> a.page_shift)];
      if (id >= 0 && id < a.n_pages)
        row = (((long long)id * a.Hk + hk) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
      else set_flag(a.flags, kDevBadPage);
      s = 0.f;
      for (int g = 0; g < kD / kFp4Group && row >= 0; ++g) {
        const uint2 w = *(const uint2*)(a.k_codes + row * (kD / 2) + g * 8);
        const float unit = fp4_scale(a.k_scales[row * (kD / kFp4Group) + g]);
        uint32_t r[8];
        fp4_unpack(w.x, r);
        fp4_unpack(w.y, r + 4);
        float part = 0.f;
        for (int x = 0; x < 8; ++x) {
          const float2 f = __half22float2(*(const __half2*)&r[x]);
          part += q_row[warp][g * 16 + 2 * x] * f.x + q_row[warp][g * 16 + 2 * x + 1] * f.y;
        }
        s += part * unit;
      }
      s *= a.scale_log2;
    }
    float top = s;
    for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(top, m);
    const float ref = top == SV_NEG_INF ? 0.f : top, f = m == SV_NEG_INF ? 0.f : exp2f(m - ref);
    const float p = key < seen ? exp2f(s - ref) : 0.f;
    m = top;
    l = l * f + p;
    for (int x = 0; x < kD / 32; ++x) o[x] *= f;
    for (int j = 0; j < min(32, seen - key0); ++j) {
      const long long r = __shfl_sync(0xffffffffu, row, j);
      const float pj = __shfl_sync(0xffffffffu, p, j);
      if (r < 0) continue;
      const float unit = fp4_scale(a.v_scales[r * (kD / kFp4Group) + lane / (512 / kD)]);
      const uint32_t w = kD == 128 ? *(const uint16_t*)(a.v_codes + r * (kD / 2) + lane * 2)
                                   : *(const uint8_t*)(a.v_codes + r * (kD / 2) + lane);
      uint32_t v[4];
      fp4_unpack(w, v);
      for (int x = 0; x < kD / 64; ++x) {
        const float2 e = __half22float2(*(const __half2*)&v[x]);
        o[2 * x] += pj * (e.x * unit);
        o[2 * x + 1] += pj * (e.y * unit);
      }
    }
  }
  for (int x = 16; x > 0; x /= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l == 0.f ? 0.f : a.v_gain / l;
  const long long to = (long long)token * a.Hq + h;
  for (int x = 0; x < kD / 64; ++x)
    *(uint32_t*)(a.out + (to * kD + lane * (kD / 32) + 2 * x) * 2) = Element<E>::pack(o[2 * x] * inv, o[2 * x + 1] * inv);
  if (a.lse && lane == 0) a.lse[to] = l == 0.f ? SV_NEG_INF : (m + log2f(l)) * 0.693147181f;
}

}  // namespace sv
