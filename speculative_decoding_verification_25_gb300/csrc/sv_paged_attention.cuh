// Attention of each request's new tokens over its paged keys and values.
//
// With s_j = scale * log2(e) * q.k_j the softmax is a running pair (m, l) and
// a running sum o: for keys taken in any order, m' = max(m, s_j),
// l' = l 2^(m-m') + 2^(s_j-m'), o' = o 2^(m-m') + 2^(s_j-m') v_j, and the
// result is o / l.
//
// One warp per (token, query head): a lane scores one key of 32, then the
// lanes share out the head's dimensions for the product with the values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_paged.cuh"

namespace sv {

constexpr int kAttnThreads = 256;
constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.693147181f;

struct AttnArgs {
  const char* q;            // token pitch in bytes
  long long q_pitch;
  const char* k_cache;
  const char* v_cache;
  const int32_t* block_table;   // [B, max_pages]
  const int32_t* cu_new;        // [B+1]
  const int32_t* kv_len;        // [B]
  int B, T, Hq, Hk, page_shift, max_pages, n_pages;
  float scale;
  char* out;
  float* lse;               // or nullptr
  unsigned* flags;
};

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*(const __half2*)&w);
}

template <typename E, int D>
__global__ void __launch_bounds__(kAttnThreads) sv_paged_attention_kernel(AttnArgs a) {
  wait_for_preceding_grid();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += kAttnThreads)
      if (a.cu_new[b] < 0 || a.cu_new[b + 1] < a.cu_new[b] || a.cu_new[b + 1] > a.T ||
          a.kv_len[b] < 0 || a.kv_len[b] > (long long)a.max_pages << a.page_shift)
        set_flag(a.flags, kDevLength);
  const long long task = ((long long)blockIdx.x * kAttnThreads + threadIdx.x) >> 5;
  const int t = (int)(task / a.Hq), h = (int)(task % a.Hq);
  if (t >= a.T) return;
  // the token's row: the first whose end passes t
  int lo = 0, hi = a.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_new[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  int visible = 0;
  if (lo < a.B) {
    const int begin = a.cu_new[lo], end = a.cu_new[lo + 1];
    const long long most = (long long)a.max_pages << a.page_shift;
    long long L = a.kv_len[lo];
    L = min(max(L, 0ll), most);
    if (begin < 0 || begin > t || end > a.T) return;
    visible = (int)max(0ll, L - (end - begin) + (t - begin) + 1);
  }
  const int hk = h / (a.Hq / a.Hk);
  const uint4* q = (const uint4*)(a.q + t * a.q_pitch + (long long)h * D * 2);
  float qf[D];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint4 w = q[i];
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2(ws[j], E());
      qf[8 * i + 2 * j] = f.x;
      qf[8 * i + 2 * j + 1] = f.y;
    }
  }
  constexpr int W = D / 32;   // dimensions per lane
  float o[W] = {}, m = SV_NEG_INF, l = 0.f;
  for (int j0 = 0; j0 < visible; j0 += 32) {
    const int j = j0 + lane;
    long long at = -1;
    float s = SV_NEG_INF;
    if (j < visible) {
      const int id = a.block_table[(long long)lo * a.max_pages + (j >> a.page_shift)];
      s = 0.f;
      if (id >= 0 && id < a.n_pages) {
        at = ((((long long)id * a.Hk + hk) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D;
        const uint4* k = (const uint4*)(a.k_cache + at * 2);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 w = k[i];
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2(ws[e], E());
            s = fmaf(qf[8 * i + 2 * e], f.x, s);
            s = fmaf(qf[8 * i + 2 * e + 1], f.y, s);
          }
        }
        s *= a.scale * kLog2e;
      } else {
        set_flag(a.flags, kDevBadPage);
      }
    }
    const float mn = fmaxf(m, warp_max(s));
    const float p = exp2f(s - mn);
    const float c = exp2f(m - mn);
    l = l * c + warp_sum(p);
    m = mn;
#pragma unroll
    for (int w = 0; w < W; ++w) o[w] *= c;
    const int n = min(32, visible - j0);
    for (int i = 0; i < n; ++i) {
      const long long vat = __shfl_sync(0xffffffffu, at, i);
      const float pi = __shfl_sync(0xffffffffu, p, i);
      if (vat < 0) continue;
      const uint32_t* v = (const uint32_t*)(a.v_cache + vat * 2) + lane * (W / 2);
#pragma unroll
      for (int w = 0; w < W / 2; ++w) {
        const float2 f = unpack2(v[w], E());
        o[2 * w] = fmaf(pi, f.x, o[2 * w]);
        o[2 * w + 1] = fmaf(pi, f.y, o[2 * w + 1]);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  E* out = (E*)a.out + ((long long)t * a.Hq + h) * D + lane * W;
#pragma unroll
  for (int w = 0; w < W; ++w) out[w] = E(o[w] * inv);
  if (a.lse && lane == 0)
    a.lse[(long long)t * a.Hq + h] = l > 0.f ? (m + log2f(l)) * kLn2 : SV_NEG_INF;
}

}  // namespace sv
