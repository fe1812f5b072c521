// New tokens on their way into the paged cache: queries and keys are rotated by
// their positions, keys and values go to their slots, as 16-bit numbers or as
// 4-bit ones.  With (x, y) a pair of a head's columns and (c, s) cosine and sine
// of its angle at the token's position, from the caller's table,
//   x' = x c - y s,   y' = x s + y c.
//
// Bound by HBM: every element is read and written once.  kD / 16 lanes share a
// head; a lane has two pieces of 8 elements (16 bytes): of rotated columns the
// two that are each other's partners where pairs are half the rotated columns
// apart, so both kinds of pairs lie within a lane.  Adjacent lanes hold adjacent
// pieces, so two lanes share a group of 16.  A warp has kRotaryHeads passes of heads of one
// token in flight; the lane's cosines and sines serve all of them.
//
// Codes and scales are those of exact arithmetic: where a rotated value's error in
// float32 could pass the border of two codes (one of a few thousand lanes), the
// lane decides in 64 bits, in which products of the inputs are exact.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_fp4.cuh"
#include "sv_paged.cuh"

namespace sv {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryHeads = 4;   // heads per lane in flight

struct RotaryArgs {
  const char* q;         // token pitches in bytes
  const char* k_new;
  const char* v_new;
  long long q_pitch, k_pitch, v_pitch, out_pitch;
  const int32_t* positions;     // nullptr: nothing is rotated
  const float* table;           // [max_positions, rot]: cosines, then sines
  const int32_t* slot_map;
  int T, Hq, Hk, page_shift, max_positions, rot;
  bool neighbours;              // pairs (2i, 2i + 1), else (i, i + rot / 2)
  long long n_slots;
  char* q_out;
  char* k_cache;                // 16-bit elements, or codes
  char* v_cache;
  uint8_t* k_scale;             // 4-bit cache
  uint8_t* v_scale;
  float k_gain, v_gain;
  bool k_plain, v_plain;        // the gain is a power of two
  unsigned* flags;
};

template <typename E>
struct Element;
template <>
struct Element<__nv_bfloat16> {
  __device__ __forceinline__ static void unpack(uint32_t w, float* x) {
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xffff0000u);
  }
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <>
struct Element<__half> {
  __device__ __forceinline__ static void unpack(uint32_t w, float* x) {
    const float2 f = __half22float2(*(const __half2*)&w);
    x[0] = f.x;
    x[1] = f.y;
  }
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// What a lane holds of a head: 16 elements, and of a token: 8 cosines and sines.
struct RotaryAngles {
  float c[8], s[8];
};
// The i-th pair of a lane: its elements' places among the 16.
__device__ __forceinline__ int pair_x(bool neighbours, int i) { return neighbours ? 2 * i : i; }
__device__ __forceinline__ int pair_y(bool neighbours, int i) { return neighbours ? 2 * i + 1 : i + 8; }

template <typename F, bool kNeighbours>
__device__ __forceinline__ void rotate(const RotaryAngles& a, const float* in, F* out) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const F x = in[pair_x(kNeighbours, i)], y = in[pair_y(kNeighbours, i)], c = a.c[i], s = a.s[i];
    out[pair_x(kNeighbours, i)] = x * c - y * s;
    out[pair_y(kNeighbours, i)] = x * s + y * c;
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The e4m3 number nearest to x >= 0, of two the even one.
static __device__ __noinline__ uint32_t nearest_scale(double x) {
  uint32_t low = 0, high = 126;   // codes of non-negative numbers ascend
  while (high - low > 1) {
    const uint32_t mid = (low + high) / 2;
    if ((double)fp4_scale(mid) <= x) low = mid;
    else high = mid;
  }
  const double middle = 0.5 * ((double)fp4_scale(low) + (double)fp4_scale(high));
  return x > middle || (x == middle && (low & 1)) ? high : low;
}
// The e2m1 code nearest to the magnitude y.
__device__ __forceinline__ uint32_t nearest_code(double y) {
  return (y > 0.25) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0);
}

// Scales and codes of a lane's two pieces `x`, of `in` after rotation.  `exact`: the values are the
// caller's own (at most 11 significant bits) and the gain is a power of two;
// float32 division, which rounds correctly, then puts every quotient on the
// right side of every border, since a border times a scale has at most 7 bits.
// Else a value is off by at most 2^-23 (|x| + |y|) for its pair, its quotient
// by 2^-23 of itself more: where twice that could cross a border the decision
// is taken in 64 bits.
template <bool kNeighbours>
__device__ __forceinline__ void quantise(const float* x, const RotaryAngles& a, const float* in,
                                         bool rotated, bool exact, float gain, uint32_t* scale,
                                         uint32_t* codes) {
  double wide[16];   // made where it is needed
  bool have = false;
  auto widen = [&]() {
    if (have) return;
    have = true;
#pragma unroll
    for (int i = 0; i < 16; ++i) wide[i] = in[i];
    if (rotated) rotate<double, kNeighbours>(a, in, wide);
  };
  float off = 0.f;
  if (!exact) {
#pragma unroll
    for (int i = 0; i < 16; ++i) off = fmaxf(off, fabsf(in[i]));
    off *= 0x1p-20f;
  }
  const float off_pair = fmaxf(off, __shfl_xor_sync(0xffffffffu, off, 1));
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const float* v = x + 8 * p;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(v[i]));
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const float six = 6.f * gain;
    uint32_t code = fp4_scale_code(__fdiv_rn(top, six));
    const bool finite = top <= 3.402823466e38f;
    const bool unsure = !exact && finite &&
                        fp4_scale_code(__fdiv_rn(top - off_pair, six)) !=
                            fp4_scale_code(__fdiv_rn(top + off_pair, six));
    if (__any_sync(0xffffffffu, unsure)) {
      widen();
      double high = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) high = fmax(high, fabs(wide[8 * p + i]));
      high = fmax(high, __shfl_xor_sync(0xffffffffu, high, 1));
      if (unsure) code = nearest_scale(high / (6.0 * (double)gain));
    }
    if (!finite) code = kFp4NanScale;
    scale[p] = code;
    codes[p] = 0;
    if (!finite || code == 0) continue;
    const float unit = fp4_scale(code) * gain;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(v[i], unit);
    codes[p] = fp4_pack(y);
    if (!exact) {
      const float far = __fdiv_rn(off, unit);
      float less[8], more[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) less[i] = y[i] - far, more[i] = y[i] + far;
      if (fp4_pack(less) != fp4_pack(more)) {
        widen();
        const double u = (double)fp4_scale(code) * (double)gain;
        codes[p] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          codes[p] |= (nearest_code(fabs(wide[8 * p + i]) / u) | (signbit(wide[8 * p + i]) ? 8u : 0u))
                      << (4 * i);
      }
    }
  }
}

template <typename E, int kD, bool kFp4, bool kNeighbours>
__device__ __forceinline__ void rotary_token(const RotaryArgs& a, int token, int first_head) {
  constexpr int kSpan = kD / 16, kPass = 32 / kSpan;
  const int lane = threadIdx.x & 31, part = lane % kSpan;
  const int turned = a.rot / 16;   // lanes of a head whose columns are rotated
  const bool rotated = part < turned;
  const int p0 = rotated ? part : turned * 2 + part - turned;
  const int p1 = rotated ? part + turned : p0 + kSpan - turned;
  const int heads = a.Hq + 2 * a.Hk;

  const int pos = a.positions ? a.positions[token] : 0;
  const int slot = a.slot_map[token];
  const bool placed = !a.positions || (pos >= 0 && pos < a.max_positions);
  if (!placed && (pos >= 0 || slot >= 0) && lane == 0) set_flag(a.flags, kDevLength);
  const bool stored = placed && slot >= 0 && slot < a.n_slots;
  if (slot >= a.n_slots && lane == 0) set_flag(a.flags, kDevBadPage);

  uint32_t w[kRotaryHeads][8];
#pragma unroll
  for (int u = 0; u < kRotaryHeads; ++u) {
    const int h = first_head + u * kPass + lane / kSpan;
    const bool used = placed && (h < a.Hq || (stored && h < heads));
    const char* row = h < a.Hq ? a.q + token * a.q_pitch + (long long)h * kD * 2
                      : h < a.Hq + a.Hk
                          ? a.k_new + token * a.k_pitch + (long long)(h - a.Hq) * kD * 2
                          : a.v_new + token * a.v_pitch + (long long)(h - a.Hq - a.Hk) * kD * 2;
    uint32_t lo[4] = {}, hi[4] = {};
    if (used) {
      ldg_stream16(row + p0 * 16, lo);
      ldg_stream16(row + p1 * 16, hi);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[u][i] = lo[i], w[u][4 + i] = hi[i];
  }
  RotaryAngles angles;
  if (rotated && placed && first_head < a.Hq + a.Hk) {
    const float* c = a.table + (long long)pos * a.rot;
    const int at = kNeighbours ? 4 * part : 8 * part;
    const int next = kNeighbours ? at + a.rot / 4 : at + 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      angles.c[i] = c[at + i];
      angles.c[4 + i] = c[next + i];
      angles.s[i] = c[a.rot / 2 + at + i];
      angles.s[4 + i] = c[a.rot / 2 + next + i];
    }
  }
#pragma unroll
  for (int u = 0; u < kRotaryHeads; ++u) {
    const int h = first_head + u * kPass + lane / kSpan;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hk;
    float in[16], x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) Element<E>::unpack(w[u][i], in + 2 * i);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = in[i];
    const bool turn = rotated && placed && (is_q || is_k);
    if (turn) rotate<float, kNeighbours>(angles, in, x);
    if (is_q || !kFp4) {
      const int hk = is_k ? h - a.Hq : h - a.Hq - a.Hk;
      if (!is_q && (!stored || h >= heads)) continue;
      char* row = is_q ? a.q_out + token * a.out_pitch + (long long)h * kD * 2
                       : (is_k ? a.k_cache : a.v_cache) +
                             ((((slot >> a.page_shift) * (long long)a.Hk + hk) << a.page_shift) +
                              (slot & ((1 << a.page_shift) - 1))) * kD * 2;
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = turn ? Element<E>::pack(x[2 * i], x[2 * i + 1]) : w[u][i];
      *(uint4*)(row + p0 * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      *(uint4*)(row + p1 * 16) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if (kFp4) {
      if (!__any_sync(0xffffffffu, !is_q && stored && h < heads)) continue;
      uint32_t scale[2], codes[2];
      const bool exact = !turn && (is_k ? a.k_plain : a.v_plain);
      quantise<kNeighbours>(x, angles, in, turn, exact, is_k ? a.k_gain : a.v_gain, scale, codes);
      if (is_q || !stored || h >= heads) continue;
      const int hk = is_k ? h - a.Hq : h - a.Hq - a.Hk;
      const long long row = (((slot >> a.page_shift) * (long long)a.Hk + hk) << a.page_shift) +
                            (slot & ((1 << a.page_shift) - 1));
      char* code_row = (is_k ? a.k_cache : a.v_cache) + row * (kD / 2);
      uint8_t* scale_row = (is_k ? a.k_scale : a.v_scale) + row * (kD / kFp4Group);
      *(uint32_t*)(code_row + p0 * 4) = codes[0];
      *(uint32_t*)(code_row + p1 * 4) = codes[1];
      if (part % 2 == 0) {
        scale_row[p0 / 2] = (uint8_t)scale[0];
        scale_row[p1 / 2] = (uint8_t)scale[1];
      }
    }
  }
}

template <typename E, int kD, bool kFp4>
__global__ void __launch_bounds__(kRotaryThreads) sv_rotary_kernel(RotaryArgs a) {
  wait_for_preceding_grid();
  allow_dependent_launch();
  constexpr int kHeads = kRotaryHeads * 32 / (kD / 16);   // of a warp
  const long long token = (long long)blockIdx.x * (kRotaryThreads / 32) + threadIdx.x / 32;
  if (token >= a.T) return;
  if (a.neighbours) rotary_token<E, kD, kFp4, true>(a, (int)token, blockIdx.y * kHeads);
  else rotary_token<E, kD, kFp4, false>(a, (int)token, blockIdx.y * kHeads);
}

// ------------------------------------------------------------------- reading
// Cached tokens as the values that they are held as; zeros for slots that are
// none.  A thread takes a group of 16: 8 bytes of codes and a scale to 32 bytes.
struct ReadFp4Args {
  const char* codes[2];        // keys, values
  const uint8_t* scales[2];
  const int32_t* slot_map;
  int T, Hk, page_shift;
  long long n_slots;
  float gain[2];
  char* out[2];
  unsigned* flags;
};
constexpr int kReadThreads = 256;

template <typename E, int kD>
__global__ void __launch_bounds__(kReadThreads) sv_read_fp4_kernel(ReadFp4Args a) {
  wait_for_preceding_grid();
  allow_dependent_launch();
  constexpr int kGroups = kD / kFp4Group;
  const int groups = a.Hk * kGroups;
  const long long i = (long long)blockIdx.x * kReadThreads + threadIdx.x;
  if (i >= (long long)a.T * groups) return;
  const int token = (int)(i / groups), g = (int)(i - (long long)token * groups);
  const int slot = a.slot_map[token];
  const bool held = slot >= 0 && slot < a.n_slots;
  if (slot >= a.n_slots) set_flag(a.flags, kDevBadPage);
  const long long row = (((slot >> a.page_shift) * (long long)a.Hk + g / kGroups) << a.page_shift) +
                        (slot & ((1 << a.page_shift) - 1));
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint32_t r[8] = {};
    float unit = 0.f;
    if (held) {
      const uint2 w = *(const uint2*)(a.codes[s] + row * (kD / 2) + g % kGroups * 8);
      unit = fp4_scale(a.scales[s][row * kGroups + g % kGroups]);
      fp4_unpack(w.x, r);
      fp4_unpack(w.y, r + 4);
    }
    uint32_t o[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float2 f = __half22float2(*(const __half2*)&r[x]);
      o[x] = Element<E>::pack(f.x * unit * a.gain[s], f.y * unit * a.gain[s]);
    }
    uint4* to = (uint4*)(a.out[s] + i * (kFp4Group * 2));
    to[0] = make_uint4(o[0], o[1], o[2], o[3]);
    to[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace sv
