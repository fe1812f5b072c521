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
// pieces, so two lanes share a group of 16.  A warp takes kRotaryHeads passes of
// heads of one token, all in flight; the lane's cosines and sines serve all of them.
// 32768 tokens of 32/8 heads of 128, bfloat16: 130 us for 0.82 GB, 6.3 TB/s (heads
// one after the other 146).  Into 4 bits 158 us, bound by instruction issue (58% of
// slots): there one copy of the long code runs while the next head's loads are
// under way (all heads unrolled 205); without queries and rotation 75 us for 0.17 GB.
// Reading 4 bits back 38 us: short threads, HBM at 43% and issue at 45%.
//
// Codes and scales are those of exact arithmetic: where a rotated value's error in
// float32 could pass the border of two codes (one of a few hundred warps), the
// lane decides with unevaluated pairs of float32, to 2^-47 (64-bit numbers are slow
// here: 320 tokens 44 us).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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

template <bool kNeighbours>
__device__ __forceinline__ void rotate(const RotaryAngles& a, const float* in, float* out) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = in[pair_x(kNeighbours, i)], y = in[pair_y(kNeighbours, i)], c = a.c[i], s = a.s[i];
    out[pair_x(kNeighbours, i)] = x * c - y * s;
    out[pair_y(kNeighbours, i)] = x * s + y * c;
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// What a lane holds of a token, to find its values again more exactly: the head's
// row, the position's cosines, and which columns.
struct RotaryPlace {
  const char* row;
  const float* table;
  int rot, p0, p1, part;
  bool turned;
};
// Its piece p (0 or 1) as pairs high + low: products by fused multiply-adds are
// exact, and so is the difference of two rounded ones in two parts.
template <typename E, bool kNeighbours>
__device__ __forceinline__ void wide_piece(const RotaryPlace& at, int p, float2* v) {
  float in[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    Element<E>::unpack(((const uint32_t*)(at.row + at.p0 * 16))[i], in + 2 * i);
    Element<E>::unpack(((const uint32_t*)(at.row + at.p1 * 16))[i], in + 8 + 2 * i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float own = p ? in[8 + i] : in[i];
    v[i] = make_float2(own, 0.f);
    if (!at.turned) continue;
    const int pair = kNeighbours ? (p ? at.rot / 4 : 0) + 4 * at.part + i / 2 : 8 * at.part + i;
    const float c = at.table[pair], t = at.table[at.rot / 2 + pair];
    const float other = kNeighbours ? in[8 * p + (i ^ 1)] : p ? in[i] : in[8 + i];
    const bool second = kNeighbours ? i % 2 : p;   // x s + y c, else x c - y s
    const float s = second ? t : -t;
    const float a = __fmul_rn(own, c), b = __fmul_rn(other, s);
    const float a_low = __fmaf_rn(own, c, -a), b_low = __fmaf_rn(other, s, -b);
    const float sum = __fadd_rn(a, b), b_part = __fsub_rn(sum, a);
    const float sum_low = __fadd_rn(__fsub_rn(a, __fsub_rn(sum, b_part)), __fsub_rn(b, b_part));
    const float low = __fadd_rn(sum_low, __fadd_rn(a_low, b_low));
    v[i].x = low == 0.f ? sum : __fadd_rn(sum, low);   // keeps the sign of a zero
    v[i].y = __fsub_rn(low, __fsub_rn(v[i].x, sum));
  }
}
__device__ __forceinline__ float2 wide_abs(float2 v) {
  return v.x < 0.f || (v.x == 0.f && v.y < 0.f) ? make_float2(-v.x, -v.y) : v;
}
__device__ __forceinline__ float2 wide_max(float2 a, float2 b) {
  return a.x > b.x || (a.x == b.x && a.y > b.y) ? a : b;
}
// The sign of v - m u, exactly where the two are close (m has few bits).
__device__ __forceinline__ float wide_over(float2 v, float m, float2 u) {
  return __fadd_rn(__fmaf_rn(-m, u.x, v.x), __fmaf_rn(-m, u.y, v.y));
}
// The largest magnitude of the piece, and its codes for a scale times gain of `unit`.
template <typename E, bool kNeighbours>
__device__ __noinline__ float2 wide_top(RotaryPlace at, int p) {
  float2 v[8], top = make_float2(0.f, 0.f);
  wide_piece<E, kNeighbours>(at, p, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) top = wide_max(top, wide_abs(v[i]));
  return top;
}
template <typename E, bool kNeighbours>
__device__ __noinline__ uint32_t wide_codes(RotaryPlace at, int p, float2 unit) {
  float2 v[8];
  wide_piece<E, kNeighbours>(at, p, v);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = wide_abs(v[i]);
    const uint32_t code = (wide_over(x, 0.25f, unit) > 0.f) + (wide_over(x, 0.75f, unit) >= 0.f) +
                          (wide_over(x, 1.25f, unit) > 0.f) + (wide_over(x, 1.75f, unit) >= 0.f) +
                          (wide_over(x, 2.5f, unit) > 0.f) + (wide_over(x, 3.5f, unit) >= 0.f) +
                          (wide_over(x, 5.f, unit) > 0.f);
    codes |= (code | (signbit(v[i].x) ? 8u : 0u)) << (4 * i);
  }
  return codes;
}
// The e4m3 number nearest to x over `six`, of two the even one; `about` is it or next to it.
static __device__ __noinline__ uint32_t nearest_scale(float2 x, float2 six, uint32_t about) {
  auto over = [&](uint32_t low) { return wide_over(x, 0.5f * (fp4_scale(low) + fp4_scale(low + 1)), six); };
  if (about < 126) {
    const float up = over(about);
    if (up > 0.f || (up == 0.f && (about & 1))) return about + 1;
  }
  if (about > 0) {
    const float down = over(about - 1);
    if (down < 0.f || (down == 0.f && (about & 1))) return about - 1;
  }
  return about;
}
__device__ __forceinline__ float2 wide_product(float a, float b) {
  const float high = __fmul_rn(a, b);
  return make_float2(high, __fmaf_rn(a, b, -high));
}

// Scales and codes of a lane's two pieces `x`, which are `in` after rotation.
// `exact`: the values are the caller's own (A 2^p, A < 2^11) and the gain is a power
// of two, so a scale times gain is B 2^q, 8 <= B < 16.  The scale's quotient comes
// from a division that rounds correctly, and a value over 6 that is not half-way
// between two scales lies 2^-13 of itself from it.  A value's quotient A / B 2^(p-q)
// that is not a border c / 4 of two codes differs from it by at least 2^-14, the
// smallest border being 1/4; so its product with the rounded inverse, off by 2^-20,
// is rounded to steps of 2^-18, and falls on the border exactly when it should.
// Else a rotated value is off by at most 2^-23 (|x| + |y|) t for its pair and the largest
// cosine or sine t, and its quotient by 2^-22 of itself, which is at most 2 max(|x|, |y|) t;
// other values' t is 1.  Where twice that, max(|x|, |y|) times `slope`, 2^-19 t, could cross
// a border, one of some hundred warps, pairs of numbers decide.
template <typename E, bool kNeighbours>
__device__ __forceinline__ void quantise(const float* x, const float* in, const RotaryPlace& at, bool exact,
                                         float slope, float gain, uint32_t* scale, uint32_t* codes) {
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) off = fmaxf(off, fabsf(in[i]));
  off *= exact ? 0.f : slope;
  const float off_pair = fmaxf(off, __shfl_xor_sync(0xffffffffu, off, 1));
  const float six = 6.f * gain, sixth = __fdiv_rn(1.f, six);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const float* v = x + 8 * p;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(v[i]));
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    uint32_t code = fp4_scale_code(__fdiv_rn(top, six));
    const bool finite = top <= 3.402823466e38f;
    const bool unsure = !exact && finite &&
                        fp4_scale_code(fmaxf(top - off_pair, 0.f) * sixth) != fp4_scale_code((top + off_pair) * sixth);
    if (__any_sync(0xffffffffu, unsure)) {
      const float2 own = unsure ? wide_top<E, kNeighbours>(at, p) : make_float2(0.f, 0.f);
      const float2 high = wide_max(own, make_float2(__shfl_xor_sync(0xffffffffu, own.x, 1),
                                                    __shfl_xor_sync(0xffffffffu, own.y, 1)));
      if (unsure) code = nearest_scale(high, wide_product(6.f, gain), fp4_scale_code(high.x * sixth));
    }
    if (!finite) code = kFp4NanScale;
    scale[p] = code;
    codes[p] = 0;
    if (!finite || code == 0) continue;
    const float unit = fp4_scale(code) * gain, inverse = __fdiv_rn(1.f, unit);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = v[i] * inverse;
      if (exact) y[i] = copysignf(__fsub_rn(__fadd_rn(y[i], 48.f), 48.f), v[i]);
    }
    codes[p] = fp4_pack(y);
    if (!exact) {
      const float far = off * inverse;
      float less[8], more[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) less[i] = y[i] - far, more[i] = y[i] + far;
      if (fp4_pack(less) != fp4_pack(more))
        codes[p] = wide_codes<E, kNeighbours>(at, p, wide_product(fp4_scale(code), gain));
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
  const int heads = a.Hq + 2 * a.Hk, mine = first_head + lane / kSpan;

  const int pos = a.positions ? a.positions[token] : 0;
  const int slot = a.slot_map[token];
  const bool placed = !a.positions || (pos >= 0 && pos < a.max_positions);
  if (!placed && (pos >= 0 || slot >= 0) && lane == 0) set_flag(a.flags, kDevLength);
  const bool stored = placed && slot >= 0 && slot < a.n_slots;
  if (slot >= a.n_slots && lane == 0) set_flag(a.flags, kDevBadPage);
  // the slot's row of head 0 in the cache; heads are a page apart
  const long long slot_row =
      stored ? ((slot >> a.page_shift) * (long long)a.Hk << a.page_shift) + (slot & ((1 << a.page_shift) - 1)) : 0;

  auto source = [&](int h) -> const char* {
    return h < a.Hq          ? a.q + token * a.q_pitch + (long long)h * kD * 2
           : h < a.Hq + a.Hk ? a.k_new + token * a.k_pitch + (long long)(h - a.Hq) * kD * 2
                             : a.v_new + token * a.v_pitch + (long long)(h - a.Hq - a.Hk) * kD * 2;
  };
  auto load = [&](int h, uint32_t* w) {
    uint32_t lo[4] = {}, hi[4] = {};
    if (placed && (h < a.Hq || (stored && h < heads))) {
      const char* row = source(h);
      ldg_stream16(row + p0 * 16, lo);
      ldg_stream16(row + p1 * 16, hi);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = lo[i], w[4 + i] = hi[i];
  };
  RotaryAngles angles;
  float slope = 0.f;   // 2^-19 of the largest of them
  const float* table = a.table + (long long)pos * a.rot;
  auto look_up = [&]() {
    if (!rotated || !placed || first_head >= a.Hq + a.Hk) return;
    const int at = kNeighbours ? 4 * part : 8 * part;
    const int next = kNeighbours ? at + a.rot / 4 : at + 4;
    if (!in_array(a.flags, (long long)pos * a.rot + a.rot / 2 + next + 3, (long long)a.max_positions * a.rot)) return;
    *(float4*)angles.c = *(const float4*)(table + at);
    *(float4*)(angles.c + 4) = *(const float4*)(table + next);
    *(float4*)angles.s = *(const float4*)(table + a.rot / 2 + at);
    *(float4*)(angles.s + 4) = *(const float4*)(table + a.rot / 2 + next);
    if (!kFp4) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) slope = fmaxf(slope, fmaxf(fabsf(angles.c[i]), fabsf(angles.s[i])));
    slope *= 0x1p-19f;
  };
  auto finish = [&](int h, const uint32_t* w, auto coded) {   // `coded`: keys and values become codes
    constexpr bool kCoded = decltype(coded)::value;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hk;
    const int hk = is_k ? h - a.Hq : h - a.Hq - a.Hk;
    const bool goes = !is_q && stored && h < heads &&
                      in_array(a.flags, slot_row + ((long long)hk << a.page_shift), a.n_slots * a.Hk);
    float in[16], x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) Element<E>::unpack(w[i], in + 2 * i);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = in[i];
    const bool turn = rotated && placed && (is_q || is_k);
    if (turn) rotate<kNeighbours>(angles, in, x);
    const long long row = slot_row + ((long long)hk << a.page_shift);
    if (is_q || (!kCoded && goes)) {
      char* to = is_q ? a.q_out + token * a.out_pitch + (long long)h * kD * 2
                      : (is_k ? a.k_cache : a.v_cache) + row * kD * 2;
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = turn ? Element<E>::pack(x[2 * i], x[2 * i + 1]) : w[i];
      *(uint4*)(to + p0 * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      *(uint4*)(to + p1 * 16) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if constexpr (kCoded) {
      if (!__any_sync(0xffffffffu, goes)) return;
      uint32_t scale[2], codes[2];
      const bool exact = !turn && (is_k ? a.k_plain : a.v_plain);
      const RotaryPlace at = {goes ? source(h) : nullptr, table, a.rot, p0, p1, part, turn};
      // a lane whose head goes nowhere has nothing to decide
      quantise<E, kNeighbours>(x, in, at, exact || !goes, turn ? slope : 0x1p-19f, is_k ? a.k_gain : a.v_gain, scale,
                                codes);
      if (!goes) return;
      char* code_row = (is_k ? a.k_cache : a.v_cache) + row * (kD / 2);
      uint8_t* scale_row = (is_k ? a.k_scale : a.v_scale) + row * (kD / kFp4Group);
      *(uint32_t*)(code_row + p0 * 4) = codes[0];
      *(uint32_t*)(code_row + p1 * 4) = codes[1];
      if (part % 2 == 0) {
        scale_row[p0 / 2] = (uint8_t)scale[0];
        scale_row[p1 / 2] = (uint8_t)scale[1];
      }
    }
  };

  if (kFp4 && first_head + kRotaryHeads * kPass > a.Hq) {
    // the quantisation is long code: one copy of it, the next head on its way meanwhile
    uint32_t w[2][8];
    load(mine, w[0]);
    look_up();
#pragma unroll 1
    for (int u = 0; u < kRotaryHeads; ++u) {
      if (u + 1 < kRotaryHeads) load(mine + (u + 1) * kPass, w[1]);
      finish(mine + u * kPass, w[0], std::integral_constant<bool, kFp4>());
#pragma unroll
      for (int i = 0; i < 8; ++i) w[0][i] = w[1][i];
    }
  } else {
    uint32_t w[kRotaryHeads][8];
#pragma unroll
    for (int u = 0; u < kRotaryHeads; ++u) load(mine + u * kPass, w[u]);
    look_up();
#pragma unroll
    for (int u = 0; u < kRotaryHeads; ++u) finish(mine + u * kPass, w[u], std::false_type());
  }
}

template <typename E, int kD, bool kFp4>
__global__ void __launch_bounds__(kRotaryThreads, 3) sv_rotary_kernel(RotaryArgs a) {
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
