// What the forms of attention over the 4-bit cache share: their arguments, a
// packed tile in shared memory, and the warp that brings it.
#pragma once

#include "sv_fp4.cuh"
#include "sv_paged_attention.cuh"

namespace sv {

// P is float16 here whatever the queries' type, and float16 has 11 bits from 2^-14
// and steps of 2^-24: so a reference is set this far below a row's maximum (in log2),
// and P is at most 2^(kFp4Below + kSlack) = 2^15.  A probability then has its 11 bits
// down to 2^-21 of the largest, and steps of 2^-31 of it below that; with the reference at
// the maximum, keys 17.5 (natural units) below the first one gave 0 where 4096 of them
// are 1e-4 of the result.  No instruction is added.
constexpr float kFp4Below = 7.f;

// bfloat16 queries become float16 times 2^-exponent.  Brought to [2^14, 2^15), the largest
// of a unit leaves the others steps of 2^-38 of it or less.  2^126 is the most that they
// are multiplied by: then no bfloat16 number is below float16's steps.
constexpr uint32_t kBf16Infinity = 0x7f80u;
__device__ __forceinline__ int query_exponent(uint32_t top) { return max((int)(top >> 7) - 127 - 14, -126); }   // of its bits
__device__ __forceinline__ uint32_t query_factor(int exponent) { return (uint32_t)(127 - exponent) << 7 | (uint32_t)(127 - exponent) << 23; }
__device__ __forceinline__ uint32_t query_pair(uint32_t w, uint32_t factor) {
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(factor));
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u), __half());
}
// The larger magnitude of the two that a word has.
__device__ __forceinline__ uint32_t larger_half(uint32_t magnitudes) { return max(magnitudes >> 16, magnitudes & 0xffffu); }
// Magnitudes of a word; `finite`: 0 for infinities and NaN.
__device__ __forceinline__ uint32_t bf16_magnitudes(uint32_t w, bool finite) {
  w &= 0x7fff7fffu;
  if (finite && (w & 0xffffu) >= kBf16Infinity) w &= 0xffff0000u;
  if (finite && w >> 16 >= kBf16Infinity) w &= 0xffffu;
  return w;
}

// The power of two that the scores' factor takes for queries that carry 2^exponent, such
// that the factor is a normal number: with 0 a masked score of -inf would become NaN, with
// an infinity a score of 0.  Where it would be less, every score (below 2^34 times it)
// is 0 to all purposes as it is.
__device__ __forceinline__ int score_exponent(float scale_log2, int exponent) {
  const int own = (int)(__float_as_uint(scale_log2) >> 23) - 127;
  return min(max(exponent, -126 - own), 127 - own);
}

struct Fp4Args : AttnArgs {
  const char* q;
  long long q_pitch;   // bytes between tokens
  const char* k_scales;
  const char* v_scales;
};

// 128 keys: their codes in 16-byte pieces, swizzled by the copy, then their scales.
template <int kD>
struct Fp4Tile {
  static constexpr int kCodeBytes = 128 * kD / 2, kScaleBytes = 128 * kD / 16;
  static constexpr int kBytes = kCodeBytes + kScaleBytes;
};
// Byte of 16-byte piece `piece` of a key's codes in a tile.
template <int kD>
__device__ __forceinline__ uint32_t fp4_piece(int row, int piece) {
  return kD == 128 ? row * 64 + ((piece ^ (row / 2 % 4)) * 16) : row * 32 + ((piece ^ (row / 4 % 2)) * 16);
}

// ------------------------------------------------------------------- loader
// One warp for keys and one for values, or one for both: tiles as they are packed,
// which alternate in a ring of kPackedStages that `full` and `empty` tell of.  Lane
// i knows the tile's page i and brings its codes, a box; its scales are too few for
// one (a tiled copy wants 128 bytes), and all lanes bring 16-byte pieces of them.
// Rows of pages past the request's length stay as they are; a page outside the
// cache reads as zeros.  A box's issue takes about 50 clocks, so pages of 16 cost
// 400 of a tile.  (Scales by copies of a page each: 64 x 5 tokens 138 us; all by
// 16-byte pieces: 148, and 256 x 9 tokens 1219 us.)
template <int kD, typename S, typename Control>
__device__ __forceinline__ void fp4_load(const Fp4Args& a, AttnWalk<S> u, Control* c, uint64_t* full,
                                         uint64_t* empty, char* ring, const CUtensorMap* k_map,
                                         const CUtensorMap* v_map, bool keys, bool values) {
  constexpr int kStages = S::kPackedStages;
  constexpr int kAhead = 4;                      // tiles whose pages are looked up ahead
  constexpr int kPerPiece = 16 / (kD / 16);      // keys of a piece of scales
  const int lane = threadIdx.x & 31;
  const int page = 1 << a.page_shift, box = min(page, S::kKeys), boxes = S::kKeys / box;
  const int box_shift = min(a.page_shift, 7);
  const int none = (a.n_pages * a.Hk) << a.page_shift;   // one past the cache's rows
  int it = 0, end = 0;   // the next copy, and the one after the last made
  bool ok = true, bad = false;

  // First row, in the cache, of the lane's page of key tile j; -1 if it has none.
  auto box_row = [&](int j) -> int {
    if (lane >= boxes) return -1;
    const int key = j * S::kKeys + lane * box;
    if (key >= u.units.row.L) return -1;
    const int pg = key >> a.page_shift;
    if (!in_array(a.flags, u.b, a.B) || !in_array(a.flags, pg, a.max_pages)) return -1;
    const int id = a.block_table[(long long)u.b * a.max_pages + pg];
    if (id >= 0 && id < a.n_pages) return ((id * a.Hk + u.h) << a.page_shift) + (key & (page - 1));
    bad = true;
    return none;
  };
  auto bring = [&](const CUtensorMap* map, const char* scales, int y) -> bool {
    const int stage = it % kStages, lap = it / kStages;
    if (lap > 0 && !mbar_await(smem_addr(&empty[stage]), (lap - 1) & 1, &c->abort_word, naps_of(a)))
      return false;
    const uint32_t bar = smem_addr(&full[stage]), to = smem_addr(ring + stage * Fp4Tile<kD>::kBytes);
    const unsigned who = __ballot_sync(0xffffffffu, y >= 0);
    if (lane == 0) mbar_arrive_expect(bar, __popc(who) * box * (kD / 2));
    __syncwarp();
    if (y >= 0) tma_load_2d(to + lane * box * (kD / 2), map, 0, y, bar);
#pragma unroll
    for (int i = 0; i < Fp4Tile<kD>::kScaleBytes / 512; ++i) {
      const int key = (i * 32 + lane) * kPerPiece;
      const int first = __shfl_sync(0xffffffffu, y, key >> box_shift), row = first + (key & (box - 1));
      const bool held = first >= 0 && first < none;
      if (first >= 0 && (!held || in_array(a.flags, row, none)))
        lane_load(to + Fp4Tile<kD>::kCodeBytes + i * 512 + lane * 16, scales + (held ? (long long)row * (kD / 16) : 0),
                  held ? 16 : 0);
    }
    lane_loads_arrive(bar);
    end = it + 1;
    return true;
  };

#pragma unroll 1
  for (bool first = true; ok && u.next(first); first = false) {
    const int n = u.most();
    if (n == 0) continue;
    int y[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) y[i] = i < n ? box_row(u.j0 + i) : -1;
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      const int next = i + kAhead < n ? box_row(u.j0 + i + kAhead) : -1;
      if (keys) ok = bring(k_map, a.k_scales, y[0]);
      ++it;
      if (ok && values) ok = bring(v_map, a.v_scales, y[0]);
      ++it;
#pragma unroll
      for (int x = 0; x + 1 < kAhead; ++x) y[x] = y[x + 1];
      y[kAhead - 1] = next;
    }
  }
  if (bad) set_flag(a.flags, kDevBadPage);
  // copies in flight land in this CTA's memory, which has to outlive them
#pragma unroll 1
  for (int i = max(0, end - kStages); i < end; ++i)
    if (i % 2 ? values : keys)
      (void)mbar_poll(smem_addr(&full[i % kStages]), (i / kStages) & 1, &c->calm, kNaps);
  __syncwarp();
}

}  // namespace sv
