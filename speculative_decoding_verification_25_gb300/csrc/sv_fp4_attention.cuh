// Attention of each request's new tokens over its paged keys and values of 4 bits.
//
// The mathematics is that of sv_paged_attention.cuh; both products run on the
// tensor core, transposed: with the cache's part as the first operand,
//   S^T = K Q^T      128 keys x the unit's query rows,
//   O^T += V^T P^T   kD columns x query rows.
// A tile of the first operand has 128 rows whatever it holds, so the cache fills
// it and the few query rows of a token or a draft are the short side (16
// to kRows columns).  The first operand comes from tensor memory, where the CTA's
// warps write what they unpack: shared memory carries the cache as it is packed,
// 0.56 bytes a value, and would be the bound of 16-bit tiles (5 bytes a value).
//
// Operands are float16 whatever the queries' type.  A code times a scale is exact
// there.  bfloat16 queries are scaled by a power of two that a unit's rows share, and
// have steps of 2^-32 of the unit's largest magnitude or less (few or none of them
// need their rounding: eight bits are exact down to 2^-25 of it).
// Probabilities are rounded to 11 bits (see kFp4Below).  The caller's gains go into
// the scores' factor and into the results'.
//
// A thread of the softmax has a key and the scores of all rows.  A row's
// reference is common to the tile: it changes only when some score exceeds the
// maximum that set it by more than kSlack, which one vote of the warps tells; then the maxima are
// taken across the threads, and what was summed is scaled.  Row sums stay
// with the threads until the unit ends.
//
// Work is cut into ranges and joined as in sv_paged_attention.cuh.
//
// Bound by instruction issue over long contexts: 4 x 1 token over 60 k to 131 k
// keys, 64/8 heads of 128, 120 us for 426 MB, 3.5 TB/s, issue at 68% of its slots, the
// tensor pipe at 8% (one CTA per SM and products issued by a chosen lane: 204).
// It is compiled for 64 registers and spills 168 bytes a thread (16 rows, D = 128).
// Drafts (64 x 5 tokens over 203 to 4099 keys, 32/8 heads, 32 rows) 90 us for 162 MB:
// units of up to 33 tiles, whose start and end take about 10 us each.
#pragma once

#include "sv_fp4_load.cuh"

namespace sv {

template <int kD, int kRowsMost>
struct Fp4Shape {
  static constexpr bool kFp4 = true;
  static constexpr int kTiles = 1;
  static constexpr int kKeys = 128;
  static constexpr int kRows = kRowsMost;                  // query rows of a unit, at most
  static constexpr int kUnitCost = 768;
  static constexpr int kSoftThreads = 128;
  static constexpr int kThreads = kSoftThreads + 2 * 128 + 128;
  static constexpr int kBlocks = kD / 64;
  static constexpr int kQBytes = kRows * kD * 2;           // two of them
  static constexpr int kPRow = kRows * 2;                  // bytes of a row of P^T
  static constexpr int kPBytes = 128 * kPRow;              // two of them
  static constexpr int kStageBytes = Fp4Tile<kD>::kBytes;
  static constexpr int kCtasPerSm = 2;
  static constexpr int kTmemCols = 512 / kCtasPerSm;
  static constexpr int kValueScales = 128 * (kD / 16) * 2; // float16
  static constexpr int kControlBytes = 1024;
  static constexpr int kStatBytes = kRows * 4 * (4 + 3);   // of four warps, and three of a row
  static constexpr int kFixedBytes = 2 * (kQBytes + kPBytes) + kValueScales + kControlBytes + kStatBytes;
  static constexpr int kMostStages = (228 * 1024 / kCtasPerSm - 1024 - kFixedBytes) / kStageBytes;
  static constexpr int kPackedStages = kMostStages >= 16 ? 16 : kMostStages >= 8 ? 8 : 4;   // a power of two
  static constexpr int kSmemBytes = kFixedBytes + kPackedStages * kStageBytes;
  // columns of tensor memory
  static constexpr int kS = 0, kO = 2 * kRows, kK = 3 * kRows, kV = kK + 64;
  static_assert(kV + 64 <= kTmemCols, "fits");
  static_assert(kMostStages >= 4, "fits");
};

struct Fp4Control {
  uint64_t full[16], empty[16];
  uint64_t q_full[2], q_free[2], k_ready, s_full[2], pv_ready[2], pv_done[2];
  uint64_t drain, met;
  uint32_t tmem;
  int abort_word, calm, last;
  unsigned status;
  int q_exponent[2];          // for the scores' factor
  AttnStart start;
  long long sums[20];
};
static_assert(sizeof(Fp4Control) <= 1024, "fits kControlBytes");

// Four warps meet (barrier `id`); whether any, or all, of them say so.
__device__ __forceinline__ bool vote_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool vote_all(int id, bool x) { return !vote_any(id, !x); }

// Largest of the warp's values, NaN aside.
__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// row / G for rows below 128, by a product.
__device__ __forceinline__ uint32_t group_inverse(int G) { return 65536u / (uint32_t)G + 1; }
__device__ __forceinline__ int group_of(int row, uint32_t inverse) { return (int)((uint32_t)row * inverse >> 16); }

// ------------------------------------------------------------------ queries
// One warp brings a unit's rows to shared memory as float16, columns past them
// zero, a unit ahead of their use.
template <typename E, int kD, typename S>
__device__ __forceinline__ void fp4_queries(const Fp4Args& a, AttnWalk<S> u, Fp4Control* c, char* q_ptr) {
  constexpr bool kBf16 = std::is_same<E, __nv_bfloat16>::value;
  constexpr int kLanes = kD / 8, kPass = 32 / kLanes, kAhead = 4;   // rows per pass, passes in flight
  const int lane = threadIdx.x & 31, part = lane % kLanes;
  const uint32_t per_g = group_inverse(a.G);
  int rounds = 0;
#pragma unroll 1
  for (bool first = true; u.next(first); first = false) {
    if (u.count(0) == 0) continue;
    const int buf = rounds % 2, rows = u.rows(), cols = (rows + 15) / 16 * 16;
    if (rounds >= 2 && !mbar_await(smem_addr(&c->q_free[buf]), (rounds / 2 - 1) & 1, &c->abort_word, naps_of(a)))
      break;
    char* to = q_ptr + buf * S::kQBytes + (part / 8) * (S::kRows * 128);
    auto load = [&](int row, uint32_t (&w)[4]) {
      w[0] = w[1] = w[2] = w[3] = 0;
      if (row >= rows) return;
      const int i = group_of(row, per_g), t = u.units.row.begin + u.first(0) + i, h = u.h * a.G + row - i * a.G;
      if (in_array(a.flags, t, a.T)) ldg_stream16(a.q + t * a.q_pitch + h * (kD * 2) + part * 16, w);
    };
    auto store = [&](int row, const uint32_t (&w)[4]) {
      if (row < cols)
        *(uint4*)(to + row * 128 + ((part % 8) ^ (row % 8)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    };
    // The first try is right for a largest magnitude of 2^-3 to 2^5, which is 2^8 to 2^16
    // then; other units are done again, with their own exponent.
    int exponent = kBf16 ? -11 : 0;
#pragma unroll 1
    for (int again = 0; again < 2; ++again) {
      const uint32_t factor = query_factor(exponent);
      uint32_t high = 0;
#pragma unroll 1
      for (int r0 = lane / kLanes; r0 < cols; r0 += kPass * kAhead) {
        uint32_t w[kAhead][4];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(r0 + i * kPass, w[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (kBf16) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              high = __vmaxu2(high, bf16_magnitudes(w[i][x], false));
              w[i][x] = query_pair(w[i][x], factor);
            }
          }
          store(r0 + i * kPass, w[i]);
        }
      }
      if (!kBf16 || again) break;
      uint32_t top = __reduce_max_sync(0xffffffffu, larger_half(high));
      if (top >= kBf16Infinity) {   // the largest of the others
        high = 0;
#pragma unroll 1
        for (int r = lane / kLanes; r < cols; r += kPass) {
          uint32_t w[4];
          load(r, w);
          for (int x = 0; x < 4; ++x) high = __vmaxu2(high, bf16_magnitudes(w[x], true));
        }
        top = __reduce_max_sync(0xffffffffu, larger_half(high));
      }
      if (top == 0 || (top >= 0x3e00u && top < 0x4200u)) break;   // 2^-3, 2^5
      exponent = query_exponent(top);
    }
    fence_async_shared();
    if (lane == 0) c->q_exponent[buf] = score_exponent(a.scale_log2, exponent);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&c->q_full[buf]));
    ++rounds;
  }
}

// --------------------------------------------------------------- unpacking
// Within a block of 32 keys, key 16 h + 4 c + j.  The values' columns (see
// fp4_values) put it at place 8 j + 2 c + h of P^T.  The key of lane x is chosen
// so that eight lanes in a row meet no bank conflict, neither in the packed
// keys (differing key mod 8) nor in P^T (differing place mod 8).
__device__ __forceinline__ int fp4_key(int x) {
  const int c = x % 8 / 2, h = x % 2, j = (2 * (c / 2) + h + x % 32 / 8) % 4;
  return x / 32 * 32 + 16 * h + 4 * c + j;
}
__device__ __forceinline__ int fp4_place(int key) {
  return key / 32 * 32 + 8 * (key % 4) + 2 * (key % 16 / 4) + key % 32 / 16;
}
// Four warps: a thread unpacks a key to its lane of tensor memory, two columns
// of the head a column.
template <int kD, typename S>
__device__ __forceinline__ void fp4_keys(const Fp4Args& a, AttnWalk<S> u, Fp4Control* c, const char* ring,
                                         uint32_t tmem) {
  const int lane = threadIdx.x & 31, x = threadIdx.x % 128, key = fp4_key(x);
  const uint32_t to = tmem + ((uint32_t)(x / 32 * 32) << 16) + S::kK;
  int g = 0;
#pragma unroll 1
  for (bool first = true; u.next(first); first = false) {
    const int n = u.count(0);
#pragma unroll 1
    for (int i = 0; i < n; ++i, ++g) {
      const int stage = 2 * g % S::kPackedStages, lap = 2 * g / S::kPackedStages;
      if (!mbar_await(smem_addr(&c->full[stage]), lap & 1, &c->abort_word, naps_of(a))) return;
      const char* tile = ring + stage * S::kStageBytes;
      // the scores of the tile before are done, and its keys free
      if (g > 0 && !mbar_await(smem_addr(&c->s_full[(g - 1) % 2]), ((g - 1) / 2) & 1, &c->abort_word, naps_of(a)))
        return;
      tc_fence_after();
      uint4 w = *(const uint4*)(tile + fp4_piece<kD>(key, 0));
      // rolled up: a role's code is run once a tile by one warp of a scheduler, and
      // long code waits for its instructions
#pragma unroll 1
      for (int p = 0; p < kD / 32; ++p) {
        const uint32_t pair = fp4_scales(*(const uint16_t*)(tile + Fp4Tile<kD>::kCodeBytes + key * (kD / 16) + p * 2));
        const uint32_t s0 = __byte_perm(pair, 0, 0x1010), s1 = __byte_perm(pair, 0, 0x3232);
        uint32_t r[16];
        fp4_unpack(w.x, r);
        fp4_unpack(w.y, r + 4);
        fp4_unpack(w.z, r + 8);
        fp4_unpack(w.w, r + 12);
        if (p + 1 < kD / 32) w = *(const uint4*)(tile + fp4_piece<kD>(key, p + 1));
#pragma unroll
        for (int y = 0; y < 16; ++y) r[y] = mul_f16x2(r[y], y < 8 ? s0 : s1);
        tmem_store16(to + p * 16, r);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&c->empty[stage]));
      tmem_wait_store();
      hand_over(&c->k_ready);
    }
  }
}

// Four warps: 32 columns of the head each, transposed.  ldmatrix gives lane l, of
// 16 keys and 16 bytes of codes, the bytes l / 4 and l / 4 + 8 of keys 4 c to
// 4 c + 3, c = l % 4.  The halves of two blocks' bytes are put together, so that a
// byte has one column of keys 4 c + j and 16 + 4 c + j and unpacks to a column
// of tensor memory; even columns of the head go to lanes 0 to 15, odd ones to 16
// to 31.  Scales become float16 pairs of those keys in shared memory first (the
// warp's two groups): those past the request's length 0, whatever they were, so
// that the values there are 0 too.
template <int kD, typename S>
__device__ __forceinline__ void fp4_values(const Fp4Args& a, AttnWalk<S> u, Fp4Control* c, const char* ring,
                                           uint32_t tmem, char* scale_ptr) {
  constexpr uint32_t kLow = 0x0f0f0f0fu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x % 128 / 32;
  const bool active = warp < kD / 32;
  const uint32_t to = tmem + ((uint32_t)(warp * 32) << 16) + S::kV;
  uint32_t* scales = (uint32_t*)(scale_ptr + (active ? warp : 0) * 512);   // [2][64] pairs
  int g = 0;
#pragma unroll 1
  for (bool first = true; u.next(first); first = false) {
    const int n = u.count(0);
#pragma unroll 1
    for (int i = 0; i < n; ++i, ++g) {
      const int stage = (2 * g + 1) % S::kPackedStages, lap = (2 * g + 1) / S::kPackedStages;
      if (!mbar_await(smem_addr(&c->full[stage]), lap & 1, &c->abort_word, naps_of(a))) return;
      const char* tile = ring + stage * S::kStageBytes;
      if (active) {
        const int left = u.units.row.L - (u.j0 + i) * S::kKeys;   // keys of the tile within the request
#pragma unroll
        for (int y = 0; y < 2; ++y) {   // pairs lane and 32 + lane
          const int key = (y * 2 + lane / 16) * 32 + lane % 16;
          const char* from = tile + Fp4Tile<kD>::kCodeBytes + key * (kD / 16) + warp * 2;
          const uint32_t s0 = key < left ? fp4_scales(*(const uint16_t*)from) : 0;
          const uint32_t s1 = key + 16 < left ? fp4_scales(*(const uint16_t*)(from + kD)) : 0;
          scales[y * 32 + lane] = __byte_perm(s0, s1, 0x5410);
          scales[64 + y * 32 + lane] = __byte_perm(s0, s1, 0x7632);
        }
      }
      // O += P V of the tile before is done, and its values free
      if (g > 0 && !mbar_await(smem_addr(&c->pv_done[(g - 1) % 2]), ((g - 1) / 2) & 1, &c->abort_word, naps_of(a)))
        return;
      tc_fence_after();
      if (active) {
        __syncwarp();
#pragma unroll 1
        for (int block = 0; block < 4; ++block) {   // of 32 keys
          const uint32_t from = smem_addr(tile) + fp4_piece<kD>(block * 32 + lane, warp);
          uint32_t m[4];   // bytes l / 4 and l / 4 + 8 of the first 16 keys, and of the others
          asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                       : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3])
                       : "r"(from)
                       : "memory");
          uint32_t even[8], odd[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 s = *(const uint4*)(scales + h * 64 + block * 16 + lane % 4 * 4);
            uint32_t r[4];
            fp4_unpack((m[h] & kLow) | (m[2 + h] << 4 & ~kLow), r);
            even[h] = mul_f16x2(r[0], s.x);
            even[2 + h] = mul_f16x2(r[1], s.y);
            even[4 + h] = mul_f16x2(r[2], s.z);
            even[6 + h] = mul_f16x2(r[3], s.w);
            fp4_unpack((m[h] >> 4 & kLow) | (m[2 + h] & ~kLow), r);
            odd[h] = mul_f16x2(r[0], s.x);
            odd[2 + h] = mul_f16x2(r[1], s.y);
            odd[4 + h] = mul_f16x2(r[2], s.z);
            odd[6 + h] = mul_f16x2(r[3], s.w);
          }
          tmem_store_16x16(to + block * 16, even);
          tmem_store_16x16(to + (16u << 16) + block * 16, odd);
        }
        tmem_wait_store();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&c->empty[stage]));
      hand_over(&c->pv_ready[g % 2]);
    }
  }
}

// ----------------------------------------------------------------- products
// One warp.  The scores of a tile are issued before O += P V of the tile before
// it, across units, so that a softmax does not wait for that product.  In this
// order the scores of a tile come after the softmax of the tile whose buffer they
// take, and when they are done so is O += P V of that tile, which leaves P's.  (A
// wait sees a phase's parity alone: products are told by two barriers in turn, so
// that whoever waits for one knows that the one before it on its barrier is done.)
template <int kD, typename S>
__device__ __forceinline__ void fp4_multiply(const Fp4Args& a, AttnWalk<S> u, Fp4Control* c, uint32_t q_smem,
                                             uint32_t p_smem, uint32_t tmem) {
  const uint64_t q_desc = tile_desc(q_smem, 16, 1024);
  const uint64_t p_desc = tile_desc(p_smem, 128 * 128, 8 * S::kPRow, S::kPRow);
  int g = 0, rounds = 0;
  bool ok = true;
  uint32_t before = 0;   // columns of the tile before, and whether it began its unit
  bool began = false;

  auto values = [&](int t) -> bool {   // O^T (+)= V^T P^T of tile t
    if (!mbar_await(smem_addr(&c->pv_ready[t % 2]), (t / 2) & 1, &c->abort_word, naps_of(a))) return false;
    tc_fence_after();
    const uint32_t desc = mma_desc(false, 128, (int)before, true);
    const uint64_t p = p_desc + (t % 2) * (S::kPBytes / 16);
    if (elect_one()) {
#pragma unroll
      for (int x = 0; x < S::kKeys / 16; ++x)
        mma_tmem_one(tmem + S::kO, tmem + S::kV + x * 8, p + x * S::kPRow, desc, !began || x > 0);
      tc_commit_one(smem_addr(&c->pv_done[t % 2]));
    }
    __syncwarp();
    return true;
  };

#pragma unroll 1
  for (bool first = true; ok && u.next(first); first = false) {
    const int n = u.count(0);
    if (n == 0) continue;
    const uint32_t cols = (u.rows() + 15) / 16 * 16, desc = mma_desc(false, 128, (int)cols, false);
    const int q_buf = rounds % 2;
    if (!(ok = mbar_await(smem_addr(&c->q_full[q_buf]), (rounds / 2) & 1, &c->abort_word, naps_of(a)))) break;
    ++rounds;
    const uint64_t q = q_desc + q_buf * (S::kQBytes / 16);
#pragma unroll 1
    for (int i = 0; i < n; ++i, ++g) {
      if (!(ok = mbar_await(smem_addr(&c->k_ready), g & 1, &c->abort_word, naps_of(a)))) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int d = 0; d < kD / 16; ++d)
          mma_tmem_one(tmem + S::kS + g % 2 * S::kRows, tmem + S::kK + d * 8,
                       q + (d / 4) * (S::kRows * 128 / 16) + (d % 4) * 2, desc, d > 0);
        tc_commit_one(smem_addr(&c->s_full[g % 2]));
        if (i == n - 1) tc_commit_one(smem_addr(&c->q_free[q_buf]));
      }
      __syncwarp();
      if (g > 0 && !(ok = values(g - 1))) break;
      before = cols;
      began = i == 0;
    }
  }
  if (ok && g > 0) (void)values(g - 1);
  // everything issued is done before the CTA's memory goes
  if (elect_one()) tc_commit_one(smem_addr(&c->drain));
  (void)mbar_poll(smem_addr(&c->drain), 0, &c->calm, kNaps);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
// Sums over the warp of kCount values per lane: lane x gets that of v[x % kCount].
template <int kCount>
__device__ __forceinline__ float warp_sums(float* v) {
  const int lane = threadIdx.x & 31;
  if (kCount == 16)
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
#pragma unroll
  for (int o = kCount / 2; o > 0; o >>= 1) {
    const bool high = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = high ? v[i + o] : v[i], give = high ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

// Four warps; none leaves alone: what went wrong is told at the next vote.
template <typename E, int kD, typename S>
__device__ __forceinline__ void fp4_softmax(const Fp4Args& a, AttnWalk<S> u, Fp4Control* c, uint32_t tmem,
                                            char* p_ptr, float* stats, long long quota, long long w1) {
  constexpr int kCols = S::kRows, kChunk = 16;
  constexpr bool kKeep = kCols == kChunk;                 // scores stay in registers over the vote
  constexpr int id = 1;                                   // of the barrier
  const int lane = threadIdx.x & 31, x = threadIdx.x, warp = x / 32;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const int my_key = fp4_key(x), place = fp4_place(my_key);
  float* tops = stats;                                    // [warp][kCols], then of a row:
  float* refs = tops + 4 * kCols;                            // the negative reference
  float* marks = refs + kCols;                               // the reference, or its inverse sum
  float* factors = marks + kCols;
  // 16-byte pieces of the thread's row of P^T, as the product's layout swizzles them
  const int turn = S::kPRow == 64 ? place / 2 % 4 : place / 4 % 2;
  char* p_row = p_ptr + place * S::kPRow;
  const uint32_t s_col = tmem + lanes + S::kS, o_col = tmem + lanes + S::kO;
  const uint32_t per_g = group_inverse(a.G);
  int g = 0, rounds = 0, meetings = 0;
  bool ok = true;

#pragma unroll 1
  for (bool first = true; u.next(first); first = false) {
    const int n = u.count(0);
    const int rows = u.rows(), cols = (rows + 15) / 16 * 16;
    float l[kCols];
#pragma unroll
    for (int y = 0; y < kCols; ++y) l[y] = 0.f;
    float f = a.scale_log2;
    if (n > 0) {
      const int q_buf = rounds % 2;
      ok = ok && mbar_await(smem_addr(&c->q_full[q_buf]), (rounds / 2) & 1, &c->abort_word, naps_of(a));
      f = ldexpf(f, c->q_exponent[q_buf]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&c->q_free[q_buf]));
      ++rounds;
    }
    if (x < kCols) marks[x] = SV_NEG_INF;
    const unsigned long long f2 = f2_pack(f, f);
    // keys that every row sees; past them row y sees a key from (key - common) G on
    const int common = u.units.row.L - u.units.row.n + u.first(0);
#pragma unroll 1
    for (int i = 0; i < n; ++i, ++g) {
      const int buf = g % 2, key0 = (u.j0 + i) * S::kKeys;
      const int from = max(0, key0 + my_key - common) * a.G;   // the first row that sees the key
      const bool masked = key0 + S::kKeys - 1 > common;
      ok = ok && mbar_await(smem_addr(&c->s_full[buf]), (g / 2) & 1, &c->abort_word, naps_of(a));
      tc_fence_after();
      const uint32_t s_at = s_col + buf * S::kRows;
      uint32_t s[kChunk];
      // a chunk's scores, or their exponents once `refs` is set
      auto scores = [&](int y0) {
#pragma unroll
        for (int y = 0; y < kChunk; y += 16)
          if (y0 + y < cols) tmem_load16(s_at + y0 + y, s + y);
        tmem_wait_load();
        tmem_pin<kChunk>(s);
        if (masked)
#pragma unroll
          for (int y = 0; y < kChunk; ++y)
            if (y0 + y < from) s[y] = 0xff800000u;
      };
      auto exponents = [&](int y0) {
#pragma unroll
        for (int y = 0; y < kChunk; y += 4) {
          if (y0 + (y & 16) >= cols) continue;
          const float4 r = *(const float4*)(refs + y0 + y);
          float e0, e1, e2, e3;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(s[y]), __uint_as_float(s[y + 1])), f2, f2_pack(r.x, r.y)), e0, e1);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(s[y + 2]), __uint_as_float(s[y + 3])), f2, f2_pack(r.z, r.w)), e2, e3);
          s[y] = __float_as_uint(e0), s[y + 1] = __float_as_uint(e1);
          s[y + 2] = __float_as_uint(e2), s[y + 3] = __float_as_uint(e3);
        }
      };
      bool raise = i == 0 || !ok;
      if (!raise) {
        float top = SV_NEG_INF;
#pragma unroll
        for (int y0 = 0; y0 < kCols; y0 += kChunk) {
          if (y0 >= cols) continue;
          scores(y0);
          exponents(y0);
#pragma unroll
          for (int y = 0; y < kChunk; y += 2)
            if (y0 + (y & 16) < cols) top = max3(top, __uint_as_float(s[y]), __uint_as_float(s[y + 1]));
        }
        raise = top > kFp4Below + kSlack;
      }
      if (i == 0 || vote_any(id, raise)) {
        if (!vote_all(id, ok)) return;
        // maxima of the rows, over the warp's keys and then over the warps
#pragma unroll 1
        for (int y0 = 0; y0 < cols; y0 += kChunk) {
          scores(y0);
          float mine = SV_NEG_INF;
#pragma unroll
          for (int y = 0; y < kChunk; ++y) {
            if (y0 + (y & 16) >= cols) continue;
            const float top = redux_max(__uint_as_float(s[y]));
            if (lane == y) mine = top;
          }
          if (lane < kChunk) tops[warp * kCols + y0 + lane] = mine;
        }
        (void)vote_any(id, false);
        if (x < cols) {
          const float high = fmaf(fmaxf(fmaxf(tops[x], tops[kCols + x]), fmaxf(tops[2 * kCols + x], tops[3 * kCols + x])), f,
                                  -kFp4Below);
          const float old = marks[x];
          const bool up = i == 0 ? high > old : high > old + kSlack;
          const float now = up ? high : old;
          factors[x] = !up ? 1.f : old == SV_NEG_INF ? 0.f : ex2_approx(old - high);
          marks[x] = now;
          refs[x] = now == SV_NEG_INF ? 1e30f : -now;   // any finite score of such a row raises it
        }
        (void)vote_any(id, false);
        if (i > 0) {
#pragma unroll
          for (int y = 0; y < kCols; ++y)
            if (y < cols) l[y] *= factors[y];
          ok = mbar_await(smem_addr(&c->pv_done[(g - 1) % 2]), ((g - 1) / 2) & 1, &c->abort_word, naps_of(a));
          tc_fence_after();
          if (ok) {
#pragma unroll 1
            for (int y0 = 0; y0 < cols; y0 += 16) {
              uint32_t o[16];
              tmem_load16(o_col + y0, o);
              tmem_wait_load();
              tmem_pin<16>(o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * factors[y0 + y]);
              tmem_store16(o_col + y0, o);
            }
            tmem_wait_store();
          }
        }
        if (kKeep && cols > 0) {
          scores(0);
          exponents(0);
        }
      }
      if (!ok) continue;
      char* p_at = p_row + buf * S::kPBytes;
#pragma unroll
      for (int y0 = 0; y0 < kCols; y0 += kChunk) {
        if (y0 >= cols) continue;
        if (!kKeep) {
          scores(y0);
          exponents(y0);
        }
#pragma unroll
        for (int y = 0; y < kChunk; y += 8) {
          if (y0 + (y & 16) >= cols) continue;
          uint32_t p[4];
#pragma unroll
          for (int z = 0; z < 8; z += 2) {
            const float p0 = ex2_approx(__uint_as_float(s[y + z])), p1 = ex2_approx(__uint_as_float(s[y + z + 1]));
            f2_unpack(f2_add(f2_pack(l[y0 + y + z], l[y0 + y + z + 1]), f2_pack(p0, p1)), l[y0 + y + z], l[y0 + y + z + 1]);
            p[z / 2] = pack2(p0, p1, __half());
          }
          *(uint4*)(p_at + (((y0 + y) / 8) ^ turn) * 16) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&c->pv_ready[buf]));
    }
    // ---- the unit's end: sums over the threads, results or a part of them
    if (n > 0)
      ok = ok && mbar_await(smem_addr(&c->pv_done[(g - 1) % 2]), ((g - 1) / 2) & 1, &c->abort_word, naps_of(a));
    tc_fence_after();
#pragma unroll
    for (int y0 = 0; y0 < kCols; y0 += kChunk)
      if (y0 < cols) {
        const float sum = warp_sums<kChunk>(l + y0);
        if (lane < kChunk) tops[warp * kCols + y0 + lane] = sum;
      }
    if (!vote_all(id, ok)) return;
    const bool whole = u.j0 == 0 && u.j1 == u.tiles;
    const int cta = blockIdx.x;
    const long long ahead = w1 - u.left - u.pos - cta * quota;
    const int c_first = cta - ranges_back(u.pos, quota);
    const bool begins_late = ahead + (cta - c_first) * quota != 0;
    const size_t slots = (size_t)gridDim.x * 2;
    const size_t slot = (size_t)cta * 2 + (cta == c_first && begins_late ? 1 : 0);
    const long long out_rows = (long long)a.T * a.Hq, part_rows = min((long long)slots * S::kRows, kAttnRows);
    const int token0 = u.units.row.begin + u.first(0);
    if (x < rows) {
      const float sum = tops[x] + tops[kCols + x] + tops[2 * kCols + x] + tops[3 * kCols + x], mark = marks[x];
      // One factor for both: it is subnormal for gains below 2^-80 alone, and with the least,
      // 2^-100, still has 12 bits for a sum of 2^38, that of 2^31 keys of the largest score.
      // (Gain apart, where values are stored: verify 93.5 us, so 91.)
      factors[x] = whole ? row_inverse(sum) * a.v_gain : 1.f;
      if (whole) {
        const int i = group_of(x, per_g);
        const long long row = (long long)(token0 + i) * a.Hq + u.h * a.G + x - i * a.G;
        if (a.lse && in_array(a.flags, row, out_rows)) a.lse[row] = row_lse(mark, sum);
      } else {
        const long long row = (long long)slot * S::kRows + x;
        if (in_array(a.flags, row, part_rows))
          ((float2*)(a.partial + slots * S::kRows * kD))[row] = make_float2(mark, sum);
      }
    }
    (void)vote_any(id, false);
    if (warp < kD / 32) {
      // lanes 0 to 15 have even columns of the head, 16 to 31 odd ones: they trade, so that a
      // lane has two neighbours of one of two rows
      const bool upper = lane >= 16;
      const int column = warp * 32 + lane % 16 * 2;
#pragma unroll 1
      for (int y0 = 0; y0 < cols; y0 += 16) {
        uint32_t o[16];
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] = 0;
        if (n > 0) {
          tmem_load16(o_col + y0, o);
          tmem_wait_load();
          tmem_pin<16>(o);
        }
#pragma unroll
        for (int y = 0; y < 16; y += 2) {
          const float v0 = __uint_as_float(o[y]) * factors[y0 + y], v1 = __uint_as_float(o[y + 1]) * factors[y0 + y + 1];
          const float other = __shfl_xor_sync(0xffffffffu, upper ? v0 : v1, 16);
          const float lo = upper ? other : v0, hi = upper ? v1 : other;
          const int r = y0 + y + upper;
          if (r >= rows) continue;
          if (whole) {
            const int i = group_of(r, per_g);
            const long long row = (long long)(token0 + i) * a.Hq + u.h * a.G + r - i * a.G;
            if (in_array(a.flags, row, out_rows)) *(uint32_t*)(a.out + (row * kD + column) * 2) = pack2(lo, hi, E());
          } else {
            const long long row = (long long)slot * S::kRows + r;
            if (in_array(a.flags, row, part_rows)) *(float2*)(a.partial + row * kD + column) = make_float2(lo, hi);
          }
        }
      }
    }
    tc_fence_before();
    if (whole) continue;
    // the CTA that has the unit's last tile; tickets as in attn_softmax
    const long long end = ahead + (long long)(u.tiles - 1) * S::kKeys;
    const int c_last = u.j1 == u.tiles ? cta : cta + ranges_ahead(end, quota);
    ok = soft_meet(c, meetings++, naps_of(a));
    if (threadIdx.x == 0) {
      const bool last = ok && in_array(a.flags, c_first, gridDim.x) &&
                        take_ticket(&a.tickets[c_first]) == c_last - c_first;
      if (last) a.tickets[c_first] = 0;
      c->last = last;
    }
    ok = soft_meet(c, meetings++, naps_of(a)) && ok;
    if (ok && c->last) {
      const int parts = c_last - c_first + 1;
      if (u.rows() * (kD / 4) <= S::kSoftThreads)
        attn_join<E, kD, S, kD / 4, 8>(a, u, c_first, parts, begins_late);
      else
        attn_join<E, kD, S, 8, 2>(a, u, c_first, parts, begins_late);
    }
  }
}

template <typename E, int kD, int kRows>
__global__ void __launch_bounds__(Fp4Shape<kD, kRows>::kThreads, Fp4Shape<kD, kRows>::kCtasPerSm)
    sv_fp4_attention_kernel(const __grid_constant__ Fp4Args a, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ CUtensorMap v_map) {
  using S = Fp4Shape<kD, kRows>;
  extern __shared__ __align__(1024) char smem[];
  char* q_ptr = smem;
  char* p_ptr = q_ptr + 2 * S::kQBytes;
  char* ring = p_ptr + 2 * S::kPBytes;
  char* value_scales = ring + S::kPackedStages * S::kStageBytes;
  float* stats = (float*)(value_scales + S::kValueScales);
  Fp4Control* c = (Fp4Control*)((char*)stats + S::kStatBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kSoft = S::kSoftThreads / 32, kKeyWarps = kSoft, kValueWarps = kSoft + 4, kLoader = kSoft + 8;

  if (warp == kLoader && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < S::kPackedStages; ++i) {
      mbar_init(smem_addr(&c->full[i]), 33);   // the boxes' and the lanes'
      mbar_init(smem_addr(&c->empty[i]), 4);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&c->q_full[i]), 1);
      mbar_init(smem_addr(&c->q_free[i]), 1 + kSoft);
      mbar_init(smem_addr(&c->s_full[i]), 1);
      mbar_init(smem_addr(&c->pv_ready[i]), kSoft + 4);
      mbar_init(smem_addr(&c->pv_done[i]), 1);
    }
    mbar_init(smem_addr(&c->k_ready), 4);
    mbar_init(smem_addr(&c->drain), 1);
    mbar_init(smem_addr(&c->met), kSoft);
    mbar_init_fence();
    c->abort_word = c->calm = 0;
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  if (warp == kLoader + 1) tmem_alloc<S::kTmemCols>(smem_addr(&c->tmem));
  wait_for_preceding_grid();
  const AttnRange range = attn_range<S>(a, c);
  const uint32_t tmem = c->tmem;
  if (range.w0 < range.w1) {
    const AttnWalk<S> u(a, c->start, range.w1 - range.w0);
    // Launched with 64 registers a thread in four warpgroups; 16 rows 80 + 2 x 64 + 48,
    // 32 rows 96 + 2 x 56 + 48.
    if (warp < kKeyWarps) {
      if (kRows == 16) asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
      else asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
      fp4_softmax<E, kD, S>(a, u, c, tmem, p_ptr, stats, range.quota, range.w1);
    } else if (warp < kLoader) {
      if (kRows > 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      if (warp < kValueWarps) fp4_keys<kD, S>(a, u, c, ring, tmem);
      else fp4_values<kD, S>(a, u, c, ring, tmem, value_scales);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
      if (warp == kLoader) fp4_load<kD, S>(a, u, c, c->full, c->empty, ring, &k_map, &v_map, true, false);
      else if (warp == kLoader + 1) fp4_multiply<kD, S>(a, u, c, smem_addr(q_ptr), smem_addr(p_ptr), tmem);
      else if (warp == kLoader + 2) fp4_load<kD, S>(a, u, c, c->full, c->empty, ring, &k_map, &v_map, false, true);
      else fp4_queries<E, kD, S>(a, u, c, q_ptr);
    }
  }
  attn_finish<S, kD>(a, c, range.spoilt);
  if (warp == kLoader + 1) tmem_free<S::kTmemCols>(tmem);
}

}  // namespace sv
