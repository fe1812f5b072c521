// Attention of each request's new tokens over its paged keys and values.
//
// With s_j = scale * log2(e) * q.k_j and any reference r, the result is
// sum_j 2^(s_j - r) v_j / sum_j 2^(s_j - r).  Keys are taken a tile at a time;
// r follows the running maximum only when that has risen by more than
// kSlack, so a tile seldom has to scale what was summed before it, and the
// probabilities stay below 2^kSlack.  (Three whole prompts of 4000 to 8192
// tokens: 629 us; following every rise, 722 us.)
//
// Times here are of calls replayed from a graph in short bursts, the SM clock
// at 2070 MHz.  Under a load of seconds the card's power cap takes the clock to
// 1950 MHz, and prompts take 6% longer, replayed or called (670 and 671 us).
//
// Both products run on the tensor core (tcgen05).  A query tile is 128 rows:
// the G query heads of one key head for 128 / G consecutive tokens, since
// they share every key and value.  S = Q K^T goes to tensor memory; four
// warps take it a row per thread, leave P = 2^(S - r), rounded to the
// operands' type (the product takes no other), in the place of S, and
// O += P V reads P from there.  All sums are float32, that of P is of P before
// its rounding.  The rounding of P adds as much to a result's error as that of
// the result itself: normal keys and values differ from 64 bits by 0.0023
// relative in bfloat16, 0.0017 without it, and by 0.00028 and 0.00021 in
// float16 (a sum of the rounded P gives the same).  float16 has steps of 2^-24:
// probabilities below that of the reference's are lost.  Rows never meet: no
// shuffle, and unused rows may hold anything.
//
// A CTA is one or two loader warps (TMA into a ring of key and value tiles) and,
// per query tile, one warp that issues the products and four softmax warps.
// Two forms:
//   wide    two query tiles of one unit against tiles of 128 keys: while one
//           tile's softmax runs, the tensor core works on the other's.  Bound
//           by the chain of a tile, about 3000 clocks per 256 x 128 scores, of
//           which the tensor core is busy for 2048: a softmax of 1200, then
//           from P to the next S 1600 (the products' 1024, their start, the
//           hand-overs) and what the other tile's turn adds.  1.52 PFLOP/s on
//           chunks of 2048 tokens over contexts of 5000 to 7000 (1.43 under
//           the power cap).
//   narrow  one query tile against tiles of 64 keys, two S buffers, and two
//           CTAs per SM: for up to 128 rows per request, where the time is
//           that of reading the cache: 6.6 to 6.7 TB/s on long contexts.
// TMEM holds 128 lanes x 512 columns: wide fills it at D = 128 with S (P in
// its place) and O of both tiles, 4 x 128.  Tiles of 64 keys with two S
// buffers instead made prompts slower (a product of 64 columns takes 58
// clocks, one of 128 columns 64).
//
// The work is the key tiles of all (request, key head, query unit) in that
// order, cut into equal ranges of keys, one per CTA: every CTA sums the rows'
// keys to find its range, so no length is needed on the host.  A unit that
// a range's end cuts leaves unnormalised sums in the workspace; the CTA that
// takes the unit's last ticket joins them, always in the order of the CTAs,
// so results do not depend on timing and no CTA waits for another.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "sv_paged.cuh"
#include "sv_ranges.h"
#include "sv_tensor.cuh"

namespace sv {

constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.693147181f;
constexpr float kSlack = 8.f;        // in log2: probabilities up to 256, exact in both types' range
constexpr int kAttnMaxCtas = 320;    // resident CTAs that the workspace has room for (narrow)
constexpr int kAttnRowsPerSlot = 128;
// rows of partial sums in the workspace, for both forms
constexpr long long kAttnRows = 2ll * kAttnMaxCtas * kAttnRowsPerSlot;

struct AttnArgs {
  const int32_t* block_table;   // [B, max_pages]
  const int32_t* cu_new;        // [B+1]
  const int32_t* kv_len;        // [B]
  int B, T, Hq, Hk, G, page_shift, max_pages, n_pages;
  int tile_tokens;              // 128 / G
  float scale_log2;
  char* out;
  float* lse;                   // or nullptr
  int* tickets;                 // one per CTA, zero between calls
  unsigned* status;             // in the workspace: not 0 once a call has given up
  float* partial;               // [CTA][2][rows][D], then [CTA][2][rows][2]
  unsigned* flags;
  int naps;                     // checked build: polls after which a wait is given up
};
// A constant in the plain build (an argument there: verify 98.3 against 97.9 us,
// ragged chunks 54.7 against 54.2).
__device__ __forceinline__ int naps_of(const AttnArgs& a) { return kChecked ? a.naps : kNaps; }

template <int kD, bool kWide>
struct AttnShape {
  static constexpr int kTiles = kWide ? 2 : 1;
  static constexpr int kKeys = kWide ? 128 : 64;
  static constexpr int kBufs = kWide ? 1 : 2;        // S buffers per query tile
  static constexpr int kBlocks = kD / 64;            // 128-byte column blocks of a row
  static constexpr int kQBytes = 128 * kD * 2;
  static constexpr int kStageBytes = kKeys * kD * 2;
  static constexpr int kStages = kD == 128 ? 4 : 8;  // what is left of the shared memory
  static_assert(kStages % 2 == 0 || !kWide, "keys and values keep to their slots");
  static constexpr int kStagingBytes = 32 * 128;     // of a warp: rows on their way out
  static constexpr int kSoftThreads = 128 * kTiles;
  // wide: whole warpgroups, so that the softmax can take registers from the rest
  static constexpr int kThreads = kSoftThreads + (kWide ? 128 : 64);
  // A unit's start and end, in keys.  Wide, whole prompts / 37 ragged requests:
  // 687 / 68 us at 0, 637 / 57 at 192, 629 / 54.3 at 256, 631 / 55 at 320.
  // Narrow, 64 x 5 tokens
  // / 4 x 1 tokens over long caches: 99.0 / 228.5 us at 32, 98.0 / 227.9 at 64,
  // 98.0 / 228.3 at 128, 98.6 / 228.6 at 192.
  static constexpr int kUnitCost = kWide ? 256 : 64;
  static constexpr int kCtasPerSm = kWide ? 1 : 2;
  static constexpr int kTmemCols = kWide ? 512 : 256;
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kControlBytes = 512;
  static constexpr int kSmemBytes =
      kTiles * (kQBytes + 4 * kStagingBytes) + kStages * kStageBytes + kControlBytes;
};

// A request's lengths, clamped to what its arrays hold; n == 0: nothing to do.
struct AttnRow {
  int begin, n, L;
};
__device__ __forceinline__ AttnRow attn_row(const AttnArgs& a, int b, bool* bad = nullptr) {
  if (!in_array(a.flags, b, a.B)) return {0, 0, 0};
  const int begin = a.cu_new[b], end = a.cu_new[b + 1];
  const int most = a.max_pages << a.page_shift;
  const int len = a.kv_len[b];
  AttnRow r;
  r.begin = begin;
  const bool sound = begin >= 0 && end >= begin && end <= a.T;
  r.n = sound ? end - begin : 0;
  r.L = min(max(len, 0), most);
  if (bad && (!sound || r.L != len)) *bad = true;
  return r;
}
// The query units of a request: kTiles tiles of tile_tokens tokens each.  A
// unit's weight is the number of keys that its last token sees, or one key
// tile where that is more, and kUnitCost, so that weights sum in closed form;
// the last unit's keys are rounded up to key tiles, so that short contexts are
// cut between tiles.
template <typename S>
struct AttnUnits {
  AttnRow row;
  int step;      // tokens per unit
  int count;     // units

  __device__ __forceinline__ AttnUnits() {}
  __device__ __forceinline__ AttnUnits(const AttnArgs& a, const AttnRow& r)
      : row(r), step(S::kTiles * a.tile_tokens), count((r.n + step - 1) / step) {}
  // keys that the request's tokens up to t1 see
  __device__ __forceinline__ int seen(int t1) const { return max(0, row.L - row.n + t1); }
  __device__ __forceinline__ int keys(int m) const {
    if (m < count - 1) return max(S::kKeys, seen((m + 1) * step));
    return max(S::kKeys, (seen(row.n) + S::kKeys - 1) / S::kKeys * S::kKeys);
  }
  // weight of the first `units` units
  __device__ __forceinline__ long long before(int units) const {
    if (units == 0) return 0;
    const int full = min(units, count - 1);   // the last may be short
    const int context = row.L - row.n;
    // units of less than a key tile
    const int few = context < S::kKeys ? min(full, (S::kKeys - 1 - context) / step) : 0;
    const long long i0 = few + 1, i1 = full;
    return (long long)units * S::kUnitCost + (long long)few * S::kKeys + (i1 - few) * context +
           (i1 - few) * (i0 + i1) / 2 * step + (units > full ? keys(count - 1) : 0);
  }
};

// Where a CTA's range starts: `pos` keys into a unit.
struct AttnStart {
  AttnRow row;
  int count;     // units of the request
  int b, h, m, pos;
};

struct AttnControl {   // at the end of the shared memory
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty, drain, met;
  uint64_t s_full[2][2], p_ready[2][2];   // [tile][buffer]
  uint64_t pv_done[2];
  uint32_t tmem;
  volatile int past;          // units whose P the second tile's issuer has seen
  int abort_word;
  int calm;                   // an abort word that stays 0, for the waits of a CTA that gives up
  int last;
  unsigned status;            // what an earlier call left in the workspace
  AttnStart start;
  long long sums[12];
};

static_assert(sizeof(AttnControl) <= 512, "fits kControlBytes");

// A CTA's walk over its range of the work; every warp keeps its own.  A key
// tile is the CTA's whose range holds the tile's first key.
template <typename S>
struct AttnWalk {
  const AttnArgs& a;
  AttnUnits<S> units;
  int b, h, m;
  int pos;                    // where the range enters the unit
  int j0, j1;                 // key tiles of the unit that are this CTA's
  int tiles;                  // all key tiles of the unit
  long long left;             // of the range, this unit's part included

  __device__ __forceinline__ AttnWalk(const AttnArgs& args, const AttnStart& s, long long length)
      : a(args), b(s.b), h(s.h), m(s.m), pos(s.pos), left(length) {
    units.row = s.row;
    units.step = S::kTiles * a.tile_tokens;
    units.count = s.count;
  }
  // To the next unit of which the CTA has a tile, first of all to the first;
  // false at the end of the range.
  __device__ __forceinline__ bool next(bool first_of_all) {
#pragma unroll 1
    while (true) {
      if (!first_of_all) {
        left -= units.keys(m) + S::kUnitCost - pos;
        if (left <= 0) return false;
        pos = 0;
        if (++m == units.count) {
          m = 0;
          if (++h == a.Hk) {
            h = 0;
            next_row();
          }
        }
      }
      first_of_all = false;
      const int keys = units.keys(m);
      tiles = (keys + S::kKeys - 1) / S::kKeys;
      j0 = (pos + S::kKeys - 1) / S::kKeys;
      j1 = left >= keys - pos ? tiles : (pos + (int)left + S::kKeys - 1) / S::kKeys;
      if (j0 < j1) return true;
    }
  }
  // The next request with tokens (there is one: the range has not ended).
  __device__ __forceinline__ void next_row() {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (++b; b < a.B; b += 32) {
      const int mine = b + lane;
      const unsigned some =
          __ballot_sync(0xffffffffu, mine < a.B && attn_row(a, min(mine, a.B - 1)).n > 0);
      if (some) {
        b += __ffs(some) - 1;
        break;
      }
    }
    units = AttnUnits<S>(a, attn_row(a, b));
  }
  // The wide form's softmax needs its registers for the scores: its loop over the
  // tiles leaves the walk in shared memory (three whole prompts: 629 us; walk in
  // registers, 652).
  __device__ __forceinline__ void park(int4* p) const {
    if (S::kTiles == 1) return;
    if ((threadIdx.x & 31) == 0) {
      p[0] = make_int4(units.row.begin, units.row.n, units.row.L, units.count);
      p[1] = make_int4(units.step, b, h, m);
      p[2] = make_int4(pos, j0, j1, tiles);
      *(long long*)(p + 3) = left;
    }
    __syncwarp();
  }
  __device__ __forceinline__ void unpark(const int4* p) {
    if (S::kTiles == 1) return;
    const int4 x = p[0], y = p[1], z = p[2];
    left = *(const long long*)(p + 3);
    units.row.begin = x.x, units.row.n = x.y, units.row.L = x.z, units.count = x.w;
    units.step = y.x, b = y.y, h = y.z, m = y.w;
    pos = z.x, j0 = z.y, j1 = z.z, tiles = z.w;
    __syncwarp();
  }
  // Query tile t of the unit: its tokens [first, last) within the request,
  // and how many of the unit's key tiles it needs of this CTA.
  __device__ __forceinline__ int first(int t) const { return (m * S::kTiles + t) * a.tile_tokens; }
  __device__ __forceinline__ int last(int t) const {
    return min(units.row.n, first(t) + a.tile_tokens);
  }
  __device__ __forceinline__ int count(int t) const {
    if (first(t) >= units.row.n) return 0;
    return max(0, min(j1, (units.seen(last(t)) + S::kKeys - 1) / S::kKeys) - j0);
  }
  __device__ __forceinline__ int rows() const {   // query rows of the unit
    return (last(S::kTiles > 1 && first(1) < units.row.n ? 1 : 0) - first(0)) * a.G;
  }
  __device__ __forceinline__ int most() const {
    int c = count(0);
    if (S::kTiles > 1) c = max(c, count(1));
    return c;
  }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ------------------------------------------------------------------- loader
// One warp, in the wide form one for queries and keys and one for values (two
// prompt chunks, pages of 16: one warp 352 us, two 316; pages of 8: 509 and
// 344).  A key or value tile is kKeys rows of one head, a box of min(page,
// kKeys) rows per page and 128-byte column block; each lane brings one box.
// Rows of pages past the request's length stay as they are.  Keys and values
// alternate in the ring, and its slots are even in number, so a slot is always
// the same warp's.
template <typename S>
__device__ __forceinline__ void attn_load(const AttnArgs& a, AttnWalk<S> u, AttnControl* c,
                                          uint32_t q_smem, uint32_t ring, const CUtensorMap* q_map,
                                          const CUtensorMap* k_map, const CUtensorMap* v_map,
                                          bool keys, bool values) {
  const int lane = threadIdx.x & 31;
  const int page = 1 << a.page_shift;
  const int box = min(page, S::kKeys);
  const int boxes = S::kKeys / box;              // pages of a tile
  const int my_page = lane / S::kBlocks, my_block = lane % S::kBlocks;
  const uint32_t my_dst = ring + (my_block * S::kKeys + my_page * box) * 128;
  int it = 0, rounds = 0;
  bool ok = true, bad = false;

  // First row, in the cache, of the lane's box of key tile j; -1 if it has none.
  auto box_row = [&](int j) -> int {
    const int key = j * S::kKeys + my_page * box;
    if (my_page >= boxes || key >= u.units.row.L) return -1;
    const int pg = key >> a.page_shift;
    if (!in_array(a.flags, u.b, a.B) || !in_array(a.flags, pg, a.max_pages)) return -1;
    const int id = a.block_table[(long long)u.b * a.max_pages + pg];
    const bool inside = id >= 0 && id < a.n_pages;
    bad |= !inside;
    // past the last row of the cache the box fills with zeros
    return ((inside ? id * a.Hk + u.h : a.n_pages * a.Hk) << a.page_shift) + (key & (page - 1));
  };
  auto bring = [&](const CUtensorMap* map, int y, bool ours) -> bool {
    const int stage = it % S::kStages, lap = it / S::kStages;
    if (ours) {
      if (lap > 0 && !mbar_wait(smem_addr(&c->empty[stage]), (lap - 1) & 1, &c->abort_word,
                                naps_of(a)))
        return false;
      const uint32_t bar = smem_addr(&c->full[stage]);
      const unsigned who = __ballot_sync(0xffffffffu, y >= 0);
      if (lane == 0) mbar_arrive_expect(bar, __popc(who) * box * 128);
      __syncwarp();
      if (y >= 0) tma_load_2d(my_dst + stage * S::kStageBytes, map, my_block * 64, y, bar);
    }
    ++it;
    return true;
  };

#pragma unroll 1
  for (bool first = true; ok && u.next(first); first = false) {
    const int n = u.most();
    if (n == 0) continue;
    int y[S::kBufs + 1];   // tiles i .. i + kBufs
#pragma unroll
    for (int i = 0; i < S::kBufs; ++i) y[i] = box_row(u.j0 + i);
#pragma unroll
    for (int i = 0; i < S::kBufs; ++i)
      if (ok && i < n) ok = bring(k_map, y[i], keys);
    if (ok && keys) {
      if (rounds > 0 &&
          !(ok = mbar_wait(smem_addr(&c->q_empty), (rounds - 1) & 1, &c->abort_word, naps_of(a))))
        break;
      ++rounds;
      const uint32_t bar = smem_addr(&c->q_full);
      const int q_tile = lane / S::kBlocks;
      const bool mine = q_tile < S::kTiles && u.count(q_tile) > 0;
      const unsigned who = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) mbar_arrive_expect(bar, __popc(who) * a.tile_tokens * a.G * 128);
      __syncwarp();
      if (mine)
        tma_load_3d(q_smem + q_tile * S::kQBytes + my_block * 128 * 128, q_map, my_block * 64,
                    u.h * a.G, u.units.row.begin + u.first(q_tile), bar);
    }
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      const bool another = i + S::kBufs < n;
      y[S::kBufs] = another ? box_row(u.j0 + i + S::kBufs) : -1;
      ok = bring(v_map, y[0], values);
      if (ok && another) ok = bring(k_map, y[S::kBufs], keys);
#pragma unroll
      for (int x = 0; x < S::kBufs; ++x) y[x] = y[x + 1];
    }
  }
  if (bad) set_flag(a.flags, kDevBadPage);
  // Copies in flight land in this CTA's memory, which has to outlive them even
  // where the warps that would have read them have given up.  Of the ring's last
  // lap the warp waits for its own (two warps: keys the even slots, values the odd).
#pragma unroll 1
  for (int i = max(0, it - S::kStages); i < it; ++i)
    if (i % 2 == 0 ? keys : values)
      (void)mbar_poll(smem_addr(&c->full[i % S::kStages]), (i / S::kStages) & 1, &c->calm, kNaps);
  if (rounds > 0) (void)mbar_poll(smem_addr(&c->q_full), (rounds - 1) & 1, &c->calm, kNaps);
  __syncwarp();
}

// ----------------------------------------------------------------- products
// A count and not a barrier: a tile without products may be units ahead, and a
// wait for a phase sees its parity alone.  A turn sleeps about a sixteenth of
// what a poll of a barrier does.
__device__ __forceinline__ bool wait_past(AttnControl* c, int units, int naps) {
  bool ok = c->past >= units;
#pragma unroll 1
  for (int i = 0; !ok && i < 16 * naps && !*(volatile int*)&c->abort_word; ++i) {
    __nanosleep(64);
    ok = c->past >= units;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) *(volatile int*)&c->abort_word = 1;
  return ok;
}

// One warp per query tile.  A product's issue lasts as long as the tensor core
// takes to accept it, so what a warp does between products (waits, commits)
// would leave the tensor core idle; the other tile's warp fills that.  The
// two take turns, O += P V and the next scores at a time: left to themselves
// they fall into step, both tiles' softmax and then both tiles' products.
// The products of one warp run in the order of their issue: S of the next
// keys follows O += P V, whose P lies where S goes.
// Columns of tensor memory: kBufs S buffers per query tile, then one O per
// query tile.
template <typename E, int kD, typename S>
__device__ __forceinline__ void attn_multiply(const AttnArgs& a, AttnWalk<S> u, AttnControl* c,
                                              uint32_t q_smem, uint32_t ring, char* ring_ptr,
                                              uint32_t tmem, int t) {
  constexpr bool kBf16 = std::is_same<E, __nv_bfloat16>::value;
  constexpr uint32_t s_desc = mma_desc(kBf16, 128, S::kKeys, false);
  constexpr uint32_t o_desc = mma_desc(kBf16, 128, kD, true);
  const int lane = threadIdx.x & 31;
  const uint32_t issue = lane == 0;
  tmem = __shfl_sync(0xffffffffu, tmem, 0);
  t = __shfl_sync(0xffffffffu, t, 0);
  const uint32_t s_base = tmem + t * S::kBufs * S::kKeys;
  const uint32_t o = tmem + S::kTiles * S::kBufs * S::kKeys + t * kD;
  int it = 0, rounds = 0;
  int done = 0;   // tiles of S issued before this unit
  bool ok = true;

  auto s_col = [&](int k) { return s_base + (k % S::kBufs) * S::kKeys; };
  auto wait_stage = [&](int i) {
    return mbar_wait(smem_addr(&c->full[i % S::kStages]), (i / S::kStages) & 1, &c->abort_word,
                     naps_of(a));
  };
  // Descriptors step by addresses / 16, and never out of their field.
  const uint64_t q_desc = tile_desc(q_smem + t * S::kQBytes, 16, 1024);
  const uint64_t k_desc = tile_desc(ring, 16, 1024);
  const uint64_t v_desc = tile_desc(ring, S::kKeys * 128, 1024);
  // The other tile's turn: the last of the arrivals that its P waits for.
  auto pass_turn = [&](bool pass) {
    if (pass && lane == 0) mbar_arrive(smem_addr(&c->p_ready[1 - t][0]));
  };
  // S = Q K^T, the tile's k-th; the turn passes before the last two products,
  // which last about as long as the other warp takes to see it
  auto scores = [&](int k, int stage, bool pass) {
    const uint64_t k0 = k_desc + stage * (S::kStageBytes / 16);
#pragma unroll
    for (int d = 0; d < kD / 16; ++d) {
      if (S::kTiles > 1 && d == kD / 16 - 2) pass_turn(pass);
      mma_smem(s_col(k), q_desc + (d / 4) * (128 * 128 / 16) + (d % 4) * 2,
               k0 + (d / 4) * (S::kKeys * 128 / 16) + (d % 4) * 2, s_desc, d > 0, issue);
    }
    tc_commit(smem_addr(&c->s_full[t][k % S::kBufs]), issue);
  };
  // A slot is free once every issuer's products with it are done; one that
  // has none waits for the slot to be full all the same, so that its arrivals
  // keep to the slot's laps.
  auto release = [&](uint64_t* bar, bool used) {
    if (used) tc_commit(smem_addr(bar), issue);
    else if (lane == 0) mbar_arrive(smem_addr(bar));
  };

#pragma unroll 1
  for (bool first = true; ok && u.next(first); first = false) {
    const int n = u.most(), cnt = u.count(t), other = S::kTiles > 1 ? u.count(1 - t) : 0;
    if (n == 0) continue;
    if (!(ok = mbar_wait(smem_addr(&c->q_full), rounds & 1, &c->abort_word, naps_of(a)))) break;
    // The turns that the first tile gives belong to one unit: the second tile's
    // issuer must be past its last wait for P of the unit before.
    if (S::kTiles > 1 && t == 0 && !(ok = wait_past(c, rounds, naps_of(a)))) break;
    ++rounds;
    tc_fence_after();
#pragma unroll 1
    for (int i = 0; i < min(n, S::kBufs); ++i) {
      if (!(ok = wait_stage(it))) break;
      tc_fence_after();
      if (i < cnt) scores(done + i, it % S::kStages, false);
      release(&c->empty[it % S::kStages], i < cnt);
      ++it;
    }
    if (ok && cnt <= S::kBufs) release(&c->q_empty, cnt > 0);   // its last scores are issued
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      const int v_it = it++, k = done + i;
      const bool another = i + S::kBufs < n, active = i < cnt, next = i + S::kBufs < cnt;
      const int k_it = another ? it++ : 0;
      if (!(ok = wait_stage(v_it))) break;
      if (active) {
        // values past the request's length must not reach the sums: 0 * NaN is NaN
        // (the other tile's warp writes the same zeros)
        const int valid = u.units.row.L - (u.j0 + i) * S::kKeys;
        if (valid < S::kKeys) {
          char* v0 = ring_ptr + (v_it % S::kStages) * S::kStageBytes;
          const int chunks = (S::kKeys - valid) * 8;
#pragma unroll 1
          for (int x = lane; x < chunks * S::kBlocks; x += 32)
            *(uint4*)(v0 + ((x / chunks) * S::kKeys + valid) * 128 + (x % chunks) * 16) =
                make_uint4(0, 0, 0, 0);
          fence_async_shared();
          __syncwarp();
        }
      }
      // wide: every wait comes before the products, since the tensor core's queue
      // is short; narrow: O += P V does not wait for keys that are still to come
      if (S::kTiles > 1 && another && !(ok = wait_stage(k_it))) break;
      if (active) {
        // no turn to wait for: the other tile has no product before this one
        if (S::kTiles > 1 && !(t == 0 ? i > 0 && i - 1 < other : i < other) && lane == 0)
          mbar_arrive(smem_addr(&c->p_ready[t][0]));
        if (!(ok = mbar_wait(smem_addr(&c->p_ready[t][k % S::kBufs]), (k / S::kBufs) & 1,
                             &c->abort_word, naps_of(a))))
          break;
        tc_fence_after();
      }
      // the other tile's next product, if it has one
      const bool pass = active && (t == 0 ? i < other : i + 1 < other);
      if (active) {
        const uint64_t v0 = v_desc + (v_it % S::kStages) * (S::kStageBytes / 16);
#pragma unroll
        for (int x = 0; x < S::kKeys / 16; ++x)
          mma_tmem(o, s_col(k) + x * 8, v0 + x * (16 * 128 / 16), o_desc, i > 0 || x > 0, issue);
      }
      // with one S buffer the next scores tell that O is up to date
      if (active && (S::kBufs > 1 || !next)) release(&c->pv_done[t], true);
      if (S::kTiles == 1 && another) {
        if (!(ok = wait_stage(k_it))) break;
        tc_fence_after();
      }
      if (next) scores(k + S::kBufs, k_it % S::kStages, pass);
      else if (S::kTiles > 1) pass_turn(pass);
      release(&c->empty[v_it % S::kStages], active);
      if (another) release(&c->empty[k_it % S::kStages], next);
      if (next && i + S::kBufs + 1 == cnt) release(&c->q_empty, true);
    }
    done += cnt;
    if (S::kTiles > 1 && t == 1 && lane == 0) c->past = rounds;
  }
  // everything issued is done before the CTA's memory goes
  release(&c->drain, true);
  (void)mbar_poll(smem_addr(&c->drain), 0, &c->calm, kNaps);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
template <int kCount>
__device__ __forceinline__ float row_max(const uint32_t* bits) {
  float top[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) top[x] = __uint_as_float(bits[x]);
#pragma unroll
  for (int x = 4; x + 4 < kCount; x += 8)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      top[y] = max3(top[y], __uint_as_float(bits[x + y]), __uint_as_float(bits[x + 4 + y]));
#pragma unroll
  for (int y = 0; y < 4; ++y) top[y] = fmaxf(top[y], __uint_as_float(bits[kCount - 4 + y]));
  return fmaxf(max3(top[0], top[1], top[2]), top[3]);
}

// All softmax warps meet (their `phase`-th meeting); false if it was given up.
__device__ __forceinline__ bool soft_meet(AttnControl* c, int phase, int naps) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&c->met));
  return mbar_wait(smem_addr(&c->met), phase & 1, &c->abort_word, naps);
}

// What a row's sum l and reference m give.  A row that sees no key has l == 0;
// one that sees a NaN or +inf score has a NaN, which stays.
__device__ __forceinline__ float row_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? SV_NEG_INF : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ int take_ticket(int* ticket) {
  int before;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
  return before;
}

// 128 bytes of each of a warp's 32 rows, a row per lane, to global memory with
// four whole segments per instruction: they pass through shared memory, their
// 16-byte pieces placed so that neither side meets bank conflicts.  The
// lane's segment is `to` pitches from `base`, none if negative; the warp's
// first `rows` have one.  The array is the `pieces` 16-byte pieces from `array`.
__device__ __forceinline__ void stage_piece(char* stage, int piece, uint32_t x, uint32_t y,
                                            uint32_t z, uint32_t w) {
  const int lane = threadIdx.x & 31;
  *(uint4*)(stage + lane * 128 + (piece ^ (lane & 7)) * 16) = make_uint4(x, y, z, w);
}
__device__ __forceinline__ void store_staged(unsigned* flags, const char* stage, char* base, int to,
                                             int pitch, int rows, const void* array,
                                             long long pieces) {
  const int lane = threadIdx.x & 31, piece = lane % 8;
  __syncwarp();
#pragma unroll 1
  for (int i0 = 0; i0 < rows; i0 += 16) {
    uint4 v[4];
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i0 + i * 4 + lane / 8;
      v[i] = *(const uint4*)(stage + row * 128 + (piece ^ (row & 7)) * 16);
      at[i] = __shfl_sync(0xffffffffu, to, row);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      char* p = base + (long long)at[i] * pitch + piece * 16;
      if (at[i] >= 0 && in_array(flags, (p - (const char*)array) / 16, pieces)) *(uint4*)p = v[i];
    }
  }
  __syncwarp();
}

// Joins the partial sums of the unit's CTAs in their order.  kSpan threads
// share a row, each kD / kSpan of its columns, and take kAhead parts at a
// time, so that their loads are in flight together: many rows have few parts
// (a prompt's unit that a range's end cuts), few rows many (a long context).
template <typename E, int kD, typename S, int kSpan, int kAhead>
__device__ __forceinline__ void attn_join(const AttnArgs& a, const AttnWalk<S>& u, int c_first,
                                          int parts, bool begins_late) {
  constexpr int kVecs = kD / 4 / kSpan;   // 16-byte pieces per thread, kSpan apart
  const size_t slots = (size_t)gridDim.x * 2;
  const float4* sums = (const float4*)a.partial;
  const float2* stats = (const float2*)(a.partial + slots * S::kRows * kD);
  if (!in_array(a.flags, slots * S::kRows - 1, kAttnRows)) return;
  const int rows0 = (u.last(0) - u.first(0)) * a.G;   // a second tile only where the first is full
  const int items = u.rows() * kSpan, col = threadIdx.x % kSpan;
#pragma unroll 1
  for (int x = threadIdx.x; x < items; x += S::kSoftThreads) {
    const int r = x / kSpan;
    const int at = r < rows0 ? r : 128 + r - rows0;   // row of the slot
    float m = SV_NEG_INF, l = 0.f;
    float4 o[kVecs] = {};
#pragma unroll 1
    for (int p0 = 0; p0 < parts; p0 += kAhead) {
      float2 ml[kAhead];
      float4 f[kAhead][kVecs];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int p = min(p0 + q, parts - 1);
        size_t row = ((size_t)(c_first + p) * 2 + (p == 0 && begins_late ? 1 : 0)) * S::kRows + at;
        if (!in_array(a.flags, row, slots * S::kRows)) row = 0;
        ml[q] = __ldcg(&stats[row]);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) f[q][v] = __ldcg(&sums[row * (kD / 4) + v * kSpan + col]);
        if (p0 + q >= parts) ml[q].x = SV_NEG_INF;
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        // a part that sees none of the row's keys has -inf and zeros
        const float top = fmaxf(m, ml[q].x), ref = top == SV_NEG_INF ? 0.f : top;
        const float c0 = ex2_approx(m - ref), c1 = ex2_approx(ml[q].x - ref);
        m = top;
        l = l * c0 + ml[q].y * c1;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          o[v].x = o[v].x * c0 + f[q][v].x * c1;
          o[v].y = o[v].y * c0 + f[q][v].y * c1;
          o[v].z = o[v].z * c0 + f[q][v].z * c1;
          o[v].w = o[v].w * c0 + f[q][v].w * c1;
        }
      }
    }
    const int g = at % 128;
    const long long to =
        (long long)(u.units.row.begin + u.first(at / 128) + g / a.G) * a.Hq + u.h * a.G + g % a.G;
    const float inv = row_inverse(l);
    if (!in_array(a.flags, to, (long long)a.T * a.Hq)) continue;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      *(uint2*)(a.out + (to * kD + (v * kSpan + col) * 4) * 2) =
          make_uint2(pack2(o[v].x * inv, o[v].y * inv, E()), pack2(o[v].z * inv, o[v].w * inv, E()));
    if (a.lse && col == 0) a.lse[to] = row_lse(m, l);
  }
}

// The warp's part of P (and of a scaled O) is in tensor memory.
__device__ __forceinline__ void hand_over(uint64_t* bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(bar));
}

template <typename E, int kD, typename S>
__device__ __forceinline__ void attn_softmax(const AttnArgs& a, AttnWalk<S> u, AttnControl* c,
                                             uint32_t tmem, char* staging, long long quota,
                                             long long w1) {
  const int warp = threadIdx.x >> 5, t = warp / 4;
  const int r = threadIdx.x % 128;                 // the thread's row of its query tile:
  const int r_token = r / a.G, r_head = r - r_token * a.G;   // a token and a head of the group
  const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
  const uint32_t o_col = tmem + lanes + S::kTiles * S::kBufs * S::kKeys + t * kD;
  char* stage = staging + warp * S::kStagingBytes;
  int done = 0;                                    // tiles of S taken before this unit
  int meetings = 0, rounds = 0;
  bool ok = true;
#pragma unroll 1
  for (bool first = true; ok && u.next(first); first = false) {
    const int n = u.count(t);
    const int token = u.first(t) + r_token;
    const bool mine = r_token < a.tile_tokens && token < u.units.row.n;
    const int rows = __popc(__ballot_sync(0xffffffffu, mine));   // the warp's first ones
    const bool any = rows > 0;
    // keys that the row sees; rows without a token see none
    const int seen = mine ? max(0, u.units.row.L - u.units.row.n + token + 1) : 0;
    // the warp's first row sees the fewest of those with a token
    const int fewest = __shfl_sync(0xffffffffu, seen, 0);
    float m = SV_NEG_INF, l = 0.f;
    int key0 = u.j0 * S::kKeys;   // the tile's first key
    u.park((int4*)stage);
#pragma unroll 1
    for (int i = 0; i < n; ++i, key0 += S::kKeys) {
      const int k = done + i, buf = k % S::kBufs;
      if (!(ok = mbar_wait(smem_addr(&c->s_full[t][buf]), (k / S::kBufs) & 1, &c->abort_word,
                           naps_of(a))))
        break;
      tc_fence_after();
      // With two S buffers the scores do not tell that the last O += P V is
      // done; the wait keeps at most one of them open, as a wait that sees a
      // phase's parity alone needs.
      auto give = [&]() -> bool {
        if (S::kBufs > 1 && i > 0 &&
            !mbar_wait(smem_addr(&c->pv_done[t]), (k - 1) & 1, &c->abort_word, naps_of(a)))
          return false;
        hand_over(&c->p_ready[t][buf]);
        return true;
      };
      if (any) {
        const uint32_t s_col = tmem + lanes + (t * S::kBufs + buf) * S::kKeys;
        uint32_t bits[S::kKeys];
#pragma unroll
        for (int x = 0; x < S::kKeys; x += 32) tmem_load32(s_col + x, bits + x);
        tmem_wait_load();
        tmem_pin<S::kKeys>(bits);
        const int left = seen - key0;   // keys of the tile that the row sees
        if (fewest < key0 + S::kKeys) {
#pragma unroll
          for (int x = 0; x < S::kKeys; ++x)
            if (x >= left) bits[x] = 0xff800000u;
        }
        // The reference follows the maximum where that rises by more than kSlack.
        const float high = row_max<S::kKeys>(bits) * a.scale_log2;
        const bool raise = mine && (i == 0 ? high > m : high > m + kSlack);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? (m == SV_NEG_INF ? 0.f : ex2_approx(m - high)) : 1.f;
          if (raise) m = high;
          l *= f;
          if (i > 0) {   // what was summed before, once the products are done
            if (S::kBufs > 1) {
              if (!(ok = mbar_wait(smem_addr(&c->pv_done[t]), (k - 1) & 1, &c->abort_word,
                                   naps_of(a))))
                break;
              tc_fence_after();
            }
#pragma unroll 1
            for (int x = 0; x < kD; x += 32) {
              uint32_t o[32];
              tmem_load32(o_col + x, o);
              tmem_wait_load();
              tmem_pin<32>(o);
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_store32(o_col + x, o);
            }
          }
        }
        const float ref = m == SV_NEG_INF ? 0.f : m;
        const unsigned long long scale2 = f2_pack(a.scale_log2, a.scale_log2);
        const unsigned long long ref2 = f2_pack(-ref, -ref);
#pragma unroll
        for (int x = 0; x < S::kKeys; x += 32) {
          uint32_t p[16];
#pragma unroll
          for (int y = 0; y < 32; y += 2) {
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(bits[x + y]), __uint_as_float(bits[x + y + 1])),
                             scale2, ref2),
                      p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            bits[x + y] = __float_as_uint(p0);
            bits[x + y + 1] = __float_as_uint(p1);
            p[y / 2] = pack2(p0, p1, E());
          }
          tmem_store16(s_col + x / 2, p);
        }
        tmem_wait_store();
        if (!(ok = give())) break;
        // The row's sum, of P before rounding, off the chain (three whole prompts:
        // 629 us; summed along with the exponentials, 642).
        unsigned long long sums[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < S::kKeys; x += 2)
          sums[(x / 2) % 2] = f2_add(sums[(x / 2) % 2], f2_pack(__uint_as_float(bits[x]),
                                                                __uint_as_float(bits[x + 1])));
        float s0, s1;
        f2_unpack(f2_add(sums[0], sums[1]), s0, s1);
        l += s0 + s1;
      } else if (!(ok = give())) {
        break;
      }
    }
    if (!ok) break;
    u.unpark((const int4*)stage);
    done += n;
    // one S buffer: one arrival per unit, else one per tile
    if (n > 0)
      ok = mbar_wait(smem_addr(&c->pv_done[t]), (S::kBufs > 1 ? done - 1 : rounds++) & 1,
                     &c->abort_word, naps_of(a));
    if (!ok) break;
    tc_fence_after();
    // A unit that is all this CTA's is written out; a part of one goes to the
    // workspace as it is, to one of two places: a range has at most one part at
    // its start and one at its end.
    const bool whole = u.j0 == 0 && u.j1 == u.tiles;
    const int cta = blockIdx.x;
    // from the start of this range to the unit's, in keys; the unit's first CTA
    const long long ahead = w1 - u.left - u.pos - cta * quota;
    const int c_first = cta - ranges_back(u.pos, quota);
    const bool begins_late = ahead + (cta - c_first) * quota != 0;   // after its range's start
    const size_t slots = (size_t)gridDim.x * 2;
    const size_t slot = (size_t)cta * 2 + (cta == c_first && begins_late ? 1 : 0);
    if (any) {
      const float inv = row_inverse(l);
      // rows of `out` from the unit's first token and head, or rows of the slot
      const long long unit = (long long)(u.units.row.begin + u.first(0)) * a.Hq + u.h * a.G;
      const int to = !mine ? -1 : whole ? (token - u.first(0)) * a.Hq + r_head : t * 128 + r;
      char* base = whole ? a.out + unit * kD * 2 : (char*)(a.partial + slot * S::kRows * kD);
      const long long out_rows = (long long)a.T * a.Hq;
      const long long part_rows = min((long long)slots * S::kRows, kAttnRows);
#pragma unroll 1
      for (int x = 0; x < kD; x += 32) {
        uint32_t bits[32] = {};
        if (n > 0) {
          tmem_load32(o_col + x, bits);
          tmem_wait_load();
          tmem_pin<32>(bits);
        }
        if (whole) {   // 64 columns make a segment
          uint32_t p[16];
#pragma unroll
          for (int y = 0; y < 16; ++y)
            p[y] = pack2(__uint_as_float(bits[2 * y]) * inv, __uint_as_float(bits[2 * y + 1]) * inv,
                         E());
#pragma unroll
          for (int y = 0; y < 4; ++y)
            stage_piece(stage, x / 8 % 8 + y, p[4 * y], p[4 * y + 1], p[4 * y + 2], p[4 * y + 3]);
          if (x % 64 == 0) continue;
        } else {
#pragma unroll
          for (int y = 0; y < 8; ++y)
            stage_piece(stage, y, bits[4 * y], bits[4 * y + 1], bits[4 * y + 2], bits[4 * y + 3]);
        }
        store_staged(a.flags, stage, base, to, whole ? kD * 2 : kD * 4, rows,
                     whole ? (const void*)a.out : a.partial,
                     whole ? out_rows * (kD / 8) : part_rows * (kD / 4));
        base += 128;
      }
      if (mine) {
        const long long row = whole ? unit + to : (long long)slot * S::kRows + to;
        const bool good = in_array(a.flags, row, whole ? out_rows : part_rows);
        if (good && !whole) ((float2*)(a.partial + slots * S::kRows * kD))[row] = make_float2(m, l);
        if (good && whole && a.lse) a.lse[row] = row_lse(m, l);
      }
    }
    tc_fence_before();
    if (whole) continue;
    // the CTA that has the unit's last tile
    const long long end = ahead + (long long)(u.tiles - 1) * S::kKeys;
    const int c_last = u.j1 == u.tiles ? cta : cta + ranges_ahead(end, quota);
    // what all warps wrote is released by one thread's ticket, and what other
    // CTAs wrote is acquired by it
    if (!(ok = soft_meet(c, meetings++, naps_of(a)))) break;
    if (threadIdx.x == 0) {
      const bool last = in_array(a.flags, c_first, gridDim.x) &&
                        take_ticket(&a.tickets[c_first]) == c_last - c_first;
      if (last) a.tickets[c_first] = 0;
      c->last = last;
    }
    if (!(ok = soft_meet(c, meetings++, naps_of(a)))) break;
    if (c->last) {
      const int parts = c_last - c_first + 1;
      if (u.rows() * (kD / 4) <= S::kSoftThreads)
        attn_join<E, kD, S, kD / 4, 8>(a, u, c_first, parts, begins_late);
      else
        attn_join<E, kD, S, 8, 2>(a, u, c_first, parts, begins_late);
    }
  }
}

template <typename E, int kD, bool kWide>
__global__ void __launch_bounds__(AttnShape<kD, kWide>::kThreads, AttnShape<kD, kWide>::kCtasPerSm)
    sv_paged_attention_kernel(const __grid_constant__ AttnArgs a,
                              const __grid_constant__ CUtensorMap q_map,
                              const __grid_constant__ CUtensorMap k_map,
                              const __grid_constant__ CUtensorMap v_map) {
  using S = AttnShape<kD, kWide>;
  extern __shared__ __align__(1024) char smem[];
  char* ring_ptr = smem + S::kTiles * S::kQBytes;
  char* staging = ring_ptr + S::kStages * S::kStageBytes;
  AttnControl* c = (AttnControl*)(staging + S::kTiles * 4 * S::kStagingBytes);
  const uint32_t q_smem = smem_addr(smem), ring = smem_addr(ring_ptr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kLoader = S::kSoftThreads / 32, kIssuer = kLoader + 1;

  // -------- set-up that reads nothing of the caller's
  if (warp == kLoader && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_addr(&c->full[i]), 1);
      mbar_init(smem_addr(&c->empty[i]), S::kTiles);
    }
    mbar_init(smem_addr(&c->q_full), 1);
    mbar_init(smem_addr(&c->q_empty), S::kTiles);
    mbar_init(smem_addr(&c->drain), S::kTiles);
    mbar_init(smem_addr(&c->met), S::kSoftThreads / 32);
#pragma unroll 1
    for (int t = 0; t < S::kTiles; ++t) {
      for (int k = 0; k < S::kBufs; ++k) {
        mbar_init(smem_addr(&c->s_full[t][k]), 1);
        mbar_init(smem_addr(&c->p_ready[t][k]), S::kTiles > 1 ? 5 : 4);   // with the turn
      }
      mbar_init(smem_addr(&c->pv_done[t]), 1);
    }
    mbar_init_fence();
    c->abort_word = c->calm = c->past = 0;
    tma_prefetch_map(&q_map);
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  if (warp == kIssuer) tmem_alloc<S::kTmemCols>(smem_addr(&c->tmem));
  wait_for_preceding_grid();

  // -------- weights of all requests, summed: thread i has rows [r0, r1)
  const int per = (a.B + S::kThreads - 1) / S::kThreads;
  const int r0 = min(a.B, (int)threadIdx.x * per), r1 = min(a.B, r0 + per);
  // in flight with the lengths
  const unsigned status = threadIdx.x == S::kThreads - 1 ? __ldcg(a.status) : 0;
  bool bad = false;
  long long mine = 0, head = 0;   // weight of the thread's requests; of one head of the last
  AttnUnits<S> units;
#pragma unroll 1
  for (int b = r0; b < r1; ++b) {
    units = AttnUnits<S>(a, attn_row(a, b, &bad));
    head = units.before(units.count);
    mine += head * a.Hk;
  }
  if (bad && blockIdx.x == 0) set_flag(a.flags, kDevLength);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) c->sums[warp] = inc;
  if (threadIdx.x == S::kThreads - 1) c->status = status;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only now, with this CTA's tensor memory taken: a CTA of the next grid that
  // held it while it waits for this grid would keep this CTA from starting.
  allow_dependent_launch();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < S::kThreads / 32; ++w) {
    if (w < warp) before += c->sums[w];
    total += c->sums[w];
  }
  const long long quota = range_quota(total, gridDim.x, S::kKeys);
  // After a call that gave up, tickets may be anything: no work, and NaN below.
  const bool spoilt = c->status != 0;
  const long long w0 = (long long)blockIdx.x * quota, w1 = spoilt ? w0 : min(total, w0 + quota);
  long long begin = before + inc - mine;
  // One thread's rows hold the start of the range; its warp finds the place.
  const unsigned holds = __ballot_sync(0xffffffffu, w0 < w1 && begin <= w0 && w0 < begin + mine);
  if (holds) {
    int b = r0;
    if (per > 1 && (holds >> lane & 1)) {
#pragma unroll 1
      for (;; ++b) {
        units = AttnUnits<S>(a, attn_row(a, b));
        head = units.before(units.count);
        if (w0 < begin + head * a.Hk) break;
        begin += head * a.Hk;
      }
    }
    const int from = __ffs(holds) - 1;
    b = __shfl_sync(0xffffffffu, b, from);
    head = __shfl_sync(0xffffffffu, head, from);
    long long off = w0 - __shfl_sync(0xffffffffu, begin, from);
    units.row.begin = __shfl_sync(0xffffffffu, units.row.begin, from);
    units.row.n = __shfl_sync(0xffffffffu, units.row.n, from);
    units.row.L = __shfl_sync(0xffffffffu, units.row.L, from);
    units.count = __shfl_sync(0xffffffffu, units.count, from);
    units.step = S::kTiles * a.tile_tokens;
    int h = min(a.Hk - 1, (int)__fdividef((float)off, (float)head));   // about, then exactly
#pragma unroll 1
    while (h * head > off) --h;
#pragma unroll 1
    while ((h + 1) * head <= off) ++h;
    off -= h * head;
    // the last unit that starts at or before off, 32 candidates at a time
    int lo = 0, span = units.count;
#pragma unroll 1
    while (span > 1) {
      const int step = (span + 31) / 32, at = lo + lane * step;
      const unsigned under =
          __ballot_sync(0xffffffffu, at < lo + span && units.before(at) <= off);
      const int last = 31 - __clz(under);   // lane 0 is always under
      span = min(step, span - last * step);
      lo += last * step;
    }
    if (lane == 0) {
      c->start.row = units.row;
      c->start.count = units.count;
      c->start.b = b;
      c->start.h = h;
      c->start.m = lo;
      c->start.pos = (int)(off - units.before(lo));
    }
  }
  __syncthreads();
  const uint32_t tmem = c->tmem;

  if (w0 < w1) {
    const AttnWalk<S> u(a, c->start, w1 - w0);
    // Wide: three warpgroups launched with 168 registers a thread, and
    // 2 x 216 + 72 = 3 x 168.  Three whole prompts: 633 us with 208 and 88, 629
    // so, 798 with 224 and 56, which the issuers cannot do with.
    if (warp >= kLoader) {
      if (kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      if (warp >= kIssuer && warp < kIssuer + S::kTiles)
        attn_multiply<E, kD, S>(a, u, c, q_smem, ring, ring_ptr, tmem, warp - kIssuer);
      else
        attn_load<S>(a, u, c, q_smem, ring, &q_map, &k_map, &v_map, warp == kLoader,
                     !kWide || warp != kLoader);
    } else {
      if (kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      attn_softmax<E, kD, S>(a, u, c, tmem, staging, quota, w1);
    }
  }
  // tokens past the last request's, or all of them
  const int used = spoilt ? 0 : min(max(a.cu_new[a.B], 0), a.T);
  const long long spare = (long long)(a.T - used) * a.Hq;
  if (spare > 0) {
    const long long first = (long long)used * a.Hq;
    const uint32_t fill = spoilt ? 0x7fff7fffu : 0u;   // two NaN of either type
#pragma unroll 1
    for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < spare * (kD / 8);
         x += (long long)gridDim.x * blockDim.x)
      ((uint4*)a.out)[first * (kD / 8) + x] = make_uint4(fill, fill, fill, fill);
    if (a.lse)
#pragma unroll 1
      for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < spare;
           x += (long long)gridDim.x * blockDim.x)
        a.lse[first + x] = spoilt ? __int_as_float(0x7fffffff) : SV_NEG_INF;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && (c->abort_word || spoilt)) {
    set_flag(a.flags, kDevTimeout);
    set_flag(a.status, kDevTimeout);
  }
  if (warp == kIssuer) tmem_free<S::kTmemCols>(tmem);
}

}  // namespace sv
