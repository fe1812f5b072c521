// Attention over the 4-bit cache for more than a few query rows a request: the
// products and the softmax of sv_paged_attention.cuh, in its wide and narrow forms,
// over tiles that four warps unpack to 16 bits in shared memory, from a ring of
// packed ones.
//
// Operands are float16 as in sv_fp4_attention.cuh: bfloat16 queries are converted in
// shared memory, each query tile with a power of two of its own (steps of 2^-38 of its
// largest magnitude).
//
// Bound by a tile's chain.  Narrow, 256 x 9 tokens over 2 k to 10 k keys, 64/8
// heads of 128: 768 us for 1.87 GB, about 2400 clocks per tile of 128 keys: 1716 of
// them are waits and handing over (measured without unpacking, exponentials and all
// but one step of each product), the rest is what unpacking and softmax add
// (transposed as in sv_fp4_attention.cuh 1726 us).  Wide, 2 x 2048 tokens over 5 k
// to 7 k: 371 us, 1.27 PFLOP/s, beside 310 of 16 bits: the unpacking shares the
// schedulers with the softmax.
#pragma once

#include "sv_fp4_load.cuh"

namespace sv {

// The wide form's shape, and a narrow one: one query tile against tiles of 128 keys
// with two S buffers, one CTA per SM.
template <int kD, bool kWide>
struct Fp4RowsShape : AttnShape<kD, true> {
  using Base = AttnShape<kD, true>;
  static constexpr bool kFp4 = true;
  static constexpr float kBelow = kFp4Below;
  // wide: a fourth unpacked tile in place of the staging (prompt chunks 446 and 392 us)
  static constexpr bool kStaged = !kWide;
  static constexpr int kChunk = kWide ? 128 : 64;
  // the unpacking's loads a step ahead: narrow 816 and 780 us (256 x 9 tokens); wide the
  // softmax of two tiles is the longer, and loses what it gains: chunks 392 and 404
  static constexpr bool kAhead = !kWide;
  static constexpr int kStagingBytes = kWide ? 64 : Base::kStagingBytes;
  static constexpr int kTiles = kWide ? 2 : 1;
  static constexpr int kBufs = kWide ? 1 : 2;
  static constexpr int kStages = (kWide ? 4 : 3) * (128 / kD);   // unpacked
  static constexpr int kPackedStages = kWide ? (kD == 128 ? 3 : 8) : kD == 128 ? 8 : 16;
  static constexpr int kSoftThreads = 128 * kTiles;
  static constexpr int kThreads = kSoftThreads + 256;   // whole warpgroups
  static constexpr int kUnitCost = kWide ? 256 : 512;
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kControlBytes = 1024;
  static constexpr int kSmemBytes = kTiles * (Base::kQBytes + 4 * kStagingBytes) +
                                    kStages * Base::kStageBytes + kPackedStages * Fp4Tile<kD>::kBytes +
                                    kControlBytes;
};

struct Fp4RowsControl {   // as AttnControl, and:
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty, drain, met;
  uint64_t s_full[2][2], p_ready[2][2];
  uint64_t pv_done[2];
  uint64_t q_raw;             // queries have arrived, not converted
  uint64_t packed_full[16], packed_empty[16];
  uint32_t tmem;
  volatile int past;
  int abort_word, calm, last;
  unsigned status;
  int q_exponent[2][2];       // for the scores' factor: [unit % 2][query tile]
  AttnStart start;
  long long sums[16];
};
static_assert(sizeof(Fp4RowsControl) <= 1024, "fits kControlBytes");

// One warp brings a unit's queries and converts its rows in place where they are
// bfloat16.
template <typename E, int kD, typename S>
__device__ __forceinline__ void fp4_rows_queries(const Fp4Args& a, AttnWalk<S> u, Fp4RowsControl* c,
                                                 char* q_ptr, const CUtensorMap* q_map) {
  const int lane = threadIdx.x & 31;
  int rounds = 0, brought = 0;
#pragma unroll 1
  for (bool first = true; u.next(first); first = false) {
    if (u.most() == 0) continue;
    if (rounds > 0 && !mbar_wait(smem_addr(&c->q_empty), (rounds - 1) & 1, &c->abort_word, naps_of(a)))
      break;
    const uint32_t bar = smem_addr(&c->q_raw);
    const int q_tile = lane / S::kBlocks, block = lane % S::kBlocks;
    const bool mine = q_tile < S::kTiles && u.count(q_tile) > 0;
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) mbar_arrive_expect(bar, __popc(who) * a.tile_tokens * a.G * 128);
    __syncwarp();
    if (mine)
      tma_load_3d(smem_addr(q_ptr) + q_tile * S::kQBytes + block * 128 * 128, q_map, block * 64, u.h * a.G,
                  u.units.row.begin + u.first(q_tile), bar);
    ++brought;
    if (!mbar_wait(bar, rounds & 1, &c->abort_word, naps_of(a))) break;
#pragma unroll 1
    for (int t = 0; t < S::kTiles; ++t) {
      int exponent = 0;
      if (std::is_same<E, __nv_bfloat16>::value && u.count(t) > 0) {
        const int pieces = (u.last(t) - u.first(t)) * a.G * 8;   // of 16 bytes in a block of 64 columns
        char* tile = q_ptr + t * S::kQBytes;
        auto largest = [&](bool finite) {
          uint32_t high = 0;
#pragma unroll 1
          for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll 8
            for (int x = lane; x < pieces; x += 32) {
              const uint4 w = *(const uint4*)(tile + b * 128 * 128 + x * 16);
              high = __vmaxu2(__vmaxu2(high, bf16_magnitudes(w.x, finite)), bf16_magnitudes(w.y, finite));
              high = __vmaxu2(__vmaxu2(high, bf16_magnitudes(w.z, finite)), bf16_magnitudes(w.w, finite));
            }
          return __reduce_max_sync(0xffffffffu, larger_half(high));
        };
        uint32_t top = largest(false);
        if (top >= kBf16Infinity) top = largest(true);   // of the others
        exponent = query_exponent(top);
        const uint32_t factor = query_factor(exponent);
#pragma unroll 1
        for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll 4
          for (int x = lane; x < pieces; x += 32) {
            uint4* at = (uint4*)(tile + b * 128 * 128 + x * 16);
            const uint4 w = *at;
            *at = make_uint4(query_pair(w.x, factor), query_pair(w.y, factor), query_pair(w.z, factor), query_pair(w.w, factor));
          }
      }
      if (lane == 0) c->q_exponent[rounds % 2][t] = score_exponent(a.scale_log2, exponent);
    }
    fence_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&c->q_full));
    ++rounds;
  }
  // a copy in flight lands in this CTA's memory
  if (brought > 0) (void)mbar_poll(smem_addr(&c->q_raw), (brought - 1) & 1, &c->calm, kNaps);
  __syncwarp();
}

// Four warps unpack, a key per thread, in the order in which the products take tiles:
// kBufs tiles of keys, then values and keys in turn.  The two rings need not keep
// step: keys have the packed one's even places, values the odd.  (A group of four
// warps each for keys and values is slower: 256 x 9 tokens 816 and 843 us.)
template <int kD, typename S>
__device__ __forceinline__ void fp4_rows_unpack(const Fp4Args& a, AttnWalk<S> u, Fp4RowsControl* c,
                                                const char* packed, char* ring) {
  const int key = threadIdx.x % 128, lane = threadIdx.x & 31;
  int it = 0, done = 0;   // unpacked tiles; key tiles of the units before
  auto unpack = [&](int tile, bool values) -> bool {
    const int from = 2 * (done + tile) + values, slot = from % S::kPackedStages;
    const int stage = it % S::kStages, lap = it / S::kStages;
    if (!mbar_await(smem_addr(&c->packed_full[slot]), (from / S::kPackedStages) & 1, &c->abort_word, naps_of(a)))
      return false;
    const char* codes = packed + slot * Fp4Tile<kD>::kBytes;
    const char* scales = codes + Fp4Tile<kD>::kCodeBytes + key * (kD / 16);
    auto load = [&](int p) { return *(const uint4*)(codes + fp4_piece<kD>(key, p)); };
    uint4 w4;
    uint2 bytes;
    if (S::kAhead) {
      w4 = load(0);
      bytes = kD == 128 ? *(const uint2*)scales : make_uint2(*(const uint32_t*)scales, 0);
    }
    if (lap > 0 && !mbar_await(smem_addr(&c->empty[stage]), (lap - 1) & 1, &c->abort_word, naps_of(a))) return false;
    char* to = ring + stage * S::kStageBytes + key * 128;
    // rolled up as in fp4_keys
#pragma unroll(S::kAhead ? 2 : 1)
    for (int p = 0; p < kD / 32; ++p) {
      if (!S::kAhead) w4 = load(p);
      const uint32_t pair = fp4_scales(S::kAhead ? bytes.x & 0xffff : *(const uint16_t*)(scales + p * 2));
      if (S::kAhead) {
        bytes.x = __funnelshift_r(bytes.x, bytes.y, 16);
        bytes.y >>= 16;
      }
      const uint32_t s[2] = {__byte_perm(pair, 0, 0x1010), __byte_perm(pair, 0, 0x3232)};
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      if (S::kAhead && p + 1 < kD / 32) w4 = load(p + 1);
      char* block = to + (p / 2) * (S::kKeys * 128);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t v[4];
        fp4_unpack(w[x], v);
#pragma unroll
        for (int y = 0; y < 4; ++y) v[y] = mul_f16x2(v[y], s[x / 2]);
        *(uint4*)(block + ((p % 2 * 4 + x) ^ (key % 8)) * 16) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_addr(&c->packed_empty[slot]));
      mbar_arrive(smem_addr(&c->full[stage]));
    }
    ++it;
    return true;
  };
#pragma unroll 1
  for (bool first = true; u.next(first); first = false) {
    const int n = u.most(), lead = min(n, S::kBufs);
#pragma unroll 1
    for (int i = -lead; i < n; ++i) {
      // values of tile i, then keys of the one kBufs ahead; keys alone at first
      if (i >= 0 && !unpack(i, true)) return;
      if (i + lead < n && !unpack(i + lead, false)) return;
    }
    done += n;
  }
}

// The narrow form's products, one warp: attn_multiply for one query tile, with as
// little between the products as can be, and P handed over before the last
// product is done (256 x 9 tokens 871 and 816 us).
template <int kD, typename S>
__device__ __forceinline__ void fp4_rows_multiply(const Fp4Args& a, AttnWalk<S> u, Fp4RowsControl* c,
                                                  uint32_t q_smem, uint32_t ring, char* ring_ptr, uint32_t tmem) {
  constexpr uint32_t s_desc = mma_desc(false, 128, S::kKeys, false);
  constexpr uint32_t o_desc = mma_desc(false, 128, kD, true);
  const int lane = threadIdx.x & 31;
  const uint64_t q_desc = tile_desc(q_smem, 16, 1024);
  const uint64_t k_desc = tile_desc(ring, 16, 1024);
  const uint64_t v_desc = tile_desc(ring, S::kKeys * 128, 1024);
  const uint32_t o = tmem + S::kBufs * S::kKeys;
  int it = 0, rounds = 0, k = 0;   // unpacked tiles, units, tiles of S whose values are next
  bool ok = true;
  auto arrived = [&](int i) {
    const bool there = mbar_await(smem_addr(&c->full[i % S::kStages]), (i / S::kStages) & 1, &c->abort_word, naps_of(a));
    tc_fence_after();
    return there;
  };
  auto scores = [&](int tile, int i, bool last) {
    const uint64_t from = k_desc + i % S::kStages * (S::kStageBytes / 16);
    if (elect_one()) {
#pragma unroll
      for (int d = 0; d < kD / 16; ++d)
        mma_smem_one(tmem + tile % S::kBufs * S::kKeys, q_desc + (d / 4) * (128 * 128 / 16) + (d % 4) * 2,
                     from + (d / 4) * (S::kKeys * 128 / 16) + (d % 4) * 2, s_desc, d > 0);
      tc_commit_one(smem_addr(&c->s_full[0][tile % S::kBufs]));
      tc_commit_one(smem_addr(&c->empty[i % S::kStages]));
      if (last) tc_commit_one(smem_addr(&c->q_empty));
    }
    __syncwarp();
  };
#pragma unroll 1
  for (bool first = true; ok && u.next(first); first = false) {
    const int n = u.count(0);
    if (n == 0) continue;
    if (!(ok = mbar_await(smem_addr(&c->q_full), rounds++ & 1, &c->abort_word, naps_of(a)))) break;
#pragma unroll 1
    for (int i = 0; i < min(n, S::kBufs); ++i, ++it) {
      if (!(ok = arrived(it))) break;
      scores(k + i, it, i + 1 == n);
    }
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i, ++k) {
      const int stage = it % S::kStages;
      if (!(ok = arrived(it++))) break;
      const int valid = u.units.row.L - (u.j0 + i) * S::kKeys;
      if (valid < S::kKeys) {   // values past the request's length: 0 * NaN is NaN
        char* v0 = ring_ptr + stage * S::kStageBytes;
        const int pieces = (S::kKeys - valid) * 8;
#pragma unroll 1
        for (int x = lane; x < pieces * S::kBlocks; x += 32)
          *(uint4*)(v0 + ((x / pieces) * S::kKeys + valid) * 128 + (x % pieces) * 16) = make_uint4(0, 0, 0, 0);
        fence_async_shared();
        __syncwarp();
      }
      if (!(ok = mbar_await(smem_addr(&c->p_ready[0][k % S::kBufs]), (k / S::kBufs) & 1, &c->abort_word, naps_of(a))))
        break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t from = v_desc + stage * (S::kStageBytes / 16);
#pragma unroll
        for (int x = 0; x < S::kKeys / 16; ++x)
          mma_tmem_one(o, tmem + k % S::kBufs * S::kKeys + x * 8, from + x * (16 * 128 / 16), o_desc, i > 0 || x > 0);
        tc_commit_one(smem_addr(&c->pv_done[k % 2]));
        tc_commit_one(smem_addr(&c->empty[stage]));
      }
      __syncwarp();
      if (i + S::kBufs < n) {
        if (!(ok = arrived(it))) break;
        scores(k + S::kBufs, it++, i + S::kBufs + 1 == n);
      }
    }
  }
  // everything issued is done before the CTA's memory goes
  if (elect_one()) tc_commit_one(smem_addr(&c->drain));
  (void)mbar_poll(smem_addr(&c->drain), 0, &c->calm, kNaps);
  __syncwarp();
}

template <typename E, int kD, bool kWide>
__global__ void __launch_bounds__(Fp4RowsShape<kD, kWide>::kThreads, Fp4RowsShape<kD, kWide>::kCtasPerSm)
    sv_fp4_rows_attention_kernel(const __grid_constant__ Fp4Args a, const __grid_constant__ CUtensorMap q_map,
                                 const __grid_constant__ CUtensorMap k_map,
                                 const __grid_constant__ CUtensorMap v_map) {
  using S = Fp4RowsShape<kD, kWide>;
  extern __shared__ __align__(1024) char smem[];
  char* ring = smem + S::kTiles * S::kQBytes;
  char* staging = ring + S::kStages * S::kStageBytes;
  char* packed = staging + S::kTiles * 4 * S::kStagingBytes;
  Fp4RowsControl* c = (Fp4RowsControl*)(packed + S::kPackedStages * Fp4Tile<kD>::kBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kQueries = S::kSoftThreads / 32, kLoader = kQueries + 1, kIssuer = kQueries + 2;
  constexpr int kUnpack = kQueries + 4;

  if (warp == kQueries && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_addr(&c->full[i]), 4);
      mbar_init(smem_addr(&c->empty[i]), S::kTiles);
    }
#pragma unroll 1
    for (int i = 0; i < S::kPackedStages; ++i) {
      mbar_init(smem_addr(&c->packed_full[i]), 33);   // the boxes' and the lanes'
      mbar_init(smem_addr(&c->packed_empty[i]), 4);
    }
    mbar_init(smem_addr(&c->q_raw), 1);
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
    }
#pragma unroll 1
    for (int t = 0; t < 2; ++t) mbar_init(smem_addr(&c->pv_done[t]), 1);
    mbar_init_fence();
    c->abort_word = c->calm = c->past = 0;
    tma_prefetch_map(&q_map);
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  if (warp == kIssuer) tmem_alloc<S::kTmemCols>(smem_addr(&c->tmem));
  wait_for_preceding_grid();
  const AttnRange range = attn_range<S>(a, c);
  const uint32_t tmem = c->tmem;
  if (range.w0 < range.w1) {
    const AttnWalk<S> u(a, c->start, range.w1 - range.w0);
    // Wide: launched with 128 registers a thread, and 2 x 176 + 80 + 80 = 4 x 128 (chunks 375
    // us; 184 and 72: 385, 168 and 88: 404); narrow: 168, and 232 + 2 x 136 = 3 x 168.
    if (warp >= kUnpack) {
      if (kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      else asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
      fp4_rows_unpack<kD, S>(a, u, c, packed, ring);
    } else if (warp >= kQueries) {
      if (kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      else asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
      // narrow: a loader each for keys and values
      if (!kWide && warp == kIssuer)
        fp4_rows_multiply<kD, S>(a, u, c, smem_addr(smem), smem_addr(ring), ring, tmem);
      else if (kWide && warp >= kIssuer && warp < kIssuer + S::kTiles)
        attn_multiply<__half, kD, S>(a, u, c, smem_addr(smem), smem_addr(ring), ring, tmem, warp - kIssuer);
      else if (warp == kQueries)
        fp4_rows_queries<E, kD, S>(a, u, c, smem, &q_map);
      else
        fp4_load<kD, S>(a, u, c, c->packed_full, c->packed_empty, packed, &k_map, &v_map, warp == kLoader,
                        kWide || warp != kLoader);
    } else {
      if (kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
      else asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
      attn_softmax<__half, E, kD, S>(a, u, c, tmem, staging, range.quota, range.w1);
    }
  }
  attn_finish<S, kD>(a, c, range.spoilt);
  if (warp == kIssuer) tmem_free<S::kTmemCols>(tmem);
}

}  // namespace sv
