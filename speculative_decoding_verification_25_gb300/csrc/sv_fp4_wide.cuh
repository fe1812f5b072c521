// Attention over the 4-bit cache for many query rows a request: the wide form of
// sv_paged_attention.cuh, its products and its softmax, over tiles that four
// warps unpack to 16 bits.  A unit's 256 rows share a tile's unpacking, which is
// 400 instructions of a warp beside the softmax's 1700, and the few packed bytes come
// straight from global memory to registers, a tile ahead.
//
// Operands are float16 as in sv_fp4_attention.cuh: bfloat16 queries are
// converted in shared memory, each query tile with a power of two of its own.
#pragma once

#include "sv_fp4.cuh"
#include "sv_paged_attention.cuh"

namespace sv {

struct Fp4WideArgs : AttnArgs {
  const char* k_codes;
  const uint8_t* k_scales;
  const char* v_codes;
  const uint8_t* v_scales;
};

template <int kD>
struct Fp4WideShape : AttnShape<kD, true> {
  using Base = AttnShape<kD, true>;
  static constexpr bool kFp4 = true;
  static constexpr int kThreads = Base::kThreads + 128;
  static constexpr int kControlBytes = 1024;
  static constexpr int kSmemBytes = Base::kSmemBytes - Base::kControlBytes + kControlBytes;
};

struct Fp4WideControl {   // as AttnControl, and:
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty, drain, met;
  uint64_t s_full[2][2], p_ready[2][2];
  uint64_t pv_done[2];
  uint64_t q_raw;             // queries have arrived, not converted
  uint32_t tmem;
  volatile int past;
  int abort_word, calm, last;
  unsigned status;
  int q_exponent[2][2];       // [unit % 2][query tile]
  AttnStart start;
  long long sums[16];
};
static_assert(sizeof(Fp4WideControl) <= 1024, "fits kControlBytes");

// Two warps, one per query tile: the first brings a unit's queries, each converts
// its tile in place where it is bfloat16.
template <typename E, int kD, typename S>
__device__ __forceinline__ void fp4_wide_queries(const Fp4WideArgs& a, AttnWalk<S> u, Fp4WideControl* c,
                                                 char* q_ptr, const CUtensorMap* q_map, int t) {
  const int lane = threadIdx.x & 31;
  char* tile = q_ptr + t * S::kQBytes;
  int rounds = 0;
  bool ok = true;
#pragma unroll 1
  for (bool first = true; ok && u.next(first); first = false) {
    if (u.most() == 0) continue;
    if (t == 0) {
      if (rounds > 0 &&
          !(ok = mbar_wait(smem_addr(&c->q_empty), (rounds - 1) & 1, &c->abort_word, naps_of(a))))
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
    }
    if (!(ok = mbar_wait(smem_addr(&c->q_raw), rounds & 1, &c->abort_word, naps_of(a)))) break;
    int exponent = 0;
    if (std::is_same<E, __nv_bfloat16>::value && u.count(t) > 0) {
      // the tile's rows, all of its pieces: columns past the unit's rows may be anything
      constexpr int kPieces = 128 * kD * 2 / 16;
      const int rows = (u.last(t) - u.first(t)) * a.G;
      float top = 0.f;
#pragma unroll 4
      for (int x = lane; x < kPieces; x += 32) {
        const uint4 w = *(const uint4*)(tile + x * 16);
        if (x / 8 % 128 >= rows) continue;
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float lo = fabsf(__uint_as_float(v[y] << 16)), hi = fabsf(__uint_as_float(v[y] & 0xffff0000u));
          if (lo < 3.4e38f) top = fmaxf(top, lo);   // neither infinities nor NaN
          if (hi < 3.4e38f) top = fmaxf(top, hi);
        }
      }
      top = warp_max(top);
      if (!(top == 0.f || (top >= 0.25f && top < 32768.f)))
        exponent = (int)(__float_as_uint(top) >> 23) - 127 - 14;   // subnormal: as if 2^-127
      // 2^-exponent in two factors, each of which is a normal number
      const float f0 = ldexpf(1.f, -exponent / 2), f1 = ldexpf(1.f, -exponent - -exponent / 2);
#pragma unroll 4
      for (int x = lane; x < kPieces; x += 32) {
        const uint4 w = *(const uint4*)(tile + x * 16);
        uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
          v[y] = pack2(__uint_as_float(v[y] << 16) * f0 * f1, __uint_as_float(v[y] & 0xffff0000u) * f0 * f1,
                       __half());
        *(uint4*)(tile + x * 16) = make_uint4(v[0], v[1], v[2], v[3]);
      }
      fence_async_shared();
    }
    if (lane == 0) c->q_exponent[rounds % 2][t] = exponent;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&c->q_full));
    ++rounds;
  }
  // a copy in flight lands in this CTA's memory
  if (t == 0 && rounds > 0 && !ok) (void)mbar_poll(smem_addr(&c->q_raw), (rounds - 1) & 1, &c->calm, kNaps);
  __syncwarp();
}

// Four warps unpack, a key per thread: its codes and scales come to registers while
// the tile before is stored.  Keys past the request's length and those of a page
// outside the cache are zeros.
template <int kD, typename S>
__device__ __forceinline__ void fp4_wide_unpack(const Fp4WideArgs& a, AttnWalk<S> u, Fp4WideControl* c,
                                                char* ring) {
  constexpr int kWords = kD / 32;   // 16-byte pieces of a row's codes
  const int key = threadIdx.x % 128, lane = threadIdx.x & 31;
  struct Row {
    uint4 codes[kWords];
    uint32_t scales[kD / 64];
  };
  bool bad = false;
  int n = 0, i = 0, it = 0;
  long long row = -1;      // of the key in the cache's arrays, -1 if there is none
  bool more = true, first = true;
  // To the next tile; its row.
  auto advance = [&]() {
    if (!more) return;
    ++i;
    while (i >= n) {
      if (!(more = u.next(first))) return;
      first = false;
      n = u.most();
      i = 0;
    }
    const int at = (u.j0 + i) * S::kKeys + key, pg = at >> a.page_shift;
    row = -1;
    if (at < u.units.row.L && in_array(a.flags, u.b, a.B) && in_array(a.flags, pg, a.max_pages)) {
      const int id = a.block_table[(long long)u.b * a.max_pages + pg];
      if (id >= 0 && id < a.n_pages)
        row = (((long long)id * a.Hk + u.h) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
      else bad = true;
    }
  };
  auto fetch = [&](const char* codes, const uint8_t* scales, Row& r) {
#pragma unroll
    for (int p = 0; p < kWords; ++p)
      r.codes[p] = row < 0 ? make_uint4(0, 0, 0, 0) : __ldg((const uint4*)(codes + row * (kD / 2)) + p);
#pragma unroll
    for (int p = 0; p < kD / 64; ++p)
      r.scales[p] = row < 0 ? 0 : __ldg((const uint32_t*)(scales + row * (kD / 16)) + p);
  };
  auto put = [&](const Row& r) -> bool {
    const int stage = it % S::kStages, lap = it / S::kStages;
    if (lap > 0 && !mbar_await(smem_addr(&c->empty[stage]), (lap - 1) & 1, &c->abort_word, naps_of(a)))
      return false;
    char* to = ring + stage * S::kStageBytes + key * 128;
#pragma unroll
    for (int p = 0; p < kWords; ++p) {
      const uint32_t pair = fp4_scales(r.scales[p / 2] >> (p % 2 * 16));
      const uint32_t s[2] = {__byte_perm(pair, 0, 0x1010), __byte_perm(pair, 0, 0x3232)};
      const uint32_t w[4] = {r.codes[p].x, r.codes[p].y, r.codes[p].z, r.codes[p].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t v[4];
        fp4_unpack(w[x], v);
#pragma unroll
        for (int y = 0; y < 4; ++y) v[y] = mul_f16x2(v[y], s[x / 2]);
        const int piece = p * 4 + x;   // of 8 columns
        *(uint4*)(to + (piece / 8) * (S::kKeys * 128) + ((piece % 8) ^ (key % 8)) * 16) =
            make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    fence_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&c->full[stage]));
    ++it;
    return true;
  };
  Row k, v;
  advance();
  if (more) fetch(a.k_codes, a.k_scales, k);
  bool ok = true;
#pragma unroll 1
  while (ok && more) {
    fetch(a.v_codes, a.v_scales, v);
    if (!(ok = put(k))) break;
    advance();
    if (more) fetch(a.k_codes, a.k_scales, k);
    ok = put(v);
  }
  if (bad) set_flag(a.flags, kDevBadPage);
}

template <typename E, int kD>
__global__ void __launch_bounds__(Fp4WideShape<kD>::kThreads, 1)
    sv_fp4_wide_attention_kernel(const __grid_constant__ Fp4WideArgs a, const __grid_constant__ CUtensorMap q_map) {
  using S = Fp4WideShape<kD>;
  extern __shared__ __align__(1024) char smem[];
  char* ring = smem + S::kTiles * S::kQBytes;
  char* staging = ring + S::kStages * S::kStageBytes;
  Fp4WideControl* c = (Fp4WideControl*)(staging + S::kTiles * 4 * S::kStagingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kQueries = S::kSoftThreads / 32, kIssuer = kQueries + 2, kUnpack = kQueries + 4;

  if (warp == kQueries && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_addr(&c->full[i]), 4);
      mbar_init(smem_addr(&c->empty[i]), S::kTiles);
    }
    mbar_init(smem_addr(&c->q_raw), 1);
    mbar_init(smem_addr(&c->q_full), S::kTiles);
    mbar_init(smem_addr(&c->q_empty), S::kTiles);
    mbar_init(smem_addr(&c->drain), S::kTiles);
    mbar_init(smem_addr(&c->met), S::kSoftThreads / 32);
#pragma unroll 1
    for (int t = 0; t < S::kTiles; ++t) {
      mbar_init(smem_addr(&c->s_full[t][0]), 1);
      mbar_init(smem_addr(&c->p_ready[t][0]), 5);   // with the turn
      mbar_init(smem_addr(&c->pv_done[t]), 1);
    }
    mbar_init_fence();
    c->abort_word = c->calm = c->past = 0;
    tma_prefetch_map(&q_map);
  }
  if (warp == kIssuer) tmem_alloc<S::kTmemCols>(smem_addr(&c->tmem));
  wait_for_preceding_grid();
  const AttnRange range = attn_range<S>(a, c);
  const uint32_t tmem = c->tmem;
  if (range.w0 < range.w1) {
    const AttnWalk<S> u(a, c->start, range.w1 - range.w0);
    // launched with 128 registers a thread, and 2 x 184 + 72 + 72 = 4 x 128
    if (warp >= kUnpack) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      fp4_wide_unpack<kD, S>(a, u, c, ring);
    } else if (warp >= kQueries) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      if (warp >= kIssuer)
        attn_multiply<__half, kD, S>(a, u, c, smem_addr(smem), smem_addr(ring), ring, tmem, warp - kIssuer);
      else
        fp4_wide_queries<E, kD, S>(a, u, c, smem, &q_map, warp - kQueries);
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
      attn_softmax<__half, E, kD, S>(a, u, c, tmem, staging, range.quota, range.w1);
    }
  }
  attn_finish<S, kD>(a, c, range.spoilt);
  if (warp == kIssuer) tmem_free<S::kTmemCols>(tmem);
}

}  // namespace sv
