// Pages, slots and packed offsets of a step, from the request lengths.
//
// Everything follows from three exclusive sums over the rows: new tokens,
// pages given back, pages taken.  Every CTA forms all of them (a thread owns
// consecutive rows; warp shuffles join the threads) and keeps a row's sums in
// shared memory; then the CTAs share out the tokens, the taken pages and the
// pages that go on the stack, each index finding its row by bisection of the
// sums.  The k-th page taken is a closed form of k, so no CTA waits for
// another's work.  Where the counts are updated in place the grid is one
// cluster, whose barrier stands between the last read and the first write;
// else it is as large as the tokens ask for.
//
// Bound by latency: the chain load lengths -> two block sums -> bisect ->
// load page -> store: 3.2 us for one row, 5.9 us for 64 rows of five tokens,
// 10 us for 1024 rows and half a million tokens, whose 4 MB over 118 CTAs add
// what one CTA per cluster of eight took 60 us for.
#pragma once

#include "sv_paged.cuh"

namespace sv {

constexpr int kPlanThreads = 1024;     // at most
constexpr int kPlanChunk = 256;        // consecutive tokens of a warp, at most
constexpr int kPlanRowBytes = 5 * 4;   // shared memory per row

struct PlanArgs {
  const int32_t* seq_len;      // [B]
  const int32_t* num_new;      // [B]
  const int32_t* page_count;   // [B]
  int32_t* block_table;        // [B, max_pages]
  int32_t* free_pages;         // [n_pages]
  const int32_t* free_count;   // [1]
  int B, page_shift, max_pages, n_pages, max_tokens;
  int chunk;                   // consecutive tokens of a warp, a multiple of 32
  int32_t* cu_new;             // [B+1]
  int32_t* kv_len;             // [B]
  int32_t* slot_map;           // [max_tokens]
  int32_t* positions;          // [max_tokens]
  int32_t* page_count_out;     // [B], may be page_count
  int32_t* free_count_out;     // [1], may be free_count
  bool in_place;               // a count's output is its input: the grid is one cluster
  unsigned* flags;
};

// Exclusive sum over the block's threads; `total` is the block's sum.
// `parts` has one entry per warp and is free again on return.
template <typename V>
__device__ __forceinline__ V block_exclusive_sum(V v, V* parts, V* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) parts[warp] = inc;
  __syncthreads();
  V p = lane < blockDim.x / 32 ? parts[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, p, o);
    if (lane >= o) p += u;
  }
  const V before = __shfl_sync(0xffffffffu, p, warp > 0 ? warp - 1 : 0);
  *total = __shfl_sync(0xffffffffu, p, 31);
  __syncthreads();
  return inc - v + (warp > 0 ? before : 0);
}

__device__ __forceinline__ int block_max(int v, int* parts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = __reduce_max_sync(0xffffffffu, v);
  if (lane == 0) parts[warp] = v;
  __syncthreads();
  v = __reduce_max_sync(0xffffffffu, parts[lane < blockDim.x / 32 ? lane : 0]);
  __syncthreads();
  return v;
}

// First row whose inclusive sum passes i (ends is non-decreasing, i < ends[n-1]).
__device__ __forceinline__ int row_of(const int* ends, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) sv_paged_plan_kernel(PlanArgs a) {
  extern __shared__ int plan_rows[];
  int* s_cu = plan_rows;             // inclusive sums: new tokens,
  int* s_need = s_cu + a.B;          // pages taken,
  int* s_back = s_need + a.B;        // pages given back
  int* s_have = s_back + a.B;        // pages held before, -1 for rows not served
  int* s_seq = s_have + a.B;
  __shared__ long long parts[32];
  const int tid = threadIdx.x;
  const int cta = blockIdx.x, n_ctas = gridDim.x, threads = blockDim.x;
  const int page = 1 << a.page_shift;

  wait_for_preceding_grid();
  allow_dependent_launch();

  unsigned bad = 0;
  int F = *a.free_count;
  if (F < 0 || F > a.n_pages) {
    bad |= kDevLength;
    F = F < 0 ? 0 : a.n_pages;
  }
  // -------- new tokens.  Rows of the thread: [r0, r1)
  const int per = (a.B + threads - 1) / threads;
  const int r0 = min(a.B, tid * per), r1 = min(a.B, r0 + per);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) {
    const int seq = a.seq_len[r], have = a.page_count[r];
    int fresh = a.num_new[r];
    const bool valid = seq >= 0 && fresh >= 0 && have >= 0 && have <= a.max_pages &&
                       (long long)seq + fresh <= ((long long)a.max_pages << a.page_shift);
    if (!valid) {
      bad |= kDevLength;
      fresh = 0;
    }
    s_seq[r] = seq;
    s_have[r] = valid ? have : -1;
    s_cu[r] = fresh;
    mine += fresh;
  }
  long long sum64;
  long long end = block_exclusive_sum(mine, parts, &sum64);
  int last_fit = 0;   // the largest sum that max_tokens admits
  for (int r = r0; r < r1; ++r) {
    const int fresh = s_cu[r];
    end += fresh;
    if (end <= a.max_tokens) {
      last_fit = (int)end;
    } else if (fresh > 0) {   // its tokens do not fit, so no later row's do
      bad |= kDevTokensClipped;
      s_have[r] = -1;
    }
    s_cu[r] = end <= a.max_tokens ? (int)end : INT32_MAX;
  }
  last_fit = block_max(last_fit, (int*)parts);
  // -------- pages given back and taken
  int back = 0, need = 0;
  for (int r = r0; r < r1; ++r) {
    s_cu[r] = min(s_cu[r], last_fit);
    s_back[r] = s_need[r] = 0;
  }
  __syncthreads();   // a row's tokens are the difference of two threads' sums
  for (int r = r0; r < r1; ++r) {
    if (s_have[r] < 0) continue;
    const int fresh = s_cu[r] - (r > 0 ? s_cu[r - 1] : 0);
    const int want = (int)(((long long)s_seq[r] + fresh + page - 1) >> a.page_shift);
    const int more = want - s_have[r];
    if (more > 0) need += s_need[r] = more;
    else back += s_back[r] = -more;
  }
  long long total;
  const long long before =
      block_exclusive_sum((long long)back << 32 | (unsigned)need, parts, &total);
  const int R = (int)(total >> 32);
  const long long avail = (long long)F + R;
  int back_end = (int)(before >> 32);
  int need_end = (int)(unsigned)before;
  int served_end = 0;
  for (int r = r0; r < r1; ++r) {
    const int d = s_need[r];
    back_end += s_back[r];
    s_back[r] = back_end;
    if (d > 0) {
      need_end += d;
      if (need_end <= avail) {
        served_end = need_end;
      } else {
        bad |= kDevNoPages;
        s_have[r] = -1;
      }
    }
    s_need[r] = need_end <= avail ? need_end : INT32_MAX;
  }
  const int N = block_max(served_end, (int*)parts);   // pages taken
  for (int r = r0; r < r1; ++r) s_need[r] = min(s_need[r], N);
  __syncthreads();

  // entry pg of row r's block table, and whether the checked build admits it
  auto entry = [&](int r, int pg) { return (long long)r * a.max_pages + pg; };
  auto has_entry = [&](int r, int pg) {
    return in_array(a.flags, r, a.B) && in_array(a.flags, pg, a.max_pages);
  };
  // k-th page taken, k < F + R: those given back in order, then the stack from its top
  auto taken = [&](int k) -> int {
    if (k >= R) {
      const int at = F - 1 - (k - R);
      return in_array(a.flags, at, a.n_pages) ? a.free_pages[at] : -1;
    }
    const int r = row_of(s_back, a.B, k);
    const int first = r > 0 ? s_back[r - 1] : 0;
    const int pg = s_have[r] - (s_back[r] - first) + (k - first);
    return has_entry(r, pg) ? a.block_table[entry(r, pg)] : -1;
  };

  // -------- the CTAs of the cluster share out what is left
  const unsigned first = cta * threads + tid, step = n_ctas * threads;   // sums stay below 2^31
  for (unsigned k = first; k < (unsigned)N; k += step) {   // the tables' new entries
    const int r = row_of(s_need, a.B, k);
    const int pg = s_have[r] + (k - (r > 0 ? s_need[r - 1] : 0));
    if (has_entry(r, pg)) a.block_table[entry(r, pg)] = taken(k);
  }
  for (unsigned j = first; (long long)j < R - N; j += step) {   // given back and not taken
    if (F + j < (unsigned)a.n_pages) a.free_pages[F + j] = taken(R - 1 - j);   // bounded here
    else bad |= kDevLength;
  }
  const int tokens = a.B > 0 ? s_cu[a.B - 1] : 0;
  const int lane = tid & 31;
  for (unsigned t0 = first / 32 * a.chunk; t0 < (unsigned)a.max_tokens; t0 += step / 32 * a.chunk) {
    unsigned t = t0 + lane;
    int r = t < (unsigned)tokens ? row_of(s_cu, a.B, t) : 0;
    for (int i = 0; i < a.chunk; i += 32, t += 32) {
      if (t >= (unsigned)a.max_tokens) break;
      int slot = -1, pos = -1;
      if (t < (unsigned)tokens) {
        while (s_cu[r] <= (int)t) ++r;
        pos = s_seq[r] + t - (r > 0 ? s_cu[r - 1] : 0);
        const int have = s_have[r];
        if (have >= 0) {
          const int pg = pos >> a.page_shift;
          const int id = pg >= have         ? taken((r > 0 ? s_need[r - 1] : 0) + pg - have)
                         : has_entry(r, pg) ? a.block_table[entry(r, pg)]
                                            : -1;
          if (id >= 0 && id < a.n_pages) slot = (id << a.page_shift) | (pos & (page - 1));
          else bad |= kDevBadPage;
        }
      }
      if (in_array(a.flags, t, a.max_tokens)) {
        a.slot_map[t] = slot;
        a.positions[t] = pos;
      }
    }
  }
  if (bad) set_flag(a.flags, bad);
  // -------- lengths and counts, in place if the caller likes: every CTA has read them
  if (a.in_place && n_ctas > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (cta == 0) {
    for (int r = tid; r < a.B; r += threads) {
      const int begin = r > 0 ? s_cu[r - 1] : 0, fresh = s_cu[r] - begin;
      const int have = s_have[r];
      a.cu_new[r + 1] = s_cu[r];
      a.kv_len[r] = have >= 0 ? s_seq[r] + fresh : 0;
      a.page_count_out[r] = have >= 0 ? have + (s_need[r] - (r > 0 ? s_need[r - 1] : 0)) -
                                            (s_back[r] - (r > 0 ? s_back[r - 1] : 0))
                                      : a.page_count[r];
    }
    if (tid == 0) {
      a.cu_new[0] = 0;
      *a.free_count_out = (int)min(avail - N, (long long)a.n_pages);
    }
  }
}

}  // namespace sv
