// decode_plan.cuh -- the split plan of the paged decodes, made on the device
// from the batch's own positions: the split length, the item count and the
// per-sequence item prefix (an item is a (sequence, split, KV head)).
//
// ITEM_KEYS is an item's fixed cost in keys, MAX_LEN the longest split; both
// are the kernel's own (measured there).
#pragma once

#include "common.cuh"

namespace kvr {

// int32 words of the plan ahead of the item prefix: the split length, the item count
constexpr int DECODE_PLAN_PREFIX = 64;

namespace {

constexpr int DP_CANDS = 16;

// The plan by one CTA of NT threads: the split length (returned), the item
// count (*nitems) and the per-sequence item prefix (prefix[0..B]).  Flags bad
// entries when `status` is not null.
template <int NT, long long ITEM_KEYS, long long MAX_LEN>
__device__ int decode_plan_block(const int64_t *__restrict__ pos, const int32_t *__restrict__ seq, int B, int hkv,
                                 int num_seqs, int64_t max_pos, long long max_ctx, int R, int32_t *prefix,
                                 int *nitems, unsigned *status) {
  constexpr int NW = NT / 32;
  __shared__ long long s_tot[NW], s_mx[NW];
  __shared__ int s_cnt[NW][DP_CANDS];
  __shared__ int s_scan[NW];
  __shared__ int s_L;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto ctx_of = [&](int b) -> long long {
    const long long p = pos[b];
    const int s = seq[b];
    return (p >= 0 && p < max_pos && p + 1 <= max_ctx && s >= 0 && s < num_seqs) ? p + 1 : 0;
  };
  // 1. total keys, longest context, bad entries
  long long tot = 0, mx = 0;
  unsigned bad = 0;
  for (int b = tid; b < B; b += NT) {
    const long long p = pos[b];
    const int s = seq[b];
    const bool bp = p < 0 || p >= max_pos || p + 1 > max_ctx, bs = s < 0 || s >= num_seqs;
    if (bp || bs) {
      bad |= (bp ? ST_BAD_POS : 0u) | (bs ? ST_BAD_SEQ : 0u);
    } else {
      tot += p + 1;
      mx = p + 1 > mx ? p + 1 : mx;
    }
  }
  if (bad && status) flag(status, bad);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tot += __shfl_xor_sync(0xffffffffu, tot, o);
    const long long y = __shfl_xor_sync(0xffffffffu, mx, o);
    mx = y > mx ? y : mx;
  }
  if (lane == 0) {
    s_tot[warp] = tot;
    s_mx[warp] = mx;
  }
  __syncthreads();
  tot = 0;
  mx = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    tot += s_tot[i];
    mx = s_mx[i] > mx ? s_mx[i] : mx;
  }
  // 2. candidate split lengths: lane c of every warp derives candidate c and
  // the warp shares them by shuffles (GB300's FP64 rate is a small fraction of
  // its integer rate, so no double arithmetic here; one 64-bit division per
  // lane, the rest in 32 bits as contexts and split lengths fit)
  unsigned mine_L;
  {
    const unsigned k = lane % 8 + 1;
    unsigned L;
    if (lane < 8) {  // about k items per resident CTA for the longest context
      unsigned n = k * (unsigned)R / ((unsigned)B * (unsigned)hkv);
      if (n < 1) n = 1;
      L = ((unsigned)mx + n - 1) / n;
    } else {         // ... for the batch's total keys
      const unsigned long long d = (unsigned long long)k * (unsigned)R;
      const unsigned long long l = ((unsigned long long)tot * (unsigned)hkv + d - 1) / d;
      L = l > (unsigned long long)MAX_LEN ? (unsigned)MAX_LEN : (unsigned)l;
    }
    L = (L + 63) / 64 * 64;
    mine_L = L < 64 ? 64u : (L > (unsigned)MAX_LEN ? (unsigned)MAX_LEN : L);
  }
  unsigned cand[DP_CANDS];
#pragma unroll
  for (int c = 0; c < DP_CANDS; ++c) cand[c] = __shfl_sync(0xffffffffu, mine_L, c);
  // 3. items of every candidate, one combined reduction
  int cnt[DP_CANDS];
#pragma unroll
  for (int c = 0; c < DP_CANDS; ++c) cnt[c] = 0;
  for (int b = tid; b < B; b += NT) {
    const unsigned ctx = (unsigned)ctx_of(b);
#pragma unroll
    for (int c = 0; c < DP_CANDS; ++c) cnt[c] += (int)((ctx + cand[c] - 1) / cand[c]);
  }
#pragma unroll
  for (int c = 0; c < DP_CANDS; ++c) cnt[c] = __reduce_add_sync(0xffffffffu, cnt[c]);
  if (lane == 0) {
#pragma unroll
    for (int c = 0; c < DP_CANDS; ++c) s_cnt[warp][c] = cnt[c];
  }
  __syncthreads();
  // 4. choose: the least cost, ties to fewer items (one thread: measured
  // quicker here than a warp-wide argmin)
  if (tid == 0) {
    unsigned best_L = (unsigned)MAX_LEN, best_items = 0;
    long long best_cost = -1;
    for (int c = 0; c < DP_CANDS; ++c) {
      unsigned items = 0;
      for (int i = 0; i < NW; ++i) items += (unsigned)s_cnt[i][c];
      items *= (unsigned)hkv;
      const long long cost = (long long)((items + (unsigned)R - 1) / (unsigned)R) * (cand[c] + ITEM_KEYS);
      if (best_cost < 0 || cost < best_cost || (cost == best_cost && items < best_items)) {
        best_cost = cost;
        best_L = cand[c];
        best_items = items;
      }
    }
    s_L = (int)best_L;
  }
  __syncthreads();
  const unsigned L = (unsigned)s_L;
  // 5. per-sequence item prefix (exclusive scan, NT sequences at a time)
  int running = 0;
  for (int b0 = 0; b0 < B; b0 += NT) {
    const int b = b0 + tid;
    const int mine = b < B ? (int)(((unsigned)ctx_of(b) + L - 1) / L) * hkv : 0;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      before += i < warp ? s_scan[i] : 0;
      all += s_scan[i];
    }
    if (b < B) prefix[b] = running + before + x - mine;
    running += all;
    __syncthreads();  // s_scan is rewritten by the next round
  }
  if (tid == 0) prefix[B] = running;
  *nitems = running;
  return (int)L;
}

// The same plan made by one warp for a batch of at most 32 sequences (lane b
// is sequence b): warp reductions and shuffles only, no block barrier.  Ties
// between candidates of equal cost go to the lower candidate index.  The
// split length and the item count go to prefix[B + 1] and prefix[B + 2].
// Lane b < B passes sequence b's position p and id s (the other lanes
// anything).
template <long long ITEM_KEYS, long long MAX_LEN>
__device__ void decode_plan_warp(long long p, int s, int B, int hkv,
                                 int num_seqs, int64_t max_pos, long long max_ctx, int R, int32_t *prefix,
                                 unsigned *status) {
  constexpr unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  unsigned ctx = 0, bad = 0;
  if (lane < B) {
    const bool bp = p < 0 || p >= max_pos || p + 1 > max_ctx, bs = s < 0 || s >= num_seqs;
    if (bp || bs)
      bad = (bp ? ST_BAD_POS : 0u) | (bs ? ST_BAD_SEQ : 0u);
    else
      ctx = (unsigned)(p + 1);
  }
  if (bad && status) flag(status, bad);
  const unsigned mx = __reduce_max_sync(FULL, ctx);
  const unsigned long long tot = ((unsigned long long)__reduce_add_sync(FULL, ctx >> 16) << 16) +
                                 __reduce_add_sync(FULL, ctx & 0xffffu);
  // candidate `lane` (lanes 0 .. 15), as in decode_plan_block
  unsigned mine_L;
  {
    const unsigned k = lane % 8 + 1;
    unsigned L;
    if (lane < 8) {
      unsigned n = k * (unsigned)R / ((unsigned)B * (unsigned)hkv);
      if (n < 1) n = 1;
      L = (mx + n - 1) / n;
    } else {
      const unsigned long long d = (unsigned long long)k * (unsigned)R;
      const unsigned long long l = (tot * (unsigned)hkv + d - 1) / d;
      L = l > (unsigned long long)MAX_LEN ? (unsigned)MAX_LEN : (unsigned)l;
    }
    L = (L + 63) / 64 * 64;
    mine_L = L < 64 ? 64u : (L > (unsigned)MAX_LEN ? (unsigned)MAX_LEN : L);
  }
  unsigned items_mine = 0;  // items of candidate `lane`
#pragma unroll
  for (int c = 0; c < DP_CANDS; ++c) {
    const unsigned L = __shfl_sync(FULL, mine_L, c);
    const unsigned n = __reduce_add_sync(FULL, (ctx + L - 1) / L);
    if (lane == c) items_mine = n * (unsigned)hkv;
  }
  unsigned key = FULL;
  if (lane < DP_CANDS) {
    unsigned cost = (items_mine + (unsigned)R - 1) / (unsigned)R * (mine_L + ITEM_KEYS);
    cost = cost > 0x7ffffffu ? 0x7ffffffu : cost;
    key = (cost << 4) | (unsigned)lane;
  }
  const unsigned L = __shfl_sync(FULL, mine_L, (int)(__reduce_min_sync(FULL, key) & 15u));
  // per-sequence item prefix
  const int mine = lane < B ? (int)((ctx + L - 1) / L) * hkv : 0;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  if (lane < B) prefix[lane] = x - mine;
  if (lane == 31) {
    prefix[B] = x;
    prefix[B + 1] = (int)L;
    prefix[B + 2] = x;
  }
}

// Batches too large for the split kernel's own plan: a kernel of its own,
// written to the workspace for the split and merge kernels.
constexpr int DP_THREADS = 256;

template <long long ITEM_KEYS, long long MAX_LEN>
__global__ void __launch_bounds__(DP_THREADS)
    decode_plan_kernel(const int64_t *__restrict__ pos, const int32_t *__restrict__ seq, int B, int hkv,
                            int num_seqs, int64_t max_pos, long long max_ctx, int R, int32_t *__restrict__ plan,
                            unsigned *status) {
  pdl_wait();
  pdl_trigger();
  int nitems;
  const int L = decode_plan_block<DP_THREADS, ITEM_KEYS, MAX_LEN>(pos, seq, B, hkv, num_seqs, max_pos, max_ctx, R,
                                                                  plan + DECODE_PLAN_PREFIX, &nitems, status);
  if (threadIdx.x == 0) {
    plan[0] = L;
    plan[1] = nitems;
  }
}

}  // namespace
}  // namespace kvr
