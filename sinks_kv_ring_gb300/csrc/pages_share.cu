// pages_share.cu -- pages held by more than one sequence: forking a sequence,
// giving pages up, and moving the pool's used blocks together (the Full pool of
// Xiaomi "Full-Pipeline Inference Optimization for MiMo-V2.5 Series", section
// 2.1, whose prefixes are kept and shared; kv_pages_grow takes blocks from the
// same free list).
//
// refs[b] counts the holders of block b beyond the first, so a pool that never
// forked has zeros, and the calls that know nothing of sharing leave it right.
// Giving a block up subtracts one: what ends at -1 has no holder left.  Then the
// blocks at -1, in ascending order, go to the free list -- an order that does not
// hang on which holder came first, so atomics decide nothing.
//
// Each call is one cluster of CTAs (or one CTA, where there is little to do: its
// barrier is cheaper): the steps of a call wait for one another, and a cluster's
// barrier is cheaper than a launch.
//
// What bounds them: the latency of a launch and of a few dependent loads and
// atomics, and of a cluster's barriers.  Giving up 4 beams of 10 blocks and forking
// them again takes 1.8 and 2.6 us (one CTA; with the cluster 9.3 in all), 128 of up
// to 257 blocks 4.1 and 6.4 (a cluster of eight; of four 3.7 and 5.3, one CTA 15 and
// 6.8: there four would do better, and all calls have eight, which compaction was
// measured with and larger pools' counts are spread over); compacting 6000 blocks under 96 sequences 5.1, where a plan in global memory
// with a barrier between its steps and a second launch for the tables took 13.2.
#include <cooperative_groups.h>

#include "launch.h"

namespace kvr {
namespace {

constexpr int SH_CTAS = 8;
constexpr int SH_THREADS = 1024;
constexpr int SH_WARPS = SH_THREADS / 32;
constexpr int SH_SMALL = 4;  // rounds of one CTA's threads up to which it does a call alone (16 measured the same)
constexpr unsigned FULLW = 0xffffffffu;

// Barrier of the call's CTAs: all that they wrote, to global memory too, is seen behind it.
template <int CTAS>
__device__ __forceinline__ void call_sync() {
  if (CTAS == 1) {
    __syncthreads();
  } else {
    __threadfence();
    cooperative_groups::this_cluster().sync();
  }
}
template <int CTAS>
__device__ __forceinline__ int call_rank() {
  return CTAS == 1 ? 0 : (int)cooperative_groups::this_cluster().block_rank();
}

// Exclusive prefix of x over the CTA's threads, in order; `total` is their sum.
__device__ __forceinline__ int cta_prefix(int x, int &total) {
  __shared__ int s_sum[SH_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(FULLW, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();  // s_sum of the call before is read
  if (lane == 31) s_sum[warp] = y;
  __syncthreads();
  // every warp takes the sums' prefix
  int z = s_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULLW, z, o);
    if (lane >= o) z += v;
  }
  total = __shfl_sync(FULLW, z, 31);
  const int before = __shfl_sync(FULLW, z, (warp + 31) & 31);
  return (warp ? before : 0) + y - x;
}
// The same for a truth value: two ballots in place of the shuffles.
__device__ __forceinline__ int cta_rank(bool x, int &total) {
  __shared__ int s_sum[SH_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(FULLW, x);
  __syncthreads();
  if (lane == 0) s_sum[warp] = __popc(m);
  __syncthreads();
  int z = s_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULLW, z, o);
    if (lane >= o) z += v;
  }
  total = __shfl_sync(FULLW, z, 31);
  const int before = __shfl_sync(FULLW, z, (warp + 31) & 31);
  return (warp ? before : 0) + __popc(m & ((1u << lane) - 1u));
}

struct FreeArgs {
  int32_t *table;
  int num_seqs, max_blocks, block_size, num_blocks;
  int32_t *refs;
  const int32_t *seqs;
  const int64_t *keep_lo, *keep_hi;
  int n;
  int32_t *free_ids, *free_count;
  int free_cap;
  unsigned *status;
};

// Entries of the call that thread `me` of `all` sees to: they are given up
// unless they hold a position of [keep_lo, keep_hi).
__device__ __forceinline__ void drop_entries(const FreeArgs &A, long long me, long long all) {
  // a warp's lanes take neighbouring entries of one request
  const int lane = threadIdx.x & 31, rounds = (A.max_blocks + 31) >> 5;
  for (long long w = me >> 5; w < (long long)A.n * rounds; w += all >> 5) {
    const int i = (int)(w / rounds), bi = (int)(w - (long long)i * rounds) * 32 + lane;
    const int s = A.seqs[i];
    if (s < 0 || s >= A.num_seqs) {
      if (bi == 0) flag(A.status, ST_BAD_SEQ);
      continue;
    }
    if (bi >= A.max_blocks) continue;
    const long long p = (long long)bi * A.block_size;
    const long long k0 = A.keep_lo ? A.keep_lo[i] : 0, k1 = A.keep_hi ? A.keep_hi[i] : 0;
    if (k0 < k1 && p < k1 && p + A.block_size > k0) continue;
    int32_t *e = A.table + (long long)s * A.max_blocks + bi;
    const int id = *e;
    if (id < 0) continue;
    if (id >= A.num_blocks) {
      flag(A.status, ST_BAD_BLOCK);
      continue;
    }
    // (taken by an exchange: a sequence that the call names twice gives up once)
    if (atomicExch(e, -1) == id) atomicSub(A.refs + id, 1);
  }
}

__global__ void __launch_bounds__(SH_THREADS) pages_drop_kernel(FreeArgs A) {
  pdl_wait();
  pdl_trigger();
  drop_entries(A, (long long)blockIdx.x * SH_THREADS + threadIdx.x, (long long)gridDim.x * SH_THREADS);
}

template <int CTAS, bool DROP>
__device__ __forceinline__ void pages_free_body(const FreeArgs &A) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, rank = call_rank<CTAS>();
  const int count = *A.free_count;
  if (DROP) {
    drop_entries(A, (long long)rank * SH_THREADS + tid, CTAS * SH_THREADS);
    call_sync<CTAS>();
  }
  // blocks without a holder: counted by the CTA that sees to them, then listed in order
  const int each = (A.num_blocks + CTAS - 1) / CTAS;
  const int lo = (int)min((long long)rank * each, (long long)A.num_blocks), hi = (int)min((long long)lo + each, (long long)A.num_blocks);
  __shared__ int s_mine;
  int before = 0, all = 0;
  if (CTAS > 1) {
    cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
    int mine = 0;
    for (int b0 = lo; b0 < hi; b0 += 4 * SH_THREADS) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int b = b0 + u * SH_THREADS + tid;
        mine += b < hi && __ldcg(A.refs + b) < 0;
      }
    }
    int total;
    cta_prefix(mine, total);
    if (tid == 0) s_mine = total;
    cl.sync();  // (and every CTA has read the count)
    for (int r = 0; r < CTAS; ++r) {
      const int x = *cl.map_shared_rank(&s_mine, r);
      before += r < rank ? x : 0;
      all += x;
    }
    cl.sync();  // (no CTA leaves while another reads its count)
    if (all == 0) return;
    if (count < 0 || (long long)count + all > A.free_cap) {
      if (rank == 0 && tid == 0) flag(A.status, ST_FREE_FULL);
      return;
    }
  } else {
    for (int b0 = 0; b0 < hi; b0 += SH_THREADS) all += __syncthreads_count(b0 + tid < hi && __ldcg(A.refs + b0 + tid) < 0);
    if (all == 0) return;
    if (count < 0 || (long long)count + all > A.free_cap) {
      if (tid == 0) flag(A.status, ST_FREE_FULL);
      return;
    }
  }
  int at = count + before;
  for (int b0 = lo; b0 < hi; b0 += SH_THREADS) {
    const bool dead = b0 + tid < hi && __ldcg(A.refs + b0 + tid) < 0;
    int total;
    const int k = cta_rank(dead, total);
    if (dead) {
      A.free_ids[at + k] = b0 + tid;
      A.refs[b0 + tid] = 0;
    }
    at += total;
  }
  if (rank == 0 && tid == 0) *A.free_count = count + all;
}
template <bool DROP>
__global__ void __cluster_dims__(SH_CTAS, 1, 1) __launch_bounds__(SH_THREADS) pages_free_kernel(FreeArgs A) {
  pages_free_body<SH_CTAS, DROP>(A);
}
__global__ void __launch_bounds__(SH_THREADS) pages_free_one_kernel(FreeArgs A) { pages_free_body<1, true>(A); }

struct ForkArgs {
  int32_t *table;
  int num_seqs, max_blocks, block_size, num_blocks;
  int32_t *refs;
  const int32_t *src_seqs, *dst_seqs;
  const int64_t *lens;
  int n;
  const int32_t *free_ids, *count_in;
  int32_t *count_out;
  int free_cap;
  int32_t *copy_src, *copy_dst, *copy_count;
  unsigned *status;
};

template <int CTAS>
__device__ __forceinline__ void pages_fork_body(const ForkArgs &A) {
  extern __shared__ int32_t s_tail[];  // [n] entry i's new block: its number in the call, or -1 (none) or -2 (not served)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, rank = call_rank<CTAS>();
  const int count = *A.count_in;
  const long long cap_pos = (long long)A.max_blocks * A.block_size;
  int need = 0;
  unsigned bad = 0;
  for (int i0 = 0; i0 < A.n; i0 += SH_THREADS) {  // (every CTA takes the same sums)
    const int i = i0 + tid;
    int code = -2;
    if (i < A.n) {
      const int s = A.src_seqs[i], d = A.dst_seqs[i];
      const long long len = A.lens[i];
      if (s < 0 || s >= A.num_seqs || d < 0 || d >= A.num_seqs || s == d) bad |= ST_BAD_SEQ;
      else if (len < 0 || len > cap_pos) bad |= ST_BAD_POS;
      else code = len % A.block_size ? 0 : -1;
    }
    int total;
    const int k = cta_rank(code == 0, total);
    if (i < A.n) s_tail[i] = code == 0 ? need + k : code;
    need += total;
  }
  __syncthreads();
  const bool none = count < 0 || count > A.free_cap || need > count;  // too few free blocks: nothing changes
  if (rank == 0) {
    if (bad) flag(A.status, bad);
    if (tid == 0 && none) flag(A.status, ST_NO_BLOCKS);
  }
  if (!none) {
    for (int i = rank * SH_WARPS + (tid >> 5); i < A.n; i += CTAS * SH_WARPS) {  // a warp an entry
      const int k = s_tail[i];
      if (k == -2) continue;
      const int32_t *from = A.table + (long long)A.src_seqs[i] * A.max_blocks;
      int32_t *to = A.table + (long long)A.dst_seqs[i] * A.max_blocks;
      const long long len = A.lens[i];
      const int whole = (int)(len / A.block_size);
      for (int bi = lane; bi < whole; bi += 32) {
        int id = from[bi];
        if (id >= 0 && id < A.num_blocks) {
          atomicAdd(A.refs + id, 1);
        } else {
          flag(A.status, ST_BAD_BLOCK);
          id = -1;
        }
        to[bi] = id;
      }
      if (k >= 0 && lane == 0) {
        int old = from[whole], id = A.free_ids[count - 1 - k];
        const bool ob = old < 0 || old >= A.num_blocks, nb = id < 0 || id >= A.num_blocks;
        if (ob || nb) flag(A.status, ST_BAD_BLOCK);
        if (nb) id = -1;
        to[whole] = id;
        A.copy_src[k] = ob || nb ? -1 : old;
        A.copy_dst[k] = ob ? -1 : id;
      }
    }
  }
  call_sync<CTAS>();  // every CTA has read the free count
  if (rank == 0 && tid == 0) {
    *A.copy_count = none ? 0 : need;
    *A.count_out = none ? count : count - need;
  }
}
__global__ void __cluster_dims__(SH_CTAS, 1, 1) __launch_bounds__(SH_THREADS) pages_fork_kernel(ForkArgs A) {
  pages_fork_body<SH_CTAS>(A);
}
__global__ void __launch_bounds__(SH_THREADS) pages_fork_one_kernel(ForkArgs A) { pages_fork_body<1>(A); }

struct CompactArgs {
  const int32_t *table;
  int32_t *table_out;
  long long entries;
  int num_blocks, limit;
  const int32_t *refs;
  int32_t *refs_out;
  const int32_t *free_ids, *free_count;
  int32_t *free_out;
  int free_cap;
  int32_t *copy_src, *copy_dst, *copy_count;
  unsigned *status;
};

// The free blocks of a pool as bits in shared memory, and how many there are below
// any id: per 32 words (1024 blocks) the total before them, per word the number
// since those (16 bits).  Six bytes for 32 blocks.
struct FreeSet {
  uint32_t *bits;    // [groups * 32]
  int *group;        // [groups + 1]
  uint16_t *since;   // [groups * 32]
  int groups;
  __device__ __forceinline__ bool has(int b) const { return bits[b >> 5] >> (b & 31) & 1; }
  __device__ __forceinline__ int below(int b) const {  // b < 1024 groups
    return group[b >> 10] + since[b >> 5] + __popc(bits[b >> 5] & ((1u << (b & 31)) - 1u));
  }
  __device__ __forceinline__ int nth(int k) const {  // the k-th free block (k < their number)
    int lo = 0, hi = groups;  // group[lo] <= k < group[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (group[mid] <= k) lo = mid; else hi = mid;
    }
    k -= group[lo];
    int w = lo * 32;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
      if (since[w + step] <= k) w += step;
    k -= since[w];
    uint32_t x = bits[w];
    for (; k > 0; --k) x &= x - 1;
    return w * 32 + __ffs(x) - 1;
  }
};

// Every CTA makes the whole set of free blocks by itself, so where a block goes is
// known everywhere without a word between the CTAs: the k-th used block at or past
// the limit takes the k-th free place.  The one barrier stands between the last
// read of the free list and its new form, which may be in place.
__global__ void __cluster_dims__(SH_CTAS, 1, 1) __launch_bounds__(SH_THREADS) pages_compact_kernel(CompactArgs A) {
  extern __shared__ uint32_t s_set[];
  __shared__ int s_wrong;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, num = A.num_blocks;
  FreeSet F;
  F.groups = (num + 1023) >> 10;
  F.bits = s_set;
  F.group = reinterpret_cast<int *>(s_set + F.groups * 32);
  F.since = reinterpret_cast<uint16_t *>(F.group + F.groups + 1);
  for (int w = tid; w < F.groups * 32; w += SH_THREADS) F.bits[w] = 0;
  if (tid == 0) s_wrong = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int me = call_rank<SH_CTAS>() * SH_THREADS + tid;
  constexpr int ALL = SH_CTAS * SH_THREADS;
  const int count = *A.free_count;
  const bool sane = count >= 0 && count <= A.free_cap && count <= num;
  // a free list that names a block twice, or none of the pool's, moves nothing
  bool odd = !sane;
  for (int j0 = tid; sane && j0 < count; j0 += 4 * SH_THREADS) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u * SH_THREADS;
      if (j >= count) break;
      const int id = A.free_ids[j];
      if (id < 0 || id >= num) odd = true;
      else odd |= atomicOr(F.bits + (id >> 5), 1u << (id & 31)) >> (id & 31) & 1;
    }
  }
  if (odd) s_wrong = 1;
  call_sync<SH_CTAS>();  // (every CTA has read the list)
  for (int g = warp; g < F.groups; g += SH_WARPS) {
    const int n = __popc(F.bits[g * 32 + lane]);
    int y = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(FULLW, y, o);
      if (lane >= o) y += z;
    }
    F.since[g * 32 + lane] = (uint16_t)(y - n);
    if (lane == 31) F.group[g] = y;
  }
  __syncthreads();
  int sum;  // (up to 1024 groups: one each)
  const int mine = tid < F.groups ? F.group[tid] : 0, before = cta_prefix(mine, sum);
  if (tid < F.groups) F.group[tid] = before;
  if (tid == 0) F.group[F.groups] = sum;
  __syncthreads();
  const bool wrong = s_wrong != 0;
  const int used = num - sum, limit = A.limit > 0 ? min(A.limit, num) : used;
  const bool none = wrong || limit < used;
  if (me == 0 && none) flag(A.status, wrong ? ST_BAD_BLOCK : ST_NO_BLOCKS);
  if (none) {  // as it was
    if (A.refs_out != A.refs)
      for (long long b = me; b < num; b += ALL) A.refs_out[b] = A.refs[b];
    if (A.free_out != A.free_ids)  // (a count that is none of the list's names all of it, or nothing)
      for (long long j = me; j < min(count, A.free_cap); j += ALL) A.free_out[j] = A.free_ids[j];
    if (A.table_out != A.table)
      for (long long e = me; e < A.entries; e += ALL) A.table_out[e] = A.table[e];
    if (me == 0) *A.copy_count = 0;
    return;
  }
  const int H = limit < num ? F.below(limit) : sum, M = used - (limit - H);  // free places below the limit; blocks that move
  for (long long bb = me; bb < num; bb += ALL) {
    const int b = (int)bb, k = F.below(b);
    const bool gone = F.has(b);
    // the free list afterwards, in descending order: all from the limit on, then what is left below it
    if (b >= limit) {
      A.free_out[num - 1 - b] = b;
      if (!gone) {
        const int m = b - limit - (k - H), to = F.nth(m), r = A.refs[b];
        A.copy_src[m] = b;
        A.copy_dst[m] = to;
        A.refs_out[to] = r;  // (nobody else writes a place that is taken)
      }
      A.refs_out[b] = 0;
    } else if (!gone) {
      if (A.refs_out != A.refs) A.refs_out[b] = A.refs[b];
    } else if (k >= M) {
      A.free_out[num - limit + H - 1 - k] = b;
      A.refs_out[b] = 0;
    }
  }
  // table entries after the move; one that names a free block names none
  for (long long e = me; e < A.entries; e += ALL) {
    int id = A.table[e];
    if (id >= 0 && id < num) {
      if (F.has(id)) id = -1;
      else if (id >= limit) id = F.nth(id - limit - (F.below(id) - H));
    }
    A.table_out[e] = id;
  }
  if (me == 0) *A.copy_count = M;
}

}  // namespace

cudaError_t launch_pages_free(int32_t *table, int num_seqs, int max_blocks, int block_size, int num_blocks, int32_t *refs,
                              const int32_t *seqs, const int64_t *keep_lo, const int64_t *keep_hi, int n,
                              int32_t *free_ids, int32_t *free_count, int free_cap, unsigned *status, cudaStream_t st) {
  const FreeArgs A{table, num_seqs, max_blocks, block_size, num_blocks, refs, seqs, keep_lo, keep_hi, n, free_ids,
                   free_count, free_cap, status};
  const long long warps = (long long)n * ((max_blocks + 31) / 32), ctas = (warps + SH_WARPS - 1) / SH_WARPS;
  if (ctas <= SH_SMALL && num_blocks <= SH_SMALL * SH_THREADS)
    return launch_pdl(pages_free_one_kernel, dim3(1), dim3(SH_THREADS), 0, st, A);
  // many entries: spread over the GPU by a launch of their own first
  if (ctas <= 4 * SH_CTAS) return launch_pdl(pages_free_kernel<true>, dim3(SH_CTAS), dim3(SH_THREADS), 0, st, A);
  const long long most = 2LL * num_sms();
  cudaError_t e = launch_pdl(pages_drop_kernel, dim3((unsigned)(ctas < most ? ctas : most)), dim3(SH_THREADS), 0, st, A);
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_free_kernel<false>, dim3(SH_CTAS), dim3(SH_THREADS), 0, st, A);
}

cudaError_t launch_pages_fork(int32_t *table, int num_seqs, int max_blocks, int block_size, int num_blocks, int32_t *refs,
                              const int32_t *src_seqs, const int32_t *dst_seqs, const int64_t *lens, int n,
                              const int32_t *free_ids, const int32_t *count_in, int32_t *count_out, int free_cap,
                              int32_t *copy_src, int32_t *copy_dst, int32_t *copy_count, unsigned *status,
                              cudaStream_t st) {
  const ForkArgs A{table, num_seqs, max_blocks, block_size, num_blocks, refs, src_seqs, dst_seqs, lens, n, free_ids,
                   count_in, count_out, free_cap, copy_src, copy_dst, copy_count, status};
  if ((long long)n * ((max_blocks + 31) / 32) <= SH_SMALL * SH_WARPS)
    return launch_pdl(pages_fork_one_kernel, dim3(1), dim3(SH_THREADS), sizeof(int32_t) * (size_t)n, st, A);
  return launch_pdl(pages_fork_kernel, dim3(SH_CTAS), dim3(SH_THREADS), sizeof(int32_t) * (size_t)n, st, A);
}

cudaError_t launch_pages_compact(const int32_t *table, int32_t *table_out, long long entries, int num_blocks, int limit,
                                 const int32_t *refs, int32_t *refs_out, const int32_t *free_ids,
                                 const int32_t *free_count, int32_t *free_out, int free_cap, int32_t *copy_src,
                                 int32_t *copy_dst, int32_t *copy_count, unsigned *status, cudaStream_t st) {
  const CompactArgs A{table, table_out, entries, num_blocks, limit, refs, refs_out, free_ids, free_count, free_out,
                      free_cap, copy_src, copy_dst, copy_count, status};
  auto bytes = [](int blocks) {
    const size_t groups = ((size_t)blocks + 1023) / 1024;
    return groups * 32 * 6 + (groups + 1) * 4;
  };
  cudaError_t e = ensure_smem_limit(23, (const void *)pages_compact_kernel, (int)bytes(COMPACT_MAX_BLOCKS));
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_compact_kernel, dim3(SH_CTAS), dim3(SH_THREADS), bytes(num_blocks), st, A);
}

}  // namespace kvr
