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
// Each call is one cluster of SH_CTAS CTAs (the table entries that a call reads
// may be spread over more of them first): the steps of a call wait for one
// another, and a cluster's barrier is cheaper than a launch.
#include <cooperative_groups.h>

#include "launch.h"

namespace kvr {
namespace {

constexpr int SH_CTAS = 8;
constexpr int SH_THREADS = 1024;
constexpr int SH_ALL = SH_CTAS * SH_THREADS;
constexpr int SH_WARPS = SH_THREADS / 32;
constexpr unsigned FULLW = 0xffffffffu;

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
  int before = 0, all = s_sum[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(FULLW, all, o);
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  total = all;
  return before + y - x;
}

// Sums of two counts of every CTA ahead of this one in the cluster, and of all of them.
struct Two {
  int a, b;
};
__device__ __forceinline__ void cluster_prefix(int a, int b, Two &before, Two &all) {
  __shared__ Two s_mine;
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  cl.sync();  // the counts of the call before are read
  if (threadIdx.x == 0) s_mine = Two{a, b};
  cl.sync();
  before = all = Two{0, 0};
  for (int r = 0; r < SH_CTAS; ++r) {
    const Two x = *cl.map_shared_rank(&s_mine, r);
    if (r < (int)cl.block_rank()) {
      before.a += x.a;
      before.b += x.b;
    }
    all.a += x.a;
    all.b += x.b;
  }
  cl.sync();  // (no CTA leaves while another reads its count)
}

// This CTA's blocks: [lo, hi) of num_blocks, in the cluster's order.
__device__ __forceinline__ void my_blocks(int num_blocks, int &lo, int &hi) {
  const int rank = (int)cooperative_groups::this_cluster().block_rank();
  const int each = (num_blocks + SH_CTAS - 1) / SH_CTAS;
  lo = (int)min((long long)rank * each, (long long)num_blocks);
  hi = (int)min((long long)lo + each, (long long)num_blocks);
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

template <bool DROP>
__global__ void __cluster_dims__(SH_CTAS, 1, 1) __launch_bounds__(SH_THREADS) pages_free_kernel(FreeArgs A) {
  pdl_wait();
  pdl_trigger();
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  const int tid = threadIdx.x;
  if (DROP) {
    drop_entries(A, (long long)cl.block_rank() * SH_THREADS + tid, SH_ALL);
    __threadfence();
    cl.sync();
  }
  // blocks without a holder: counted, then listed in order
  int lo, hi;
  my_blocks(A.num_blocks, lo, hi);
  int mine = 0;
  for (int b0 = lo; b0 < hi; b0 += SH_THREADS) mine += __syncthreads_count(b0 + tid < hi && __ldcg(A.refs + b0 + tid) < 0);
  const int count = *A.free_count;
  Two before, all;
  cluster_prefix(mine, 0, before, all);  // (every CTA has read the count)
  if (all.a == 0) return;
  if (count < 0 || (long long)count + all.a > A.free_cap) {
    if (cl.block_rank() == 0 && tid == 0) flag(A.status, ST_FREE_FULL);
    return;
  }
  int at = count + before.a;
  for (int b0 = lo; b0 < hi; b0 += SH_THREADS) {
    const bool dead = b0 + tid < hi && __ldcg(A.refs + b0 + tid) < 0;
    int total;
    const int k = cta_prefix(dead ? 1 : 0, total);
    if (dead) {
      A.free_ids[at + k] = b0 + tid;
      A.refs[b0 + tid] = 0;
    }
    at += total;
  }
  if (cl.block_rank() == 0 && tid == 0) *A.free_count = count + all.a;
}

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

__global__ void __cluster_dims__(SH_CTAS, 1, 1) __launch_bounds__(SH_THREADS) pages_fork_kernel(ForkArgs A) {
  extern __shared__ int32_t s_tail[];  // [n] entry i's new block: its number in the call, or -1 (none) or -2 (not served)
  pdl_wait();
  pdl_trigger();
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, rank = (int)cl.block_rank();
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
    const int k = cta_prefix(code == 0, total);
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
    for (int i = rank * SH_WARPS + (tid >> 5); i < A.n; i += SH_CTAS * SH_WARPS) {  // a warp an entry
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
  cl.sync();  // every CTA has read the free count
  if (rank == 0 && tid == 0) {
    *A.copy_count = none ? 0 : need;
    *A.count_out = none ? count : count - need;
  }
}

struct CompactArgs {
  int num_blocks, limit;
  const int32_t *refs;
  int32_t *refs_out;
  const int32_t *free_ids, *free_count;
  int32_t *free_out;
  int free_cap;
  int32_t *copy_src, *copy_dst, *copy_count;
  int32_t *map;  // [num_blocks]: a block's id afterwards, -1 where it is free
  unsigned *status;
};

__global__ void __cluster_dims__(SH_CTAS, 1, 1) __launch_bounds__(SH_THREADS) pages_compact_kernel(CompactArgs A) {
  pdl_wait();
  pdl_trigger();
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  const int tid = threadIdx.x, rank = (int)cl.block_rank(), me = rank * SH_THREADS + tid, num = A.num_blocks;
  const int count = *A.free_count;
  const bool sane = count >= 0 && count <= A.free_cap && count <= num;
  for (long long b = me; b < num; b += SH_ALL) A.map[b] = (int)b;
  __threadfence();
  cl.sync();
  if (sane)
    for (int j = me; j < count; j += SH_ALL) {
      const int id = A.free_ids[j];
      if (id >= 0 && id < num) A.map[id] = -1;
    }
  __threadfence();
  cl.sync();
  int lo, hi;
  my_blocks(num, lo, hi);
  int mine = 0;
  for (int b0 = lo; b0 < hi; b0 += SH_THREADS) mine += __syncthreads_count(b0 + tid < hi && __ldcg(A.map + b0 + tid) < 0);
  Two before, all;
  cluster_prefix(mine, 0, before, all);
  const int used = num - all.a, limit = A.limit > 0 ? min(A.limit, num) : used;
  // a free list that names a block twice or none of the pool's, or a limit below what is used: nothing moves
  const bool wrong = !sane || all.a != count, low = !wrong && limit < used, none = wrong || low;
  if (me == 0 && none) flag(A.status, wrong ? ST_BAD_BLOCK : ST_NO_BLOCKS);
  // holes below the limit, and used blocks at or past it, in order: the k-th of these goes to the k-th hole
  int holes = 0, movers = 0;
  for (int b0 = lo; b0 < hi; b0 += SH_THREADS) {
    const int b = b0 + tid;
    const bool gone = b < hi && __ldcg(A.map + b) < 0;
    holes += __syncthreads_count(b < hi && gone && b < limit);
    movers += __syncthreads_count(b < hi && !gone && b >= limit);
  }
  cluster_prefix(holes, movers, before, all);
  const int M = none ? 0 : all.b, H = all.a;
  int ha = before.a, ma = before.b;
  for (int b0 = lo; b0 < hi; b0 += SH_THREADS) {
    const int b = b0 + tid;
    const bool gone = b < hi && __ldcg(A.map + b) < 0;
    const bool hole = b < hi && gone && b < limit, mover = b < hi && !gone && b >= limit;
    int th, tm;
    const int kh = ha + cta_prefix(hole, th), km = ma + cta_prefix(mover, tm);
    ha += th;
    ma += tm;
    if (!none) {
      if (hole && kh < M) A.copy_dst[kh] = b;
      if (mover) A.copy_src[km] = b;
      // the free list afterwards, in descending order: the lowest ids are taken first
      if (b < hi && b >= limit) A.free_out[num - 1 - b] = b;
      if (hole && kh >= M) A.free_out[num - limit + H - 1 - kh] = b;
      if (hole && kh >= M) A.refs_out[b] = 0;
      if (mover) A.map[b] = -2 - km;  // (its place is looked up when all are known)
      else if (b < hi && !gone) A.refs_out[b] = A.refs[b];
      else if (b < hi && b >= limit) A.refs_out[b] = 0;
    }
  }
  if (none) {  // as it was
    for (long long b = me; b < num; b += SH_ALL) {
      if (A.refs_out != A.refs) A.refs_out[b] = A.refs[b];
      if (A.free_out != A.free_ids && sane && b < count) A.free_out[b] = A.free_ids[b];
      A.map[b] = (int)b;
    }
  }
  __threadfence();
  cl.sync();
  for (int b = lo + tid; b < hi && M > 0; b += SH_THREADS) {
    const int x = __ldcg(A.map + b);
    if (x > -2) continue;
    const int to = __ldcg(A.copy_dst + (-2 - x));
    A.map[b] = to;
    // (the hole's own thread wrote nothing there; in place, the old word is read ahead of its zero)
    const int r = A.refs[b];
    A.refs_out[to] = r;
    A.refs_out[b] = 0;
  }
  if (me == 0) *A.copy_count = M;
}

// Table entries after the move; one that names a free block names none.
__global__ void __launch_bounds__(256)
    pages_remap_kernel(const int32_t *table, int32_t *table_out, long long entries, const int32_t *__restrict__ map, int num) {
  pdl_wait();
  pdl_trigger();
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < entries; e += step) {
    const int id = table[e];
    table_out[e] = id >= 0 && id < num ? map[id] : id;
  }
}

}  // namespace

cudaError_t launch_pages_free(int32_t *table, int num_seqs, int max_blocks, int block_size, int num_blocks, int32_t *refs,
                              const int32_t *seqs, const int64_t *keep_lo, const int64_t *keep_hi, int n,
                              int32_t *free_ids, int32_t *free_count, int free_cap, unsigned *status, cudaStream_t st) {
  const FreeArgs A{table, num_seqs, max_blocks, block_size, num_blocks, refs, seqs, keep_lo, keep_hi, n, free_ids,
                   free_count, free_cap, status};
  // many entries: spread over the GPU by a launch of their own first
  const long long warps = (long long)n * ((max_blocks + 31) / 32), ctas = (warps + SH_WARPS - 1) / SH_WARPS;
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
  return launch_pdl(pages_fork_kernel, dim3(SH_CTAS), dim3(SH_THREADS), sizeof(int32_t) * (size_t)n, st, A);
}

cudaError_t launch_pages_compact(const int32_t *table, int32_t *table_out, long long entries, int num_blocks, int limit,
                                 const int32_t *refs, int32_t *refs_out, const int32_t *free_ids,
                                 const int32_t *free_count, int32_t *free_out, int free_cap, int32_t *copy_src,
                                 int32_t *copy_dst, int32_t *copy_count, int32_t *map, unsigned *status,
                                 cudaStream_t st) {
  const CompactArgs A{num_blocks, limit, refs, refs_out, free_ids, free_count, free_out, free_cap, copy_src, copy_dst,
                      copy_count, map, status};
  cudaError_t e = launch_pdl(pages_compact_kernel, dim3(SH_CTAS), dim3(SH_THREADS), 0, st, A);
  if (e != cudaSuccess) return e;
  const long long blocks = (entries + 255) / 256, most = 8LL * num_sms();
  return launch_pdl(pages_remap_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, st, table,
                    table_out, entries, static_cast<const int32_t *>(map), num_blocks);
}

}  // namespace kvr
