// pages_grow.cu -- block tables and slot maps of a batch's next step, made on
// the GPU from the requests' lengths (the pool "grown on demand" of Xiaomi
// "Full-Pipeline Inference Optimization for MiMo-V2.5 Series", section 2.1).
//
// Request i holds len[i] positions and gains add[i].  With ceil(len / bs)
// blocks held, it needs blocks ceil(len / bs) .. ceil((len + add) / bs) - 1:
// the k-th block of the call, in (request, block) order, is the k-th id from
// the end of the free list.  A row's block is either held already (read from
// the table) or one of those ids, so no row waits for a table write and the
// whole step is one launch.
//
// Clusters of GROW_CTAS CTAs: every CTA takes the same prefix sums over the
// requests (rows and blocks) into shared memory.  The first cluster then fills
// the batch's rows and the new table entries; its barrier stands between the
// last read of the free count and its update, which may be in place.  The
// other clusters, as many as the row arrays ask for, write the -1 of the rows
// behind the last token, which depend on no count.
//
// What bounds it: 64 requests of one token take 4.5 us, the latency of a launch
// and of a chain of dependent loads (sequence id, table entry or free id).  1000
// requests of mixed lengths with 400,000 rows, 40,000 of them filled, take
// 12.5 us: the rows' searches on the first cluster's eight SMs (25 us with one
// cluster, which wrote the padding as well; 20 us with clusters of four; two to
// eight rows of a thread at a time, and 32-bit divisions, changed nothing).
#include <cooperative_groups.h>

#include "launch.h"

namespace kvr {
namespace {

constexpr int GROW_CTAS = 8;
constexpr int GROW_THREADS = 1024;
constexpr int GROW_WARPS = GROW_THREADS / 32;
constexpr unsigned FULLW = 0xffffffffu;

struct GrowArgs {
  int32_t *table;
  int num_seqs, max_blocks, block_size, num_blocks;
  const int32_t *seqs;
  const int64_t *lens;
  const int32_t *add;
  int n;
  const int32_t *free_ids;
  const int32_t *count_in;
  int32_t *count_out;
  int free_cap;
  int32_t *cu_rows;
  int64_t *pos;
  int32_t *row_seq;
  int64_t *slots;
  long long T;
};

__global__ void __cluster_dims__(GROW_CTAS, 1, 1) __launch_bounds__(GROW_THREADS)
    pages_grow_kernel(GrowArgs A, unsigned *status) {
  extern __shared__ int32_t s_mem[];
  int32_t *s_row = s_mem;               // [n + 1] first row of request i
  int32_t *s_blk = s_row + A.n + 1;     // [n + 1] first new block of request i
  __shared__ int s_warp[2][GROW_WARPS];
  __shared__ int s_base[2];
  __shared__ int s_over;                // a running total left int range or the batch does not fit
  pdl_wait();
  pdl_trigger();
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int part = (int)(blockIdx.x / GROW_CTAS), parts = (int)(gridDim.x / GROW_CTAS);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = A.block_size;
  const long long cap_pos = (long long)A.max_blocks * bs;
  if (tid == 0) {
    s_base[0] = s_base[1] = 0;
    s_over = 0;
  }
  __syncthreads();
  const int count = part == 0 ? *A.count_in : 0;

  // rows and new blocks of request i (none where it cannot be served)
  auto want = [&](int i, int &rows, int &blks) -> unsigned {
    rows = blks = 0;
    const long long len = A.lens[i];
    const int ad = A.add[i], s = A.seqs[i];
    if (s < 0 || s >= A.num_seqs) return ST_BAD_SEQ;
    if (len < 0 || ad < 0 || len > cap_pos || len + ad > cap_pos) return ST_BAD_POS;
    rows = ad;
    blks = (int)((len + ad + bs - 1) / bs - (len + bs - 1) / bs);
    return 0u;
  };

  unsigned bad = 0;
  for (int i0 = 0; i0 < A.n; i0 += GROW_THREADS) {
    const int i = i0 + tid;
    int rows = 0, blks = 0;
    if (i < A.n) bad |= want(i, rows, blks);
    int x = rows, y = blks;
    bool over = false;  // sums of at most 2^31 - 1 each stay below 2^32: a wrapped one is seen as negative
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(FULLW, x, o), b = __shfl_up_sync(FULLW, y, o);
      if (lane >= o) {
        x = (int)((unsigned)x + (unsigned)a);
        y = (int)((unsigned)y + (unsigned)b);
        over |= x < 0 || y < 0;
        if (x < 0) x = 0x7fffffff;
        if (y < 0) y = 0x7fffffff;
      }
    }
    if (lane == 31) {
      s_warp[0][warp] = x;
      s_warp[1][warp] = y;
    }
    if (over) s_over = 1;
    __syncthreads();
    long long bx = s_base[0], by = s_base[1];
    for (int w = 0; w < warp; ++w) {
      bx += s_warp[0][w];
      by += s_warp[1][w];
    }
    if (bx + x > 0x7fffffffLL || by + y > 0x7fffffffLL) s_over = 1;
    if (i < A.n) {
      s_row[i] = (int)bx + x - rows;
      s_blk[i] = (int)by + y - blks;
    }
    __syncthreads();
    if (tid == GROW_THREADS - 1) {
      s_base[0] = (int)bx + x;
      s_base[1] = (int)by + y;
    }
    __syncthreads();
  }
  const int total = s_base[0], need = s_base[1];
  if (tid == 0) {
    s_row[A.n] = total;
    s_blk[A.n] = need;
  }
  __syncthreads();
  if (part > 0) {  // rows past the last token (none when there are more tokens than rows)
    if (s_over || total >= A.T) return;
    const long long step = (long long)(parts - 1) * GROW_CTAS * GROW_THREADS;
    for (long long r = total + ((long long)(part - 1) * GROW_CTAS + rank) * GROW_THREADS + tid; r < A.T; r += step) {
      A.pos[r] = -1;
      A.row_seq[r] = -1;
      A.slots[r] = -1;
    }
    return;
  }
  const long long mine = parts > 1 && !s_over && total < A.T ? total : A.T;  // rows of this cluster
  // all or nothing: too many rows, or too few free blocks, make an empty step
  const bool rows_over = s_over || total > A.T;
  const bool short_of = !rows_over && (count < 0 || count > A.free_cap || need > count);
  const bool none = rows_over || short_of;
  if (rank == 0) {
    if (bad) flag(status, bad);
    if (tid == 0 && rows_over) flag(status, ST_BAD_ROWS);
    if (tid == 0 && short_of) flag(status, ST_NO_BLOCKS);
    for (int i = tid; i <= A.n; i += GROW_THREADS) A.cu_rows[i] = none ? 0 : s_row[i];
  }
  // the id of the call's k-th new block, -1 (flagged) when the list holds no id of the pool there
  auto new_id = [&](int k) -> int {
    const int id = A.free_ids[count - 1 - k];
    return id >= 0 && id < A.num_blocks ? id : -1;
  };
  const int stride = GROW_CTAS * GROW_THREADS, me = rank * GROW_THREADS + tid;
  if (!none) {
    // new table entries
    for (long long kk = me; kk < need; kk += stride) {
      const int k = (int)kk;
      int lo = 0, hi = A.n;  // s_blk[lo] <= k < s_blk[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_blk[mid] <= k) lo = mid; else hi = mid;
      }
      const int id = new_id(k);
      if (id < 0) flag(status, ST_BAD_BLOCK);
      const int bi = (int)((A.lens[lo] + bs - 1) / bs) + (k - s_blk[lo]);
      A.table[(long long)A.seqs[lo] * A.max_blocks + bi] = id;
    }
  }
  for (long long r = me; r < mine; r += stride) {
    long long p = -1, slot = -1;
    int s = -1;
    if (!none && r < total) {
      int lo = 0, hi = A.n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_row[mid] <= (int)r) lo = mid; else hi = mid;
      }
      const long long len = A.lens[lo];
      s = A.seqs[lo];
      p = len + (r - s_row[lo]);
      const int bi = (int)(p / bs), held = (int)((len + bs - 1) / bs);
      int id;
      if (bi < held) {
        id = A.table[(long long)s * A.max_blocks + bi];
        if (id < 0 || id >= A.num_blocks) {
          flag(status, ST_BAD_BLOCK);
          id = -1;
        }
      } else {
        id = new_id(s_blk[lo] + (bi - held));
      }
      slot = id < 0 ? -1 : (long long)id * bs + (p - (long long)bi * bs);
    }
    A.pos[r] = p;
    A.row_seq[r] = s;
    A.slots[r] = slot;
  }
  cluster.sync();  // every CTA has read the free count
  if (rank == 0 && tid == 0) *A.count_out = none ? count : count - need;
}

}  // namespace

cudaError_t launch_pages_grow(int32_t *table, int num_seqs, int max_blocks, int block_size, int num_blocks,
                              const int32_t *seqs, const int64_t *lens, const int32_t *add, int n,
                              const int32_t *free_ids, const int32_t *count_in, int32_t *count_out, int free_cap,
                              int32_t *cu_rows, int64_t *pos, int32_t *row_seq, int64_t *slots, long long T,
                              unsigned *status, cudaStream_t st) {
  const GrowArgs A{table, num_seqs, max_blocks, block_size, num_blocks, seqs, lens, add, n, free_ids, count_in,
                   count_out, free_cap, cu_rows, pos, row_seq, slots, T};
  const size_t smem = 2 * sizeof(int32_t) * ((size_t)GROW_MAX_N + 1);
  cudaError_t e = ensure_smem_limit(16, (const void *)pages_grow_kernel, (int)smem);
  if (e != cudaSuccess) return e;
  // one cluster writes 16K rows about as fast as the launch itself takes; beyond, more of them up to the GPU's SMs
  long long parts = 1 + T / 16384;
  const long long most = num_sms() / GROW_CTAS;
  if (parts > most) parts = most > 1 ? most : 1;
  return launch_pdl(pages_grow_kernel, dim3((unsigned)(GROW_CTAS * parts)), dim3(GROW_THREADS),
                    2 * sizeof(int32_t) * ((size_t)n + 1), st, A, status);
}

}  // namespace kvr
