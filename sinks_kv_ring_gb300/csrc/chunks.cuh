// chunks.cuh -- calls over batches of chunks of rows (the 8-bit append, the unpacks of
// both quantised pools): which chunk a unit of the call's work belongs to, and whether
// the chunks are in order.
#pragma once

#include "common.cuh"

namespace kvr {

// Chunk i of a call over n chunks: its rows [c0, c1), its first position and its
// sequence.
struct Chunk {
  int i, c0, c1, seq;
  long long pos;
};
// Units of a call over chunks: chunk i owns units cu[i] / 16 + 2i onwards (rows [cu[i],
// cu[i+1]) touch at most rows / 16 + 2 tiles), or, a unit a row, units cu[i] onwards
// (rows touch no more tiles than there are rows).
struct ChunkUnits {
  int shift, each;
  __host__ __device__ __forceinline__ long long first(int cu, int i) const { return (cu >> shift) + (long long)each * i; }
};
constexpr ChunkUnits CHUNKS_BY_TILE{4, 2}, CHUNKS_BY_ROW{0, 0};
// Whether a chunk's rows are out of order, or not among the call's T.
__device__ __forceinline__ bool rows_odd(int c0, int c1, long long T) { return c0 < 0 || c1 < c0 || c1 > T; }
// Flags such chunks of a call.  The units may leave one out (no unit is its own, or the search
// passes it by), so each is looked at once: by threads `me` of `all` of each of `ctas` CTAs.
__device__ __forceinline__ void rows_check(const int32_t *__restrict__ cu, int n, long long T, unsigned cta, unsigned ctas,
                                           unsigned me, unsigned all, unsigned *status) {
  for (long long i = (long long)cta * all + me; i < n; i += (long long)ctas * all)
    if (rows_odd(cu[i], cu[i + 1], T)) flag(status, ST_BAD_ROWS);
}
// Whether unit `unit` lies behind all chunks, by a warp: none of the last 64 ends past it (so up to 64 chunks it holds of all of
// them, in order or not).
__device__ __forceinline__ bool behind_chunks(const int32_t *__restrict__ cu, int n, ChunkUnits units, long long unit) {
  const int i = max(n - (int)(threadIdx.x & 31), 1), j = max(i - 32, 1);
  return !__any_sync(0xffffffffu, units.first(cu[i], i) > unit || (n > 32 && units.first(cu[j], j) > unit));
}
constexpr int CHECK_CHUNKS = 1024;  // that a CTA looks at where CTAs do nothing else
__device__ __forceinline__ int zeros_from_below(unsigned m) { return __clz(__brev(m)); }  // (32 of none)
// The chunk that owns unit `unit`, by a warp: a search over cu_rows, and no plan is
// made first.  A round narrows the chunks down by 32; the last 64 are read whole, with
// their positions and sequences, so that a batch of up to 64 waits for one load where
// a binary search waits for one a step and then for the chunk's own.
//
// It is the one ahead of the first that begins past the unit.  So where cu_rows is out of
// order, a unit of a chunk ahead of the place finds its chunk all the same, up to 64
// chunks: all from the first to its own begin no later, and the next one does.  (Of more,
// the ones that a round looks at may lie behind the place.)
__device__ __forceinline__ Chunk chunk_of(const int32_t *__restrict__ cu, const int64_t *__restrict__ pos,
                                              const int32_t *__restrict__ seqs, int n, ChunkUnits units, long long unit) {
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;  // the chunk is in [lo, lo + len)
  while (len > 64) {
    const int step = (len + 31) >> 5, i = lo + lane * step;
    const bool in = lane * step < len;
    const unsigned m = __ballot_sync(full, !(in && units.first(in ? cu[i] : 0, i) <= unit));
    const int last = max(zeros_from_below(m), 1) - 1;  // (chunk 0 always counts)
    len = min(step, len - last * step);
    lo += last * step;
  }
  const int ia = lo + lane, ib = ia + 32, ie = lo + len;
  const bool in_a = ia < ie, in_b = ib < ie;
  const int ca = in_a ? cu[ia] : 0, cb = in_b ? cu[ib] : 0, ce = cu[ie];
  const long long pa = in_a ? pos[ia] : 0, pb = in_b ? pos[ib] : 0;
  const int sa = in_a ? seqs[ia] : 0, sb = in_b ? seqs[ib] : 0;
  const unsigned ma = __ballot_sync(full, !(in_a && units.first(ca, ia) <= unit));
  const unsigned mb = __ballot_sync(full, !(in_b && units.first(cb, ib) <= unit));
  const int at = max(ma ? zeros_from_below(ma) : 32 + zeros_from_below(mb), 1) - 1, l = at & 31, l1 = (at + 1) & 31;
  const int n_a = __shfl_sync(full, ca, l1), n_b = __shfl_sync(full, cb, l1);
  Chunk C;
  C.i = lo + at;
  C.c0 = __shfl_sync(full, at < 32 ? ca : cb, l);
  C.c1 = at + 1 == len ? ce : at + 1 < 32 ? n_a : n_b;
  C.pos = __shfl_sync(full, at < 32 ? pa : pb, l);
  C.seq = __shfl_sync(full, at < 32 ? sa : sb, l);
  return C;
}

}  // namespace kvr
