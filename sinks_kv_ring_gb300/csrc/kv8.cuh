// kv8.cuh -- the 8-bit form of the Full pool: the tile format and its device
// view.
//
// Sixteen consecutive positions of one KV head form a tile: signed codes u in
// -127..127 (stored as u + 128) with one scale for the tile's K and one for its
// V, value = s u.  The scale is the least bf16 number s with 127 s >= |x| for
// every value of the tile, so u s is exact in fp32, no value is off by more than
// s / 2, and quotients that lie half way between two codes are seen as such.
//
// Positions are appended in order.  A position that asks for a larger scale
// makes the tile's scale grow: the codes there become rint(u s_old / s_new),
// another half step at most.  Rows behind the last appended one mean nothing.
//
// A tile is contiguous, so one bulk copy brings codes and scales together, and
// its bytes lie in the order in which the lanes of a warp feed the m16n8k16
// products: lane 4a + t of a K load holds dims 16t..16t+15 of a group of 64 of
// position a (or a + 8), lane 4a + t of a V load dims 4a..4a+3 of a group of 32
// of positions 2t, 2t+1, 2t+8 and 2t+9, each one 16-byte read without a bank
// conflict.  A row (K or V of one position) that is not finite has its codes at
// zero and a bit in a mask; it reads as NaN.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace kvr {

constexpr int KV8_OFF_V = 16 * DQK;                // V codes [4][8][4][4 dims][2][2]
constexpr int KV8_OFF_TAIL = KV8_OFF_V + 16 * DV;  // 5120: K scale, V scale (fp32), K mask, V mask (16 bits), a zero word
constexpr int KV8_TILE = KV8_OFF_TAIL + 16;        // 5136
static_assert(KV8_TILE == 5136, "tile size of the pool format");

// Device view of an 8-bit pool (see kvr_kv8_layout).
struct Kv8View {
  uint8_t *data;
  const int32_t *block_table;
  int hkv;
  int num_seqs;
  int max_blocks;
  int block_size;
  int num_blocks;
};

// First byte of the tile of row `row` of block blk, KV head h.
__device__ __forceinline__ long long kv8_tile(const Kv8View &P, int blk, int h, int row) {
  return (((long long)blk * P.hkv + h) * (P.block_size >> 4) + (row >> 4)) * KV8_TILE;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
__device__ __forceinline__ __half2 bits_half2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }

// The codes in the low (HI = 0) or high two bytes of w as a pair of fp16
// numbers: byte b under the high byte 0x64 is 1024 + b, less 1152 it is u
// (exact): two instructions a pair.
template <int HI>
__device__ __forceinline__ uint32_t kv8_pair(uint32_t w) {
  const uint32_t x = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140);
  return half2_bits(__hadd2(bits_half2(x), bits_half2(0xe480e480u)));
}

// Chunk i of a call over n chunks: its rows [c0, c1), its first position and its
// sequence.
struct Kv8Chunk {
  int i, c0, c1, seq;
  long long pos;
};
// Units of a call over chunks: chunk i owns units cu[i] / 16 + 2i onwards (rows [cu[i],
// cu[i+1]) touch at most rows / 16 + 2 tiles), or, a unit a row, units cu[i] onwards
// (rows touch no more tiles than there are rows).
struct Kv8Units {
  int shift, each;
  __host__ __device__ __forceinline__ long long first(int cu, int i) const { return (cu >> shift) + (long long)each * i; }
};
constexpr Kv8Units KV8_BY_TILE{4, 2}, KV8_BY_ROW{0, 0};
// Whether a chunk's rows are out of order, or not among the call's T.
__device__ __forceinline__ bool kv8_rows_odd(int c0, int c1, long long T) { return c0 < 0 || c1 < c0 || c1 > T; }
// Flags such chunks of a call.  The units may leave one out (no unit is its own, or the search
// passes it by), so each is looked at by one thread of the grid: thread `me` of a CTA's `all`.
__device__ __forceinline__ void kv8_rows_check(const int32_t *__restrict__ cu, int n, long long T, unsigned me, unsigned all,
                                               unsigned *status) {
  for (long long i = (long long)blockIdx.x * all + me; i < n; i += (long long)gridDim.x * all)
    if (kv8_rows_odd(cu[i], cu[i + 1], T)) flag(status, ST_BAD_ROWS);
}
__device__ __forceinline__ int ones_from_below(unsigned m) { return __clz(__brev(~m)); }
// The chunk that owns unit `unit`, by a warp: a search over cu_rows, and no plan is
// made first.  A round narrows the chunks down by 32; the last 64 are read whole, with
// their positions and sequences, so that a batch of up to 64 waits for one load where
// a binary search waits for one a step and then for the chunk's own.
//
// It is the one ahead of the first that begins past the unit.  So where cu_rows is out of
// order, a unit of a chunk ahead of the place finds its chunk all the same, up to 64
// chunks: all from the first to its own begin no later, and the next one does.  (Of more,
// the ones that a round looks at may lie behind the place.)
__device__ __forceinline__ Kv8Chunk kv8_chunk(const int32_t *__restrict__ cu, const int64_t *__restrict__ pos,
                                              const int32_t *__restrict__ seqs, int n, Kv8Units units, long long unit) {
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;  // the chunk is in [lo, lo + len)
  while (len > 64) {
    const int step = (len + 31) >> 5, i = lo + lane * step;
    const bool in = lane * step < len;
    const unsigned m = __ballot_sync(full, in && units.first(in ? cu[i] : 0, i) <= unit);
    const int last = max(ones_from_below(m), 1) - 1;  // (chunk 0 always counts)
    len = min(step, len - last * step);
    lo += last * step;
  }
  const int ia = lo + lane, ib = ia + 32, ie = lo + len;
  const bool in_a = ia < ie, in_b = ib < ie;
  const int ca = in_a ? cu[ia] : 0, cb = in_b ? cu[ib] : 0, ce = cu[ie];
  const long long pa = in_a ? pos[ia] : 0, pb = in_b ? pos[ib] : 0;
  const int sa = in_a ? seqs[ia] : 0, sb = in_b ? seqs[ib] : 0;
  const unsigned ma = __ballot_sync(full, in_a && units.first(ca, ia) <= unit);
  const unsigned mb = __ballot_sync(full, in_b && units.first(cb, ib) <= unit);
  const int at = max(ma == full ? 32 + ones_from_below(mb) : ones_from_below(ma), 1) - 1, l = at & 31, l1 = (at + 1) & 31;
  const int n_a = __shfl_sync(full, ca, l1), n_b = __shfl_sync(full, cb, l1);
  Kv8Chunk C;
  C.i = lo + at;
  C.c0 = __shfl_sync(full, at < 32 ? ca : cb, l);
  C.c1 = at + 1 == len ? ce : at + 1 < 32 ? n_a : n_b;
  C.pos = __shfl_sync(full, at < 32 ? pa : pb, l);
  C.seq = __shfl_sync(full, at < 32 ? sa : sb, l);
  return C;
}

}  // namespace kvr
