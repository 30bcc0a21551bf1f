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

#include "chunks.cuh"
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

}  // namespace kvr
