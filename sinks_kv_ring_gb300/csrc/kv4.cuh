// kv4.cuh -- the 4-bit form of the Full pool: the tile format, its device
// view and the quantiser.
//
// One group is 64 dims of one token's K (three groups; group 0 holds the
// rotary dims) or V (two groups).  A group's values are m + s * u with codes
// u in 0..15: m is its least value rounded down to fp16, s the fp16 step
// rounded up, so m + 15 s reaches its greatest value and no value inside
// fp16's range is off by more than s / 2.  fp16 keeps three bits more of m
// and s than bf16 would; values past +-65504 saturate.
//
// Sixteen consecutive positions of one KV head form a tile of KV4_TILE bytes,
// contiguous in memory, so one bulk copy brings codes and scales together.
// Inside it the bytes lie in the order in which the lanes of a warp feed the
// m16n8k16 products: lane 4a + t of a K load holds positions a and a + 8 and
// dims 16t..16t+15 of a group, lane 4a + t of a V load dims 8a..8a+7 of
// positions 2t, 2t+1, 2t+8 and 2t+9, each one 16-byte read without a bank
// conflict.  A V code pair of two neighbouring positions shares a 32-bit
// word, one position in each half, so a mask leaves the two halves of an MMA
// operand in place.  No byte belongs to two positions: tokens of one position
// are written without reading what lies beside them.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace kvr {

constexpr int KV4_GROUP = 64;                   // dims of one scale
constexpr int KV4_KG = DQK / KV4_GROUP;         // 3 groups of K
constexpr int KV4_VG = DV / KV4_GROUP;          // 2 groups of V
constexpr int KV4_OFF_V = 16 * DQK / 2;         // 1536: V codes
constexpr int KV4_OFF_KS = KV4_OFF_V + 16 * DV / 2;      // 2560: K scales   [3][16] fp16
constexpr int KV4_OFF_VS = KV4_OFF_KS + 16 * KV4_KG * 2; // 2656: V scales   [2][16] fp16
constexpr int KV4_OFF_VM = KV4_OFF_VS + 16 * KV4_VG * 2; // 2720: V minima   [2][16] fp16
constexpr int KV4_OFF_KM = KV4_OFF_VM + 16 * KV4_VG * 2; // 2784: K minima   [16][3 + a zero] fp16
constexpr int KV4_TILE = KV4_OFF_KM + 16 * 8;            // 2912
static_assert(KV4_TILE == 2912 && KV4_TILE % 32 == 0, "tile size of the pool format");

// Index of position r (0..15) within a [16] row of scales: the four
// positions 2t, 2t+1, 2t+8, 2t+9 of lane t lie together.
__host__ __device__ constexpr int kv4_quad(int r) { return ((r >> 1) & 3) * 4 + (r >> 3) * 2 + (r & 1); }
// Byte of the tile where the 16 dims 16t..16t+15 of K group g of position r start (8 bytes).
__host__ __device__ constexpr int kv4_k_at(int g, int r, int t) {
  return g * 512 + ((r & 7) * 4 + t) * 16 + (r >> 3) * 8;
}
// Byte where dims 8a + 4w .. +3 of V group g of position r lie (2 bytes).
__host__ __device__ constexpr int kv4_v_at(int g, int r, int a, int w) {
  return KV4_OFF_V + g * 512 + (a * 4 + ((r >> 1) & 3)) * 16 + (r >> 3) * 8 + w * 4 + (r & 1) * 2;
}

// Device view of a 4-bit pool (see kvr_kv4_layout).
struct Kv4View {
  uint8_t *data;
  const int32_t *block_table;
  int hkv;
  int num_seqs;
  int max_blocks;
  int block_size;
  int num_blocks;
};

// First byte of the tile of position p % block_size (a multiple of 16 or not)
// in block blk, KV head h.
__device__ __forceinline__ long long kv4_tile(const Kv4View &P, int blk, int h, int row) {
  return (((long long)blk * P.hkv + h) * (P.block_size >> 4) + (row >> 4)) * KV4_TILE;
}

__device__ __forceinline__ uint32_t h2_as_u32(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
__device__ __forceinline__ __half2 u32_as_h2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }

}  // namespace kvr
