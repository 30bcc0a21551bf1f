// kv8_append.cu -- fused KV write into an 8-bit pool: rotate-half RoPE of k
// (dims 0..63), value scale of v, quantisation with one scale per tile of 16
// positions (colibri "MiMo-V2.6", "What the engine implements": partial RoPE,
// values multiplied by attention_value_scale, as kv_ring_append_rope).
//
// For the K, and apart from it the V, of one tile and KV head, with x the new
// rows' fp32 values and s_old the tile's scale (0 where the chunk starts the
// tile):
//   s = max(s_old, least bf16 with 127 s >= max |x|),  u = rint(x / s),
//   rows ahead in the tile: u = rint(u s_old / s).
// The quotient is the correctly rounded one, so exact ties, which bf16 values over a
// bf16 scale meet often, round to even: with the reciprocal in two numbers, r + r' =
// 1/s (1 + d), |d| < 2^-47, it is RN(x r + RN(x r')), within 2^-46 of x / s ahead of
// the rounding.  A point m halfway between two fp32 numbers has 25 bits and s has 8:
// x = m s is no fp32 number (m is odd in its last place, so the product has 25 bits
// or more), and x - m s is no less than the last place of a product of 33 bits, 2^-33
// of x: what is within 2^-46 of x / s rounds as x / s does.
//
// A CTA takes one tile: two warps half of a head's K rows each, two half of its V
// dims each, with 16 bytes of codes a lane and store; two of a kind exchange their
// largest magnitudes through shared memory.  A first warp finds the tile's chunk and
// rows for all, while the others look at a part of cu_rows each CTA (rows_check).  A chunk that starts inside a tile finds the rows ahead of it there:
// their V codes share 16 bytes with the new ones and are read in any case, their K
// codes only where the scale grows.  Large calls take up to four heads of a tile
// one after the other (MANY), for one search and one look at the RoPE rows; where that
// leaves fewer than 16 CTAs an SM, two rounds, a CTA has one head (64 tokens of 4 KV
// heads: 3.0 us, by four heads 6.4; 8192: 7.5 and 8.1; 37 x 1021 of 8: 57.4 and 52.3).
//
// What bounds it: the latency of a warp's chain (rows, largest magnitude, scale,
// stores) at the 32 warps an SM that its registers leave, over the memory it moves: 37
// x 1021 tokens of 8 KV heads take 52 us, 0.82 of what their 961 bytes each take at the
// copy rate; 30 x 4096 of 4, 82 us, 0.85; 8192 tokens of 4 KV heads 7.4 us, 64 tokens
// 3.0.  The first form took 145, 17 and 7.4: quotients two to an instruction, all
// loads out before the block is looked up, and one chunk search for all took the large
// case to 80; the rotary group as pairs in one lane (no partner's loads, half the RoPE
// loads) and 32-byte loads to 63, as the requests to L1 had bound it; a tile's K by one
// warp and its V by another, 20 warps an SM of 96 registers, stood at 59.
// Measured and left out: the rows of tiles further on, or of a CTA's next heads, into
// L2 by bulk prefetches (58 for 59, and 59 for 54); V by one warp beside two for K
// (57); eight heads a CTA (52.6).
#include "kv8.cuh"
#include "launch.h"

namespace kvr {
namespace {

constexpr int K8A_WARPS = 4;  // two for a tile's K, two for its V
constexpr int K8A_CTAS = 8;   // per SM
constexpr int K8A_HEADS = 4;  // that a CTA takes one after the other, at most
constexpr unsigned FULLW = 0xffffffffu;

__device__ __forceinline__ void prefetch_line(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The least bf16 number s with 127 s >= a (a finite, >= 0): the quotient
// rounded up to bf16, one step more where fp32 rounded it down onto it.
__device__ __forceinline__ float kv8_scale(float a) {
  uint32_t b = (__float_as_uint(__fdiv_rn(a, 127.f)) + 0xffffu) & 0xffff0000u;
  if (__fmul_rn(__uint_as_float(b), 127.f) < a) b += 0x10000u;
  return __uint_as_float(b);
}

// What the quotients by a scale are made with.
struct Kv8Div {
  uint64_t r, rest;  // the reciprocal in two numbers (0 for a scale of 0), in both halves
  float f;           // `far`: of a scale so small, or large, that one of the two leaves fp32's normal numbers, they are
  bool far;          // the reciprocal of f times the scale, for values times f
};
__device__ __forceinline__ Kv8Div kv8_div(float s) {
  Kv8Div D;
  D.far = (s < 0x1p-90f || s > 0x1p60f) && s > 0.f;
  D.f = s < 1.f ? 0x1p64f : 0x1p-64f;
  if (D.far) s *= D.f;
  const float r = s > 0.f ? __frcp_rn(s) : 0.f, rest = __fmul_rn(__fmaf_rn(-s, r, 1.f), r);
  D.r = f32x2(r, r);
  D.rest = f32x2(rest, rest);
  return D;
}
// Stored codes (u + 128) of four values in two pairs: the quotients are rounded by
// adding 1.5 2^23 and the 128 (an even number: halves go to even as without it),
// which leaves them in the low bytes.
template <bool FAR>
__device__ __forceinline__ uint32_t kv8_codes(uint64_t a, uint64_t b, const Kv8Div &D) {
  const uint64_t magic = f32x2(12583040.f, 12583040.f);
  if (FAR) {
    a = mul_f32x2(a, f32x2(D.f, D.f));
    b = mul_f32x2(b, f32x2(D.f, D.f));
  }
  float x, y, z, w;
  f32x2_split(add_f32x2(fma_f32x2(a, D.r, mul_f32x2(a, D.rest)), magic), x, y);
  f32x2_split(add_f32x2(fma_f32x2(b, D.r, mul_f32x2(b, D.rest)), magic), z, w);
  return __byte_perm(__byte_perm(__float_as_uint(x), __float_as_uint(y), 0x0040),
                     __byte_perm(__float_as_uint(z), __float_as_uint(w), 0x0040), 0x5410);
}
// Stored codes under a larger scale: the values that they stand for, quantised again.
template <bool FAR>
__device__ __forceinline__ uint32_t kv8_again(uint32_t w, float s_old, const Kv8Div &D) {
  const float2 a = __half22float2(bits_half2(kv8_pair<0>(w))), b = __half22float2(bits_half2(kv8_pair<1>(w)));
  const uint64_t s = f32x2(s_old, s_old);
  return kv8_codes<FAR>(mul_f32x2(f32x2(a.x, a.y), s), mul_f32x2(f32x2(b.x, b.y), s), D);
}

__device__ __forceinline__ uint64_t bf16_f32x2(uint32_t w) {
  return f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t word4(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// 32 bytes of input, in one load where its rows are 32-byte aligned (a lane's
// quarter of a 128-byte line: half the requests).
__device__ __forceinline__ void load32(const void *p, bool wide, uint4 &a, uint4 &b) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = reinterpret_cast<const uint4 *>(p)[0];
    b = reinterpret_cast<const uint4 *>(p)[1];
  }
}
// Largest magnitudes of a packed pair of bf16, kept apart in the two halves (a NaN above all).
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) {
  asm("{.reg .b32 a; abs.bf16x2 a, %1; max.NaN.bf16x2 %0, %0, a;}" : "+r"(m) : "r"(w));
  return m;
}

struct Kv8Append {
  const uint16_t *k, *v;
  const int32_t *cu_rows;
  const int64_t *P0;
  const int32_t *seqs;
  int n;
  long long T;
  const float *table;
  int64_t max_pos;
  float vscale;
  Kv8View dst;
  unsigned *status;
  int heads, per_tile;  // heads of a CTA, CTAs of a tile
  ChunkUnits units;
};

// Where a warp's tile lies and which of its rows are new.
struct Kv8Item {
  int blk;         // its block (any number: checked before the tile is touched; not set by append_item)
  int row;         // first row of the tile in its block
  long long row0;  // k/v row of the tile's position 0 (may lie ahead of the chunk's first)
  int r0, r1;      // new rows [r0, r1); rows below r0 are there already
  long long p;     // position of the tile's row 0
};
// The tile, or null where its block is none of the pool's.
__device__ __forceinline__ uint8_t *tile_of(const Kv8Append &A, const Kv8Item &I, int h) {
  return I.blk < 0 || I.blk >= A.dst.num_blocks ? nullptr : A.dst.data + kv8_tile(A.dst, I.blk, h, I.row);
}

// A K row of a lane under the tile's scale: row r, dims 16t .. of the groups of 64 that are not rotated, and 8t .. and
// 32 + 8t .. of the rotary one.
template <bool FAR>
__device__ __forceinline__ void put_k(const uint64_t (&x0)[8], const uint4 (&raw)[2][2], bool is_new, bool again, float s_old,
                                      const Kv8Div &D, uint8_t *tile, int r, int t) {
  uint8_t *at = tile + r * 64 + 16 * t;
  if (is_new) {
    uint8_t *rot = tile + r * 64 + 8 * t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint2 *>(rot + 32 * i) =
          make_uint2(kv8_codes<FAR>(x0[4 * i], x0[4 * i + 1], D), kv8_codes<FAR>(x0[4 * i + 2], x0[4 * i + 3], D));
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // four dims each
        const uint4 &w = raw[g][j >> 1];
        c[j] = kv8_codes<FAR>(bf16_f32x2(j & 1 ? w.z : w.x), bf16_f32x2(j & 1 ? w.w : w.y), D);
      }
      *reinterpret_cast<uint4 *>(at + 1024 + 1024 * g) = make_uint4(c[0], c[1], c[2], c[3]);
    }
  } else if (again) {
    uint4 w[3];
#pragma unroll
    for (int g = 0; g < 3; ++g) w[g] = *reinterpret_cast<const uint4 *>(at + 1024 * g);
#pragma unroll
    for (int g = 0; g < 3; ++g)
      *reinterpret_cast<uint4 *>(at + 1024 * g) =
          make_uint4(kv8_again<FAR>(w[g].x, s_old, D), kv8_again<FAR>(w[g].y, s_old, D), kv8_again<FAR>(w[g].z, s_old, D),
                     kv8_again<FAR>(w[g].w, s_old, D));
  }
}

// Rows 8 half .. 8 half + 7 of the tile's K for heads h0 .. h1 - 1, by one of two warps.
template <bool MANY>
__device__ __forceinline__ void kv8_append_k(const Kv8Append &A, const Kv8Item &I, int h0, int h1, int half, int lane) {
  __shared__ uint32_t s_top[2][2];  // of a head, and of the next one
  const int t = lane & 3, gr = lane >> 2, r = gr + 8 * half, H = A.dst.hkv;
  const bool wide = (reinterpret_cast<uintptr_t>(A.k) & 31u) == 0, wide_t = (reinterpret_cast<uintptr_t>(A.table) & 31u) == 0;
  const bool is_new = r >= I.r0 && r < I.r1;
  // the row's cosines and sines, of all heads: kept by each thread for itself
  __shared__ uint4 s_cs[MANY ? 4 : 1][64];
  uint4 cs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = make_uint4(0, 0, 0, 0);
  if (is_new) {
    const float *tr = A.table + (I.p + r) * 64 + 16 * t;
#pragma unroll
    for (int i = 0; i < 2; ++i) load32(tr + 8 * i, wide_t, cs[2 * i], cs[2 * i + 1]);
  }
  if (MANY) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s_cs[i][32 * half + lane] = cs[i];
  }
  for (int h = h0; h < (MANY ? h1 : h0 + 1); ++h) {
    uint4 raw[2][2];  // dims 16t .. 16t + 15 of the groups of 64 that are not rotated
    uint64_t x0[8];   // dims 8t .. and 32 + 8t .. of the rotary one, in pairs
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i >> 1][i & 1] = make_uint4(0, 0, 0, 0);
    if (is_new) {
      const uint16_t *src = A.k + ((I.row0 + r) * H + h) * DQK;
      a = *reinterpret_cast<const uint4 *>(src + 8 * t);
      b = *reinterpret_cast<const uint4 *>(src + 32 + 8 * t);
#pragma unroll
      for (int i = 0; i < 2; ++i) load32(src + 64 + 64 * i + 16 * t, wide, raw[i][0], raw[i][1]);
    }
    uint8_t *const tile = tile_of(A, I, h);
    if (!tile) return;  // (both warps)
    uint4 tail = make_uint4(0, 0, 0, 0);
    if (I.r0 > 0) {
      tail = *reinterpret_cast<const uint4 *>(tile + KV8_OFF_TAIL);
      // (K rows ahead in the tile, in case the scale grows)
      if (lane < 12) prefetch_line(tile + 512 * half + 1024 * (lane >> 2) + 128 * (lane & 3));
    }
    // the rotary group: products and sums rounded one by one, so the result does not hang on contraction
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // two pairs (d, d + 32)
      float x[2], y[2];
      const uint4 w = MANY ? s_cs[MANY ? i : 0][32 * half + lane] : cs[i];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t wa = word4(a, i), wb = word4(b, i);
        const float va = __uint_as_float(u ? wa & 0xffff0000u : wa << 16);
        const float vb = __uint_as_float(u ? wb & 0xffff0000u : wb << 16);
        const float c = __uint_as_float(u ? w.z : w.x), sn = __uint_as_float(u ? w.w : w.y);
        x[u] = __fsub_rn(__fmul_rn(va, c), __fmul_rn(vb, sn));
        y[u] = __fadd_rn(__fmul_rn(vb, c), __fmul_rn(va, sn));
      }
      x0[i] = f32x2(x[0], x[1]);
      x0[4 + i] = f32x2(y[0], y[1]);
    }
    // the row's largest magnitude (as bits: infinities and NaN above all), the rows that are not finite, the tile's largest
    uint32_t bad = 0, m2 = 0, m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 &w = raw[i >> 1][i & 1];
      m2 = abs_max2(abs_max2(abs_max2(abs_max2(m2, w.x), w.y), w.z), w.w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x, y;
      f32x2_split(x0[i], x, y);
      m = max(max(m, __float_as_uint(x) & 0x7fffffffu), __float_as_uint(y) & 0x7fffffffu);
    }
    m = max(m, max(m2 << 16, m2 & 0xffff0000u));
    m = max(m, __shfl_xor_sync(FULLW, m, 1));
    m = max(m, __shfl_xor_sync(FULLW, m, 2));
    const bool odd = m >= 0x7f800000u;
    const unsigned rows = __ballot_sync(FULLW, odd && t == 0);  // bit 4 gr
    if (rows) {
#pragma unroll
      for (int i = 0; i < 8; ++i) bad |= (rows >> (4 * i) & 1u) << i;
      if (odd) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) x0[i] = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) raw[g][0] = raw[g][1] = make_uint4(0, 0, 0, 0);
      }
    }
    m = __reduce_max_sync(FULLW, m);
    uint32_t *top = s_top[(h - h0) & 1];
    if (lane == 0) top[half] = m;
    __syncwarp();
    asm volatile("bar.sync 1, 64;" ::: "memory");  // (both warps have the tail, too)
    const float s_old = __uint_as_float(tail.x), s_need = kv8_scale(__uint_as_float(max(top[0], top[1])));
    const bool grow = I.r0 > 0 && s_need > s_old;
    const float s = I.r0 > 0 && !grow ? s_old : s_need;
    const Kv8Div D = kv8_div(s);
    if (D.far) put_k<true>(x0, raw, is_new, grow && r < I.r0, s_old, D, tile, r, t);
    else put_k<false>(x0, raw, is_new, grow && r < I.r0, s_old, D, tile, r, t);
    if (lane == 0) {
      tile[KV8_OFF_TAIL + 8 + half] = (uint8_t)((tail.z & ((1u << I.r0) - 1u)) >> (8 * half) | bad);
      if (half == 0) {
        *reinterpret_cast<float *>(tile + KV8_OFF_TAIL) = s;
        *reinterpret_cast<uint32_t *>(tile + KV8_OFF_TAIL + 12) = 0u;
      }
    }
  }
}

// V of a lane under its scale: positions 2t, 2t + 1, 2t + 8, 2t + 9, dims 4 gr .. of each of its two groups of 32 (`to`: its
// codes of the first).
template <bool FAR>
__device__ __forceinline__ void put_v(const uint2 (&raw)[4][2], const uint4 (&old)[2], float vscale, bool grow, float s_old,
                                      const Kv8Div &D, const Kv8Item &I, uint8_t *to, int t) {
  const uint64_t vs = f32x2(vscale, vscale);
  uint32_t keep = 0;  // bytes of positions that are there already
#pragma unroll
  for (int j = 0; j < 4; ++j) keep |= 2 * t + (j & 1) + 8 * (j >> 1) < I.r0 ? 0xffu << (8 * j) : 0u;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t c[4];  // of position j: four dims
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = kv8_codes<FAR>(mul_f32x2(bf16_f32x2(raw[j][g].x), vs), mul_f32x2(bf16_f32x2(raw[j][g].y), vs), D);
    // to a word per dim: positions in its bytes
    uint32_t w[4];
    const uint32_t a = __byte_perm(c[0], c[1], 0x5140), b = __byte_perm(c[2], c[3], 0x5140);  // dims 0, 1 of both
    const uint32_t e = __byte_perm(c[0], c[1], 0x7362), f = __byte_perm(c[2], c[3], 0x7362);  // dims 2, 3
    w[0] = __byte_perm(a, b, 0x5410);
    w[1] = __byte_perm(a, b, 0x7632);
    w[2] = __byte_perm(e, f, 0x5410);
    w[3] = __byte_perm(e, f, 0x7632);
    if (I.r0 > 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o = word4(old[g], i);
        if (grow) o = kv8_again<FAR>(o, s_old, D);
        w[i] = (o & keep) | (w[i] & ~keep);
      }
    }
    *reinterpret_cast<uint4 *>(to + 512 * g) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Groups 2 half and 2 half + 1 of the tile's V for heads h0 .. h1 - 1, by one of two warps.
template <bool MANY>
__device__ __forceinline__ void kv8_append_v(const Kv8Append &A, const Kv8Item &I, int h0, int h1, int half, int lane) {
  __shared__ uint4 s_max[2][2][4];  // of a head, and of the next one
  const int t = lane & 3, gr = lane >> 2, H = A.dst.hkv;
  for (int h = h0; h < (MANY ? h1 : h0 + 1); ++h) {
    // positions 2t, 2t + 1, 2t + 8, 2t + 9 (j), dims 4 gr .. 4 gr + 3 of each group of 32
    uint2 raw[4][2];
    uint4 old[2];
    bool is_new[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 2 * t + (j & 1) + 8 * (j >> 1);
      is_new[j] = r >= I.r0 && r < I.r1;
      const uint16_t *src = A.v + ((I.row0 + r) * H + h) * DV + 64 * half + 4 * gr;
#pragma unroll
      for (int g = 0; g < 2; ++g) raw[j][g] = is_new[j] ? *reinterpret_cast<const uint2 *>(src + 32 * g) : make_uint2(0, 0);
    }
    uint8_t *const tile = tile_of(A, I, h);
    if (!tile) return;  // (both warps)
    uint8_t *const to = tile + KV8_OFF_V + 1024 * half + 16 * lane;
    uint4 tail = make_uint4(0, 0, 0, 0);
    if (I.r0 > 0) {
      tail = *reinterpret_cast<const uint4 *>(tile + KV8_OFF_TAIL);
#pragma unroll
      for (int g = 0; g < 2; ++g) old[g] = *reinterpret_cast<const uint4 *>(to + 512 * g);
    }
    uint32_t mx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t m2 = 0;
#pragma unroll
      for (int g = 0; g < 2; ++g) m2 = abs_max2(abs_max2(m2, raw[j][g].x), raw[j][g].y);
      uint32_t m = max(m2 << 16, m2 & 0xffff0000u);
      m = max(m, __shfl_xor_sync(FULLW, m, 4));
      m = max(m, __shfl_xor_sync(FULLW, m, 8));
      mx[j] = max(m, __shfl_xor_sync(FULLW, m, 16));
    }
    uint4(*mine)[4] = s_max[(h - h0) & 1];
    if (gr == 0) mine[half][t] = make_uint4(mx[0], mx[1], mx[2], mx[3]);
    __syncwarp();
    asm volatile("bar.sync 2, 64;" ::: "memory");  // (both warps have the tail, too)
    const uint4 other = mine[half ^ 1][t];
    uint32_t top = 0, bad = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t m = max(mx[j], word4(other, j));
      // the largest of the scaled values is the largest's product (a NaN stays one)
      uint32_t y = __float_as_uint(__fmul_rn(__uint_as_float(m), A.vscale)) & 0x7fffffffu;
      const bool odd = is_new[j] && y >= 0x7f800000u;
      const unsigned rows = __ballot_sync(FULLW, odd && gr == 0);  // bits t
      if (rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= (rows >> i & 1u) << (2 * i + (j & 1) + 8 * (j >> 1));
        if (odd) {
          y = 0;
          raw[j][0] = raw[j][1] = make_uint2(0, 0);
        }
      }
      top = max(top, is_new[j] ? y : 0u);
    }
    top = __reduce_max_sync(FULLW, top);
    const float s_old = __uint_as_float(tail.y), s_need = kv8_scale(__uint_as_float(top));
    const bool grow = I.r0 > 0 && s_need > s_old;
    const float s = I.r0 > 0 && !grow ? s_old : s_need;
    const Kv8Div D = kv8_div(s);
    if (D.far) put_v<true>(raw, old, A.vscale, grow, s_old, D, I, to, t);
    else put_v<false>(raw, old, A.vscale, grow, s_old, D, I, to, t);
    if (lane == 0 && half == 0) {
      *reinterpret_cast<float *>(tile + KV8_OFF_TAIL + 4) = s;
      *reinterpret_cast<uint16_t *>(tile + KV8_OFF_TAIL + 10) = (uint16_t)(((tail.z >> 16) & ((1u << I.r0) - 1u)) | bad);
    }
  }
}

// The tile of unit `unit` of the call, by a warp; false: none.
__device__ __forceinline__ bool append_item(const Kv8Append &A, long long unit, bool say, Kv8Item &I, const int32_t *&entry) {
  const Chunk C = chunk_of(A.cu_rows, A.P0, A.seqs, A.n, A.units, unit);
  const int i = C.i, c0 = C.c0, c1 = C.c1, s = C.seq;
  const long long a = C.pos;
  if (rows_odd(c0, c1, A.T)) return false;
  const long long u = unit - A.units.first(c0, i);
  if (u < 0 || c1 == c0 || s == -1) return false;
  const bool bs = s < 0 || s >= A.dst.num_seqs;
  const long long most = min((long long)A.max_pos, (long long)A.dst.max_blocks * A.dst.block_size);
  const bool bp = a < 0 || a > most - (c1 - c0);
  if (bs || bp) {
    if (say && u == 0) flag(A.status, (bs ? ST_BAD_SEQ : 0u) | (bp ? ST_BAD_POS : 0u));
    return false;
  }
  I.p = ((a >> 4) + u) << 4;
  const long long end = a + (c1 - c0);
  if (I.p >= end) return false;
  I.r0 = (int)max(a - I.p, 0LL);
  I.r1 = (int)min(end - I.p, 16LL);
  I.row0 = c0 + (I.p - a);
  const unsigned tile = (unsigned)(I.p >> 4), per_block = (unsigned)A.dst.block_size >> 4, bi = tile / per_block;
  entry = A.dst.block_table + (long long)s * A.dst.max_blocks + bi;
  I.row = (int)(16 * (tile - bi * per_block));
  return true;
}

template <bool MANY>
__global__ void __launch_bounds__(K8A_WARPS * 32, K8A_CTAS) kv8_append_kernel(Kv8Append A) {
  __shared__ Kv8Item s_item;
  __shared__ const int32_t *s_entry;  // of the block table; null: nothing to do
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const unsigned per_tile = MANY ? A.per_tile : A.dst.hkv, unit = blockIdx.x / per_tile;
  const int h0 = (int)(blockIdx.x - unit * per_tile) * (MANY ? A.heads : 1), h1 = min(h0 + A.heads, A.dst.hkv);
  const bool say = threadIdx.x == 0 && h0 == 0;
  pdl_wait();
  pdl_trigger();
  if (part == 0) {
    Kv8Item I;
    const int32_t *entry = nullptr;
    append_item(A, unit, say, I, entry);
    if (lane == 0) s_item = I, s_entry = entry;
  } else {
    rows_check(A.cu_rows, A.n, A.T, blockIdx.x, gridDim.x, threadIdx.x - 32, 32 * (K8A_WARPS - 1), A.status);
  }
  __syncthreads();
  if (!s_entry) return;
  Kv8Item I = s_item;
  I.blk = *s_entry;
  if (part & 1) kv8_append_v<MANY>(A, I, h0, h1, part >> 1, lane); else kv8_append_k<MANY>(A, I, h0, h1, part >> 1, lane);
  if (say && (I.blk < 0 || I.blk >= A.dst.num_blocks)) flag(A.status, ST_BAD_BLOCK);
}

}  // namespace

cudaError_t launch_kv8_append(const uint16_t *k, const uint16_t *v, const int32_t *cu_rows, const int64_t *P0,
                              const int32_t *seqs, int n, long long T, const float *table, int64_t max_pos,
                              float value_scale, const Kv8View &dst, unsigned *status, cudaStream_t st) {
  if (dst.hkv > (1 << 24)) return cudaErrorInvalidValue;  // (a position alone would be 5 GB)
  Kv8Append A{k, v, cu_rows, P0, seqs, n, T, table, max_pos, value_scale, dst, status, 1, dst.hkv, CHUNKS_BY_TILE};
  long long units = (T >> 4) + 2LL * n;  // tiles that the call could have: by row the fewer for chunks of one or two
  if (T <= units) A.units = CHUNKS_BY_ROW, units = T;  // (256 chunks of one row, 8 KV heads: 7.1 us, by tile 9.0)
  while (2 * A.heads <= K8A_HEADS && A.heads < dst.hkv &&
         units * ((dst.hkv + 2 * A.heads - 1) / (2 * A.heads)) >= 2LL * K8A_CTAS * num_sms())
    A.heads *= 2;
  A.per_tile = (dst.hkv + A.heads - 1) / A.heads;
  const long long blocks = units * A.per_tile;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;  // (rows of 88 TB, or 2^28 chunks)
  return launch_pdl(A.heads > 1 ? kv8_append_kernel<true> : kv8_append_kernel<false>, dim3((unsigned)blocks),
                    dim3(K8A_WARPS * 32), 0, st, A);
}

}  // namespace kvr
