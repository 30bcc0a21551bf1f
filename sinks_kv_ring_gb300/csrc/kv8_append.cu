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
// The quotient is the correctly rounded one: r = RN(1/s), q = RN(x r), and one
// residual step RN(q + r (x - s q)) (the division by Newton correction of P.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990), so exact ties, which bf16 values over a bf16 scale meet
// often, round to even.
//
// A warp takes the K, another the V, of one tile and KV head, whole: 16 bytes of
// codes a lane and store, the tile's largest magnitude a few shuffles away.  A
// chunk that starts inside a tile finds the rows ahead of it there: their V
// codes share 16 bytes with the new ones and are read in any case, their K codes
// only where the scale grows.
#include "kv8.cuh"
#include "launch.h"

namespace kvr {
namespace {

constexpr int K8A_WARPS = 8;
constexpr unsigned FULLW = 0xffffffffu;

__device__ __forceinline__ float abs_bits(uint32_t m) { return __uint_as_float(m); }

// The least bf16 number s with 127 s >= a (a finite, >= 0): the quotient
// rounded up to bf16, one step more where fp32 rounded it down onto it.
__device__ __forceinline__ float kv8_scale(float a) {
  uint32_t b = (__float_as_uint(__fdiv_rn(a, 127.f)) + 0xffffu) & 0xffff0000u;
  if (__fmul_rn(__uint_as_float(b), 127.f) < a) b += 0x10000u;
  return __uint_as_float(b);
}

// Stored codes (u + 128) of four values: rint(x / s) by the residual step,
// rounded by adding 1.5 2^23, which leaves it in the low bits.  s = 0 has r = 0.
struct Kv8Div {
  float s, r;
  bool slow;  // a scale so small that its reciprocal or the residual leaves fp32
};
__device__ __forceinline__ Kv8Div kv8_div(float s) {
  Kv8Div D;
  D.s = s;
  D.slow = s < 0x1p-100f && s > 0.f;
  D.r = s > 0.f && !D.slow ? __frcp_rn(s) : 0.f;
  return D;
}
__device__ __forceinline__ uint32_t kv8_codes(const float (&x)[4], const Kv8Div &D) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q0 = __fmul_rn(x[i], D.r);
    float v = fmaf(fmaf(-D.s, q0, x[i]), D.r, q0);
    if (D.slow) v = __fdiv_rn(x[i], D.s);
    q[i] = __float_as_uint(__fadd_rn(v, 12582912.f));
  }
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410) ^ 0x80808080u;
}
// Stored codes under a larger scale: the values that they stand for, quantised again.
__device__ __forceinline__ uint32_t kv8_again(uint32_t w, float s_old, const Kv8Div &D) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __fmul_rn((float)((int)((w >> (8 * i)) & 255u) - 128), s_old);
  return kv8_codes(x, D);
}

__device__ __forceinline__ void unpack_bf16(uint32_t w, float &lo, float &hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
// Largest magnitudes of a packed pair of bf16, kept apart in the two halves.
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

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
  long long warps;  // 2 hkv warps for each tile that the call could have
  unsigned *status;
};

// Where a warp's tile lies and which of its rows are new.
struct Kv8Item {
  uint8_t *tile;
  long long row0;  // k/v row of the tile's position 0 (may lie ahead of the chunk's first)
  int r0, r1;      // new rows [r0, r1); rows below r0 are there already
  long long p;     // position of the tile's row 0
};

__device__ __forceinline__ void kv8_append_k(const Kv8Append &A, const Kv8Item &I, int h, int lane) {
  const int t = lane & 3, gr = lane >> 2, H = A.dst.hkv;
  // rows gr and gr + 8, dims 16t .. 16t + 15 of each group of 64; and of the rotary group the other half of the pairs
  uint4 raw[2][3][2], mate[2][2];
  float4 cs[2][8];
  bool is_new[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = gr + 8 * e;
    is_new[e] = r >= I.r0 && r < I.r1;
    const uint16_t *src = A.k + ((I.row0 + r) * H + h) * DQK + 16 * t;
    const float *tr = A.table + (I.p + r) * 64 + 32 * (t & 1);
#pragma unroll
    for (int g = 0; g < 3; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) raw[e][g][i] = is_new[e] ? reinterpret_cast<const uint4 *>(src + 64 * g)[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      mate[e][i] = is_new[e] ? reinterpret_cast<const uint4 *>(src + (t < 2 ? 32 : -32))[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[e][i] = is_new[e] ? reinterpret_cast<const float4 *>(tr)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const uint4 tail = I.r0 > 0 ? *reinterpret_cast<const uint4 *>(I.tile + KV8_OFF_TAIL) : make_uint4(0, 0, 0, 0);
  // the rotary group: products and sum rounded one by one, so the result does not hang on contraction
  float x0[2][16];
  const float sign = t < 2 ? -1.f : 1.f;  // a c - b s, or b c + a s
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 &w4 = raw[e][0][i >> 2], &m4 = mate[e][i >> 2];
      const uint32_t w = (i & 3) == 0 ? w4.x : (i & 3) == 1 ? w4.y : (i & 3) == 2 ? w4.z : w4.w;
      const uint32_t m = (i & 3) == 0 ? m4.x : (i & 3) == 1 ? m4.y : (i & 3) == 2 ? m4.z : m4.w;
      float a, b, c, d;
      unpack_bf16(w, a, b);
      unpack_bf16(m, c, d);
      x0[e][2 * i] = __fadd_rn(__fmul_rn(a, cs[e][i].x), sign * __fmul_rn(c, cs[e][i].y));
      x0[e][2 * i + 1] = __fadd_rn(__fmul_rn(b, cs[e][i].z), sign * __fmul_rn(d, cs[e][i].w));
    }
  // a row's largest magnitude (as bits: infinities and NaN above all), the rows that are not finite, the tile's largest
  uint32_t top = 0, bad = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t m2 = 0, m = 0;
#pragma unroll
    for (int g = 1; g < 3; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 &w = raw[e][g][i];
        m2 = abs_max2(abs_max2(abs_max2(abs_max2(m2, w.x), w.y), w.z), w.w);
      }
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x0[e][i]) & 0x7fffffffu);
    m = max(m, max(m2 << 16, m2 & 0xffff0000u));
    m = max(m, __shfl_xor_sync(FULLW, m, 1));
    m = max(m, __shfl_xor_sync(FULLW, m, 2));
    const bool odd = m >= 0x7f800000u;
    const unsigned rows = __ballot_sync(FULLW, odd && t == 0);  // bit 4 gr
#pragma unroll
    for (int i = 0; i < 8; ++i) bad |= (rows >> (4 * i) & 1u) << (i + 8 * e);
    if (odd) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x0[e][i] = 0.f;
#pragma unroll
      for (int g = 1; g < 3; ++g) raw[e][g][0] = raw[e][g][1] = make_uint4(0, 0, 0, 0);
    } else {
      top = max(top, m);
    }
  }
  top = __reduce_max_sync(FULLW, top);
  const float s_old = __uint_as_float(tail.x), s_need = kv8_scale(abs_bits(top));
  const bool grow = I.r0 > 0 && s_need > s_old;
  const float s = I.r0 > 0 && !grow ? s_old : s_need;
  const Kv8Div D = kv8_div(s);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = gr + 8 * e;
    uint8_t *at = I.tile + e * 512 + lane * 16;
    if (is_new[e]) {
#pragma unroll
      for (int g = 0; g < 3; ++g) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // four dims each
          float x[4];
          if (g == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = x0[e][4 * j + i];
          } else {
            const uint4 &w = raw[e][g][j >> 1];
            unpack_bf16(j & 1 ? w.z : w.x, x[0], x[1]);
            unpack_bf16(j & 1 ? w.w : w.y, x[2], x[3]);
          }
          c[j] = kv8_codes(x, D);
        }
        *reinterpret_cast<uint4 *>(at + 1024 * g) = make_uint4(c[0], c[1], c[2], c[3]);
      }
    } else if (grow && r < I.r0) {
      uint4 w[3];
#pragma unroll
      for (int g = 0; g < 3; ++g) w[g] = *reinterpret_cast<const uint4 *>(at + 1024 * g);
#pragma unroll
      for (int g = 0; g < 3; ++g)
        *reinterpret_cast<uint4 *>(at + 1024 * g) = make_uint4(kv8_again(w[g].x, s_old, D), kv8_again(w[g].y, s_old, D),
                                                               kv8_again(w[g].z, s_old, D), kv8_again(w[g].w, s_old, D));
    }
  }
  if (lane == 0) {
    *reinterpret_cast<float *>(I.tile + KV8_OFF_TAIL) = s;
    *reinterpret_cast<uint16_t *>(I.tile + KV8_OFF_TAIL + 8) = (uint16_t)((tail.z & ((1u << I.r0) - 1u)) | bad);
    *reinterpret_cast<uint32_t *>(I.tile + KV8_OFF_TAIL + 12) = 0u;
  }
}

__device__ __forceinline__ void kv8_append_v(const Kv8Append &A, const Kv8Item &I, int h, int lane) {
  const int t = lane & 3, gr = lane >> 2, H = A.dst.hkv;
  // positions 2t, 2t + 1, 2t + 8, 2t + 9 (j), dims 4 gr .. 4 gr + 3 of each group of 32
  uint2 raw[4][4];
  uint4 old[4];
  bool is_new[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 2 * t + (j & 1) + 8 * (j >> 1);
    is_new[j] = r >= I.r0 && r < I.r1;
    const uint16_t *src = A.v + ((I.row0 + r) * H + h) * DV + 4 * gr;
#pragma unroll
    for (int g = 0; g < 4; ++g) raw[j][g] = is_new[j] ? *reinterpret_cast<const uint2 *>(src + 32 * g) : make_uint2(0, 0);
  }
  const bool any_old = I.r0 > 0;
  uint4 tail = make_uint4(0, 0, 0, 0);
  if (any_old) {
    tail = *reinterpret_cast<const uint4 *>(I.tile + KV8_OFF_TAIL);
#pragma unroll
    for (int g = 0; g < 4; ++g) old[g] = *reinterpret_cast<const uint4 *>(I.tile + KV8_OFF_V + 512 * g + 16 * lane);
  }
  uint32_t top = 0, bad = 0;
  bool odd[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t m2 = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) m2 = abs_max2(abs_max2(m2, raw[j][g].x), raw[j][g].y);
    uint32_t m = max(m2 << 16, m2 & 0xffff0000u);
    m = max(m, __shfl_xor_sync(FULLW, m, 4));
    m = max(m, __shfl_xor_sync(FULLW, m, 8));
    m = max(m, __shfl_xor_sync(FULLW, m, 16));
    // the largest of the scaled values is the largest's product (a NaN stays one)
    const uint32_t y = __float_as_uint(__fmul_rn(__uint_as_float(m), A.vscale)) & 0x7fffffffu;
    odd[j] = m >= 0x7f800000u || y >= 0x7f800000u;
    if (is_new[j]) {
      if (!odd[j]) top = max(top, y);
    }
    const unsigned rows = __ballot_sync(FULLW, is_new[j] && odd[j] && gr == 0);  // bits t
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (rows >> i & 1u) << (2 * i + (j & 1) + 8 * (j >> 1));
  }
  top = __reduce_max_sync(FULLW, top);
  const float s_old = __uint_as_float(tail.y), s_need = kv8_scale(abs_bits(top));
  const bool grow = any_old && s_need > s_old;
  const float s = any_old && !grow ? s_old : s_need;
  const Kv8Div D = kv8_div(s);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t c[4];  // of position j: four dims
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[4];
      unpack_bf16(raw[j][g].x, x[0], x[1]);
      unpack_bf16(raw[j][g].y, x[2], x[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = odd[j] ? 0.f : __fmul_rn(x[i], A.vscale);
      c[j] = kv8_codes(x, D);
    }
    // to a word per dim: positions in its bytes
    uint32_t w[4];
    const uint32_t a = __byte_perm(c[0], c[1], 0x5140), b = __byte_perm(c[2], c[3], 0x5140);  // dims 0, 1 of both
    const uint32_t e = __byte_perm(c[0], c[1], 0x7362), f = __byte_perm(c[2], c[3], 0x7362);  // dims 2, 3
    w[0] = __byte_perm(a, b, 0x5410);
    w[1] = __byte_perm(a, b, 0x7632);
    w[2] = __byte_perm(e, f, 0x5410);
    w[3] = __byte_perm(e, f, 0x7632);
    if (any_old) {
      uint32_t keep = 0;  // bytes of positions that are there already
#pragma unroll
      for (int j = 0; j < 4; ++j) keep |= 2 * t + (j & 1) + 8 * (j >> 1) < I.r0 ? 0xffu << (8 * j) : 0u;
      uint32_t o[4] = {old[g].x, old[g].y, old[g].z, old[g].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (grow) o[i] = kv8_again(o[i], s_old, D);
        w[i] = (o[i] & keep) | (w[i] & ~keep);
      }
    }
    *reinterpret_cast<uint4 *>(I.tile + KV8_OFF_V + 512 * g + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lane == 0) {
    *reinterpret_cast<float *>(I.tile + KV8_OFF_TAIL + 4) = s;
    *reinterpret_cast<uint16_t *>(I.tile + KV8_OFF_TAIL + 10) = (uint16_t)(((tail.z >> 16) & ((1u << I.r0) - 1u)) | bad);
  }
}

__global__ void __launch_bounds__(K8A_WARPS * 32) kv8_append_kernel(Kv8Append A) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, per = 2 * A.dst.hkv;
  const long long w = (long long)blockIdx.x * K8A_WARPS + (threadIdx.x >> 5);
  if (w >= A.warps) return;
  const long long unit = w / per;
  const int part = (int)(w - unit * per), h = part >> 1;
  const bool say = lane == 0 && part == 0;
  const int i = kv8_chunk(A.cu_rows, A.n, unit);
  const int c0 = A.cu_rows[i], c1 = A.cu_rows[i + 1], s = A.seqs[i];
  const long long a = A.P0[i];
  if (c0 < 0 || c1 < c0 || c1 > A.T) {
    if (say) flag(A.status, ST_BAD_ROWS);
    return;
  }
  const long long u = unit - ((c0 >> 4) + 2LL * i);
  if (u < 0 || c1 == c0 || s == -1) return;
  const bool bs = s < 0 || s >= A.dst.num_seqs;
  const long long most = min((long long)A.max_pos, (long long)A.dst.max_blocks * A.dst.block_size);
  const bool bp = a < 0 || a > most - (c1 - c0);
  if (bs || bp) {
    if (say && u == 0) flag(A.status, (bs ? ST_BAD_SEQ : 0u) | (bp ? ST_BAD_POS : 0u));
    return;
  }
  Kv8Item I;
  I.p = ((a >> 4) + u) << 4;
  const long long end = a + (c1 - c0);
  if (I.p >= end) return;
  I.r0 = (int)max(a - I.p, 0LL);
  I.r1 = (int)min(end - I.p, 16LL);
  I.row0 = c0 + (I.p - a);
  const unsigned tile = (unsigned)(I.p >> 4), per_block = (unsigned)A.dst.block_size >> 4, bi = tile / per_block;
  const int blk = A.dst.block_table[(long long)s * A.dst.max_blocks + bi];
  if (blk < 0 || blk >= A.dst.num_blocks) {
    if (say) flag(A.status, ST_BAD_BLOCK);
    return;
  }
  I.tile = A.dst.data + kv8_tile(A.dst, blk, h, (int)(16 * (tile - bi * per_block)));
  if (part & 1) kv8_append_v(A, I, h, lane); else kv8_append_k(A, I, h, lane);
}

}  // namespace

cudaError_t launch_kv8_append(const uint16_t *k, const uint16_t *v, const int32_t *cu_rows, const int64_t *P0,
                              const int32_t *seqs, int n, long long T, const float *table, int64_t max_pos,
                              float value_scale, const Kv8View &dst, unsigned *status, cudaStream_t st) {
  if (dst.hkv > (1 << 24)) return cudaErrorInvalidValue;  // (a position alone would be 5 GB)
  Kv8Append A{k, v, cu_rows, P0, seqs, n, T, table, max_pos, value_scale, dst, 0, status};
  A.warps = ((T >> 4) + 2LL * n) * 2 * dst.hkv;
  const long long blocks = (A.warps + K8A_WARPS - 1) / K8A_WARPS;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;  // (2^34 warps: rows of 22 TB)
  return launch_pdl(kv8_append_kernel, dim3((unsigned)blocks), dim3(K8A_WARPS * 32), 0, st, A);
}

}  // namespace kvr
