// kv4_append.cu -- fused KV write into a 4-bit pool: rotate-half RoPE of k
// (dims 0..63), value scale of v, quantisation in groups of 64 dims.
//
// colibri "MiMo-V2.6", "What the engine implements" (partial RoPE, values
// multiplied by attention_value_scale), as kv_ring_append_rope, with
//   m = fp16 down(min x), s = fp16 up((max x - m) / 15),
//   u = clamp(rint((x - m) / s), 0, 15)
// per group, all in fp32.  The quotient is the correctly rounded one:
// r = RN(1/s), q = RN(d r), and one residual step RN(q + r (d - s q)) (the
// division by Newton correction of P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): one reciprocal per
// group instead of 64 divisions, and exact ties round to even as they should
// (bf16 keys meet them often).
//
// A warp takes four tokens of one KV head at a time: lane 8i + c holds dims
// 8c..8c+7 of a group of token i, so the group's extrema are three shuffles
// away and a 16-byte load brings a lane's values, all five in flight before
// the destination is looked up.
//
// What bounds it: a warp's own chain (loads, the RoPE row, some 480 instructions
// per four tokens of a head, stores), with too few warps an SM to fill either
// side: 52 us for 302,216 (token, KV head) pairs, 0.70 of what their 820 bytes
// each take at the copy rate, 64% of the issue slots, and waits for loads the
// largest of the stalls.  The extrema of the five groups go through one butterfly that halves
// what a lane carries at each step, a group's scale is taken by one lane of its
// token (2 divisions instead of 10 per lane) and the codes come in packed
// pairs.  Loading the next head's values ahead of their use, into registers or
// shared memory, gained nothing (54 us or more).  The stores are 2 and 4 bytes
// wide (a position's V codes lie apart) and merge in L2; putting whole tiles
// together in shared memory first, for full-sector stores, measured slower (73
// us against 64 at the time): they are not what bounds it.
#include "kv4.cuh"
#include "launch.h"

namespace kvr {
namespace {

constexpr int K4A_WARPS = 4;
// From this many (token, KV head) pairs on a warp takes four KV heads, not one
// (one head against four, in us: 32,768 pairs 10.6 / 10.8; 49,152 14.3 / 15.6;
// 65,536 17.4 / 15.9; 131,072 31.2 / 26.7; 302,216 63.5 / 51.8): the look-up of
// the destination and the start of its dependent loads are paid once, but too
// few warps start at small sizes (64 tokens: 2.6 / 5.2).
constexpr long long K4A_MANY = 65536;
constexpr unsigned FULLW = 0xffffffffu;

// min and max that hand a NaN on
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// Least and negated greatest of a lane's 8 bf16 values, as a packed pair.
__device__ __forceinline__ uint32_t extrema_bf16(const uint4 &x) {
  const uint32_t a = min_nan_bf16x2(min_nan_bf16x2(x.x, x.y), min_nan_bf16x2(x.z, x.w));
  const uint32_t b = max_nan_bf16x2(max_nan_bf16x2(x.x, x.y), max_nan_bf16x2(x.z, x.w)) ^ 0x80008000u;
  return min_nan_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
}

// Scale and minimum of a group (packed, scale in the low half) and the
// reciprocal of the scale; the reciprocal is -1 where values lie past fp16
// (their codes need a clamp) and -2 where one is not finite.
__device__ __forceinline__ void kv4_scale(float lo, float hi, uint32_t &sm, float &r) {
  const __half m = __float2half_rd(fminf(fmaxf(lo, -65504.f), 65504.f));
  const float mf = __half2float(m);
  const __half s = __float2half_ru(fminf(__fdiv_rn(__fsub_rn(hi, mf), 15.f), 65504.f));
  const float sf = __half2float(s);
  sm = __half_as_ushort(s) | ((uint32_t)__half_as_ushort(m) << 16);
  r = sf > 0.f ? __frcp_rn(sf) : 0.f;
  if (!(lo >= -65504.f && hi <= 65504.f)) {  // (so for a NaN)
    r = -1.f;
    if (!(lo >= -3.4028235e38f && hi <= 3.4028235e38f)) {
      sm = 0x7fff7fffu;
      r = -2.f;
    }
  }
}

// Codes of a lane's 8 values (dim i in nibble i, pairs of dims in x) under
// scale, minimum and reciprocal.  The quotient lies in [0, 15] and is rounded
// by adding 1.5 2^23, which leaves it in the low bits; multiply-adds join the
// nibbles.
__device__ __forceinline__ uint32_t kv4_codes(const uint64_t (&x)[4], uint32_t sm, float r) {
  const float sf = __half2float(__ushort_as_half((uint16_t)sm)), mf = __half2float(__ushort_as_half((uint16_t)(sm >> 16)));
  const uint64_t nm = f32x2(-mf, -mf), ns = f32x2(-sf, -sf), rr = f32x2(r, r), magic = f32x2(12582912.f, 12582912.f);
  uint32_t w = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const uint64_t d = add_f32x2(x[i], nm);
    const uint64_t q0 = mul_f32x2(d, rr);
    float a, b;
    f32x2_split(add_f32x2(fma_f32x2(fma_f32x2(ns, q0, d), rr, q0), magic), a, b);
    w = (w * 16u + __float_as_uint(b)) * 16u + __float_as_uint(a);
  }
  return w - 0x4b400000u * 0x11111111u;  // less the eight exponents
}
// The same where values may lie past fp16 (r = -1) or one is not finite (-2).
__device__ __forceinline__ uint32_t kv4_codes_any(const uint64_t (&x)[4], uint32_t sm, float r) {
  if (r >= 0.f) return kv4_codes(x, sm, r);
  uint32_t w = 0;
  if (r == -1.f) {
    const float sf = __half2float(__ushort_as_half((uint16_t)sm)), mf = __half2float(__ushort_as_half((uint16_t)(sm >> 16)));
    r = sf > 0.f ? __frcp_rn(sf) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      f32x2_split(x[i >> 1], a, b);
      const float d = __fsub_rn(i & 1 ? b : a, mf);
      const float q0 = __fmul_rn(d, r);
      const float q = fmaf(fmaf(-sf, q0, d), r, q0);
      w |= (uint32_t)__float2int_rn(fminf(fmaxf(q, 0.f), 15.f)) << (4 * i);
    }
  }
  return w;
}

// Where token t goes: block (-1: nowhere) and row in it; flags a token that
// cannot be written where `say` is set.
__device__ __forceinline__ void look_up(const int64_t *__restrict__ pos, const int32_t *__restrict__ seq,
                                        const int64_t *__restrict__ slots, long long t, int T, int64_t max_pos,
                                        const Kv4View &dst, bool say, unsigned *status, int &blk, int &row, int &p) {
  blk = -1;
  row = p = 0;
  if (t >= T) return;
  const long long pp = pos[t];
  const int s = slots ? 0 : seq[t];
  unsigned bad = 0;
  bool pad = s == -1;
  if (slots) {
    const long long slot = slots[t];
    pad = slot < 0;
    if (!pad) {
      if (slot < (long long)dst.num_blocks * dst.block_size) {
        // (a pool of 2^32 positions would be 781 GB)
        blk = (int)((unsigned)slot / (unsigned)dst.block_size);
        row = (int)((unsigned)slot - (unsigned)blk * (unsigned)dst.block_size);
      } else {
        bad = ST_BAD_BLOCK;
      }
    }
  }
  if (!pad && !bad) {
    if (pp < 0 || pp >= max_pos) {
      bad = ST_BAD_POS;
    } else if (!slots) {
      if (s < 0 || s >= dst.num_seqs) {
        bad = ST_BAD_SEQ;
      } else {
        const unsigned bi = (unsigned)pp / (unsigned)dst.block_size;  // (max_pos < 2^31)
        blk = bi < (unsigned)dst.max_blocks ? dst.block_table[(long long)s * dst.max_blocks + bi] : -1;
        row = (int)((unsigned)pp - bi * (unsigned)dst.block_size);
        if (blk < 0 || blk >= dst.num_blocks) bad = ST_BAD_BLOCK;
      }
    }
  }
  if (bad) {
    blk = -1;
    if (say) flag(status, bad);
  }
  if (blk >= 0) p = (int)pp;  // (a token that goes nowhere rotates by row 0: its position may be anything)
}

__device__ __forceinline__ uint64_t bf16x2_f32x2(uint32_t x) {
  return f32x2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// Quantise and store a lane's values of all five groups; r >= 0 for all where
// ANY is not set.
template <bool ANY>
__device__ __forceinline__ void put_codes(const uint64_t (&x0)[4], const uint4 (&raw)[5], float vscale, uint32_t mysm,
                                          float myr, uint8_t *kd, uint8_t *vd, bool put, int lane) {
#pragma unroll
  for (int g = 0; g < 5; ++g) {
    const int from = (lane & 24) + (g == 0 ? 1 : 2 * g - 2);
    const uint32_t sm = __shfl_sync(FULLW, mysm, from);
    const float rc = __shfl_sync(FULLW, myr, from);
    uint64_t x[4];
    const uint32_t e[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (g < KV4_KG) {
        x[i] = g == 0 ? x0[i] : bf16x2_f32x2(e[i]);
      } else {  // (a packed product would be joined with the subtraction that follows, and not be rounded)
        x[i] = f32x2(__fmul_rn(__uint_as_float(e[i] << 16), vscale), __fmul_rn(__uint_as_float(e[i] & 0xffff0000u), vscale));
      }
    }
    const uint32_t w = ANY ? kv4_codes_any(x, sm, rc) : kv4_codes(x, sm, rc);
    if (put) {
      if (g < KV4_KG) {
        *reinterpret_cast<uint32_t *>(kd + 512 * g) = w;
      } else {
        *reinterpret_cast<uint16_t *>(vd + 512 * (g - KV4_KG)) = (uint16_t)w;
        *reinterpret_cast<uint16_t *>(vd + 512 * (g - KV4_KG) + 4) = (uint16_t)(w >> 16);
      }
    }
  }
}

// One token of four (lane 8i + c: token i): rotate, quantise and store to
// position r of `tile` (null: nothing); tr points to the (cos, sin) of the
// lane's 8 dims.
__device__ __forceinline__ void put_token(const uint4 (&raw)[5], const float *tr, float vscale, uint8_t *tile,
                                          int r, int lane) {
  const int c = lane & 7;
  // group 0: rotate.  The other half of the pair lies four lanes away;
  // products and sum are rounded one by one, so the result does not hang on
  // contraction.
  uint64_t x0[4];
  {
    float cs[16];  // (cos, sin) of the lane's dims; not kept across heads: 16 registers
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(cs[4 * u]), "=f"(cs[4 * u + 1]), "=f"(cs[4 * u + 2]), "=f"(cs[4 * u + 3])
                   : "l"(tr + 4 * u));
    }
    const uint32_t neg = c < 4 ? 0x80008000u : 0u;  // a - b, or a + b
    const uint32_t e[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t o = __shfl_xor_sync(FULLW, e[i], 4) ^ neg;
      const float a0 = __fmul_rn(__uint_as_float(e[i] << 16), cs[4 * i]);
      const float b0 = __fmul_rn(__uint_as_float(o << 16), cs[4 * i + 1]);
      const float a1 = __fmul_rn(__uint_as_float(e[i] & 0xffff0000u), cs[4 * i + 2]);
      const float b1 = __fmul_rn(__uint_as_float(o & 0xffff0000u), cs[4 * i + 3]);
      x0[i] = f32x2(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
    }
  }
  // Extrema.  Each step of a butterfly over the token's eight lanes halves
  // what a lane still carries: of four packed pairs to two, one, one, and of
  // group 0's two to one.  Lane c ends with group 1 + c / 2, lane 1 with group
  // 0 besides, and takes that group's scale (the divisions are most of a
  // group's cost).
  float lo, hi;
  {
    const uint32_t m1 = extrema_bf16(raw[1]), m2 = extrema_bf16(raw[2]);
    const uint32_t m3 = extrema_bf16(raw[3]), m4 = extrema_bf16(raw[4]);
    const bool b2 = c & 4, b1 = c & 2, b0 = c & 1;
    const uint32_t ma = min_nan_bf16x2(b2 ? m3 : m1, __shfl_xor_sync(FULLW, b2 ? m1 : m3, 4));
    const uint32_t mb = min_nan_bf16x2(b2 ? m4 : m2, __shfl_xor_sync(FULLW, b2 ? m2 : m4, 4));
    uint32_t m = min_nan_bf16x2(b1 ? mb : ma, __shfl_xor_sync(FULLW, b1 ? ma : mb, 2));
    m = min_nan_bf16x2(m, __shfl_xor_sync(FULLW, m, 1));
    lo = __uint_as_float(m << 16);
    hi = -__uint_as_float(m & 0xffff0000u);
    if (c >= 4) {  // the scaled values' extrema are the extrema's products (swapped under a negative scale)
      const float a = __fmul_rn(lo, vscale), b = __fmul_rn(hi, vscale);
      lo = min_nan(a, b);
      hi = max_nan(a, b);
    }
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f32x2_split(x0[i], y[2 * i], y[2 * i + 1]);
    const float l = min_nan(min_nan(y[0], y[1], y[2]), min_nan(y[3], y[4], y[5]), min_nan(y[6], y[7]));
    const float h = -max_nan(max_nan(y[0], y[1], y[2]), max_nan(y[3], y[4], y[5]), max_nan(y[6], y[7]));
    float z = min_nan(b0 ? h : l, __shfl_xor_sync(FULLW, b0 ? l : h, 1));
    z = min_nan(z, __shfl_xor_sync(FULLW, z, 2));
    z = min_nan(z, __shfl_xor_sync(FULLW, z, 4));
    const float other = __shfl_xor_sync(FULLW, z, 1);
    if (c == 1) {
      lo = other;
      hi = -z;
    }
  }
  uint32_t mysm;
  float myr;
  kv4_scale(lo, hi, mysm, myr);
  if (tile) {
    if (c == 1 || !(c & 1)) {  // the group's scale and minimum
      const int g = c == 1 ? 0 : 1 + (c >> 1), q = kv4_quad(r) * 2;
      const int at_s = g < KV4_KG ? KV4_OFF_KS + g * 32 + q : KV4_OFF_VS + (g - KV4_KG) * 32 + q;
      const int at_m = g < KV4_KG ? KV4_OFF_KM + r * 8 + g * 2 : KV4_OFF_VM + (g - KV4_KG) * 32 + q;
      *reinterpret_cast<uint16_t *>(tile + at_s) = (uint16_t)mysm;
      *reinterpret_cast<uint16_t *>(tile + at_m) = (uint16_t)(mysm >> 16);
    } else if (c == 3) {
      *reinterpret_cast<uint16_t *>(tile + KV4_OFF_KM + r * 8 + 6) = 0;
    }
  }
  uint8_t *kd = tile + kv4_k_at(0, r, c >> 1) + (c & 1) * 4, *vd = tile + kv4_v_at(0, r, c, 0);
  if (__any_sync(FULLW, myr < 0.f)) {
    put_codes<true>(x0, raw, vscale, mysm, myr, kd, vd, tile != nullptr, lane);
  } else {
    put_codes<false>(x0, raw, vscale, mysm, myr, kd, vd, tile != nullptr, lane);
  }
}

__device__ __forceinline__ void load_token(const uint16_t *__restrict__ k, const uint16_t *__restrict__ v, size_t item,
                                           bool have, int c, uint4 (&raw)[5]) {
#pragma unroll
  for (int g = 0; g < 5; ++g) raw[g] = make_uint4(0, 0, 0, 0);
  if (have) {
    const uint4 *k4 = reinterpret_cast<const uint4 *>(k) + item * (DQK / 8);
    const uint4 *v4 = reinterpret_cast<const uint4 *>(v) + item * (DV / 8);
#pragma unroll
    for (int g = 0; g < KV4_KG; ++g) raw[g] = k4[g * 8 + c];
#pragma unroll
    for (int g = 0; g < KV4_VG; ++g) raw[KV4_KG + g] = v4[g * 8 + c];
  }
}

// A warp takes HEADS KV heads of four tokens, one after the other (a token's
// last ones may be fewer).
template <int HEADS, int CTAS>
__global__ void __launch_bounds__(K4A_WARPS * 32, CTAS)
    kv4_append_kernel(const uint16_t *__restrict__ k, const uint16_t *__restrict__ v, const int64_t *__restrict__ pos,
                      const int32_t *__restrict__ seq, const int64_t *__restrict__ slots, int T, unsigned warps,
                      const float *__restrict__ table, int64_t max_pos, float vscale, Kv4View dst, unsigned *status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 7;
  const unsigned w = blockIdx.x * K4A_WARPS + (threadIdx.x >> 5);
  if (w >= warps) return;
  const unsigned parts = ((unsigned)dst.hkv + HEADS - 1) / HEADS, four = w / parts;
  const int h0 = (int)(w - four * parts) * HEADS, h1 = min(h0 + HEADS, dst.hkv);
  const long long t = 4LL * four + (lane >> 3);
  const size_t item = (size_t)t * dst.hkv;
  uint4 raw[5];
  load_token(k, v, item + h0, t < T, c, raw);
  int blk, row, p;
  look_up(pos, seq, slots, t, T, max_pos, dst, h0 == 0 && c == 0, status, blk, row, p);
  const float *tr = table + (long long)p * 64 + 16 * (c & 3);
#pragma unroll 1
  for (int h = h0;;) {
    put_token(raw, tr, vscale, blk >= 0 ? dst.data + kv4_tile(dst, blk, h, row) : nullptr, row & 15, lane);
    if (HEADS == 1 || ++h >= h1) break;
    load_token(k, v, item + h, t < T, c, raw);
  }
}

template <int HEADS, int CTAS>
cudaError_t launch_heads(const uint16_t *k, const uint16_t *v, const int64_t *pos, const int32_t *seq,
                         const int64_t *slots, int T, const float *table, int64_t max_pos, float value_scale,
                         const Kv4View &dst, unsigned *status, cudaStream_t st) {
  const long long warps = ((long long)T + 3) / 4 * ((dst.hkv + HEADS - 1) / HEADS);
  const long long ctas = (warps + K4A_WARPS - 1) / K4A_WARPS;
  if (warps > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(kv4_append_kernel<HEADS, CTAS>, dim3((unsigned)ctas), dim3(K4A_WARPS * 32), 0, st, k, v, pos, seq,
                    slots, T, (unsigned)warps, table, max_pos, value_scale, dst, status);
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t *k, const uint16_t *v, const int64_t *pos, const int32_t *seq,
                              const int64_t *slots, int T, const float *table, int64_t max_pos, float value_scale,
                              const Kv4View &dst, unsigned *status, cudaStream_t st) {
  if (dst.hkv > 1 && (long long)T * dst.hkv >= K4A_MANY)
    return launch_heads<4, 8>(k, v, pos, seq, slots, T, table, max_pos, value_scale, dst, status, st);
  return launch_heads<1, 10>(k, v, pos, seq, slots, T, table, max_pos, value_scale, dst, status, st);
}

}  // namespace kvr
