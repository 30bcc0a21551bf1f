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
// A warp takes four tokens of one KV head: lane 8i + c holds dims 8c..8c+7 of
// a group of token i, so the group's extrema are three shuffles away and a
// 16-byte load brings a lane's values, all five in flight before the
// destination is looked up.
//
// What bounds it: instructions, about 750 per four tokens (unpacking, extrema,
// the exact quotient; the schedulers issue in 75% of the cycles): 302,216
// (token, KV head) pairs take 64 us where their 820 bytes each take 37 us at
// the copy rate.  The scales of a token's five groups are taken by five of its
// lanes at once (2 divisions instead of 10 per lane), the codes in packed
// pairs.  The stores are 2 and 4 bytes wide (a position's V codes lie apart)
// and merge in L2; putting whole tiles together in shared memory first, for
// full-sector stores, measured slower (73 us against 64): they are not what
// bounds it.
#include "kv4.cuh"
#include "launch.h"

namespace kvr {
namespace {

constexpr int K4A_WARPS = 4;
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

// Least and greatest of a group's 64 bf16 values over its eight lanes: in
// packed pairs, the greatest as the least of the negated ones.
__device__ __forceinline__ void extrema_bf16(const uint4 &x, float &lo, float &hi) {
  const uint32_t a = min_nan_bf16x2(min_nan_bf16x2(x.x, x.y), min_nan_bf16x2(x.z, x.w));
  const uint32_t b = max_nan_bf16x2(max_nan_bf16x2(x.x, x.y), max_nan_bf16x2(x.z, x.w)) ^ 0x80008000u;
  uint32_t m = min_nan_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));  // (least, -greatest)
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = min_nan_bf16x2(m, __shfl_xor_sync(FULLW, m, o));
  lo = __uint_as_float(m << 16);
  hi = -__uint_as_float(m & 0xffff0000u);
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

// Codes of a lane's 8 values (dim i in nibble i) under scale, minimum and
// reciprocal.  The quotient lies in [0, 15] and is rounded by adding 1.5 2^23,
// which leaves it in the low bits; multiply-adds join the nibbles.
__device__ __forceinline__ uint32_t kv4_codes(const float (&x)[8], uint32_t sm, float r) {
  const float sf = __half2float(__ushort_as_half((uint16_t)sm)), mf = __half2float(__ushort_as_half((uint16_t)(sm >> 16)));
  uint32_t w = 0;
  if (r >= 0.f) {  // (the group's eight lanes agree)
    const uint64_t nm = f32x2(-mf, -mf), ns = f32x2(-sf, -sf), rr = f32x2(r, r), magic = f32x2(12582912.f, 12582912.f);
#pragma unroll
    for (int i = 6; i >= 0; i -= 2) {
      const uint64_t d = add_f32x2(f32x2(x[i], x[i + 1]), nm);
      const uint64_t q0 = mul_f32x2(d, rr);
      float a, b;
      f32x2_split(add_f32x2(fma_f32x2(fma_f32x2(ns, q0, d), rr, q0), magic), a, b);
      w = (w * 16u + __float_as_uint(b)) * 16u + __float_as_uint(a);
    }
    return w - 0x4b400000u * 0x11111111u;  // less the eight exponents
  }
  if (r == -1.f) {  // values past fp16
    r = sf > 0.f ? __frcp_rn(sf) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = __fsub_rn(x[i], mf);
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

// One token of four (lane 8i + c: token i): rotate, quantise and store to
// position r of `tile` (null: nothing); p is its position.
__device__ __forceinline__ void put_token(const uint4 (&raw)[5], const float *__restrict__ table, int p, float vscale,
                                          uint8_t *tile, int r, int lane) {
  const int c = lane & 7;
  // group 0: rotate.  The other half of the pair lies four lanes away;
  // products and sum are rounded one by one, so the result does not hang on
  // contraction.
  float x0[8];
  {
    float cs[16];
    const float4 *tr = reinterpret_cast<const float4 *>(table + (long long)p * 64 + 16 * (c & 3));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4 f = tr[u];
      cs[4 * u] = f.x; cs[4 * u + 1] = f.y; cs[4 * u + 2] = f.z; cs[4 * u + 3] = f.w;
    }
    uint4 o;
    o.x = __shfl_xor_sync(FULLW, raw[0].x, 4);
    o.y = __shfl_xor_sync(FULLW, raw[0].y, 4);
    o.z = __shfl_xor_sync(FULLW, raw[0].z, 4);
    o.w = __shfl_xor_sync(FULLW, raw[0].w, 4);
    const uint16_t *e = reinterpret_cast<const uint16_t *>(&raw[0]), *oe = reinterpret_cast<const uint16_t *>(&o);
    const uint32_t neg = c < 4 ? 0x80000000u : 0u;  // a - b, or a + b
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = __fmul_rn(bf2f(e[i]), cs[2 * i]), b = __fmul_rn(bf2f(oe[i]), cs[2 * i + 1]);
      x0[i] = __fadd_rn(a, __uint_as_float(__float_as_uint(b) ^ neg));
    }
  }
  // extrema of all groups, then lane g of the token's eight takes group g's
  // scale (the divisions are most of a group's cost) and hands it round
  float lo = x0[0], hi = x0[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x0[i]);
    hi = max_nan(hi, x0[i]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(FULLW, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(FULLW, hi, o));
  }
#pragma unroll
  for (int g = 1; g < 5; ++g) {
    float a, b;
    extrema_bf16(raw[g], a, b);
    lo = c == g ? a : lo;
    hi = c == g ? b : hi;
  }
  if (c >= KV4_KG) {  // the scaled values' extrema are the extrema's products (swapped under a negative scale)
    const float a = __fmul_rn(lo, vscale), b = __fmul_rn(hi, vscale);
    lo = min_nan(a, b);
    hi = max_nan(a, b);
  }
  uint32_t mysm;
  float myr;
  kv4_scale(lo, hi, mysm, myr);
  if (tile && c < 5) {  // lane c writes group c's scale and minimum
    const int q = kv4_quad(r) * 2;
    const int at_s = c < KV4_KG ? KV4_OFF_KS + c * 32 + q : KV4_OFF_VS + (c - KV4_KG) * 32 + q;
    const int at_m = c < KV4_KG ? KV4_OFF_KM + r * 8 + c * 2 : KV4_OFF_VM + (c - KV4_KG) * 32 + q;
    *reinterpret_cast<uint16_t *>(tile + at_s) = (uint16_t)mysm;
    *reinterpret_cast<uint16_t *>(tile + at_m) = (uint16_t)(mysm >> 16);
  } else if (tile && c == 5) {
    *reinterpret_cast<uint16_t *>(tile + KV4_OFF_KM + r * 8 + 6) = 0;
  }
  uint8_t *kd = tile + kv4_k_at(0, r, c >> 1) + (c & 1) * 4, *vd = tile + kv4_v_at(0, r, c, 0);
#pragma unroll
  for (int g = 0; g < 5; ++g) {
    const uint32_t sm = __shfl_sync(FULLW, mysm, (lane & 24) + g);
    const float rc = __shfl_sync(FULLW, myr, (lane & 24) + g);
    float x[8];
    const uint16_t *e = reinterpret_cast<const uint16_t *>(&raw[g]);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = g == 0 ? x0[i] : g < KV4_KG ? bf2f(e[i]) : __fmul_rn(bf2f(e[i]), vscale);
    const uint32_t w = kv4_codes(x, sm, rc);
    if (tile) {
      if (g < KV4_KG) {
        *reinterpret_cast<uint32_t *>(kd + 512 * g) = w;
      } else {
        *reinterpret_cast<uint16_t *>(vd + 512 * (g - KV4_KG)) = (uint16_t)w;
        *reinterpret_cast<uint16_t *>(vd + 512 * (g - KV4_KG) + 4) = (uint16_t)(w >> 16);
      }
    }
  }
}

__global__ void __launch_bounds__(K4A_WARPS * 32)
    kv4_append_kernel(const uint16_t *__restrict__ k, const uint16_t *__restrict__ v, const int64_t *__restrict__ pos,
                      const int32_t *__restrict__ seq, const int64_t *__restrict__ slots, int T, unsigned warps,
                      const float *__restrict__ table, int64_t max_pos, float vscale, Kv4View dst, unsigned *status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 7;
  const unsigned w = blockIdx.x * K4A_WARPS + (threadIdx.x >> 5);
  if (w >= warps) return;
  const unsigned four = w / (unsigned)dst.hkv;
  const int h = (int)(w - four * (unsigned)dst.hkv);
  const long long t = 4LL * four + (lane >> 3);
  uint4 raw[5];
#pragma unroll
  for (int g = 0; g < 5; ++g) raw[g] = make_uint4(0, 0, 0, 0);
  if (t < T) {
    const size_t item = (size_t)t * dst.hkv + h;
    const uint4 *k4 = reinterpret_cast<const uint4 *>(k) + item * (DQK / 8);
    const uint4 *v4 = reinterpret_cast<const uint4 *>(v) + item * (DV / 8);
#pragma unroll
    for (int g = 0; g < KV4_KG; ++g) raw[g] = k4[g * 8 + c];
#pragma unroll
    for (int g = 0; g < KV4_VG; ++g) raw[KV4_KG + g] = v4[g * 8 + c];
  }
  int blk, row, p;
  look_up(pos, seq, slots, t, T, max_pos, dst, h == 0 && c == 0, status, blk, row, p);
  put_token(raw, table, p, vscale, blk >= 0 ? dst.data + kv4_tile(dst, blk, h, row) : nullptr, row & 15, lane);
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t *k, const uint16_t *v, const int64_t *pos, const int32_t *seq,
                              const int64_t *slots, int T, const float *table, int64_t max_pos, float value_scale,
                              const Kv4View &dst, unsigned *status, cudaStream_t st) {
  const long long warps = ((long long)T + 3) / 4 * dst.hkv, ctas = (warps + K4A_WARPS - 1) / K4A_WARPS;
  if (warps > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(kv4_append_kernel, dim3((unsigned)ctas), dim3(K4A_WARPS * 32), 0, st, k, v, pos, seq, slots, T,
                    (unsigned)warps, table, max_pos, value_scale, dst, status);
}

}  // namespace kvr
