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
// A warp takes four (token, KV head) items: lane 8i + c holds dims 8c..8c+7
// of a group of item i, five groups in turn, so the group's extrema are three
// shuffles away and a 16-byte load brings a lane's values.  All five loads
// are in flight before the destination is looked up.
#include "kv4.cuh"
#include "launch.h"

namespace kvr {
namespace {

constexpr int K4A_WARPS = 8;
constexpr int K4A_ITEMS = 4;
constexpr unsigned FULLW = 0xffffffffu;

// Codes of a lane's 8 values (dim i in nibble i) and the group's scale and
// minimum; the 8 lanes of the group call together.
__device__ __forceinline__ uint32_t kv4_quantise(const float (&x)[8], int lane, uint16_t &s16, uint16_t &m16) {
  float lo = x[0], hi = x[0], odd = 0.f;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) odd = fmaf(x[i], 0.f, odd);  // NaN when a value is infinite or NaN
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(FULLW, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(FULLW, hi, o));
  }
  const bool bad = (__ballot_sync(FULLW, odd != odd) >> (lane & 24)) & 0xffu;
  const __half m = __float2half_rd(fminf(fmaxf(lo, -65504.f), 65504.f));
  const float mf = __half2float(m);
  const __half s = __float2half_ru(fminf(__fdiv_rn(__fsub_rn(hi, mf), 15.f), 65504.f));
  const float sf = __half2float(s);
  const float r = sf > 0.f ? __frcp_rn(sf) : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fsub_rn(x[i], mf);
    const float q0 = __fmul_rn(d, r);
    const float q = fmaf(fmaf(-sf, q0, d), r, q0);
    w |= (uint32_t)__float2int_rn(fminf(fmaxf(q, 0.f), 15.f)) << (4 * i);
  }
  s16 = bad ? 0x7fff : __half_as_ushort(s);
  m16 = bad ? 0x7fff : __half_as_ushort(m);
  return bad ? 0u : w;
}

__global__ void __launch_bounds__(K4A_WARPS * 32)
    kv4_append_kernel(const uint16_t *__restrict__ k, const uint16_t *__restrict__ v, const int64_t *__restrict__ pos,
                      const int32_t *__restrict__ seq, const int64_t *__restrict__ slots, long long total,
                      const float *__restrict__ table, int64_t max_pos, float vscale, Kv4View dst, unsigned *status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 7;
  const long long item =
      ((long long)blockIdx.x * K4A_WARPS + (threadIdx.x >> 5)) * K4A_ITEMS + (lane >> 3);
  const bool have = item < total;

  uint4 raw[5];
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

  // where the item goes: the tile's first byte and the position within it
  // (every lane of the item the same; lane c = 0 flags)
  uint8_t *tile = nullptr;
  int r = 0;
  long long p = 0;
  unsigned bad = 0;
  if (have) {
    const long long t = item / dst.hkv;
    const int h = (int)(item - t * dst.hkv);
    p = pos[t];
    long long slot = -1;
    const int s = slots ? 0 : seq[t];
    if (slots) {
      slot = slots[t];
      if (slot >= (long long)dst.num_blocks * dst.block_size) {
        bad = ST_BAD_BLOCK;
        slot = -1;
      }
    }
    const bool skip = slots ? slot < 0 : s == -1;  // padding
    if (!skip && !bad) {
      if (p < 0 || p >= max_pos) {
        bad = ST_BAD_POS;
      } else if (!slots) {
        if (s < 0 || s >= dst.num_seqs) {
          bad = ST_BAD_SEQ;
        } else {
          const long long bi = p / dst.block_size;
          const int blk = bi < dst.max_blocks ? dst.block_table[(long long)s * dst.max_blocks + bi] : -1;
          if (blk < 0 || blk >= dst.num_blocks)
            bad = ST_BAD_BLOCK;
          else
            slot = (long long)blk * dst.block_size + (p - bi * dst.block_size);
        }
      }
    }
    if (bad) {
      if (c == 0 && h == 0) flag(status, bad);
    } else if (slot >= 0) {
      const int blk = (int)(slot / dst.block_size), row = (int)(slot % dst.block_size);
      tile = dst.data + kv4_tile(dst, blk, h, row);
      r = row & 15;
    }
  }
  if (!__any_sync(FULLW, tile != nullptr)) return;

  // RoPE row: frequencies 8(c & 3) .. +7
  float cs[16];
  if (tile) {
    const float4 *tr = reinterpret_cast<const float4 *>(table + p * 64 + 16 * (c & 3));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4 f = tr[u];
      cs[4 * u] = f.x; cs[4 * u + 1] = f.y; cs[4 * u + 2] = f.z; cs[4 * u + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int u = 0; u < 16; ++u) cs[u] = 0.f;
  }

#pragma unroll
  for (int g = 0; g < 5; ++g) {
    const uint16_t *e = reinterpret_cast<const uint16_t *>(&raw[g]);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bf2f(e[i]);
    if (g == 0) {
      // the other half of the rotated pair lies four lanes away; products and
      // sum are rounded one by one, so the result does not hang on contraction
      uint4 o;
      o.x = __shfl_xor_sync(FULLW, raw[0].x, 4);
      o.y = __shfl_xor_sync(FULLW, raw[0].y, 4);
      o.z = __shfl_xor_sync(FULLW, raw[0].z, 4);
      o.w = __shfl_xor_sync(FULLW, raw[0].w, 4);
      const uint16_t *oe = reinterpret_cast<const uint16_t *>(&o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = __fmul_rn(x[i], cs[2 * i]), b = __fmul_rn(bf2f(oe[i]), cs[2 * i + 1]);
        x[i] = c < 4 ? __fsub_rn(a, b) : __fadd_rn(a, b);
      }
    } else if (g >= KV4_KG) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], vscale);
    }
    uint16_t s16, m16;
    const uint32_t w = kv4_quantise(x, lane, s16, m16);
    if (tile) {
      if (g < KV4_KG) {
        *reinterpret_cast<uint32_t *>(tile + kv4_k_at(g, r, c >> 1) + (c & 1) * 4) = w;
        if (c == 0) {
          *reinterpret_cast<uint16_t *>(tile + KV4_OFF_KS + (g * 16 + kv4_quad(r)) * 2) = s16;
          if (g < 2)
            *reinterpret_cast<uint16_t *>(tile + KV4_OFF_KM + r * 8 + g * 2) = m16;
          else
            *reinterpret_cast<uint32_t *>(tile + KV4_OFF_KM + r * 8 + 4) = m16;  // and the row's zero
        }
      } else {
        const int vg = g - KV4_KG;
        *reinterpret_cast<uint16_t *>(tile + kv4_v_at(vg, r, c, 0)) = (uint16_t)w;
        *reinterpret_cast<uint16_t *>(tile + kv4_v_at(vg, r, c, 1)) = (uint16_t)(w >> 16);
        if (c == 0) {
          *reinterpret_cast<uint16_t *>(tile + KV4_OFF_VS + (vg * 16 + kv4_quad(r)) * 2) = s16;
          *reinterpret_cast<uint16_t *>(tile + KV4_OFF_VM + (vg * 16 + kv4_quad(r)) * 2) = m16;
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t *k, const uint16_t *v, const int64_t *pos, const int32_t *seq,
                              const int64_t *slots, int T, const float *table, int64_t max_pos, float value_scale,
                              const Kv4View &dst, unsigned *status, cudaStream_t st) {
  const long long items = (long long)T * dst.hkv;
  const long long per_block = (long long)K4A_WARPS * K4A_ITEMS;
  const long long blocks = (items + per_block - 1) / per_block;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(kv4_append_kernel, dim3((unsigned)blocks), dim3(K4A_WARPS * 32), 0, st, k, v, pos, seq, slots,
                    items, table, max_pos, value_scale, dst, status);
}

}  // namespace kvr
