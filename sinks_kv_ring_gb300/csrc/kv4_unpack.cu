// kv4_unpack.cu -- positions of a 4-bit pool back to bf16, into pages or
// rows: what the prefill and varlen calls read when a sequence kept in 4 bits
// goes on.
//
// Value = m + s * u: the product is exact in fp32, the sum is rounded once to
// fp32 and once to bf16.  Entry i of the call is cu_rows[i+1] - cu_rows[i]
// positions from lo[i] on.  A work unit is one tile of 16 positions of one KV
// head, taken by one warp; entry i owns units cu_rows[i] / 16 + 2i onwards
// (an entry of n rows touches at most n / 16 + 2 tiles), so a unit finds its
// entry by a search over cu_rows and no plan is made first.  A call of more than
// K4U_ONCE CTAs goes round with fewer of them instead, and a warp stops behind
// the last entry's rows: a T far above the rows there are (all that a block
// table spans) costs neither CTAs nor searches.
//
// What bounds it: HBM, 180 bytes in and 640 out per (position, KV head), as
// long as every store fills its sectors: 122,880 positions of 4 KV heads take
// 64 us (6.3 TB/s, 0.93 of the copy rate), 70 with K stored 16 bytes at a time
// and 76 with codes converted by integer-to-float instructions.
#include "kv4.cuh"
#include "launch.h"

namespace kvr {
namespace {

constexpr int K4U_WARPS = 8;
// Going round takes 16 registers more a thread (600,002 positions of 4 KV heads:
// 293 us at once, 300 in rounds).  1000 rows of 4 KV heads: 4.6 us with T = 1000,
// 21 with T = 2^19 and 79 with 2^21 (empty CTAs), 9.5 beyond (in rounds).
constexpr int K4U_ONCE = 1 << 16;
constexpr int K4U_CTAS = 32;  // CTAs per SM of a call that goes round

// The values of a word of codes (dim i in nibble i) as bf16.  A code masked
// out of the word in place is the fp16 number u 2^-24 (or 16 u 2^-24), so the
// conversion to fp32 is the fp16 one and the power of two goes into the scale
// (exactly): s24 = s 2^24, s20 = s 2^20.
__device__ __forceinline__ uint4 kv4_word(uint32_t w, float s24, float s20, float m) {
  const uint32_t w8 = w >> 8;
  const float2 a = __half22float2(u32_as_h2(w & 0x000f000fu)), b = __half22float2(u32_as_h2(w & 0x00f000f0u));
  const float2 c = __half22float2(u32_as_h2(w8 & 0x000f000fu)), d = __half22float2(u32_as_h2(w8 & 0x00f000f0u));
  return make_uint4(pack_bf16(fmaf(a.x, s24, m), fmaf(b.x, s20, m)), pack_bf16(fmaf(c.x, s24, m), fmaf(d.x, s20, m)),
                    pack_bf16(fmaf(a.y, s24, m), fmaf(b.y, s20, m)), pack_bf16(fmaf(c.y, s24, m), fmaf(d.y, s20, m)));
}
// 32 bytes, in one store where the destination's rows are 32-byte aligned (two
// 16-byte stores of a warp each fill half of every sector they touch).
__device__ __forceinline__ void store32(uint16_t *p, const uint4 &a, const uint4 &b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = a;
    reinterpret_cast<uint4 *>(p)[1] = b;
  }
}
__device__ __forceinline__ float kv4_half(uint32_t w, int hi) {
  return __half2float(__ushort_as_half((uint16_t)(hi ? w >> 16 : w)));
}

// Unit `unit` of KV head h, by a warp.  False when it lies behind all rows of
// the call, as every later one does: the entry found does not come earlier for
// a later unit (even where cu_rows is out of order), and the last one's rows
// have ended or are none.
__device__ __forceinline__ bool unpack_unit(const Kv4View &src, const int32_t *__restrict__ src_seqs,
                                            const int64_t *__restrict__ lo, const int32_t *__restrict__ cu_rows, int n,
                                            long long T, const int32_t *__restrict__ dst_seqs, const KvView &dst,
                                            long long unit, int h, unsigned *status) {
  const int lane = threadIdx.x & 31;
  // the last entry whose first unit is not past this one
  int i = 0, hi = n;
  while (hi - i > 1) {
    const int mid = i + ((hi - i) >> 1);
    if ((long long)(cu_rows[mid] >> 4) + 2LL * mid <= unit) i = mid; else hi = mid;
  }
  const int c0 = cu_rows[i], c1 = cu_rows[i + 1];
  if (c0 < 0 || c1 < c0 || c1 > T) {
    if (lane == 0) flag(status, ST_BAD_ROWS);
    return i < n - 1;
  }
  long long a = lo[i];
  const int s = src_seqs[i];
  const bool mine = lane == 0 && h == 0;
  const long long u = unit - ((c0 >> 4) + 2LL * i);
  if (u < 0) return true;
  if (c1 == c0) return i < n - 1;
  // an entry that names no source has its rows written as zeros
  bool ok = true;
  if (a < 0 || a > (long long)src.max_blocks * src.block_size) {
    if (mine) flag(status, ST_BAD_POS);
    if (dst.kind != 3) return i < n - 1;  // (no position: no page either)
    a = 0;
    ok = false;
  }
  if (s < 0 || s >= src.num_seqs) {
    if (mine) flag(status, ST_BAD_SEQ);
    ok = false;
  }
  const long long p0 = ((a >> 4) + u) << 4;  // the first position of the unit's tile
  const long long end = a + (c1 - c0);
  if (p0 >= end) return i < n - 1;

  // (in tiles, which 32 bits hold: a sequence has at most 2^35 positions, an entry 2^31)
  const unsigned tile0 = (unsigned)(p0 >> 4), stb = (unsigned)src.block_size >> 4, sbi = tile0 / stb;
  int sblk = 0;
  if (ok) {
    sblk = sbi < (unsigned)src.max_blocks ? src.block_table[(long long)s * src.max_blocks + sbi] : -1;
    ok = sblk >= 0 && sblk < src.num_blocks;
    if (!ok && mine) flag(status, ST_BAD_BLOCK);
  }
  // destination head-row of position p0 + j: rows of a tile are `step` apart
  long long drow;
  long long step = 1;
  if (dst.kind == 3) {
    drow = ((long long)c0 + (p0 - a)) * dst.hkv + h;  // may start below the entry's first row: those positions are not written
    step = dst.hkv;
  } else {
    const int ds = dst_seqs[i];
    if (ds < 0 || ds >= dst.num_seqs) {
      if (mine) flag(status, ST_BAD_SEQ);
      return true;
    }
    const unsigned dtb = (unsigned)dst.block_size >> 4, dbi = tile0 / dtb;  // a tile lies in one block
    const int dblk = dbi < (unsigned)dst.max_blocks ? dst.block_table[(long long)ds * dst.max_blocks + dbi] : -1;
    if (dblk < 0 || dblk >= dst.num_blocks) {
      if (mine) flag(status, ST_BAD_BLOCK);
      return true;
    }
    drow = ((long long)dblk * dst.hkv + h) * dst.block_size + 16 * (tile0 - dbi * dtb);
  }

  const uint8_t *tile = src.data + (ok ? kv4_tile(src, sblk, h, (int)(16 * (tile0 - sbi * stb))) : 0);
  uint4 kc[KV4_KG], vc[KV4_VG];
#pragma unroll
  for (int g = 0; g < KV4_KG; ++g)
    kc[g] = ok ? *reinterpret_cast<const uint4 *>(tile + g * 512 + lane * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int g = 0; g < KV4_VG; ++g)
    vc[g] = ok ? *reinterpret_cast<const uint4 *>(tile + KV4_OFF_V + g * 512 + lane * 16) : make_uint4(0, 0, 0, 0);
  const int q = lane >> 2, t = lane & 3;
  const bool wide = (reinterpret_cast<uintptr_t>(dst.k) & 31u) == 0;  // (a row is 384 bytes)
  // K minima of positions q and q + 8 (three and a zero), K scales of the same
  uint2 km[2];
  uint16_t ks[2][KV4_KG];
  // V scales and minima of positions 2t, 2t + 1, 2t + 8, 2t + 9
  uint2 vs[KV4_VG], vm[KV4_VG];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int r = q + 8 * nt;
    km[nt] = ok ? *reinterpret_cast<const uint2 *>(tile + KV4_OFF_KM + r * 8) : make_uint2(0, 0);
#pragma unroll
    for (int g = 0; g < KV4_KG; ++g)
      ks[nt][g] = ok ? *reinterpret_cast<const uint16_t *>(tile + KV4_OFF_KS + (g * 16 + kv4_quad(r)) * 2) : (uint16_t)0;
  }
#pragma unroll
  for (int g = 0; g < KV4_VG; ++g) {
    vs[g] = ok ? *reinterpret_cast<const uint2 *>(tile + KV4_OFF_VS + g * 32 + t * 8) : make_uint2(0, 0);
    vm[g] = ok ? *reinterpret_cast<const uint2 *>(tile + KV4_OFF_VM + g * 32 + t * 8) : make_uint2(0, 0);
  }
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {  // K: positions q and q + 8, dims 16t .. of each group
    const int r = q + 8 * nt;
    const long long p = p0 + r;
    if (p < a || p >= end) continue;
    uint16_t *kd = dst.k + (drow + r * step) * DQK + 16 * t;
#pragma unroll
    for (int g = 0; g < KV4_KG; ++g) {
      const float sc = __half2float(__ushort_as_half(ks[nt][g])), mn = kv4_half(g == 2 ? km[nt].y : km[nt].x, g & 1);
      const float s24 = sc * 0x1p24f, s20 = sc * 0x1p20f;
      store32(kd + 64 * g, kv4_word(nt ? kc[g].z : kc[g].x, s24, s20, mn), kv4_word(nt ? kc[g].w : kc[g].y, s24, s20, mn),
              wide);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // V: positions 2t + (j & 1) + 8 (j >> 1), dims 8q .. of each group
    const int e = j & 1, nt = j >> 1, r = 8 * nt + 2 * t + e;
    const long long p = p0 + r;
    if (p < a || p >= end) continue;
    uint16_t *vd = dst.v + (drow + r * step) * DV + 8 * q;
#pragma unroll
    for (int g = 0; g < KV4_VG; ++g) {
      const float sc = kv4_half(nt ? vs[g].y : vs[g].x, e), mn = kv4_half(nt ? vm[g].y : vm[g].x, e);
      const uint32_t w0 = nt ? vc[g].z : vc[g].x, w1 = nt ? vc[g].w : vc[g].y;
      *reinterpret_cast<uint4 *>(vd + 64 * g) = kv4_word(__byte_perm(w0, w1, e ? 0x7632 : 0x5410), sc * 0x1p24f, sc * 0x1p20f, mn);
    }
  }
  return true;
}

template <bool ROUND>
__global__ void __launch_bounds__(K4U_WARPS * 32)
    kv4_unpack_kernel(Kv4View src, const int32_t *__restrict__ src_seqs, const int64_t *__restrict__ lo,
                      const int32_t *__restrict__ cu_rows, int n, long long T, const int32_t *__restrict__ dst_seqs,
                      KvView dst, long long units, unsigned *status) {
  pdl_wait();
  pdl_trigger();
  const unsigned w = blockIdx.x * K4U_WARPS + (threadIdx.x >> 5), first = w / (unsigned)src.hkv;
  int h = (int)(w - first * (unsigned)src.hkv);
  for (long long unit = first; unit < units;) {
    if (!unpack_unit(src, src_seqs, lo, cu_rows, n, T, dst_seqs, dst, unit, h, status) || !ROUND) return;
    // on by gridDim.x * K4U_WARPS (unit, head) pairs
    const unsigned step = gridDim.x * K4U_WARPS, su = step / (unsigned)src.hkv;
    unit += su;
    h += (int)(step - su * (unsigned)src.hkv);
    if (h >= src.hkv) {
      h -= src.hkv;
      ++unit;
    }
  }
}

}  // namespace

cudaError_t launch_kv4_unpack(const Kv4View &src, const int32_t *src_seqs, const int64_t *lo, const int32_t *cu_rows,
                              int n, long long T, const int32_t *dst_seqs, const KvView &dst, unsigned *status,
                              cudaStream_t st) {
  const long long units = (T >> 4) + 2LL * n;
  long long blocks = (units * src.hkv + K4U_WARPS - 1) / K4U_WARPS;  // (units < 2^33)
  if (src.hkv > (1 << 24)) return cudaErrorInvalidValue;  // (a position alone would be 3 GB)
  const bool round = blocks > K4U_ONCE;
  if (round) blocks = (long long)K4U_CTAS * num_sms();
  return launch_pdl(round ? kv4_unpack_kernel<true> : kv4_unpack_kernel<false>, dim3((unsigned)blocks),
                    dim3(K4U_WARPS * 32), 0, st, src, src_seqs, lo, cu_rows, n, T, dst_seqs, dst, units, status);
}

}  // namespace kvr
