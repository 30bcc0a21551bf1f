// kv8_unpack.cu -- positions of an 8-bit pool back to bf16, into pages or rows:
// what the prefill and varlen calls read when a sequence kept in 8 bits goes on.
//
// Value = s u: exact in fp32 (a code of 7 bits, a scale of 8), one rounding to
// bf16.  Entry i of the call is cu_rows[i+1] - cu_rows[i] positions from lo[i]
// on.  A work unit is one tile of 16 positions of one KV head, taken by one
// warp; which entry's it is comes from a search over cu_rows (chunk_of), and no
// plan is made first.  A call of more than K8U_ONCE CTAs goes round with fewer of
// them instead, and a warp stops behind the last entry's rows: a T far above the
// rows there are (all that a block table spans) costs neither CTAs nor searches
// (1000 rows of 4 KV heads: 3.6 us with T = 1000, 17 with 2^19, 7 with 2^21 or 2^23).
//
// What bounds it: HBM, 321 bytes in and 640 out per (position, KV head): 122,880
// positions of 4 KV heads take 72 us, 0.96 of the copy rate.
#include "kv8.cuh"
#include "launch.h"

namespace kvr {
namespace {

constexpr int K8U_WARPS = 8;
constexpr int K8U_ONCE = 1 << 16;
// CTAs per SM past which a warp asks ahead of the search whether its unit lies behind all rows: 1000 rows with T = 2^19 27 us
// without it, 17 with it.  A call of fewer is a wave or two, which would wait for one load more.
constexpr int K8U_MANY = 8;
constexpr int K8U_CTAS = 32;  // CTAs per SM of a call that goes round

// Values of the four codes of a word, as bf16: (byte 0, 1) and (2, 3).
__device__ __forceinline__ uint2 kv8_word(uint32_t w, float s) {
  const float2 a = __half22float2(bits_half2(kv8_pair<0>(w))), b = __half22float2(bits_half2(kv8_pair<1>(w)));
  return make_uint2(pack_bf16(a.x * s, a.y * s), pack_bf16(b.x * s, b.y * s));
}
// 32 bytes, in one store where the destination's rows are 32-byte aligned.
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

// Unit `unit`, of entry C of the call's n, and KV head h, by a warp.  False when it lies
// behind all rows of the call, as every later one does: the entry found does not
// come earlier for a later unit (even where cu_rows is out of order), and the last
// one's rows have ended or are none.
__device__ __forceinline__ bool unpack_unit(const Kv8View &src, const Chunk &C, int n, long long T,
                                            const int32_t *__restrict__ dst_seqs, const KvView &dst, long long unit, int h,
                                            unsigned *status) {
  const int lane = threadIdx.x & 31;
  const ChunkUnits units = CHUNKS_BY_TILE;
  const int i = C.i, c0 = C.c0, c1 = C.c1, s = C.seq;
  if (rows_odd(c0, c1, T)) return i < n - 1;
  long long a = C.pos;
  const bool mine = lane == 0 && h == 0;
  const long long u = unit - units.first(c0, i);
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

  const uint8_t *tile = src.data + (ok ? kv8_tile(src, sblk, h, (int)(16 * (tile0 - sbi * stb))) : 0);
  // (codes of a tile that is not there are zero: byte 128)
  const uint4 none = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
  uint4 kc[2][3], vc[4];
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int g = 0; g < 3; ++g) kc[e][g] = ok ? *reinterpret_cast<const uint4 *>(tile + g * 1024 + e * 512 + lane * 16) : none;
#pragma unroll
  for (int g = 0; g < 4; ++g) vc[g] = ok ? *reinterpret_cast<const uint4 *>(tile + KV8_OFF_V + g * 512 + lane * 16) : none;
  const uint4 tail = ok ? *reinterpret_cast<const uint4 *>(tile + KV8_OFF_TAIL) : make_uint4(0, 0, 0, 0);
  const float ks = __uint_as_float(tail.x), vs = __uint_as_float(tail.y);
  const float nan = __uint_as_float(0x7fffffffu);
  const int q = lane >> 2, t = lane & 3;
  const bool wide = (reinterpret_cast<uintptr_t>(dst.k) & 31u) == 0;  // (a row is 384 bytes)
#pragma unroll
  for (int e = 0; e < 2; ++e) {  // K: positions q and q + 8, dims 16t .. of each group of 64
    const int r = q + 8 * e;
    const long long p = p0 + r;
    if (p < a || p >= end) continue;
    const float s1 = tail.z >> r & 1 ? nan : ks;
    uint16_t *kd = dst.k + (drow + r * step) * DQK + 16 * t;
#pragma unroll
    for (int g = 0; g < 3; ++g) {
      const uint2 w0 = kv8_word(kc[e][g].x, s1), w1 = kv8_word(kc[e][g].y, s1);
      const uint2 w2 = kv8_word(kc[e][g].z, s1), w3 = kv8_word(kc[e][g].w, s1);
      store32(kd + 64 * g, make_uint4(w0.x, w0.y, w1.x, w1.y), make_uint4(w2.x, w2.y, w3.x, w3.y), wide);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // V: positions 2t + (j & 1) + 8 (j >> 1), dims 4q .. of each group of 32
    const int r = 2 * t + (j & 1) + 8 * (j >> 1);
    const long long p = p0 + r;
    if (p < a || p >= end) continue;
    const float s1 = tail.z >> (16 + r) & 1 ? nan : vs;
    uint16_t *vd = dst.v + (drow + r * step) * DV + 4 * q;
    const uint32_t sel = 0x40u + 0x11u * (uint32_t)j;  // byte j of two words
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t w = __byte_perm(__byte_perm(vc[g].x, vc[g].y, sel), __byte_perm(vc[g].z, vc[g].w, sel), 0x5410);
      *reinterpret_cast<uint2 *>(vd + 32 * g) = kv8_word(w, s1);
    }
  }
  return true;
}

template <bool ROUND>
__global__ void __launch_bounds__(K8U_WARPS * 32, ROUND ? 2 : 4)
    kv8_unpack_kernel(Kv8View src, const int32_t *__restrict__ src_seqs, const int64_t *__restrict__ lo,
                      const int32_t *__restrict__ cu_rows, int n, long long T, const int32_t *__restrict__ dst_seqs,
                      KvView dst, long long units, unsigned ctas, unsigned many, unsigned *status) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= ctas) {  // the grid's last CTAs look whether cu_rows is in order, and the others do not wait for it
    rows_check(cu_rows, n, T, blockIdx.x - ctas, gridDim.x - ctas, threadIdx.x, K8U_WARPS * 32, status);
    return;
  }
  const unsigned w = blockIdx.x * K8U_WARPS + (threadIdx.x >> 5), first = w / (unsigned)src.hkv;
  int h = (int)(w - first * (unsigned)src.hkv);
  if ((ROUND || ctas > many) && behind_chunks(cu_rows, n, CHUNKS_BY_TILE, first)) return;
  Chunk C = chunk_of(cu_rows, lo, src_seqs, n, CHUNKS_BY_TILE, first);
  for (long long unit = first; unit < units;) {
    if (!unpack_unit(src, C, n, T, dst_seqs, dst, unit, h, status) || !ROUND) return;
    // on by ctas * K8U_WARPS (unit, head) pairs
    const unsigned step = ctas * K8U_WARPS, su = step / (unsigned)src.hkv;
    unit += su;
    h += (int)(step - su * (unsigned)src.hkv);
    if (h >= src.hkv) {
      h -= src.hkv;
      ++unit;
    }
    C = chunk_of(cu_rows, lo, src_seqs, n, CHUNKS_BY_TILE, unit);
  }
}

}  // namespace

cudaError_t launch_kv8_unpack(const Kv8View &src, const int32_t *src_seqs, const int64_t *lo, const int32_t *cu_rows,
                              int n, long long T, const int32_t *dst_seqs, const KvView &dst, unsigned *status,
                              cudaStream_t st) {
  const long long units = (T >> 4) + 2LL * n;
  long long blocks = (units * src.hkv + K8U_WARPS - 1) / K8U_WARPS;  // (units < 2^33)
  if (src.hkv > (1 << 24)) return cudaErrorInvalidValue;  // (a position alone would be 5 GB)
  const bool round = blocks > K8U_ONCE;
  if (round) blocks = (long long)K8U_CTAS * num_sms();
  const long long check = ((long long)n + CHECK_CHUNKS - 1) / CHECK_CHUNKS;
  return launch_pdl(round ? kv8_unpack_kernel<true> : kv8_unpack_kernel<false>, dim3((unsigned)(blocks + check)),
                    dim3(K8U_WARPS * 32), 0, st, src, src_seqs, lo, cu_rows, n, T, dst_seqs, dst, units, (unsigned)blocks,
                    (unsigned)(K8U_MANY * num_sms()), status);
}

}  // namespace kvr
