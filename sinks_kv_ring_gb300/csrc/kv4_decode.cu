// kv4_decode.cu -- one-token decode over a full-attention layer kept in 4
// bits: split-K with a log-sum-exp merge, as the bf16 decode.
//
// Mathematics.  With values m + s u, a key's score takes its scales out of
// the product, and the values theirs:
//   score_j = sum_g s_jg (q_g . u_jg) + sum_g m_jg sum(q_g)
//   o       = sum_j (p_j s_jg) u_jg + sum_j p_j m_jg
// so the tensor cores multiply codes, and a scale costs one multiply per
// (head, key, group), not one per element.  All products are m16n8k16 f16
// with fp32 accumulators; groups of more than 8 query heads per KV head put
// the heads in the 16 rows, smaller ones in the 8 columns (SMALL, below):
//   * Codes as operands.  A code u masked out of a word in place, w &
//     0x000f000f, is the pair of fp16 numbers u 2^-24 (subnormal, exact in the
//     product), and w & 0x00f000f0 is 16 u 2^-24: two instructions give two
//     operand registers and one shift serves the next two, 5 per 8 codes, with
//     no conversion, no bias and no rounding.  The factor 16 of every other
//     dim is divided out of q beforehand (K) or of the sums afterwards (V).
//     (e4m3 operands would take 3 per 8 codes, but their m16n8k32 product runs
//     at 20 cycles here: 470 us at batch 64 where this takes 285.)
//   * Queries are rotated, scaled by softmax_scale log2(e), brought by a power
//     of two to a largest magnitude in [2^14, 2^15) per head, and rounded once
//     to fp16 (2^-11 of a value, where the bf16 decode rounds to 2^-8).
//   * The minima enter as one more k = 8 product, of the stored fp16 minima
//     with sum(q_g) in two fp16 parts, which starts the score.  The sum is stored
//     times 2^-24, below 2^-3, so the low part ends at fp16's least step: off by
//     2^-25 at most, max|q| 2^-15 of the sum, far less than the rounding of q to
//     fp16 moves the same product.
//   * Weights p 2^bias are fp16, with bias + 4 = 14 as long as the value scales
//     stay below 2 and less by the scales' exponent beyond; a group's scales that
//     are all below 2^-9 are brought up by a power of two.  So weight times scale
//     (one packed fp16 multiply) stays in range at both ends: beside scales up to
//     2^9, as a group's largest are, it is above fp16's least number for weights
//     down to 2^-26 of the largest, and what the 2^15 keys that a warp has at
//     most weigh below that is 2^-11 together.  A long flat tail keeps its mass.  Both roundings are 2^-11 of a weight, eight times finer
//     than the bf16 weights of the other decode.
//   * sum p m and sum p come out of one more product, with the two groups'
//     minima and ones as its other operand.
// The running maximum is a reference that moves (with a rescale of the sums)
// only when a score passes it by more than 4: the check is one vote per 32
// keys.
//
// Work.  Each warp streams its own 32-key units through its own ring of bulk
// copies (one copy brings two tiles' codes and scales), with no barrier
// between warps inside a piece; 12 warps an SM, three CTAs, hold the sums in
// registers.
//
// What bounds it.  180 bytes and 2 (192 + 128) G flops per key and KV head.
// Up to 8 heads: HBM (batch 64 at 32769 keys, 4 x 8 heads: 229 us, 6.60 TB/s,
// 0.97 of the copy rate).  At 16 heads the products alone take 153 us (86 of
// them per unit at 8.2 cycles an SM quarter) and every other instruction of a
// quarter about 0.75 cycles on top, as masks, loads and softmax share its
// register ports with them: 287 us (5.27 TB/s, 0.78).  Measured and left out:
// two CTAs of 255 registers (322 us), 16-key units with four CTAs (335), scores
// of one unit interleaved with the sums of the one before (323), queries held
// in registers (327).
//
// A single row at 32769 keys, 4 x 16 heads, takes 13.5 us: about 2 of launch,
// 2.5 until the first tile is there, 5 of products, 1 of joining the CTA's
// warps and 3 of merging 104 pieces a row (shares of 10 units).  The plan made before the wait for
// the kernel ahead and in the merge kernel while the split kernel ends took 1.4
// us off that and 1 to 2 off ragged batches; requesting the first tiles into L2
// before the wait changed nothing.
#include <cooperative_groups.h>

#include "kv4.cuh"
#include "line.cuh"
#include "tc_ptx.cuh"

namespace kvr {
namespace {

constexpr unsigned ST_TIMEOUT = 8u;  // KVR_DEV_TIMEOUT
constexpr int K4_WARPS = 4;
constexpr int K4_CTAS = 3;           // per SM
constexpr int K4_TILES = 2;          // tiles of a unit
constexpr int K4_UNIT = 16 * K4_TILES;
constexpr int K4_NT = 2 * K4_TILES;  // its 8-key column tiles
constexpr int K4_STAGES = 2;
constexpr int K4_STAGE = K4_TILES * KV4_TILE;
constexpr float K4_PBIAS = 10.f;     // weights are p 2^10 as long as the value scales are below 2 (times 2^14: fp16's end)
constexpr int K4_FOLD = 16;          // units between foldings of the minima's sum (1 us at batch 64; 4 units: 4 us)
constexpr float K4_SLACK = 4.f;      // how far a score may pass the reference maximum
// The work line (line.cuh) in units of K4_UNIT keys.  A row's set-up and merge,
// in units (48 ragged rows, 8 heads a group: 8 -> 49 us, 12 -> 43, 16 -> 41, 24
// -> 42; 16 heads: 59, 53, 53, 55); the least share is a unit a warp (8 and 12
// units measured the same).  The greatest: the tensor cores cut a sum off below
// its last bit at every product (2^-23 of it as measured: rows of 2^24 keys, one
// a CTA, came out 3% too large), two a unit; at 1024 units a warp that is 2^-12
// of the sum, a sixteenth of the output's half step.
struct K4Line {
  static constexpr int UNIT = K4_UNIT, ROW = 16, MIN = K4_WARPS, MOST = 1024 * K4_WARPS, CTAS = K4_CTAS;
  static constexpr bool SHARE = false;
};
// shared memory: query operands (12 steps), their group sums, row factors, barriers, abort flag, stages
constexpr int K4_OFF_QX = 12 * 512;
constexpr int K4_OFF_ROW = K4_OFF_QX + 256;
constexpr int K4_OFF_ONES = K4_OFF_ROW + 64;  // four fp16 ones, four zeros
constexpr int K4_OFF_BAR = K4_OFF_ONES + 16;
constexpr int K4_OFF_STALL = K4_OFF_BAR + 8 * K4_WARPS * K4_STAGES;  // a barrier that nothing completes (test hook)
constexpr int K4_OFF_ABORT = K4_OFF_STALL + 8;
constexpr int K4_OFF_L = (K4_OFF_ABORT + 4 + 7) / 8 * 8;
constexpr int K4_OFF_PLAN = (K4_OFF_L + 8 + 15) / 16 * 16;
constexpr int K4_PLAN_BYTES = (LINE_INLINE_MAX + 2) * 8;
constexpr int K4_OFF_STAGE = (K4_OFF_PLAN + K4_PLAN_BYTES + 127) / 128 * 128;
constexpr int K4_SMEM = K4_OFF_STAGE + K4_WARPS * K4_STAGES * K4_STAGE;
static_assert(K4_WARPS * K4_STAGES * K4_STAGE >= (K4_WARPS * 16 * (MO_STRIDE + 2) + K4_WARPS * 16 + 32 + 16 * DV) * 4,
              "merge area");
static_assert(K4_CTAS * (K4_SMEM + 1024) <= 228 * 1024, "CTAs per SM");

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};\n"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(b0));
}
// the transpose of an 8 x 8 matrix of 16-bit elements held as an MMA fragment
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint4 lds128(const uint8_t *a) { return *reinterpret_cast<const uint4 *>(a); }
__device__ __forceinline__ uint2 lds64(const uint8_t *a) { return *reinterpret_cast<const uint2 *>(a); }
__device__ __forceinline__ uint32_t lds32(const uint8_t *a) { return *reinterpret_cast<const uint32_t *>(a); }

// The query operands of one item: thread (row r, eighth c) rotates and scales
// 24 dims of head r, the row's eight threads share its power of two and its
// group sums.  Operand order: step 4g + j holds, for lane 4a + t, the halves
// of dims 64 g + 16 t + 8 (j / 2) + 2 (j % 2) + {0, 4} (registers 0, 1: rows a
// and a + 8) and + {1, 5}, divided by 16 (registers 2, 3): what masking word
// j / 2, shifted by 8 (j % 2), leaves.
struct K4Query {
  uint2 lo, hi;
  uint4 g1, g2;
  float4 t0, t1;
};
__device__ __forceinline__ K4Query kv4_query_load(const uint16_t *__restrict__ qh, int G,
                                                  const float *__restrict__ cs_row, int tid) {
  const int r = tid >> 3, c = tid & 7;
  K4Query Q = {};
  if (r < G) {
    const uint16_t *qr = qh + r * DQK;
    Q.lo = *reinterpret_cast<const uint2 *>(qr + 4 * c);
    Q.hi = *reinterpret_cast<const uint2 *>(qr + 32 + 4 * c);
    Q.g1 = *reinterpret_cast<const uint4 *>(qr + 64 + 8 * c);
    Q.g2 = *reinterpret_cast<const uint4 *>(qr + 128 + 8 * c);
    Q.t0 = *reinterpret_cast<const float4 *>(cs_row + 8 * c);
    Q.t1 = *reinterpret_cast<const float4 *>(cs_row + 8 * c + 4);
  }
  return Q;
}
__device__ __forceinline__ void kv4_query(const K4Query &Q, int G, float scale_log2, uint8_t *smem, int tid) {
  const int r = tid >> 3, c = tid & 7;
  float y[24];
#pragma unroll
  for (int i = 0; i < 24; ++i) y[i] = 0.f;
  if (r < G) {
    const float cs[8] = {Q.t0.x, Q.t0.y, Q.t0.z, Q.t0.w, Q.t1.x, Q.t1.y, Q.t1.z, Q.t1.w};
    const uint16_t *a = reinterpret_cast<const uint16_t *>(&Q.lo), *b = reinterpret_cast<const uint16_t *>(&Q.hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v1 = bf2f(a[i]), v2 = bf2f(b[i]);
      y[i] = (v1 * cs[2 * i] - v2 * cs[2 * i + 1]) * scale_log2;
      y[4 + i] = (v2 * cs[2 * i] + v1 * cs[2 * i + 1]) * scale_log2;
    }
    const uint16_t *e1 = reinterpret_cast<const uint16_t *>(&Q.g1), *e2 = reinterpret_cast<const uint16_t *>(&Q.g2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[8 + i] = bf2f(e1[i]) * scale_log2;
      y[16 + i] = bf2f(e2[i]) * scale_log2;
    }
  }
  uint32_t mx = 0;  // largest magnitude's bits (NaN and infinity above all)
#pragma unroll
  for (int i = 0; i < 24; ++i) mx = max(mx, __float_as_uint(y[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(FULLW, mx, o));
  // y 2^a has its largest magnitude in [2^14, 2^15); not finite, or zero: as it is
  const int ex = (int)(mx >> 23);
  int a = (ex == 255 || mx == 0) ? 0 : 14 + 127 - ex;
  a = a > 126 ? 126 : a;  // (values below 2^-112 stay smaller than that)
  const float up = __uint_as_float((uint32_t)(127 + (a > 0 ? a : 0)) << 23);   // 2^max(a, 0)
  const float dn = a < 0 ? __uint_as_float((uint32_t)max(127 + a, 1) << 23) : 1.f;  // 2^min(a, 0)  (a >= -113)
  float sum[3] = {0.f, 0.f, 0.f};
  __half hs[24];
#pragma unroll
  for (int i = 0; i < 24; ++i) {
    const int g = i >> 3;
    // the thread's dims of a group: for group 0 4c..4c+3 and 32+4c.., else 8c..8c+7
    const int d = g == 0 ? ((i & 4) ? 32 + 4 * c + (i & 3) : 4 * c + (i & 3)) : 8 * c + (i & 7);
    const int nib = d & 7, j = ((d >> 3) & 1) * 2 + ((nib >> 1) & 1);
    const float v = y[i] * up * dn;
    const __half h = __float2half_rn((nib & 1) ? v * 0.0625f : v);
    sum[g] += __half2float(h) * ((nib & 1) ? 16.f : 1.f);
    const int at = ((g * 4 + j) * 32 + (r & 7) * 4 + (d >> 4)) * 16 + ((nib & 1) * 2 + (r >> 3)) * 4 + (nib >> 2) * 2;
    hs[i] = h;
    if (g == 0) *reinterpret_cast<__half *>(smem + at) = h;
    else if (nib >= 4) *reinterpret_cast<__half2 *>(smem + at - 2) = __halves2half2(hs[i - 4], h);
  }
#pragma unroll
  for (int g = 0; g < 3; ++g)
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum[g] += __shfl_xor_sync(FULLW, sum[g], o);
  if (c < 4) {  // k = 2c, 2c + 1 of the minima's product: (s0, s1), (s2, 0), and the low parts of both
    __half2 w;
    const float s0 = (c & 1) ? sum[2] * 0x1p-24f : sum[0] * 0x1p-24f, s1 = (c & 1) ? 0.f : sum[1] * 0x1p-24f;
    __half h0 = __float2half_rn(s0), h1 = __float2half_rn(s1);
    if (c >= 2) {
      h0 = __float2half_rn(s0 - __half2float(h0));
      h1 = __float2half_rn(s1 - __half2float(h1));
    }
    w = __halves2half2(h0, h1);
    *reinterpret_cast<__half2 *>(smem + K4_OFF_QX + ((r & 7) * 4 + c) * 8 + (r >> 3) * 4) = w;
  }
  // a score's unit: the sums hold (y . k) 2^(a - 24)
  if (c == 0) {
    const int e = 24 - a;  // >= -102
    *reinterpret_cast<float *>(smem + K4_OFF_ROW + 4 * r) = __uint_as_float((uint32_t)min(max(127 + e, 1), 254) << 23);
  }
}

struct K4Args : LineArgs {
  const uint16_t *q;
  Kv4View pool;
  const float *table;
  float scale_log2;
  unsigned *status;
  unsigned long long stall_ns;  // test hook: warp 0's first wait is on a barrier that nothing completes (0: no stall)
  int cs;                      // DIRECT: CTAs of a row
  unsigned long long tpb_mul;  // ceil(2^36 / tiles per block): tile / tiles per block = tile * tpb_mul >> 36 (tile < 2^28)
};

// The size of the value scales, seen from both ends of fp16.  A weight times a
// scale has to stay in range: above, the weights' exponent bias gives way (the
// scales of both groups together); below, the scales of a group whose largest so
// far is under 2^-9 are multiplied by a power of two that brings it to [1, 2),
// and the group's sums count in that (a weight of 2^-17 beside a scale of 2^-18
// was below fp16's least number, and a batch's 8,000 such keys a warp, 5% of a
// row, were lost).  Both only ever move one way, as larger scales turn up.  Costs
// 0.1% at batch 64 and 16 heads, 0.4% at 8, 0.9% on 48 ragged rows.
constexpr uint32_t K4_PLAIN = 15;  // e of a group whose scales are used as they are
constexpr uint32_t K4_TINY = 6;    // fp16's exponent field of 2^-9
struct K4Scales {
  uint32_t e;     // of group 0 (low half) and 1: scales are multiplied by 2^(15 - e); 0 before the first keys
  __half2 limit;  // the largest scale that this lane's share of the check may meet
};
__device__ __forceinline__ bool kv4_plain(const K4Scales &k) { return k.e == (K4_PLAIN << 16 | K4_PLAIN); }
__device__ __forceinline__ uint32_t kv4_e(const K4Scales &k, int g) { return g ? k.e >> 16 : k.e & 0xffffu; }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// Takes in a unit's scales (`big`: this lane's two, zeros where they do not
// count; lanes 0..7 and 16..23 hold group 0's; NaN ones aside): lowers `bias`,
// updates `k`, and leaves in r[g] what group g's sums are multiplied by.
__device__ __forceinline__ void kv4_take_scales(__half2 big, int lane, float &bias, K4Scales &k, float (&r)[KV4_VG]) {
  const uint32_t lo = h2_as_u32(big) & 0xffffu, hi = h2_as_u32(big) >> 16;
  const uint32_t x = max(lo > 0x7c00u ? 0u : lo, hi > 0x7c00u ? 0u : hi);
  // exponent field of a group's largest: it is below 2^(hb - 14)
  const uint32_t hb[KV4_VG] = {__reduce_max_sync(FULLW, (lane & 8) ? 0u : x) >> 10,
                               __reduce_max_sync(FULLW, (lane & 8) ? x : 0u) >> 10};
  // the least power of two above the largest scale, times 2^(bias + slack), fits fp16
  bias = fminf(bias, 15.f - K4_SLACK - (float)((int)max(hb[0], hb[1]) - 14));
  uint32_t e[KV4_VG];
#pragma unroll
  for (int g = 0; g < KV4_VG; ++g) {
    e[g] = max(kv4_e(k, g), hb[g] < K4_TINY ? hb[g] : K4_PLAIN);
    r[g] = pow2((int)kv4_e(k, g) - (int)e[g]);
  }
  k.e = e[1] << 16 | e[0];
  const uint32_t mine = (lane & 8) ? e[1] : e[0];
  k.limit = u32_as_h2((((mine < K4_PLAIN ? mine : 25u - (uint32_t)(int)bias) << 10) + 0x3ffu) * 0x10001u);
}
// A unit's scales times their groups' powers of two (exact: the largest is below 2).
__device__ __forceinline__ void kv4_raise(uint32_t (&sv)[KV4_VG][K4_NT], const K4Scales &k) {
#pragma unroll
  for (int g = 0; g < KV4_VG; ++g) {
    const __half2 b = u32_as_h2(((30u - kv4_e(k, g)) << 10) * 0x10001u);
#pragma unroll
    for (int nt = 0; nt < K4_NT; ++nt) sv[g][nt] = h2_as_u32(__hmul2(u32_as_h2(sv[g][nt]), b));
  }
}

// SMALL: groups of up to 8 query heads.  The keys are then the 16 rows of the
// products and the heads their 8 columns (scores K Q^T, sums V^T P^T): half
// the products, and half the registers for the sums (four CTAs an SM, at 128
// registers, measured slower than three: 241 us against 230 at batch 64 and 8
// heads).
// The codes' operands are the same registers; a weight's row and column change
// places between the two products by an 8 x 8 transposition (movmatrix).
//
// FORM: the work line, a share a CTA (K4_LINE) or several (K4_TURNS: the loop
// over them costs the line 0.5%, so batches that cannot need it go without);
// or DIRECT: short contexts of few rows, where a launch costs more than the
// work.  A cluster of A.cs CTAs takes one row, each an equal share of its units,
// and the CTAs merge their parts through each other's shared memory: one
// launch, no plan and no workspace.
enum K4Form { K4_LINE, K4_TURNS, K4_DIRECT };
template <bool SMALL, K4Form FORM>
__global__ void __launch_bounds__(K4_WARPS * 32, K4_CTAS) kv4_decode_kernel(K4Args A) {
  constexpr bool DIRECT = FORM == K4_DIRECT, TURNS = FORM == K4_TURNS;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hkv = A.pool.hkv, G = A.G;
  const uint32_t sBase = smem_u32(smem);
  const uint32_t sBar = sBase + K4_OFF_BAR + 8 * K4_STAGES * warp;
  volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + K4_OFF_ABORT);
  uint8_t *const sStage = smem + K4_OFF_STAGE + warp * K4_STAGES * K4_STAGE;
  int64_t *sPrefix = reinterpret_cast<int64_t *>(smem + K4_OFF_PLAN);
  if (tid < 4) *reinterpret_cast<uint32_t *>(smem + K4_OFF_ONES + 4 * tid) = tid < 2 ? 0x3c003c00u : 0u;
  if (lane == 0) {
    for (int j = 0; j < K4_STAGES; ++j) tc::mbar_init(sBar + 8 * j, 1);
    if (warp == 0) {
      tc::mbar_init(sBase + K4_OFF_STALL, 1);
      *abort_flag = 0;
    }
    tc::fence_mbar_init();
  }
  // The plan: every CTA makes it for small batches.  For up to a sequence a
  // thread it is made before the wait for the kernel ahead, with the CTA's
  // first part, from positions and ids read early (ld_early_s32); after the
  // wait it stands if they read the same, else it is made again.
  const bool early = !DIRECT && A.B <= K4_WARPS * 32;
  const int64_t *prefix = A.B <= LINE_INLINE_MAX ? sPrefix : A.plan + LINE_PLAN;
  long long x = 0, line_end = 0, early_p = 0;
  int b = 0, kv = 0, lo = 0, hi = 0, early_s = 0;
  bool ready = DIRECT;  // b, kv, lo, hi hold the next part
  auto plan = [&](auto get, unsigned *status) {
    return line_plan<K4Line, K4_WARPS * 32>(get, A.B, hkv, A.pool.num_seqs, A.max_pos, A.max_ctx, gridDim.x, sPrefix, status);
  };
  long long *const sL = reinterpret_cast<long long *>(smem + K4_OFF_L);  // TURNS: L, for the shares after the first
  int turn = 0;                                                          // and the shares done
  auto share = [&](long long L) {
    x = blockIdx.x * L;
    line_end = min(x + L, (long long)prefix[A.B]);
    ready = x < line_end;
    if (TURNS && tid == 0) *sL = L;  // (a barrier follows each call)
    if (ready) line_part<K4Line>(prefix, A.B, hkv, line_end, x, b, kv, lo, hi);
  };
  if (early) {
    if (tid < A.B) {
      early_p = ld_early_s64(A.pos + tid);
      early_s = ld_early_s32(A.seq + tid);
    }
    share(plan([&](int, long long &p, int &s) { p = early_p, s = early_s; }, nullptr));
  }
  pdl_wait();
  pdl_trigger();
  bool same = early;
  if (early && tid < A.B) {
    const long long p = A.pos[tid];
    const int s = A.seq[tid];
    same = p == early_p && s == early_s;
    if (blockIdx.x == 0) line_units<K4Line>(p, s, A.pool.num_seqs, A.max_pos, A.max_ctx, A.status);
  }
  same = __syncthreads_and(same);
  if (!DIRECT && !same) {
    share(A.B <= LINE_INLINE_MAX
              ? plan([&](int i, long long &p, int &s) { p = A.pos[i], s = A.seq[i]; }, blockIdx.x == 0 ? A.status : nullptr)
              : A.plan[0]);
    if (TURNS) __syncthreads();  // *sL
  }

  const int tpb = A.pool.block_size >> 4;
  const int t = lane & 3, gr = lane >> 2;
  uint32_t seen = 0;  // this warp's loads waited for so far: stage seen % K4_STAGES, phase (seen / K4_STAGES) & 1
  uint32_t sent = 0;  // and issued
  bool gave_up = false;

  while (TURNS || ready || x < line_end) {
    if (TURNS && !ready && x >= line_end) {  // the share is done: the next one lies gridDim.x shares on
      const long long total = prefix[A.B];
      if (line_end >= total) break;
      const long long L = *sL;
      x = line_end + (gridDim.x - 1) * L;
      if (x >= total) break;
      line_end = min(x + L, total);
      ++turn;
    }
    int w = 0, key_lo, key_hi;
    long long p;
    if (DIRECT) {
      ready = false;
      const int row = (int)blockIdx.x / A.cs, rank = (int)blockIdx.x - row * A.cs;
      b = row / hkv;
      kv = row - b * hkv;
      p = A.pos[b];
      const int units = line_units<K4Line>(p, A.seq[b], A.pool.num_seqs, A.max_pos, A.max_ctx,
                                  kv == 0 && rank == 0 && tid == 0 ? A.status : nullptr);
      if (units == 0) {  // (so for the whole cluster)
        uint16_t *o = A.out + ((long long)b * A.hq + (long long)kv * G) * DV;
        for (int i = rank * (K4_WARPS * 32) + tid; i < G * DV; i += A.cs * (K4_WARPS * 32)) o[i] = 0;
        return;
      }
      const int each = (units + A.cs - 1) / A.cs;
      key_lo = min(rank * each, units) * K4_UNIT;
      key_hi = (int)min((long long)min((rank + 1) * each, units) * K4_UNIT, p + 1);
      if (key_hi < key_lo) key_hi = key_lo;
    } else {
      if (!ready) line_part<K4Line>(prefix, A.B, hkv, line_end, x, b, kv, lo, hi);
      ready = false;
      if (hi <= 0) continue;  // set-up alone: no piece
      w = (int)blockIdx.x + b * hkv + kv;
      if (TURNS) w += turn * (int)gridDim.x;
      p = A.pos[b];
      key_lo = lo * K4_UNIT;
      key_hi = (int)min((long long)hi * K4_UNIT, p + 1);
    }
    const int s = A.seq[b];  // (a row that gets here has a valid position and id)
    const int nunit = (key_hi - key_lo + K4_UNIT - 1) / K4_UNIT;
    const int my_n = nunit > warp ? (nunit - warp + K4_WARPS - 1) / K4_WARPS : 0;
    const int32_t *bt = A.pool.block_table + (long long)s * A.pool.max_blocks;
    const K4Query Q = kv4_query_load(A.q + ((long long)b * A.hq + (long long)kv * G) * DQK, G, A.table + p * 64, tid);
    tc::fence_proxy_async_smem();                   // the last piece's merge area lies over the stages:
    if (__syncthreads_or(*abort_flag != 0)) break;  // it is free again, its accesses ahead of the copies'

    // Units go out 32 at a time: lane l looks up unit base + l's tiles (a
    // block that is none of the pool's gives -1) and issues its copies when
    // its turn comes; `ok` has the warp's units with every tile in range.
    int ids[2];
    uint3 ok = make_uint3(0, 0, 0), next_ok = ok;  // x: whole units; y, z: units with their first, second tile
    auto fetch_ids = [&](int base) {
      const int key0 = key_lo + K4_UNIT * (warp + (base + lane) * K4_WARPS);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int key = key0 + 16 * k;
        ids[k] = -1;
        if (base + lane < my_n && key < key_hi) {
          const unsigned tile = (unsigned)key >> 4, bi = (unsigned)((tile * A.tpb_mul) >> 36);
          const int blk = bt[bi];
          if (blk >= 0 && blk < A.pool.num_blocks)
            ids[k] = (blk * hkv + kv) * tpb + (int)(tile - bi * tpb);
          else
            flag(A.status, ST_BAD_BLOCK);
        }
      }
      next_ok.x = __ballot_sync(FULLW, ids[0] >= 0 && ids[1] >= 0 && key0 + K4_UNIT <= key_hi);
      next_ok.y = __ballot_sync(FULLW, ids[0] >= 0);
      next_ok.z = __ballot_sync(FULLW, ids[1] >= 0);
    };
    auto issue = [&](int i) {
      if ((i & 31) == 0) fetch_ids(i);
      const uint32_t st = sent % K4_STAGES;
      ++sent;
      if (lane == (i & 31)) {
        const uint32_t bar = sBar + 8 * st, dst = smem_u32(sStage + st * K4_STAGE);
        if (ids[0] >= 0 && ids[1] == ids[0] + 1) {
          tc::mbar_expect_tx(bar, 2 * KV4_TILE);
          tc::bulk_load(dst, A.pool.data + (long long)ids[0] * KV4_TILE, 2 * KV4_TILE, bar);
        } else {
          int n = 0;
#pragma unroll
          for (int k = 0; k < K4_TILES; ++k) n += ids[k] >= 0;
          tc::mbar_expect_tx(bar, n * KV4_TILE);
#pragma unroll
          for (int k = 0; k < K4_TILES; ++k)
            if (ids[k] >= 0)
              tc::bulk_load(dst + k * KV4_TILE, A.pool.data + (long long)ids[k] * KV4_TILE, KV4_TILE, bar);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < K4_STAGES - 1; ++i)
      if (i < my_n) issue(i);

    kv4_query(Q, G, A.scale_log2, smem, tid);
    __syncthreads();
    int run_n = my_n;
    if (A.stall_ns && warp == 0 && !gave_up && !tc::mbar_wait(sBase + K4_OFF_STALL, 0, abort_flag, A.stall_ns)) {
      gave_up = true;
      run_n = 0;
    }
    // of a masked unit from key0 on: which of this lane's two value scales of the check count
    auto kept_of = [&](int i, int key0) {
      const int k = key0 + 16 * (lane >> 4) + 2 * ((lane & 7) >> 1) + 8 * (lane & 1);
      const bool in = ((lane >> 4 ? ok.z : ok.y) >> (i & 31)) & 1;
      return (in && k < key_hi ? 0xffffu : 0u) | (in && k + 1 < key_hi ? 0xffff0000u : 0u);
    };
    // merge area, over the stages once all warps are done with them: per warp, reference and sum per row, and numerators
    // in true units (times 2 to the bias, as the sums)
    float *mml = reinterpret_cast<float *>(smem + K4_OFF_STAGE);  // [4][16][2]
    float *mo = mml + K4_WARPS * 16 * 2;                          // [4][16][MO_STRIDE]
    if constexpr (!SMALL) {
      const float crow0 = *reinterpret_cast<const float *>(smem + K4_OFF_ROW + 4 * gr);
      const float crow1 = *reinterpret_cast<const float *>(smem + K4_OFF_ROW + 4 * (gr + 8));
      const uint2 qx = lds64(smem + K4_OFF_QX + lane * 8);

      float O[16][4], E[4];
#pragma unroll
      for (int n = 0; n < 16; ++n) O[n][0] = O[n][1] = O[n][2] = O[n][3] = 0.f;
      E[0] = E[1] = E[2] = E[3] = 0.f;
      // per row, the exponent that a weight is counted from (its maximum so far
      // less the bias); -inf, and 0 in its place, before the first keys
      float mb0 = NEG_INF, mb1 = NEG_INF, r0 = 0.f, r1 = 0.f;
      float limit = NEG_INF;                   // how large a score less r may get before the reference moves (bias + slack)
      K4Scales vs = {0u, __float2half2_rn(0.f)};

      // The sums of codes (all positive) and of minima grow together and cancel
      // in the end, while the tensor cores cut every sum off below its last bit:
      // every K4_FOLD units the minima's sum goes into the codes' (rounded to
      // nearest), so neither gets large.  Without it the output of 18,000 keys a
      // CTA was off by 0.3%, twice its rounding.
      auto fold = [&]() {
        const int src = lane & ~3;
        const float g00 = __shfl_sync(FULLW, E[0], src), g01 = __shfl_sync(FULLW, E[1], src);
        const float g10 = __shfl_sync(FULLW, E[2], src), g11 = __shfl_sync(FULLW, E[3], src);
        if (t == 0) E[0] = E[1] = E[2] = E[3] = 0.f;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float k = pow2(((n & 1) ? -5 : -9) - (int)kv4_e(vs, n >> 3)), m0 = n < 8 ? g00 : g01, m1 = n < 8 ? g10 : g11;
          O[n][0] = fmaf(m0, k, O[n][0]);
          O[n][1] = fmaf(m0, k, O[n][1]);
          O[n][2] = fmaf(m1, k, O[n][2]);
          O[n][3] = fmaf(m1, k, O[n][3]);
        }
      };
      for (int i = 0; i < run_n; ++i) {
        if ((i & 31) == 0) ok = next_ok;  // (the units of this round were looked up no later than with their first)
        if (i + K4_STAGES - 1 < my_n) issue(i + K4_STAGES - 1);
        const uint32_t st = seen % K4_STAGES;
        const bool got = __all_sync(FULLW, tc::mbar_wait(sBar + 8 * st, (seen / K4_STAGES) & 1u, abort_flag));
        if (!got) {
          gave_up = true;
          break;
        }
        ++seen;
        const uint8_t *sT = sStage + st * K4_STAGE;
        const bool whole = (ok.x >> (i & 31)) & 1;  // both tiles there, every key in range
        if (!whole && !(((ok.y | ok.z) >> (i & 31)) & 1)) continue;  // no block of the pool

        // scores
        float S[K4_NT][4];
#pragma unroll
        for (int nt = 0; nt < K4_NT; ++nt) {
          S[nt][0] = S[nt][1] = S[nt][2] = S[nt][3] = 0.f;
          mma_f16_k8(S[nt], qx.x, qx.y, lds32(sT + (nt >> 1) * KV4_TILE + KV4_OFF_KM + (gr + 8 * (nt & 1)) * 8 + (t & 1) * 4));
        }
#pragma unroll
        for (int g = 0; g < KV4_KG; ++g) {
          uint4 kw[K4_TILES];
#pragma unroll
          for (int k = 0; k < K4_TILES; ++k) kw[k] = lds128(sT + k * KV4_TILE + g * 512 + lane * 16);
          float acc[K4_NT][4];
#pragma unroll
          for (int nt = 0; nt < K4_NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 a = lds128(smem + (g * 4 + j) * 512 + lane * 16);
#pragma unroll
            for (int nt = 0; nt < K4_NT; ++nt) {
              const uint4 &kk = kw[nt >> 1];
              uint32_t x = (nt & 1) ? ((j >> 1) ? kk.w : kk.z) : ((j >> 1) ? kk.y : kk.x);
              if (j & 1) x >>= 8;
              mma_f16(acc[nt], a.x, a.y, a.z, a.w, x & 0x000f000fu, x & 0x00f000f0u);
            }
          }
#pragma unroll
          for (int h = 0; h < K4_TILES; ++h) {
            const uint2 sc = lds64(sT + h * KV4_TILE + KV4_OFF_KS + g * 32 + t * 8);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float2 f = __half22float2(u32_as_h2(n ? sc.y : sc.x));
              float(&Sn)[4] = S[2 * h + n];
              const float(&an)[4] = acc[2 * h + n];
              const uint64_t ff = f32x2(f.x, f.y);
              f32x2_split(fma_f32x2(f32x2(an[0], an[1]), ff, f32x2(Sn[0], Sn[1])), Sn[0], Sn[1]);
              f32x2_split(fma_f32x2(f32x2(an[2], an[3]), ff, f32x2(Sn[2], Sn[3])), Sn[2], Sn[3]);
            }
          }
        }
        // value scales and minima of this lane's keys (2t, 2t+1, 2t+8, 2t+9 of both tiles)
        uint32_t sv[KV4_VG][K4_NT], vm[K4_NT];
#pragma unroll
        for (int h = 0; h < K4_TILES; ++h) {
          const uint8_t *at = sT + h * KV4_TILE;
#pragma unroll
          for (int g = 0; g < KV4_VG; ++g) {
            const uint2 x = lds64(at + KV4_OFF_VS + g * 32 + t * 8);
            sv[g][2 * h] = x.x;
            sv[g][2 * h + 1] = x.y;
          }
          // columns of the sums' product: group 0's minima, group 1's, ones, nothing
          const uint2 x = lds64(gr < 2 ? at + KV4_OFF_VM + gr * 32 + t * 8 : smem + K4_OFF_ONES + (gr == 2 ? 0 : 8));
          vm[2 * h] = x.x;
          vm[2 * h + 1] = x.y;
        }
        // each lane looks at two of the unit's 64 value scales (masked ones,
        // which may be anything, left out)
        __half2 big = u32_as_h2(lds32(sT + (lane >> 4) * KV4_TILE + KV4_OFF_VS + (lane & 15) * 4));
        if (!whole) {
          // keys past the range or of a bad block: what lies there (any bits) must not be met
          const int key0 = key_lo + K4_UNIT * (warp + i * K4_WARPS);
#pragma unroll
          for (int nt = 0; nt < K4_NT; ++nt) {
            const int k = key0 + 8 * nt + 2 * t;
            const bool in = ((nt >> 1 ? ok.z : ok.y) >> (i & 31)) & 1;
            const bool v0 = in && k < key_hi, v1 = in && k + 1 < key_hi;
            if (!v0) S[nt][0] = S[nt][2] = NEG_INF;
            if (!v1) S[nt][1] = S[nt][3] = NEG_INF;
            const uint32_t keep = (v0 ? 0xffffu : 0u) | (v1 ? 0xffff0000u : 0u);
            sv[0][nt] &= keep;
            sv[1][nt] &= keep;
            vm[nt] &= keep;
          }
          big = u32_as_h2(h2_as_u32(big) & kept_of(i, key0));
        }
        // scores less the reference, base 2; does one pass it, or a value scale its bound?
        float X[K4_NT][4];
        float top0 = NEG_INF, top1 = NEG_INF;
#pragma unroll
        for (int nt = 0; nt < K4_NT; ++nt) {
          f32x2_split(fma_f32x2(f32x2(S[nt][0], S[nt][1]), f32x2(crow0, crow0), f32x2(-r0, -r0)), X[nt][0], X[nt][1]);
          f32x2_split(fma_f32x2(f32x2(S[nt][2], S[nt][3]), f32x2(crow1, crow1), f32x2(-r1, -r1)), X[nt][2], X[nt][3]);
          top0 = fmax3(top0, X[nt][0], X[nt][1]);
          top1 = fmax3(top1, X[nt][2], X[nt][3]);
        }
        const bool move = fmaxf(top0, top1) > limit || __hgt2_mask(big, vs.limit) != 0u || limit == NEG_INF;
        const bool rare = move || !kv4_plain(vs);
        // weights, taken before the vote on them is in
        uint32_t P[K4_NT][2];  // [8 keys][row gr, row gr + 8]
#pragma unroll
        for (int nt = 0; nt < K4_NT; ++nt) {
          P[nt][0] = h2_as_u32(__floats2half2_rn(ex2(X[nt][0]), ex2(X[nt][1])));
          P[nt][1] = h2_as_u32(__floats2half2_rn(ex2(X[nt][2]), ex2(X[nt][3])));
        }
        if (__any_sync(FULLW, rare)) {
          if (__any_sync(FULLW, move)) {
            // new reference per row: the larger of the old one and this unit's maximum
            float t0 = top0 + r0, t1 = top1 + r1;
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              t0 = fmaxf(t0, __shfl_xor_sync(FULLW, t0, o));
              t1 = fmaxf(t1, __shfl_xor_sync(FULLW, t1, o));
            }
            const bool fresh = limit == NEG_INF;  // the first keys: nothing to scale yet
            const float was = fresh ? K4_PBIAS : limit - K4_SLACK;
            float bias = was, rv[KV4_VG];
            kv4_take_scales(big, lane, bias, vs, rv);
            mb0 += was - bias;  // (-inf stays)
            mb1 += was - bias;
            // (a unit has a key in range: no maximum means that its scores are NaN, and the row will be)
            const float n0 = fmaxf(mb0, (t0 == NEG_INF ? 0.f : t0) - bias);
            const float n1 = fmaxf(mb1, (t1 == NEG_INF ? 0.f : t1) - bias);
            const float c0 = fresh ? 0.f : ex2(r0 - n0), c1 = fresh ? 0.f : ex2(r1 - n1);
            mb0 = r0 = n0;
            mb1 = r1 = n1;
            limit = bias + K4_SLACK;
#pragma unroll
            for (int n = 0; n < 16; ++n) {
              O[n][0] *= c0 * rv[n >> 3];
              O[n][1] *= c0 * rv[n >> 3];
              O[n][2] *= c1 * rv[n >> 3];
              O[n][3] *= c1 * rv[n >> 3];
            }
            E[0] *= c0;
            E[1] *= c0;
            E[2] *= c1;
            E[3] *= c1;
#pragma unroll
            for (int nt = 0; nt < K4_NT; ++nt) {
              X[nt][0] = fmaf(S[nt][0], crow0, -n0);
              X[nt][1] = fmaf(S[nt][1], crow0, -n0);
              X[nt][2] = fmaf(S[nt][2], crow1, -n1);
              X[nt][3] = fmaf(S[nt][3], crow1, -n1);
              P[nt][0] = h2_as_u32(__floats2half2_rn(ex2(X[nt][0]), ex2(X[nt][1])));
              P[nt][1] = h2_as_u32(__floats2half2_rn(ex2(X[nt][2]), ex2(X[nt][3])));
            }
          }
          if (!kv4_plain(vs)) kv4_raise(sv, vs);
        }
        // sums
#pragma unroll
        for (int h = 0; h < K4_TILES; ++h) {
          // (a tile that is not there has no weight, and any code is a finite operand)
          const uint8_t *at = sT + h * KV4_TILE + KV4_OFF_V;
          const uint32_t *p0 = P[2 * h], *p1 = P[2 * h + 1];
          mma_f16(E, p0[0], p0[1], p1[0], p1[1], vm[2 * h], vm[2 * h + 1]);
#pragma unroll
          for (int g = 0; g < KV4_VG; ++g) {
            const uint4 x = lds128(at + g * 512 + lane * 16);
            const __half2 s0 = u32_as_h2(sv[g][2 * h]), s1 = u32_as_h2(sv[g][2 * h + 1]);
            const uint32_t a0 = h2_as_u32(__hmul2(u32_as_h2(p0[0]), s0)), a1 = h2_as_u32(__hmul2(u32_as_h2(p0[1]), s0));
            const uint32_t a2 = h2_as_u32(__hmul2(u32_as_h2(p1[0]), s1)), a3 = h2_as_u32(__hmul2(u32_as_h2(p1[1]), s1));
#pragma unroll
            for (int ww = 0; ww < 2; ++ww) {
              uint32_t y0 = ww ? x.y : x.x, y1 = ww ? x.w : x.z;
              float(*On)[4] = &O[g * 8 + ww * 4];
              mma_f16(On[0], a0, a1, a2, a3, y0 & 0x000f000fu, y1 & 0x000f000fu);
              mma_f16(On[1], a0, a1, a2, a3, y0 & 0x00f000f0u, y1 & 0x00f000f0u);
              y0 >>= 8;
              y1 >>= 8;
              mma_f16(On[2], a0, a1, a2, a3, y0 & 0x000f000fu, y1 & 0x000f000fu);
              mma_f16(On[3], a0, a1, a2, a3, y0 & 0x00f000f0u, y1 & 0x00f000f0u);
            }
          }
        }
        __syncwarp();  // the stage is read: the next copy into it may go out
        if ((i & (K4_FOLD - 1)) == K4_FOLD - 1) fold();
      }
      __syncthreads();  // all warps done with their stages: reuse them as the merge area

      {
        const int src = lane & ~3;
        const float g00 = __shfl_sync(FULLW, E[0], src), g01 = __shfl_sync(FULLW, E[1], src);  // sum p m, groups 0, 1
        const float g10 = __shfl_sync(FULLW, E[2], src), g11 = __shfl_sync(FULLW, E[3], src);
        if (t == 1) {
          float *m = mml + warp * 32;
          m[gr * 2] = mb0;
          m[gr * 2 + 1] = E[0];
          m[(gr + 8) * 2] = mb1;
          m[(gr + 8) * 2 + 1] = E[2];
        }
        float *o = mo + warp * 16 * MO_STRIDE;
#pragma unroll
        for (int g = 0; g < KV4_VG; ++g)
#pragma unroll
          for (int ww = 0; ww < 2; ++ww)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float(*On)[4] = &O[g * 8 + ww * 4];
              const float m0 = g ? g01 : g00, m1 = g ? g11 : g10;
              const float un = pow2(9 + (int)kv4_e(vs, g)), un16 = pow2(5 + (int)kv4_e(vs, g));  // even and odd dims' units
              const int d = 64 * g + 8 * (2 * t + c) + 4 * ww;
              *reinterpret_cast<float4 *>(o + gr * MO_STRIDE + d) =
                  make_float4(fmaf(On[0][c], un, m0), fmaf(On[1][c], un16, m0), fmaf(On[2][c], un, m0), fmaf(On[3][c], un16, m0));
              *reinterpret_cast<float4 *>(o + (gr + 8) * MO_STRIDE + d) =
                  make_float4(fmaf(On[0][2 + c], un, m1), fmaf(On[1][2 + c], un16, m1), fmaf(On[2][2 + c], un, m1),
                              fmaf(On[3][2 + c], un16, m1));
            }
      }
    } else {
      // a head's column: this lane has heads 2t and 2t + 1
      const float crow0 = *reinterpret_cast<const float *>(smem + K4_OFF_ROW + 8 * t);
      const float crow1 = *reinterpret_cast<const float *>(smem + K4_OFF_ROW + 8 * t + 4);
      const uint32_t qx = lds32(smem + K4_OFF_QX + lane * 8);
      uint2 qb[12];
#pragma unroll
      for (int j = 0; j < 12; ++j) qb[j] = make_uint2(lds32(smem + j * 512 + lane * 16), lds32(smem + j * 512 + lane * 16 + 8));

      float O[8][4], E[4];  // O[4g + i]: dims 64g + 8 gr + i (rows gr) and + 4 (rows gr + 8)
#pragma unroll
      for (int n = 0; n < 8; ++n) O[n][0] = O[n][1] = O[n][2] = O[n][3] = 0.f;
      E[0] = E[1] = E[2] = E[3] = 0.f;
      float mb0 = NEG_INF, mb1 = NEG_INF, r0 = 0.f, r1 = 0.f;  // of the two heads (see the other form)
      float limit = NEG_INF;
      K4Scales vs = {0u, __float2half2_rn(0.f)};
      // which scales of a 4-position word are this lane's keys gr and gr + 8
      const uint32_t pick = (gr & 1) ? 0x7632u : 0x5410u;

      auto fold = [&]() {
        const float m00 = __shfl_sync(FULLW, E[0], t), m01 = __shfl_sync(FULLW, E[1], t);          // group 0, both heads
        const float m10 = __shfl_sync(FULLW, E[0], 4 + t), m11 = __shfl_sync(FULLW, E[1], 4 + t);  // group 1
        if (gr < 2) E[0] = E[1] = 0.f;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float k = pow2(((n & 1) ? -5 : -9) - (int)kv4_e(vs, n >> 2)), m0 = n < 4 ? m00 : m10, m1 = n < 4 ? m01 : m11;
          O[n][0] = fmaf(m0, k, O[n][0]);
          O[n][1] = fmaf(m1, k, O[n][1]);
          O[n][2] = fmaf(m0, k, O[n][2]);
          O[n][3] = fmaf(m1, k, O[n][3]);
        }
      };
      for (int i = 0; i < run_n; ++i) {
        if ((i & 31) == 0) ok = next_ok;  // (the units of this round were looked up no later than with their first)
        if (i + K4_STAGES - 1 < my_n) issue(i + K4_STAGES - 1);
        const uint32_t st = seen % K4_STAGES;
        const bool got = __all_sync(FULLW, tc::mbar_wait(sBar + 8 * st, (seen / K4_STAGES) & 1u, abort_flag));
        if (!got) {
          gave_up = true;
          break;
        }
        ++seen;
        const uint8_t *sT = sStage + st * K4_STAGE;
        const bool whole = (ok.x >> (i & 31)) & 1;  // both tiles there, every key in range
        if (!whole && !(((ok.y | ok.z) >> (i & 31)) & 1)) continue;  // no block of the pool

        // scores: rows keys gr and gr + 8 of each tile, columns heads 2t, 2t + 1
        float S[K4_TILES][4];
#pragma unroll
        for (int h = 0; h < K4_TILES; ++h) {
          const uint8_t *at = sT + h * KV4_TILE;
          S[h][0] = S[h][1] = S[h][2] = S[h][3] = 0.f;
          mma_f16_k8(S[h], lds32(at + KV4_OFF_KM + gr * 8 + (t & 1) * 4), lds32(at + KV4_OFF_KM + (gr + 8) * 8 + (t & 1) * 4), qx);
        }
#pragma unroll
        for (int g = 0; g < KV4_KG; ++g)
#pragma unroll
          for (int h = 0; h < K4_TILES; ++h) {
            const uint4 kw = lds128(sT + h * KV4_TILE + g * 512 + lane * 16);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t lo = (j >> 1) ? kw.y : kw.x, hi = (j >> 1) ? kw.w : kw.z;
              if (j & 1) {
                lo >>= 8;
                hi >>= 8;
              }
              mma_f16(acc, lo & 0x000f000fu, hi & 0x000f000fu, lo & 0x00f000f0u, hi & 0x00f000f0u, qb[g * 4 + j].x, qb[g * 4 + j].y);
            }
            const uint2 sc4 = lds64(sT + h * KV4_TILE + KV4_OFF_KS + g * 32 + (gr >> 1) * 8);
            const float2 sc = __half22float2(u32_as_h2(__byte_perm(sc4.x, sc4.y, pick)));
            S[h][0] = fmaf(acc[0], sc.x, S[h][0]);
            S[h][1] = fmaf(acc[1], sc.x, S[h][1]);
            S[h][2] = fmaf(acc[2], sc.y, S[h][2]);
            S[h][3] = fmaf(acc[3], sc.y, S[h][3]);
          }
        // value scales of keys 2t, 2t+1, 2t+8, 2t+9, and the rows of the sums' product (minima of both groups, ones)
        uint32_t sv[KV4_VG][K4_NT], vm[K4_NT];
#pragma unroll
        for (int h = 0; h < K4_TILES; ++h) {
          const uint8_t *at = sT + h * KV4_TILE;
#pragma unroll
          for (int g = 0; g < KV4_VG; ++g) {
            const uint2 x = lds64(at + KV4_OFF_VS + g * 32 + t * 8);
            sv[g][2 * h] = x.x;
            sv[g][2 * h + 1] = x.y;
          }
          const uint2 x = lds64(gr < 2 ? at + KV4_OFF_VM + gr * 32 + t * 8 : smem + K4_OFF_ONES + (gr == 2 ? 0 : 8));
          vm[2 * h] = x.x;
          vm[2 * h + 1] = x.y;
        }
        // each lane looks at two of the unit's 64 value scales (masked ones,
        // which may be anything, left out)
        __half2 big = u32_as_h2(lds32(sT + (lane >> 4) * KV4_TILE + KV4_OFF_VS + (lane & 15) * 4));
        if (!whole) {  // (see the other form)
          const int key0 = key_lo + K4_UNIT * (warp + i * K4_WARPS);
#pragma unroll
          for (int nt = 0; nt < K4_NT; ++nt) {
            const bool in = ((nt >> 1 ? ok.z : ok.y) >> (i & 31)) & 1;
            if (!in || key0 + 8 * nt + gr >= key_hi) S[nt >> 1][2 * (nt & 1)] = S[nt >> 1][2 * (nt & 1) + 1] = NEG_INF;
            const int k = key0 + 8 * nt + 2 * t;
            const uint32_t keep = (in && k < key_hi ? 0xffffu : 0u) | (in && k + 1 < key_hi ? 0xffff0000u : 0u);
            sv[0][nt] &= keep;
            sv[1][nt] &= keep;
            vm[nt] &= keep;
          }
          big = u32_as_h2(h2_as_u32(big) & kept_of(i, key0));
        }
        float top0 = NEG_INF, top1 = NEG_INF;
        float X[K4_TILES][4];
#pragma unroll
        for (int h = 0; h < K4_TILES; ++h) {
          f32x2_split(fma_f32x2(f32x2(S[h][0], S[h][1]), f32x2(crow0, crow1), f32x2(-r0, -r1)), X[h][0], X[h][1]);
          f32x2_split(fma_f32x2(f32x2(S[h][2], S[h][3]), f32x2(crow0, crow1), f32x2(-r0, -r1)), X[h][2], X[h][3]);
          top0 = fmax3(top0, X[h][0], X[h][2]);
          top1 = fmax3(top1, X[h][1], X[h][3]);
        }
        const bool move = fmaxf(top0, top1) > limit || __hgt2_mask(big, vs.limit) != 0u || limit == NEG_INF;
        const bool rare = move || !kv4_plain(vs);
        if (__any_sync(FULLW, rare)) {
          if (__any_sync(FULLW, move)) {
            float t0 = top0 + r0, t1 = top1 + r1;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              t0 = fmaxf(t0, __shfl_xor_sync(FULLW, t0, o));
              t1 = fmaxf(t1, __shfl_xor_sync(FULLW, t1, o));
            }
            const bool fresh = limit == NEG_INF;
            const float was = fresh ? K4_PBIAS : limit - K4_SLACK;
            float bias = was, rv[KV4_VG];
            kv4_take_scales(big, lane, bias, vs, rv);
            mb0 += was - bias;
            mb1 += was - bias;
            const float n0 = fmaxf(mb0, (t0 == NEG_INF ? 0.f : t0) - bias);
            const float n1 = fmaxf(mb1, (t1 == NEG_INF ? 0.f : t1) - bias);
            const float c0 = fresh ? 0.f : ex2(r0 - n0), c1 = fresh ? 0.f : ex2(r1 - n1);
            mb0 = r0 = n0;
            mb1 = r1 = n1;
            limit = bias + K4_SLACK;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              O[n][0] *= c0 * rv[n >> 2];
              O[n][1] *= c1 * rv[n >> 2];
              O[n][2] *= c0 * rv[n >> 2];
              O[n][3] *= c1 * rv[n >> 2];
            }
            E[0] *= c0;
            E[1] *= c1;
#pragma unroll
            for (int h = 0; h < K4_TILES; ++h) {
              X[h][0] = fmaf(S[h][0], crow0, -n0);
              X[h][1] = fmaf(S[h][1], crow1, -n1);
              X[h][2] = fmaf(S[h][2], crow0, -n0);
              X[h][3] = fmaf(S[h][3], crow1, -n1);
            }
          }
          if (!kv4_plain(vs)) kv4_raise(sv, vs);
        }
        // weights: row head gr, columns keys 2t, 2t + 1 (nt even: of the tile's first eight, odd: of the others)
        uint32_t P[K4_NT];
#pragma unroll
        for (int h = 0; h < K4_TILES; ++h) {
          P[2 * h] = transpose8(h2_as_u32(__floats2half2_rn(ex2(X[h][0]), ex2(X[h][1]))));
          P[2 * h + 1] = transpose8(h2_as_u32(__floats2half2_rn(ex2(X[h][2]), ex2(X[h][3]))));
        }
#pragma unroll
        for (int h = 0; h < K4_TILES; ++h) {
          const uint8_t *at = sT + h * KV4_TILE + KV4_OFF_V;
          mma_f16(E, vm[2 * h], 0u, vm[2 * h + 1], 0u, P[2 * h], P[2 * h + 1]);
#pragma unroll
          for (int g = 0; g < KV4_VG; ++g) {
            const uint4 x = lds128(at + g * 512 + lane * 16);
            const uint32_t b0 = h2_as_u32(__hmul2(u32_as_h2(P[2 * h]), u32_as_h2(sv[g][2 * h])));
            const uint32_t b1 = h2_as_u32(__hmul2(u32_as_h2(P[2 * h + 1]), u32_as_h2(sv[g][2 * h + 1])));
            mma_f16(O[4 * g], x.x & 0x000f000fu, x.y & 0x000f000fu, x.z & 0x000f000fu, x.w & 0x000f000fu, b0, b1);
            mma_f16(O[4 * g + 1], x.x & 0x00f000f0u, x.y & 0x00f000f0u, x.z & 0x00f000f0u, x.w & 0x00f000f0u, b0, b1);
            const uint32_t y0 = x.x >> 8, y1 = x.y >> 8, y2 = x.z >> 8, y3 = x.w >> 8;
            mma_f16(O[4 * g + 2], y0 & 0x000f000fu, y1 & 0x000f000fu, y2 & 0x000f000fu, y3 & 0x000f000fu, b0, b1);
            mma_f16(O[4 * g + 3], y0 & 0x00f000f0u, y1 & 0x00f000f0u, y2 & 0x00f000f0u, y3 & 0x00f000f0u, b0, b1);
          }
        }
        __syncwarp();  // the stage is read: the next copy into it may go out
        if ((i & (K4_FOLD - 1)) == K4_FOLD - 1) fold();
      }
      __syncthreads();  // all warps done with their stages: reuse them as the merge area
      {
        const float m00 = __shfl_sync(FULLW, E[0], t), m01 = __shfl_sync(FULLW, E[1], t);
        const float m10 = __shfl_sync(FULLW, E[0], 4 + t), m11 = __shfl_sync(FULLW, E[1], 4 + t);
        if (gr == 2) {  // the ones' row: sums of weights
          *reinterpret_cast<float4 *>(mml + warp * 32 + 4 * t) = make_float4(mb0, E[0], mb1, E[1]);
        }
        float *o = mo + warp * 16 * MO_STRIDE + 2 * t * MO_STRIDE + 8 * gr;
#pragma unroll
        for (int g = 0; g < KV4_VG; ++g)
#pragma unroll
          for (int ww = 0; ww < 2; ++ww)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float m = c ? (g ? m11 : m01) : (g ? m10 : m00);
              const float un = pow2(9 + (int)kv4_e(vs, g)), un16 = pow2(5 + (int)kv4_e(vs, g));
              const int e = 2 * ww + c;
              *reinterpret_cast<float4 *>(o + c * MO_STRIDE + 64 * g + 4 * ww) =
                  make_float4(fmaf(O[4 * g][e], un, m), fmaf(O[4 * g + 1][e], un16, m), fmaf(O[4 * g + 2][e], un, m),
                              fmaf(O[4 * g + 3][e], un16, m));
            }
      }
    }
    __syncthreads();
    float *fac = mo + K4_WARPS * 16 * MO_STRIDE;  // [4 warps][16 heads]
    float *own_ml = fac + K4_WARPS * 16;          // DIRECT: the CTA's merged part, [16][2] and [16][128]
    float *own_o = own_ml + 32;
    if (tid < G) {
      float M = NEG_INF;
#pragma unroll
      for (int ww = 0; ww < K4_WARPS; ++ww) M = fmaxf(M, mml[ww * 32 + tid * 2]);
      const float base = M == NEG_INF ? 0.f : M;
      float L = 0.f;
#pragma unroll
      for (int ww = 0; ww < K4_WARPS; ++ww) {
        const float mw = mml[ww * 32 + tid * 2];
        const float f = mw == NEG_INF ? 0.f : ex2(mw - base);
        fac[ww * 16 + tid] = f;
        L += mml[ww * 32 + tid * 2 + 1] * f;
      }
      float *pml = DIRECT ? own_ml : A.part_ml + (long long)w * G * 2;
      pml[tid * 2] = M;
      pml[tid * 2 + 1] = L;
    }
    __syncthreads();
    for (int idx = tid; idx < G * (DV / 4); idx += blockDim.x) {
      const int g = idx / (DV / 4), d4 = 4 * (idx % (DV / 4));
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int ww = 0; ww < K4_WARPS; ++ww) {
        const float f = fac[ww * 16 + g];
        const float4 x = *reinterpret_cast<const float4 *>(mo + (ww * 16 + g) * MO_STRIDE + d4);
        acc.x += x.x * f;
        acc.y += x.y * f;
        acc.z += x.z * f;
        acc.w += x.w * f;
      }
      *reinterpret_cast<float4 *>(DIRECT ? own_o + g * DV + d4 : A.part_o + ((long long)w * G + g) * DV + d4) = acc;
    }
    if constexpr (DIRECT) {
      cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
      const int rank = (int)cl.block_rank();
      cl.sync();
      for (int idx = rank * (K4_WARPS * 32) + tid; idx < G * (DV / 4); idx += A.cs * (K4_WARPS * 32)) {
        const int g = idx / (DV / 4), d4 = 4 * (idx % (DV / 4));
        float M = NEG_INF, S = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < A.cs; ++c) M = fmaxf(M, cl.map_shared_rank(own_ml, c)[2 * g]);
        for (int c = 0; c < A.cs; ++c) {
          const float2 ml = *reinterpret_cast<const float2 *>(cl.map_shared_rank(own_ml, c) + 2 * g);
          if (ml.x == NEG_INF) continue;
          const float f = ex2(ml.x - M);
          const float4 o = *reinterpret_cast<const float4 *>(cl.map_shared_rank(own_o, c) + g * DV + d4);
          S += ml.y * f;
          acc.x += o.x * f;
          acc.y += o.y * f;
          acc.z += o.z * f;
          acc.w += o.w * f;
        }
        const float inv = S == 0.f ? 0.f : 1.f / S;
        *reinterpret_cast<uint2 *>(A.out + ((long long)b * A.hq + (long long)kv * G + g) * DV + d4) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      }
      cl.sync();  // no CTA leaves while another reads its part
    }
  }
  if (gave_up && lane == 0) flag(A.status, ST_TIMEOUT);
  // leave no copy in flight: only a wait that gave up left any (bounded again)
  uint32_t never = 0;
  for (; seen != sent; ++seen) tc::mbar_wait(sBar + 8 * (seen % K4_STAGES), (seen / K4_STAGES) & 1u, &never);
}

// Short contexts go by clusters in one launch.  Measured at max_ctx 1024
// (one launch against the work line's two): 1 x 2 KV heads at 4 query heads
// each 5.7 us against 7.1, 16 x 4 at 16 11.1 / 13.2, 64 x 4 23.0 / 24.3, 600
// x 4 121 / 156; at 2048 8 x 4 11.3 / 12.5 but 64 x 4 38.1 / 34.4: a row then
// needs its eight CTAs.
bool one_launch(int B, int hkv, long long max_ctx) {
  const long long R = (long long)K4_CTAS * num_sms(), units = (max_ctx + K4_UNIT - 1) / K4_UNIT;
  return units <= (8LL * B * hkv <= R ? 64 : 32);
}

}  // namespace

size_t kv4_decode_workspace(int B, int hq, int hkv, long long max_ctx) {
  if (one_launch(B, hkv, max_ctx)) return 0;
  return line_workspace<K4Line>(B, hq, hkv, max_ctx);
}

cudaError_t launch_kv4_decode(const uint16_t *q, const int64_t *pos, const int32_t *seq, int B, int hq,
                              const Kv4View &pool, const float *table, int64_t max_pos, float softmax_scale,
                              long long max_ctx, void *ws, uint16_t *out, unsigned *status, cudaStream_t st) {
  const int hkv = pool.hkv, G = hq / hkv, R = K4_CTAS * num_sms();
  const long long rows = (long long)B * hkv, units = (max_ctx + K4_UNIT - 1) / K4_UNIT;
  if (rows > 0x7ffffffLL) return cudaErrorInvalidValue;  // (its queries alone would fill the GPU)
  const bool direct = one_launch(B, hkv, max_ctx);
  static void (*const kernels[2][3])(K4Args) = {
      {kv4_decode_kernel<false, K4_LINE>, kv4_decode_kernel<false, K4_TURNS>, kv4_decode_kernel<false, K4_DIRECT>},
      {kv4_decode_kernel<true, K4_LINE>, kv4_decode_kernel<true, K4_TURNS>, kv4_decode_kernel<true, K4_DIRECT>}};
  const int form = direct ? K4_DIRECT : line_turns<K4Line>(B, hkv, max_ctx) > 1 ? K4_TURNS : K4_LINE;
  void (*const kernel)(K4Args) = kernels[G <= 8][form];
  cudaError_t e = ensure_smem_limit(17 + 3 * (G <= 8) + form, (const void *)kernel, K4_SMEM, true);
  if (e != cudaSuccess) return e;
  K4Args A;
  line_args<K4Line>(A, pos, seq, B, hq, hkv, pool.num_seqs, max_pos, max_ctx, ws, out);
  A.q = q;
  A.pool = pool;
  A.table = table;
  A.scale_log2 = softmax_scale * LOG2E;
  A.status = status;
  A.stall_ns = take_stall();
  const unsigned long long tpb = (unsigned long long)(pool.block_size >> 4);
  A.tpb_mul = ((1ull << 36) + tpb - 1) / tpb;
  A.cs = 1;
  if (direct) {
    // as many CTAs a row as the longest row gives every warp a unit, as a
    // cluster may have, and as the GPU holds of all rows at once
    while (A.cs < 8 && A.cs * K4_WARPS < units && 2 * A.cs * rows <= R) A.cs *= 2;
    return launch_pdl_cluster(kernel, dim3((unsigned)(rows * A.cs)), dim3(K4_WARPS * 32), (size_t)K4_SMEM, A.cs, st, A);
  }
  return line_launch<K4Line>(kernel, K4_WARPS * 32, (size_t)K4_SMEM, A, status, st);
}

}  // namespace kvr
