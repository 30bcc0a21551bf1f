// kv8_decode.cu -- one-token decode over a full-attention layer kept in 8
// bits: split-K with a log-sum-exp merge over the work line (line.cuh), as the
// 4-bit decode.
//
// Mathematics.  With values s u, one scale s for a tile's K and one for its V,
//   score_j = ks (q . u_j),   o = sum_j (p_j vs) u_j / sum_j p_j,
// so the tensor cores multiply codes and a scale costs one multiply a tile.  All
// products are m16n8k16 f16 with fp32 accumulators; groups of more than 8 query
// heads per KV head put the heads in the 16 rows, smaller ones in the 8 columns
// (kv8_decode_kernel, below):
//   * Codes become fp16 numbers, exactly, by two instructions a pair (kv8_pair).
//   * Queries are rotated, scaled by softmax_scale log2(e), brought by a power
//     of two to a largest magnitude in [2^14, 2^15) per head, and rounded once to
//     fp16 (2^-11 of a value, where the bf16 decode rounds to 2^-8).
//   * The weights of the value product are p_j vs, taken as one power of two of
//     score + log2(vs) less a reference of its own: the largest such sum so far.
//     It is held as its distance d from the scores' reference r, and a weight's
//     exponent is (score - r) + (log2(vs) - d): no value scale is ever added to a
//     score, which may be so large (1e6 and more) that fp32 would cut the scale off.
//     Scores are rounded once, ahead of their maximum, so the largest is r exactly.
//     So a weight is at most 2^15 whatever the scales are, and one is lost to
//     fp16's least number only where it is below 2^-35 of the largest share in
//     the output, not of the largest probability: light keys with large values
//     and heavy keys with small ones both keep their part.  A weight is rounded to
//     2^-11 of itself, an eighth of the output's own rounding.
//   * sum p_j stays in fp32 beside it, under the running maximum of the scores.
// Either reference moves (with a rescale of the sums) only when a sum passes it by
// more than 4: the check is one vote a pair of tiles.
//
// Work.  Each warp streams its own tiles of 16 keys, two at a time, through its own
// ring of bulk copies (one copy brings codes and scales), with no barrier between
// warps inside a piece; 8 warps an SM, two CTAs, hold the sums in registers.
//
// What bounds it.  321 bytes and 2 (192 + 128) flops a query row per key and KV
// head.  Long contexts: HBM (batch 64 at 32769 keys, 4 KV heads: 387 to 396 us across
// GPUs, 1.0 of the copy rate, at 16 heads a group as at 8; one row of 2^20 keys 194 to
// 197 us).  With more query rows a key, a warp's own chain: 64 x 4 drafts at 32772
// keys take 567 us at 8 heads a group (32 query rows a part) and 1117 at 16 (two
// parts each), where the keys once would take 397 and the products alone 298 and 596
// (8.2 cycles each on an SM quarter); two warps a scheduler at 255 registers do not
// overlap them with the conversions and the softmax (tensor pipe 35%, issue slots
// 34%).  16 x 2 at 16384 keys and 4 heads 56 us, 99 with each row alone.  A warp needs
// about 1700 cycles for a tile at 16 query rows, 650 of them the tensor pipe's for its
// two warps; so a batch that is neither is bound by that and by the set-up of a part
// (2.4 us from the wait for the kernel ahead to the first product) and the merge: one
// row of 32769 keys, 4 x 16 heads, 14.1 us.
//
// Measured and left out (batch 64 at 32769, 16 heads, when the kernel took 401):
// query operands in registers 420, three CTAs of 168 registers without the 32-row
// form 410 (8 rows of 8192 keys: 19.8 against 21.8); the pair after the next one
// requested behind the products instead of ahead of the wait, 1% slower throughout;
// table entries, queries and RoPE rows brought into L1 ahead of the check of the
// batch, no change.
#include <cooperative_groups.h>
#include <type_traits>

#include "kv8.cuh"
#include "line.cuh"
#include "tc_ptx.cuh"

namespace kvr {
namespace {

constexpr unsigned ST_TIMEOUT = 8u;  // KVR_DEV_TIMEOUT
constexpr int K8_WARPS = 4;
constexpr int K8_CTAS = 2;           // per SM
constexpr int K8_UNIT = 16;          // keys: one tile
constexpr int K8_PAIRS = 2;           // of tiles in a warp's ring
constexpr int K8_MT = 2;
constexpr int K8_ROWS = 16 * K8_MT;  // query rows of a part: those of up to 4 batch rows of one sequence
constexpr float K8_PBIAS = 11.f;     // weights are 2^11 where they equal the reference
constexpr float K8_SLACK = 4.f;      // how far a score or weight may pass its reference
constexpr float K8_NONE = -3.402823466e38f;  // a reference before the first keys: fp32's lowest finite number, so no score is below it
constexpr float K8_FAR = -512.f;     // least distance of the weights' reference: 2^-512 of the largest probability is no fp32 number
// The work line (line.cuh) in units of one tile.  A row's set-up and merge, in units
// (48 ragged rows at 8 heads a group: 24 -> 83.9 us, 36 -> 82.8, 56 -> 83.0; at 16:
// 87.7, 89.4, 92.4; 12 x 4 drafts: 26.3, 27.2, 29.0).  The greatest share: the tensor
// cores cut a sum off below its last bit at every product (2^-23 of it as
// measured), one a tile for the values; at 2048 tiles a warp that is 2^-12 of the
// sum at most, a sixteenth of the output's half step.
struct K8Line {
  static constexpr int UNIT = K8_UNIT, ROW = 24, MIN = K8_WARPS, MOST = 2048 * K8_WARPS, CTAS = K8_CTAS;
  static constexpr bool SHARE = true;
};
// Batch rows that may go together: as many as their heads fit in K8_ROWS query rows, up to the four of a draft.
int rows_together(int G) { return K8_ROWS / G >= 4 ? 4 : K8_ROWS / G >= 2 ? 2 : 1; }
// shared memory: query operands (12 steps, twice), row factors and key counts, barriers, abort flag, plan, stages
constexpr int K8_OFF_ROW = K8_MT * 12 * 512;
constexpr int K8_OFF_KEYS = K8_OFF_ROW + 4 * K8_ROWS;
constexpr int K8_OFF_BAR = K8_OFF_KEYS + 4 * K8_ROWS;
constexpr int K8_OFF_STALL = K8_OFF_BAR + 8 * K8_WARPS * K8_PAIRS;  // a barrier that nothing completes (test hook)
constexpr int K8_OFF_ABORT = K8_OFF_STALL + 8;
constexpr int K8_OFF_L = (K8_OFF_ABORT + 4 + 7) / 8 * 8;
constexpr int K8_OFF_PLAN = (K8_OFF_L + 8 + 15) / 16 * 16;
constexpr int K8_OFF_EARLY = K8_OFF_PLAN + (LINE_INLINE_MAX + 2) * 8;  // positions and ids of a batch of up to a row a thread
constexpr int K8_OFF_INFO = K8_OFF_EARLY + K8_WARPS * 32 * 12;
constexpr int K8_OFF_STAGE = (K8_OFF_INFO + LINE_INLINE_MAX + 127) / 128 * 128;
constexpr int K8_SMEM = K8_OFF_STAGE + K8_WARPS * K8_PAIRS * 2 * KV8_TILE;
static_assert(K8_WARPS * K8_PAIRS * 2 * KV8_TILE >=
                  (K8_WARPS * 16 * (MO_STRIDE + 2) + K8_WARPS * 16 + K8_ROWS * (2 + DV)) * 4,
              "merge area");
static_assert(K8_CTAS * (K8_SMEM + 1024) <= 228 * 1024, "CTAs per SM");

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the transpose of an 8 x 8 matrix of 16-bit elements held as an MMA fragment
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint4 lds128(const uint8_t *a) { return *reinterpret_cast<const uint4 *>(a); }
__device__ __forceinline__ uint32_t lds32(const uint8_t *a) { return *reinterpret_cast<const uint32_t *>(a); }
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ float lg2(float x) {
  float y;  // (not .ftz: a tile's values may be so small that their scale is below the normal numbers)
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A score's unit: the product of a K scale and a query's, held at fp32's greatest number, so that codes of 0 under large keys
// and queries give 0 (a NaN, of a query that is not finite, stays one).
__device__ __forceinline__ float score_unit(float ks, float f) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(ks * f), "f"(3.402823466e38f));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return half2_bits(__floats2half2_rn(lo, hi)); }

// The query operands of 16 of a part's rows (row r is head r % G of batch row r / G
// of the part): thread (row, eighth c) rotates and scales 24 dims of its row, and
// the row's eight threads share its power of two.  Operand order: step 4g + w
// holds, for lane 4a + t, dims 64 g + 16 t + 4 w + {0, 1} (registers 0, 1: rows a
// and a + 8) and + {2, 3} (registers 2, 3), as word w of a lane's K codes has them.
struct K8Query {
  uint2 lo, hi;
  uint4 g1, g2;
  float4 t0, t1;
};
__device__ __forceinline__ K8Query kv8_query_load(const uint16_t *__restrict__ qr, const float *__restrict__ cs_row, int c,
                                                  bool have) {
  K8Query Q = {};
  if (have) {
    Q.lo = *reinterpret_cast<const uint2 *>(qr + 4 * c);
    Q.hi = *reinterpret_cast<const uint2 *>(qr + 32 + 4 * c);
    Q.g1 = *reinterpret_cast<const uint4 *>(qr + 64 + 8 * c);
    Q.g2 = *reinterpret_cast<const uint4 *>(qr + 128 + 8 * c);
    Q.t0 = *reinterpret_cast<const float4 *>(cs_row + 8 * c);
    Q.t1 = *reinterpret_cast<const float4 *>(cs_row + 8 * c + 4);
  }
  return Q;
}
// (Q is all zeros for a row that is not there); ops, factor: the 16 rows' operands and row factors
__device__ __forceinline__ void kv8_query(const K8Query &Q, float scale_log2, uint8_t *ops, float *factor, int tid) {
  const int r = tid >> 3, c = tid & 7;
  float y[24];
  {
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
  // y 2^a has its largest magnitude in [2^14, 2^15); zero: as it is
  const int ex = (int)(mx >> 23);
  int a = mx == 0 ? 0 : 14 + 127 - ex;
  a = a > 126 ? 126 : a;  // (values below 2^-112 stay smaller than that)
  const float up = __uint_as_float((uint32_t)(127 + (a > 0 ? a : 0)) << 23);        // 2^max(a, 0)
  const float dn = a < 0 ? __uint_as_float((uint32_t)max(127 + a, 1) << 23) : 1.f;  // 2^min(a, 0)  (a >= -114)
#pragma unroll
  for (int i = 0; i < 24; i += 4) {  // four neighbouring dims
    const int g = i >> 3;
    const int d = g == 0 ? ((i & 4) ? 32 + 4 * c : 4 * c) : 8 * c + (i & 7);
    const int at = ((g * 4 + (d >> 2 & 3)) * 32 + (r & 7) * 4 + (d >> 4)) * 16 + (r >> 3) * 4;
    *reinterpret_cast<uint32_t *>(ops + at) = pack_h2(y[i] * up * dn, y[i + 1] * up * dn);
    *reinterpret_cast<uint32_t *>(ops + at + 8) = pack_h2(y[i + 2] * up * dn, y[i + 3] * up * dn);
  }
  // a score's unit per K scale: the sums hold (y . u) 2^a.  A query that is not finite has none: its row is NaN
  if (c == 0)
    factor[r] = mx >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)min(max(127 - a, 1), 254) << 23);
}

struct K8Args : LineArgs {
  const uint16_t *q;
  Kv8View pool;
  const float *table;
  float scale_log2;
  unsigned *status;
  unsigned long long stall_ns;  // test hook: warp 0's first wait is on a barrier that nothing completes (0: no stall)
  int cs;                       // DIRECT: CTAs of a row
  uint32_t g_mul;               // ceil(2^16 / G): r / G = r * g_mul >> 16 (r < 32)
  unsigned long long tpb_mul;   // ceil(2^36 / tiles per block): tile / tiles per block = tile * tpb_mul >> 36 (tile < 2^28)
};

// A part's query rows are the G heads of a batch row, or of up to rmax of them that
// share a sequence.  Up to 8 rows: the keys are the 16 rows of the products and the
// query rows their 8 columns (scores K Q^T, sums V^T P^T): half the products of the
// other form, and a quarter of the registers for the sums; the codes' operands are
// the same registers, and a weight's row and column change places between the two
// products by an 8 x 8 transposition (movmatrix).  Up to 16, or 32: the query rows
// are the rows of one, or two, products, and a tile's codes are converted once for
// both.
//
// FORM: the work line, a share a CTA (K8_LINE) or several (K8_TURNS); or DIRECT:
// short contexts of few rows, where a launch costs more than the work.  A cluster
// of A.cs CTAs takes one row, each an equal share of its units, and the CTAs
// merge their parts through each other's shared memory: one launch, no plan and
// no workspace.
enum K8Form { K8_LINE, K8_TURNS, K8_DIRECT };
template <K8Form FORM>
__global__ void __launch_bounds__(K8_WARPS * 32, K8_CTAS) kv8_decode_kernel(K8Args A) {
  constexpr bool DIRECT = FORM == K8_DIRECT, TURNS = FORM == K8_TURNS;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hkv = A.hkv, G = A.G;
  const uint32_t sBase = smem_u32(smem);
  const uint32_t sBar = sBase + K8_OFF_BAR + 8 * K8_PAIRS * warp;
  volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + K8_OFF_ABORT);
  uint8_t *const sStage = smem + K8_OFF_STAGE + warp * K8_PAIRS * 2 * KV8_TILE;
  int64_t *sPrefix = reinterpret_cast<int64_t *>(smem + K8_OFF_PLAN);
  if (lane == 0) {
    for (int j = 0; j < K8_PAIRS; ++j) tc::mbar_init(sBar + 8 * j, 1);
    if (warp == 0) {
      tc::mbar_init(sBase + K8_OFF_STALL, 1);
      *abort_flag = 0;
    }
    tc::fence_mbar_init();
  }
  // The plan: every CTA makes it for small batches.  For up to a sequence a
  // thread it is made before the wait for the kernel ahead, with the CTA's
  // first part, from positions and ids read early (ld_early_s32); after the
  // wait it stands if they read the same, else it is made again.
  const bool early = !DIRECT && A.B <= K8_WARPS * 32;
  const int64_t *prefix = A.B <= LINE_INLINE_MAX ? sPrefix : A.plan + LINE_PLAN;
  const uint8_t *info = A.B <= LINE_INLINE_MAX ? smem + K8_OFF_INFO : reinterpret_cast<uint8_t *>(A.plan + LINE_PLAN + A.B + 1);
  long long x = 0, line_end = 0, early_p = 0;
  int b = 0, kv = 0, lo = 0, hi = 0, early_s = 0;
  bool ready = DIRECT;  // b, kv, lo, hi hold the next part
  auto plan = [&](auto get, unsigned *status) {
    return line_plan<K8Line, K8_WARPS * 32>(get, A.B, hkv, A.num_seqs, A.max_pos, A.max_ctx, gridDim.x, sPrefix, status,
                                               A.rmax, smem + K8_OFF_INFO);
  };
  long long *const sL = reinterpret_cast<long long *>(smem + K8_OFF_L);  // TURNS: L, for the shares after the first
  int turn = 0;                                                          // and the shares done
  auto share = [&](long long L) {
    x = blockIdx.x * L;
    line_end = min(x + L, (long long)prefix[A.B]);
    ready = x < line_end;
    if (TURNS && tid == 0) *sL = L;  // (a barrier follows each call)
    if (ready) line_part<K8Line>(prefix, A.B, hkv, line_end, x, b, kv, lo, hi);
  };
  int64_t *const sPos = reinterpret_cast<int64_t *>(smem + K8_OFF_EARLY);
  int32_t *const sSeq = reinterpret_cast<int32_t *>(smem + K8_OFF_EARLY + K8_WARPS * 32 * 8);
  if (early) {
    if (tid < A.B) {
      sPos[tid] = early_p = ld_early_s64(A.pos + tid);
      sSeq[tid] = early_s = ld_early_s32(A.seq + tid);
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
    if (blockIdx.x == 0) line_units<K8Line>(p, s, A.num_seqs, A.max_pos, A.max_ctx, A.status);
  }
  same = __syncthreads_and(same);
  if (!DIRECT && !same) {
    share(A.B <= LINE_INLINE_MAX
              ? plan([&](int i, long long &p, int &s) { p = A.pos[i], s = A.seq[i]; }, blockIdx.x == 0 ? A.status : nullptr)
              : A.plan[0]);
    if (TURNS) __syncthreads();  // *sL
  }

  int *const sKeys = reinterpret_cast<int *>(smem + K8_OFF_KEYS);
  const int tpb = A.pool.block_size >> 4;
  const int t = lane & 3, gr = lane >> 2;
  uint32_t seen = 0;  // this warp's pairs waited for so far: slot seen % K8_PAIRS, phase (seen / K8_PAIRS) & 1
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
    long long w = 0;                  // the piece's first partial row
    int key_lo, key_hi, rows;         // rows: of the batch, from b on
    long long at[4], top = -1;        // their positions, and the largest
    auto positions = [&]() {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        at[c] = c < rows ? (same ? sPos[b + c] : A.pos[b + c]) : -1;
        top = max(top, at[c]);
      }
    };
    if (DIRECT) {
      ready = false;
      const int row = (int)blockIdx.x / A.cs, rank = (int)blockIdx.x - row * A.cs;
      b = row / hkv;
      kv = row - b * hkv;
      // the rows that go together (as the plan has it), by every warp
      const int base = b & ~(A.rmax - 1), in = b - base;
      long long pl = -1;
      int sl = -1;
      if (lane < A.rmax && base + lane < A.B) pl = A.pos[base + lane], sl = A.seq[base + lane];
      const bool say = kv == 0 && rank == 0 && warp == 0 && lane == in;
      const int mine = line_units<K8Line>(pl, sl, A.num_seqs, A.max_pos, A.max_ctx, say ? A.status : nullptr);
      const uint8_t told = line_info(line_joined(mine > 0, sl, lane, A.rmax), in);
      if (__shfl_sync(FULLW, mine, in) == 0) {  // (so for the whole cluster)
        uint16_t *o = A.out + ((long long)b * A.hq + (long long)kv * G) * DV;
        for (int i = rank * (K8_WARPS * 32) + tid; i < G * DV; i += A.cs * (K8_WARPS * 32)) o[i] = 0;
        return;
      }
      if (line_lead(told)) return;  // (the whole cluster: the row's leader has one)
      rows = line_rows(told);
      positions();
      const int units = (int)((top + K8_UNIT) / K8_UNIT), each = (units + A.cs - 1) / A.cs;
      key_lo = min(rank * each, units) * K8_UNIT;
      key_hi = (int)min((long long)min((rank + 1) * each, units) * K8_UNIT, top + 1);
      if (key_hi < key_lo) key_hi = key_lo;
    } else {
      if (!ready) line_part<K8Line>(prefix, A.B, hkv, line_end, x, b, kv, lo, hi);
      ready = false;
      if (hi <= 0) continue;  // set-up alone: no piece
      rows = line_rows(info[b]);
      w = line_at(A, (int)blockIdx.x + (TURNS ? turn * (int)gridDim.x : 0), b, kv, rows);
      positions();
      key_lo = lo * K8_UNIT;
      key_hi = (int)min((long long)hi * K8_UNIT, top + 1);
    }
    const int s = same ? sSeq[b] : A.seq[b];  // (a row that gets here has a valid position and id)
    const int nunit = (key_hi - key_lo + K8_UNIT - 1) / K8_UNIT;
    const int my_n = nunit > warp ? (nunit - warp + K8_WARPS - 1) / K8_WARPS : 0;
    const int32_t *bt = A.pool.block_table + (long long)s * A.pool.max_blocks;
    const int nq = rows * G;  // query rows
    K8Query Q[K8_MT];
#pragma unroll
    for (int m = 0; m < K8_MT; ++m) {
      const int r = 16 * m + (tid >> 3), c = (int)((uint32_t)r * A.g_mul >> 16);
      const bool have = r < nq;
      const long long pr = c == 0 ? at[0] : c == 1 ? at[1] : c == 2 ? at[2] : at[3];
      if (m == 0 || nq > 16)
        Q[m] = kv8_query_load(A.q + ((long long)(b + c) * A.hq + (long long)kv * G + (r - c * G)) * DQK, A.table + pr * 64,
                              tid & 7, have);
      if ((tid & 7) == 0 && have) sKeys[r] = (int)pr + 1;  // keys that the row may see
    }
    tc::fence_proxy_async_smem();                   // the last piece's merge area lies over the stages:
    if (__syncthreads_or(*abort_flag != 0)) break;  // it is free again, its accesses ahead of the copies'

    // Units go two at a time, for their latencies' sake: one barrier and one wait a pair.  They are looked up 32 at a
    // time: lane l has unit base + l's tile (a block that is none of the pool's gives -1) and issues its copy when the
    // pair's turn comes; `ok` has the warp's units that lie in the pool.
    int id = -1;
    uint32_t ok = 0, next_ok = 0;
    auto fetch_ids = [&](int base) {
      const int key = key_lo + K8_UNIT * (warp + (base + lane) * K8_WARPS);
      id = -1;
      if (base + lane < my_n) {
        const unsigned tile = (unsigned)key >> 4, bi = (unsigned)((tile * A.tpb_mul) >> 36);
        const int blk = bt[bi];
        if (blk >= 0 && blk < A.pool.num_blocks)
          id = (blk * hkv + kv) * tpb + (int)(tile - bi * tpb);
        else
          flag(A.status, ST_BAD_BLOCK);
      }
      next_ok = __ballot_sync(FULLW, id >= 0);
    };
    auto issue = [&](int i) {  // units i (even) and i + 1
      if ((i & 31) == 0) fetch_ids(i);
      const uint32_t slot = sent % K8_PAIRS, bar = sBar + 8 * slot;
      ++sent;
      if ((lane ^ i) & 30) return;
      if (!(lane & 1)) tc::mbar_expect_tx(bar, __popc(next_ok >> (i & 31) & 3u) * KV8_TILE);
      if (id >= 0)
        tc::bulk_load(smem_u32(sStage + (2 * slot + (lane & 1)) * KV8_TILE), A.pool.data + (long long)id * KV8_TILE, KV8_TILE,
                      bar);
    };
#pragma unroll
    for (int i = 0; i < K8_PAIRS - 1; ++i)
      if (2 * i < my_n) issue(2 * i);

    kv8_query(Q[0], A.scale_log2, smem, reinterpret_cast<float *>(smem + K8_OFF_ROW), tid);
    if (nq > 16) kv8_query(Q[K8_MT - 1], A.scale_log2, smem + 12 * 512, reinterpret_cast<float *>(smem + K8_OFF_ROW) + 16, tid);
    __syncthreads();
    int run_n = my_n;
    if (A.stall_ns && warp == 0 && !gave_up && !tc::mbar_wait(sBase + K8_OFF_STALL, 0, abort_flag, A.stall_ns)) {
      gave_up = true;
      run_n = 0;
    }
    // Waits for units i (even) and i + 1, with the next pair on its way; null where a unit is none or has no block of the
    // pool.  False: not in time.
    auto next_tiles = [&](int i, const uint8_t *(&T)[2]) {
      if ((i & 31) == 0) ok = next_ok;  // (the units of this round were looked up no later than with their first)
      if (i + 2 * (K8_PAIRS - 1) < my_n) issue(i + 2 * (K8_PAIRS - 1));
      const uint32_t slot = seen % K8_PAIRS;
      if (!__all_sync(FULLW, tc::mbar_wait(sBar + 8 * slot, (seen / K8_PAIRS) & 1u, abort_flag))) {
        gave_up = true;
        return false;
      }
      ++seen;
#pragma unroll
      for (int u = 0; u < 2; ++u) T[u] = ok >> ((i + u) & 31) & 1 ? sStage + (2 * slot + u) * KV8_TILE : nullptr;
      return true;
    };
    // the units in turn: step(n, tiles, their first keys) takes one or two of them
    auto units = [&](auto both, auto step) {
      for (int i = 0; i < run_n; i += 2) {
        const uint8_t *T[2];
        if (!next_tiles(i, T)) break;
        const int key0 = key_lo + K8_UNIT * (warp + i * K8_WARPS), key1 = key0 + K8_UNIT * K8_WARPS;
        if (decltype(both)::value && T[0] && T[1]) {
          const uint8_t *const two[2] = {T[0], T[1]};
          const int keys[2] = {key0, key1};
          step(std::integral_constant<int, 2>(), two, keys);
        } else {
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {
            const uint8_t *const one[1] = {u ? T[1] : T[0]};
            const int keys[1] = {u ? key1 : key0};
            if (one[0]) step(std::integral_constant<int, 1>(), one, keys);
          }
        }
        __syncwarp();  // the slot is read: the next pair into it may go out
      }
    };
    // merge area, over the stages once all warps are done with them: per warp, reference and sum per row, and numerators,
    // of 16 rows at a time; behind it the CTA's merged part of all rows (DIRECT)
    float *mml = reinterpret_cast<float *>(smem + K8_OFF_STAGE);  // [4][16][2]
    float *mo = mml + K8_WARPS * 16 * 2;                          // [4][16][MO_STRIDE]
    float *fac = mo + K8_WARPS * 16 * MO_STRIDE;                  // [4 warps][16]
    float *own_ml = fac + K8_WARPS * 16;                          // [32][2]
    float *own_o = own_ml + 2 * K8_ROWS;                          // [32][128]
    // the CTA's four parts of rows 16 m .. joined
    auto join = [&](int m) {
      __syncthreads();
      const int n = min(nq - 16 * m, 16);
      if (tid < n) {
        float M = NEG_INF;
#pragma unroll
        for (int ww = 0; ww < K8_WARPS; ++ww) M = fmaxf(M, mml[ww * 32 + tid * 2]);
        const float base = M == NEG_INF ? 0.f : M;
        float L = 0.f;
#pragma unroll
        for (int ww = 0; ww < K8_WARPS; ++ww) {
          const float mw = mml[ww * 32 + tid * 2];
          const float f = mw == NEG_INF ? 0.f : ex2(mw - base);
          fac[ww * 16 + tid] = f;
          L += mml[ww * 32 + tid * 2 + 1] * f;
        }
        float *pml = DIRECT ? own_ml + 32 * m : A.part_ml + (w + 16 * m) * 2;
        pml[tid * 2] = M;
        pml[tid * 2 + 1] = L;
      }
      __syncthreads();
      float *po = DIRECT ? own_o + 16 * m * DV : A.part_o + (w + 16 * m) * DV;
      for (int idx = tid; idx < n * (DV / 4); idx += blockDim.x) {
        const int g = idx / (DV / 4), d4 = 4 * (idx % (DV / 4));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int ww = 0; ww < K8_WARPS; ++ww) {
          const float f = fac[ww * 16 + g];
          const float4 x = *reinterpret_cast<const float4 *>(mo + (ww * 16 + g) * MO_STRIDE + d4);
          acc.x += x.x * f;
          acc.y += x.y * f;
          acc.z += x.z * f;
          acc.w += x.w * f;
        }
        *reinterpret_cast<float4 *>(po + g * DV + d4) = acc;
      }
    };
    // A warp's reference of a row for the merge: none (-inf) where it saw no key of the row's.  (The largest key adds 1 to
    // the sum; where no score is a number the sum is none either, and makes the row's one, whatever the reference is.)
    auto ref = [](float r, float l) { return l == 0.f ? NEG_INF : r; };
    const float *sFac = reinterpret_cast<const float *>(smem + K8_OFF_ROW);

    // MT x 16 query rows as rows of the products; this lane has rows gr and gr + 8 (index e) of each
    auto wide = [&](auto mt) {
      constexpr int MT = decltype(mt)::value;
      float f[MT][2], O[MT][16][4];              // O[m][4g + i]: dims 32 g + 4 c + i of column c
      float rr[MT][2], dd[MT][2], ll[MT][2];     // the scores' reference, how far from it the weights' (less the bias) is; sums
      int keys[MT][2], least = 0x7fffffff;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int n = 0; n < 16; ++n) O[m][n][0] = O[m][n][1] = O[m][n][2] = O[m][n][3] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * m + gr + 8 * e;
          f[m][e] = sFac[r];
          keys[m][e] = r < nq ? sKeys[r] : 0x7fffffff;
          least = min(least, keys[m][e]);
          rr[m][e] = K8_NONE;
          dd[m][e] = K8_FAR;
          ll[m][e] = 0.f;
        }
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) least = min(least, __shfl_xor_sync(FULLW, least, o));
      least = min(least, key_hi);  // keys that every row sees
      units(std::integral_constant<bool, MT == 1>(), [&](auto nb, auto &T, auto &key0) {
        constexpr int NB = decltype(nb)::value;
        // scores: columns keys 2t, 2t + 1 (nt = 0) and + 8; where there is but one chain of products for each, two sums
        constexpr bool SPLIT = MT == 1 && NB == 1;
        float S[NB][MT][2][4], S2[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) S[n][m][nt][0] = S[n][m][nt][1] = S[n][m][nt][2] = S[n][m][nt][3] = 0.f;
          S2[nt][0] = S2[nt][1] = S2[nt][2] = S2[nt][3] = 0.f;
        }
#pragma unroll
        for (int g = 0; g < 3; ++g) {
          uint4 ka[NB], kb[NB];
#pragma unroll
          for (int n = 0; n < NB; ++n) ka[n] = lds128(T[n] + g * 1024 + lane * 16), kb[n] = lds128(T[n] + g * 1024 + 512 + lane * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 q[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) q[m] = lds128(smem + m * 12 * 512 + (g * 4 + j) * 512 + lane * 16);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              const uint32_t a0 = kv8_pair<0>(word(ka[n], j)), a1 = kv8_pair<1>(word(ka[n], j));
              const uint32_t b0 = kv8_pair<0>(word(kb[n], j)), b1 = kv8_pair<1>(word(kb[n], j));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma_f16(SPLIT && (j & 1) ? S2[0] : S[n][m][0], q[m].x, q[m].y, q[m].z, q[m].w, a0, a1);
                mma_f16(SPLIT && (j & 1) ? S2[1] : S[n][m][1], q[m].x, q[m].y, q[m].z, q[m].w, b0, b1);
              }
            }
          }
        }
        if (SPLIT) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int u = 0; u < 4; ++u) S[0][0][nt][u] += S2[nt][u];
        }
        uint4 tail[NB];
        float lv[NB], top[NB][MT][2];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          tail[n] = lds128(T[n] + KV8_OFF_TAIL);
          const float ks = __uint_as_float(tail[n].x);
          lv[n] = lg2(__uint_as_float(tail[n].y));  // -inf for a scale of 0: no weight
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float fs = score_unit(ks, f[m][e]);
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                float(&x)[4] = S[n][m][nt];
                f32x2_split(mul_f32x2(f32x2(x[2 * e], x[2 * e + 1]), f32x2(fs, fs)), x[2 * e], x[2 * e + 1]);
              }
            }
          if (!(key0[n] + 16 <= least && tail[n].z == 0)) {  // not every row sees all 16 keys, or some K row is not finite
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const int k = 8 * (u >> 1) + 2 * t + (u & 1);
                  float &x = S[n][m][u >> 1][2 * e + (u & 1)];
                  if (key0[n] + k >= min(keys[m][e], key_hi)) x = NEG_INF;
                  else if (tail[n].z >> k & 1) x = __uint_as_float(0x7fffffffu);
                }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float(&x)[2][4] = S[n][m];
              top[n][m][e] = fmaxf(fmax3(x[0][2 * e], x[0][2 * e + 1], x[1][2 * e]), x[1][2 * e + 1]);
              const float by = top[n][m][e] - rr[m][e];
              move |= by > K8_SLACK || (lv[n] - dd[m][e]) + by > K8_SLACK + K8_PBIAS;
            }
        }
        if (__any_sync(FULLW, move)) {
          // new references per row: the larger of the old one and these tiles' maximum
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float r = rr[m][e], x[NB];
#pragma unroll
              for (int n = 0; n < NB; ++n) {
                x[n] = top[n][m][e];
                x[n] = fmaxf(x[n], __shfl_xor_sync(FULLW, x[n], 1));
                x[n] = fmaxf(x[n], __shfl_xor_sync(FULLW, x[n], 2));
                r = fmaxf(r, x[n]);
              }
              const float by = rr[m][e] - r;
              float d = fmaxf(dd[m][e] + by, K8_FAR);
#pragma unroll
              for (int n = 0; n < NB; ++n) d = fmaxf(d, (x[n] - r) + lv[n] - K8_PBIAS);
              const float c = ex2((dd[m][e] - d) + by);
              ll[m][e] *= ex2(by);
              rr[m][e] = r;
              dd[m][e] = d;
#pragma unroll
              for (int d = 0; d < 16; ++d) {
                O[m][d][2 * e] *= c;
                O[m][d][2 * e + 1] *= c;
              }
            }
        }
        uint32_t P[NB][MT][2][2];  // weights [8 keys][row gr, row gr + 8]
        bool far = false;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // a weight is exp2(score - r) times exp2 of this; where it is within 2^64 either way, a product that underflows
              // is below fp16's least number all the same
              const float h = lv[n] - dd[m][e], w = ex2(h);
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                float &x = S[n][m][nt][2 * e], &y = S[n][m][nt][2 * e + 1];
                f32x2_split(add_f32x2(f32x2(x, y), f32x2(-rr[m][e], -rr[m][e])), x, y);
                const float a = ex2(x), b = ex2(y);
                ll[m][e] += a + b;
                P[n][m][nt][e] = pack_h2(a * w, b * w);
              }
              far |= !(fabsf(h) <= 64.f);
            }
        if (__any_sync(FULLW, far)) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
                  P[n][m][nt][e] = pack_h2(ex2(S[n][m][nt][2 * e] + (lv[n] - dd[m][e])),
                                           ex2(S[n][m][nt][2 * e + 1] + (lv[n] - dd[m][e])));
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if (!(tail[n].z >> 16)) continue;  // V rows that are not finite
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int k = 8 * (u >> 1) + 2 * t + (u & 1);
                if ((tail[n].z >> (16 + k) & 1) && key0[n] + k < min(keys[m][e], key_hi))
                  P[n][m][u >> 1][e] |= u & 1 ? 0x7fff0000u : 0x7fffu;
              }
        }
        // sums
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint4 v = lds128(T[n] + KV8_OFF_V + g * 512 + lane * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t v0 = kv8_pair<0>(word(v, j)), v1 = kv8_pair<1>(word(v, j));
#pragma unroll
              for (int m = 0; m < MT; ++m)
                mma_f16(O[m][4 * g + j], P[n][m][0][0], P[n][m][0][1], P[n][m][1][0], P[n][m][1][1], v0, v1);
            }
          }
      });
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        __syncthreads();  // all warps done with their stages (or the merge area): (re)use them as the merge area
        float *o = mo + warp * 16 * MO_STRIDE;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = ll[m][e];
          l += __shfl_xor_sync(FULLW, l, 1);
          l += __shfl_xor_sync(FULLW, l, 2);
          // numerators in the scores' reference, by the root of the factor twice: scales near fp32's least number
          const float r = ref(rr[m][e], l), c = ex2(0.5f * dd[m][e]);
          if (t == 0) *reinterpret_cast<float2 *>(mml + warp * 32 + (gr + 8 * e) * 2) = make_float2(r, l);
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float(*On)[4] = &O[m][4 * g];
              const int a = 2 * e + u;
              *reinterpret_cast<float4 *>(o + (gr + 8 * e) * MO_STRIDE + 32 * g + 4 * (2 * t + u)) =
                  make_float4(On[0][a] * c * c, On[1][a] * c * c, On[2][a] * c * c, On[3][a] * c * c);
            }
        }
        join(m);
      }
    };
    // up to 8 query rows as columns; this lane has columns 2t and 2t + 1 (index e)
    auto narrow = [&]() {
      uint2 qb[12];
#pragma unroll
      for (int j = 0; j < 12; ++j) qb[j] = make_uint2(lds32(smem + j * 512 + lane * 16), lds32(smem + j * 512 + lane * 16 + 8));
      float f[2], O[8][4];  // O[2g + j]: dims 32 g + 4 gr + 2 j (rows gr) and + 1 (rows gr + 8)
      float rr[2], dd[2], ll[2];
      int keys[2], least = 0x7fffffff;
#pragma unroll
      for (int n = 0; n < 8; ++n) O[n][0] = O[n][1] = O[n][2] = O[n][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[e] = sFac[2 * t + e];
        keys[e] = 2 * t + e < nq ? sKeys[2 * t + e] : 0x7fffffff;
        least = min(least, keys[e]);
        rr[e] = K8_NONE;
        dd[e] = K8_FAR;
        ll[e] = 0.f;
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) least = min(least, __shfl_xor_sync(FULLW, least, o));
      least = min(least, key_hi);
      units(std::integral_constant<bool, true>(), [&](auto nb, auto &T, auto &key0) {
        constexpr int NB = decltype(nb)::value;
        // scores: rows keys gr and gr + 8 (index h); two sums, as one chain of products waits for itself
        float S[NB][4], S2[NB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int u = 0; u < 4; ++u) S[n][u] = S2[n][u] = 0.f;
#pragma unroll
        for (int g = 0; g < 3; ++g) {
          uint4 ka[NB], kb[NB];
#pragma unroll
          for (int n = 0; n < NB; ++n) ka[n] = lds128(T[n] + g * 1024 + lane * 16), kb[n] = lds128(T[n] + g * 1024 + 512 + lane * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < NB; ++n)
              mma_f16(j & 1 ? S2[n] : S[n], kv8_pair<0>(word(ka[n], j)), kv8_pair<0>(word(kb[n], j)), kv8_pair<1>(word(ka[n], j)),
                      kv8_pair<1>(word(kb[n], j)), qb[4 * g + j].x, qb[4 * g + j].y);
        }
        uint4 tail[NB];
        float lv[NB], top[NB][2];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          tail[n] = lds128(T[n] + KV8_OFF_TAIL);
          const float ks = __uint_as_float(tail[n].x);
          lv[n] = lg2(__uint_as_float(tail[n].y));
          const uint64_t fs = f32x2(score_unit(ks, f[0]), score_unit(ks, f[1]));
#pragma unroll
          for (int h = 0; h < 4; h += 2)
            f32x2_split(mul_f32x2(add_f32x2(f32x2(S[n][h], S[n][h + 1]), f32x2(S2[n][h], S2[n][h + 1])), fs), S[n][h], S[n][h + 1]);
          if (!(key0[n] + 16 <= least && tail[n].z == 0)) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int k = gr + 8 * (u >> 1);
              if (key0[n] + k >= min(keys[u & 1], key_hi)) S[n][u] = NEG_INF;
              else if (tail[n].z >> k & 1) S[n][u] = __uint_as_float(0x7fffffffu);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[n][e] = fmaxf(S[n][e], S[n][2 + e]);
            const float by = top[n][e] - rr[e];
            move |= by > K8_SLACK || (lv[n] - dd[e]) + by > K8_SLACK + K8_PBIAS;
          }
        }
        if (__any_sync(FULLW, move)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float r = rr[e], x[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              x[n] = top[n][e];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x[n] = fmaxf(x[n], __shfl_xor_sync(FULLW, x[n], o));
              r = fmaxf(r, x[n]);
            }
            const float by = rr[e] - r;
            float d = fmaxf(dd[e] + by, K8_FAR);
#pragma unroll
            for (int n = 0; n < NB; ++n) d = fmaxf(d, (x[n] - r) + lv[n] - K8_PBIAS);
            const float c = ex2((dd[e] - d) + by);
            ll[e] *= ex2(by);
            rr[e] = r;
            dd[e] = d;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              O[d][e] *= c;
              O[d][2 + e] *= c;
            }
          }
        }
        uint32_t P[NB][2];  // weights: row query row gr, columns keys 2t, 2t + 1 and + 8
        float w[NB][2];
        bool far = false;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float h = lv[n] - dd[e];
            w[n][e] = ex2(h);
            far |= !(fabsf(h) <= 64.f);
          }
        far = __any_sync(FULLW, far);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x, y;
            f32x2_split(add_f32x2(f32x2(S[n][2 * h], S[n][2 * h + 1]), f32x2(-rr[0], -rr[1])), x, y);
            const float a = ex2(x), b = ex2(y);
            ll[0] += a;
            ll[1] += b;
            uint32_t pw = pack_h2(a * w[n][0], b * w[n][1]);
            if (far) pw = pack_h2(ex2(x + (lv[n] - dd[0])), ex2(y + (lv[n] - dd[1])));
            if (tail[n].z >> 16 && (tail[n].z >> (16 + gr + 8 * h) & 1)) {  // a V row that is not finite
              const int k = key0[n] + gr + 8 * h;
              pw |= (k < min(keys[0], key_hi) ? 0x7fffu : 0u) | (k < min(keys[1], key_hi) ? 0x7fff0000u : 0u);
            }
            P[n][h] = transpose8(pw);
          }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint4 v = lds128(T[n] + KV8_OFF_V + g * 512 + lane * 16);
            mma_f16(O[2 * g], kv8_pair<0>(v.x), kv8_pair<0>(v.y), kv8_pair<1>(v.x), kv8_pair<1>(v.y), P[n][0], P[n][1]);
            mma_f16(O[2 * g + 1], kv8_pair<0>(v.z), kv8_pair<0>(v.w), kv8_pair<1>(v.z), kv8_pair<1>(v.w), P[n][0], P[n][1]);
          }
      });
      __syncthreads();  // all warps done with their stages: reuse them as the merge area
      float c[2], r[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) ll[e] += __shfl_xor_sync(FULLW, ll[e], o);
        r[e] = ref(rr[e], ll[e]);
        c[e] = ex2(0.5f * dd[e]);  // (twice, as above)
      }
      if (gr == 0) *reinterpret_cast<float4 *>(mml + warp * 32 + 4 * t) = make_float4(r[0], ll[0], r[1], ll[1]);
      float *o = mo + warp * 16 * MO_STRIDE + 2 * t * MO_STRIDE + 4 * gr;
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4 *>(o + e * MO_STRIDE + 32 * g) =
              make_float4(O[2 * g][e] * c[e] * c[e], O[2 * g][2 + e] * c[e] * c[e], O[2 * g + 1][e] * c[e] * c[e],
                          O[2 * g + 1][2 + e] * c[e] * c[e]);
      join(0);
    };
    if (nq <= 8) narrow();
    else if (K8_MT == 1 || nq <= 16) wide(std::integral_constant<int, 1>());
    else wide(std::integral_constant<int, K8_MT>());
    if constexpr (DIRECT) {
      cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
      const int rank = (int)cl.block_rank();
      cl.sync();
      for (int idx = rank * (K8_WARPS * 32) + tid; idx < nq * (DV / 4); idx += A.cs * (K8_WARPS * 32)) {
        const int r = idx / (DV / 4), d4 = 4 * (idx % (DV / 4));
        float M = NEG_INF, S = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < A.cs; ++c) M = fmaxf(M, cl.map_shared_rank(own_ml, c)[2 * r]);
        for (int c = 0; c < A.cs; ++c) {
          const float2 ml = *reinterpret_cast<const float2 *>(cl.map_shared_rank(own_ml, c) + 2 * r);
          if (ml.x == NEG_INF) continue;
          const float f = ex2(ml.x - M);
          const float4 o = *reinterpret_cast<const float4 *>(cl.map_shared_rank(own_o, c) + r * DV + d4);
          S += ml.y * f;
          acc.x += o.x * f;
          acc.y += o.y * f;
          acc.z += o.z * f;
          acc.w += o.w * f;
        }
        const float inv = S == 0.f ? 0.f : 1.f / S;
        const int c = (int)((uint32_t)r * A.g_mul >> 16);
        *reinterpret_cast<uint2 *>(A.out + ((long long)(b + c) * A.hq + (long long)kv * G + (r - c * G)) * DV + d4) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      }
      cl.sync();  // no CTA leaves while another reads its part
    }
  }
  if (gave_up && lane == 0) flag(A.status, ST_TIMEOUT);
  // leave no copy in flight: only a wait that gave up left any (bounded again)
  uint32_t never = 0;
  for (; seen != sent; ++seen) tc::mbar_wait(sBar + 8 * (seen % K8_PAIRS), (seen / K8_PAIRS) & 1u, &never);
}

// Short contexts go by clusters in one launch.  Measured at 16 query heads per KV
// head (one launch against the work line's two): rows of 2048 keys, 1 x 4 KV heads
// 8.6 us against 7.3, 4 x 4 10.5 / 10.3, 16 x 4 14.2 / 15.8, 64 x 4 37.3 / 40.5;
// of 1024, 1 x 4 7.3 / 6.4, 4 x 4 8.4 / 9.6, 64 x 4 22.1 / 26.4; of 256, 1 x 4 6.1 /
// 6.3, 64 x 4 10.8 / 16.0; of 4096, 4 x 4 14.0 / 12.1, 64 x 4 66.2 / 65.1.  A few rows
// gain by the whole GPU's warps once eight CTAs have a few tiles each; up to 1024
// keys that is less than a second launch and a workspace cost a caller from the host.
// (A captured step does not pay those: 1 x 4 KV heads at 1024 keys costs it 0.9 us.)
bool one_launch(int B, int hkv, long long max_ctx) {
  const long long units = (max_ctx + K8_UNIT - 1) / K8_UNIT;
  return units <= ((long long)B * hkv < 8 ? 64 : 128);
}

}  // namespace

size_t kv8_decode_workspace(int B, int hq, int hkv, long long max_ctx) {
  if (one_launch(B, hkv, max_ctx)) return 0;
  return line_workspace<K8Line>(B, hq, hkv, max_ctx, rows_together(hq / hkv));
}

cudaError_t launch_kv8_decode(const uint16_t *q, const int64_t *pos, const int32_t *seq, int B, int hq,
                              const Kv8View &pool, const float *table, int64_t max_pos, float softmax_scale,
                              long long max_ctx, void *ws, uint16_t *out, unsigned *status, cudaStream_t st) {
  const int hkv = pool.hkv, G = hq / hkv, R = K8_CTAS * num_sms();
  const long long rows = (long long)B * hkv, units = (max_ctx + K8_UNIT - 1) / K8_UNIT;
  if (rows > 0x7ffffffLL) return cudaErrorInvalidValue;  // (its queries alone would fill the GPU)
  const bool direct = one_launch(B, hkv, max_ctx);
  static void (*const kernels[3])(K8Args) = {kv8_decode_kernel<K8_LINE>, kv8_decode_kernel<K8_TURNS>,
                                             kv8_decode_kernel<K8_DIRECT>};
  const int form = direct ? K8_DIRECT : line_turns<K8Line>(B, hkv, max_ctx) > 1 ? K8_TURNS : K8_LINE;
  void (*const kernel)(K8Args) = kernels[form];
  cudaError_t e = ensure_smem_limit(24 + form, (const void *)kernel, K8_SMEM, true);
  if (e != cudaSuccess) return e;
  K8Args A;
  line_args<K8Line>(A, pos, seq, B, hq, hkv, pool.num_seqs, max_pos, max_ctx, ws, out,
                    rows_together(G));
  A.q = q;
  A.pool = pool;
  A.table = table;
  A.scale_log2 = softmax_scale * LOG2E;
  A.status = status;
  A.stall_ns = take_stall();
  const unsigned long long tpb = (unsigned long long)(pool.block_size >> 4);
  A.tpb_mul = ((1ull << 36) + tpb - 1) / tpb;
  A.g_mul = (65536u + (uint32_t)G - 1) / (uint32_t)G;
  A.cs = 1;
  if (direct) {
    // as many CTAs a row as the longest row gives every warp a unit, as a
    // cluster may have, and as the GPU holds of all rows at once
    while (A.cs < 8 && A.cs * K8_WARPS < units && 2 * A.cs * rows <= R) A.cs *= 2;
    return launch_pdl_cluster(kernel, dim3((unsigned)(rows * A.cs)), dim3(K8_WARPS * 32), (size_t)K8_SMEM, A.cs, st, A);
  }
  return line_launch<K8Line>(kernel, K8_WARPS * 32, (size_t)K8_SMEM, A, status, st);
}

}  // namespace kvr
