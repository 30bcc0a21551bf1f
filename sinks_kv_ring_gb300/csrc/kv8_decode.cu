// kv8_decode.cu -- one-token decode over a full-attention layer kept in 8
// bits: split-K with a log-sum-exp merge over the work line (line.cuh), as the
// 4-bit decode.
//
// Mathematics.  With values s u, one scale s for a tile's K and one for its V,
//   score_j = ks (q . u_j),   o = sum_j (p_j vs) u_j / sum_j p_j,
// so the tensor cores multiply codes and a scale costs one multiply a tile.  All
// products are m16n8k16 f16 with fp32 accumulators; groups of more than 8 query
// heads per KV head put the heads in the 16 rows, smaller ones in the 8 columns
// (SMALL, below):
//   * Codes become fp16 numbers, exactly, by two instructions a pair (kv8_pair).
//   * Queries are rotated, scaled by softmax_scale log2(e), brought by a power
//     of two to a largest magnitude in [2^14, 2^15) per head, and rounded once to
//     fp16 (2^-11 of a value, where the bf16 decode rounds to 2^-8).
//   * The weights of the value product are p_j vs, taken as one power of two of
//     score + log2(vs) less a reference of its own: the largest such sum so far.
//     So a weight is at most 2^15 whatever the scales are, and one is lost to
//     fp16's least number only where it is below 2^-35 of the largest share in
//     the output, not of the largest probability: light keys with large values
//     and heavy keys with small ones both keep their part.  A weight is rounded to
//     2^-11 of itself, an eighth of the output's own rounding.
//   * sum p_j stays in fp32 beside it, under the running maximum of the scores.
// Either reference moves (with a rescale of the sums) only when a sum passes it by
// more than 4: the check is one vote a tile.
//
// Work.  Each warp streams its own tiles of 16 keys through its own ring of bulk
// copies (one copy brings codes and scales), with no barrier between warps
// inside a piece; 12 warps an SM, three CTAs, hold the sums in registers.
#include <cooperative_groups.h>

#include "kv8.cuh"
#include "line.cuh"
#include "tc_ptx.cuh"

namespace kvr {
namespace {

constexpr unsigned ST_TIMEOUT = 8u;  // KVR_DEV_TIMEOUT
constexpr int K8_WARPS = 4;
constexpr int K8_CTAS = 3;           // per SM
constexpr int K8_UNIT = 16;          // keys: one tile
constexpr int K8_STAGES = 3;
constexpr float K8_PBIAS = 11.f;     // weights are 2^11 where they equal the reference
constexpr float K8_SLACK = 4.f;      // how far a score or weight may pass its reference
constexpr float K8_NONE = -1e30f;    // a reference before the first keys
// The work line (line.cuh) in units of one tile.  The greatest share: the tensor
// cores cut a sum off below its last bit at every product (2^-23 of it as
// measured), one a tile for the values; at 2048 tiles a warp that is 2^-12 of the
// sum at most, a sixteenth of the output's half step.
struct K8Line {
  static constexpr int UNIT = K8_UNIT, ROW = 24, MIN = K8_WARPS, MOST = 2048 * K8_WARPS, CTAS = K8_CTAS;
};
// shared memory: query operands (12 steps), row factors, barriers, abort flag, plan, stages
constexpr int K8_OFF_ROW = 12 * 512;
constexpr int K8_OFF_BAR = K8_OFF_ROW + 64;
constexpr int K8_OFF_STALL = K8_OFF_BAR + 8 * K8_WARPS * K8_STAGES;  // a barrier that nothing completes (test hook)
constexpr int K8_OFF_ABORT = K8_OFF_STALL + 8;
constexpr int K8_OFF_L = (K8_OFF_ABORT + 4 + 7) / 8 * 8;
constexpr int K8_OFF_PLAN = (K8_OFF_L + 8 + 15) / 16 * 16;
constexpr int K8_OFF_STAGE = (K8_OFF_PLAN + (LINE_INLINE_MAX + 2) * 8 + 127) / 128 * 128;
constexpr int K8_SMEM = K8_OFF_STAGE + K8_WARPS * K8_STAGES * KV8_TILE;
static_assert(K8_WARPS * K8_STAGES * KV8_TILE >= (K8_WARPS * 16 * (MO_STRIDE + 2) + K8_WARPS * 16 + 32 + 16 * DV) * 4,
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
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return half2_bits(__floats2half2_rn(lo, hi)); }

// The query operands of one row: thread (head r, eighth c) rotates and scales 24
// dims of head r, and the head's eight threads share its power of two.  Operand
// order: step 4g + w holds, for lane 4a + t, dims 64 g + 16 t + 4 w + {0, 1}
// (registers 0, 1: heads a and a + 8) and + {2, 3} (registers 2, 3), as word w of
// a lane's K codes has them.
struct K8Query {
  uint2 lo, hi;
  uint4 g1, g2;
  float4 t0, t1;
};
__device__ __forceinline__ K8Query kv8_query_load(const uint16_t *__restrict__ qh, int G,
                                                  const float *__restrict__ cs_row, int tid) {
  const int r = tid >> 3, c = tid & 7;
  K8Query Q = {};
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
__device__ __forceinline__ void kv8_query(const K8Query &Q, int G, float scale_log2, uint8_t *smem, int tid) {
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
    *reinterpret_cast<uint32_t *>(smem + at) = pack_h2(y[i] * up * dn, y[i + 1] * up * dn);
    *reinterpret_cast<uint32_t *>(smem + at + 8) = pack_h2(y[i + 2] * up * dn, y[i + 3] * up * dn);
  }
  // a score's unit per K scale: the sums hold (y . u) 2^a.  A query that is not finite has none: its row is NaN
  if (c == 0)
    *reinterpret_cast<float *>(smem + K8_OFF_ROW + 4 * r) =
        mx >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)min(max(127 - a, 1), 254) << 23);
}

struct K8Args : LineArgs {
  const uint16_t *q;
  Kv8View pool;
  const float *table;
  float scale_log2;
  unsigned *status;
  unsigned long long stall_ns;  // test hook: warp 0's first wait is on a barrier that nothing completes (0: no stall)
  int cs;                       // DIRECT: CTAs of a row
  unsigned long long tpb_mul;   // ceil(2^36 / tiles per block): tile / tiles per block = tile * tpb_mul >> 36 (tile < 2^28)
};

// SMALL: groups of up to 8 query heads.  The keys are then the 16 rows of the
// products and the heads their 8 columns (scores K Q^T, sums V^T P^T): half the
// products, and half the registers for the sums.  The codes' operands are the
// same registers; a weight's row and column change places between the two
// products by an 8 x 8 transposition (movmatrix).
//
// FORM: the work line, a share a CTA (K8_LINE) or several (K8_TURNS); or DIRECT:
// short contexts of few rows, where a launch costs more than the work.  A cluster
// of A.cs CTAs takes one row, each an equal share of its units, and the CTAs
// merge their parts through each other's shared memory: one launch, no plan and
// no workspace.
enum K8Form { K8_LINE, K8_TURNS, K8_DIRECT };
template <bool SMALL, K8Form FORM>
__global__ void __launch_bounds__(K8_WARPS * 32, K8_CTAS) kv8_decode_kernel(K8Args A) {
  constexpr bool DIRECT = FORM == K8_DIRECT, TURNS = FORM == K8_TURNS;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hkv = A.hkv, G = A.G;
  const uint32_t sBase = smem_u32(smem);
  const uint32_t sBar = sBase + K8_OFF_BAR + 8 * K8_STAGES * warp;
  volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + K8_OFF_ABORT);
  uint8_t *const sStage = smem + K8_OFF_STAGE + warp * K8_STAGES * KV8_TILE;
  int64_t *sPrefix = reinterpret_cast<int64_t *>(smem + K8_OFF_PLAN);
  if (lane == 0) {
    for (int j = 0; j < K8_STAGES; ++j) tc::mbar_init(sBar + 8 * j, 1);
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
  long long x = 0, line_end = 0, early_p = 0;
  int b = 0, kv = 0, lo = 0, hi = 0, early_s = 0;
  bool ready = DIRECT;  // b, kv, lo, hi hold the next part
  auto plan = [&](auto get, unsigned *status) {
    return line_plan<K8Line, K8_WARPS * 32>(get, A.B, hkv, A.num_seqs, A.max_pos, A.max_ctx, gridDim.x, sPrefix, status);
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
    if (blockIdx.x == 0) line_units<K8Line>(p, s, A.num_seqs, A.max_pos, A.max_ctx, A.status);
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
  uint32_t seen = 0;  // this warp's loads waited for so far: stage seen % K8_STAGES, phase (seen / K8_STAGES) & 1
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
      const int units = line_units<K8Line>(p, A.seq[b], A.num_seqs, A.max_pos, A.max_ctx,
                                           kv == 0 && rank == 0 && tid == 0 ? A.status : nullptr);
      if (units == 0) {  // (so for the whole cluster)
        uint16_t *o = A.out + ((long long)b * A.hq + (long long)kv * G) * DV;
        for (int i = rank * (K8_WARPS * 32) + tid; i < G * DV; i += A.cs * (K8_WARPS * 32)) o[i] = 0;
        return;
      }
      const int each = (units + A.cs - 1) / A.cs;
      key_lo = min(rank * each, units) * K8_UNIT;
      key_hi = (int)min((long long)min((rank + 1) * each, units) * K8_UNIT, p + 1);
      if (key_hi < key_lo) key_hi = key_lo;
    } else {
      if (!ready) line_part<K8Line>(prefix, A.B, hkv, line_end, x, b, kv, lo, hi);
      ready = false;
      if (hi <= 0) continue;  // set-up alone: no piece
      w = (int)blockIdx.x + b * hkv + kv;
      if (TURNS) w += turn * (int)gridDim.x;
      p = A.pos[b];
      key_lo = lo * K8_UNIT;
      key_hi = (int)min((long long)hi * K8_UNIT, p + 1);
    }
    const int s = A.seq[b];  // (a row that gets here has a valid position and id)
    const int nunit = (key_hi - key_lo + K8_UNIT - 1) / K8_UNIT;
    const int my_n = nunit > warp ? (nunit - warp + K8_WARPS - 1) / K8_WARPS : 0;
    const int32_t *bt = A.pool.block_table + (long long)s * A.pool.max_blocks;
    const K8Query Q = kv8_query_load(A.q + ((long long)b * A.hq + (long long)kv * G) * DQK, G, A.table + p * 64, tid);
    tc::fence_proxy_async_smem();                   // the last piece's merge area lies over the stages:
    if (__syncthreads_or(*abort_flag != 0)) break;  // it is free again, its accesses ahead of the copies'

    // Units go out 32 at a time: lane l looks up unit base + l's tile (a block
    // that is none of the pool's gives -1) and issues its copy when its turn
    // comes; `ok` has the warp's units that lie in the pool.
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
    auto issue = [&](int i) {
      if ((i & 31) == 0) fetch_ids(i);
      const uint32_t st = sent % K8_STAGES;
      ++sent;
      if (lane == (i & 31)) {
        const uint32_t bar = sBar + 8 * st;
        tc::mbar_expect_tx(bar, id >= 0 ? KV8_TILE : 0);
        if (id >= 0)
          tc::bulk_load(smem_u32(sStage + st * KV8_TILE), A.pool.data + (long long)id * KV8_TILE, KV8_TILE, bar);
      }
    };
#pragma unroll
    for (int i = 0; i < K8_STAGES - 1; ++i)
      if (i < my_n) issue(i);

    kv8_query(Q, G, A.scale_log2, smem, tid);
    __syncthreads();
    int run_n = my_n;
    if (A.stall_ns && warp == 0 && !gave_up && !tc::mbar_wait(sBase + K8_OFF_STALL, 0, abort_flag, A.stall_ns)) {
      gave_up = true;
      run_n = 0;
    }
    // the tile of unit i, or null: no block of the pool, or (gave_up) not there in time
    auto next_tile = [&](int i) -> const uint8_t * {
      if ((i & 31) == 0) ok = next_ok;  // (the units of this round were looked up no later than with their first)
      if (i + K8_STAGES - 1 < my_n) issue(i + K8_STAGES - 1);
      const uint32_t st = seen % K8_STAGES;
      if (!__all_sync(FULLW, tc::mbar_wait(sBar + 8 * st, (seen / K8_STAGES) & 1u, abort_flag))) {
        gave_up = true;
        return nullptr;
      }
      ++seen;
      return (ok >> (i & 31)) & 1 ? sStage + st * KV8_TILE : nullptr;
    };
    // references of the scores (r) and of the weights (R, less the bias) of this
    // lane's two rows or columns, and the sums of exp2(score - r)
    float r0 = K8_NONE, r1 = K8_NONE, R0 = K8_NONE, R1 = K8_NONE, l0 = 0.f, l1 = 0.f;
    bool any = false;  // a tile was there
    // merge area, over the stages once all warps are done with them: per warp, reference and sum per row, and numerators
    float *mml = reinterpret_cast<float *>(smem + K8_OFF_STAGE);  // [4][16][2]
    float *mo = mml + K8_WARPS * 16 * 2;                          // [4][16][MO_STRIDE]
    if constexpr (!SMALL) {
      const float crow0 = *reinterpret_cast<const float *>(smem + K8_OFF_ROW + 4 * gr);
      const float crow1 = *reinterpret_cast<const float *>(smem + K8_OFF_ROW + 4 * (gr + 8));
      float O[16][4];  // O[4g + i]: dims 32 g + 4 c + i of column c
#pragma unroll
      for (int n = 0; n < 16; ++n) O[n][0] = O[n][1] = O[n][2] = O[n][3] = 0.f;
      for (int i = 0; i < run_n; ++i) {
        const uint8_t *sT = next_tile(i);
        if (!sT) {
          if (gave_up) break;
          continue;
        }
        any = true;
        // scores: rows heads gr and gr + 8, columns keys 2t, 2t + 1 (nt = 0) and + 8
        float S[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) S[nt][0] = S[nt][1] = S[nt][2] = S[nt][3] = 0.f;
#pragma unroll
        for (int g = 0; g < 3; ++g) {
          const uint4 ka = lds128(sT + g * 1024 + lane * 16), kb = lds128(sT + g * 1024 + 512 + lane * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 a = lds128(smem + (g * 4 + j) * 512 + lane * 16);
            mma_f16(S[0], a.x, a.y, a.z, a.w, kv8_pair<0>(word(ka, j)), kv8_pair<1>(word(ka, j)));
            mma_f16(S[1], a.x, a.y, a.z, a.w, kv8_pair<0>(word(kb, j)), kv8_pair<1>(word(kb, j)));
          }
        }
        const uint4 tail = lds128(sT + KV8_OFF_TAIL);
        const int left = key_hi - (key_lo + K8_UNIT * (warp + i * K8_WARPS));  // keys of the tile in range
        if (left < 16 || tail.z != 0) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = 8 * nt + 2 * t + e;
              if (k >= left) S[nt][e] = S[nt][2 + e] = NEG_INF;
              else if (tail.z >> k & 1) S[nt][e] = S[nt][2 + e] = __uint_as_float(0x7fffffffu);  // a K row that is not finite
            }
        }
        // (the least number keeps a factor of zero from making NaN of a masked score)
        const float ks = __uint_as_float(tail.x), f0 = fmaf(ks, crow0, 0x1p-126f), f1 = fmaf(ks, crow1, 0x1p-126f);
        const float lv = lg2(__uint_as_float(tail.y));  // -inf for a scale of 0: no weight
        const float top0 = fmaxf(fmax3(S[0][0], S[0][1], S[1][0]), S[1][1]) * f0;
        const float top1 = fmaxf(fmax3(S[0][2], S[0][3], S[1][2]), S[1][3]) * f1;
        const bool move = fmaxf(top0 - r0, top1 - r1) > K8_SLACK || lv + fmaxf(top0 - R0, top1 - R1) > K8_SLACK + K8_PBIAS;
        if (__any_sync(FULLW, move)) {
          // new references per row: the larger of the old one and this tile's maximum
          float t0 = top0, t1 = top1;
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(FULLW, t0, o));
            t1 = fmaxf(t1, __shfl_xor_sync(FULLW, t1, o));
          }
          const float n0 = fmaxf(r0, t0), n1 = fmaxf(r1, t1);
          l0 *= ex2(r0 - n0);
          l1 *= ex2(r1 - n1);
          r0 = n0;
          r1 = n1;
          const float N0 = fmaxf(R0, t0 + lv - K8_PBIAS), N1 = fmaxf(R1, t1 + lv - K8_PBIAS);
          const float c0 = ex2(R0 - N0), c1 = ex2(R1 - N1);
          R0 = N0;
          R1 = N1;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            O[n][0] *= c0;
            O[n][1] *= c0;
            O[n][2] *= c1;
            O[n][3] *= c1;
          }
        }
        uint32_t P[2][2];  // weights [8 keys][row gr, row gr + 8]
        const float g0 = lv - R0, g1 = lv - R1;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          l0 += ex2(fmaf(S[nt][0], f0, -r0)) + ex2(fmaf(S[nt][1], f0, -r0));
          l1 += ex2(fmaf(S[nt][2], f1, -r1)) + ex2(fmaf(S[nt][3], f1, -r1));
          P[nt][0] = pack_h2(ex2(fmaf(S[nt][0], f0, g0)), ex2(fmaf(S[nt][1], f0, g0)));
          P[nt][1] = pack_h2(ex2(fmaf(S[nt][2], f1, g1)), ex2(fmaf(S[nt][3], f1, g1)));
        }
        if (tail.z >> 16) {  // V rows that are not finite
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int k = 8 * nt + 2 * t;
            const uint32_t nan = (k < left && (tail.z >> (16 + k) & 1) ? 0x7fffu : 0u) |
                                 (k + 1 < left && (tail.z >> (17 + k) & 1) ? 0x7fff0000u : 0u);
            P[nt][0] |= nan;
            P[nt][1] |= nan;
          }
        }
        // sums
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint4 v = lds128(sT + KV8_OFF_V + g * 512 + lane * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f16(O[4 * g + j], P[0][0], P[0][1], P[1][0], P[1][1], kv8_pair<0>(word(v, j)), kv8_pair<1>(word(v, j)));
        }
        __syncwarp();  // the stage is read: the next copy into it may go out
      }
      __syncthreads();  // all warps done with their stages: reuse them as the merge area
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        l0 += __shfl_xor_sync(FULLW, l0, o);
        l1 += __shfl_xor_sync(FULLW, l1, o);
      }
      // numerators in the scores' reference (0 where no score was a number: the row will not be one)
      const float m0 = r0 == K8_NONE ? 0.f : r0, m1 = r1 == K8_NONE ? 0.f : r1;
      const float c0 = ex2(R0 - m0), c1 = ex2(R1 - m1);
      if (t == 0) {
        float *m = mml + warp * 32;
        m[gr * 2] = any ? m0 : NEG_INF;
        m[gr * 2 + 1] = l0;
        m[(gr + 8) * 2] = any ? m1 : NEG_INF;
        m[(gr + 8) * 2 + 1] = l1;
      }
      float *o = mo + warp * 16 * MO_STRIDE;
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float(*On)[4] = &O[4 * g];
          const int d = 32 * g + 4 * (2 * t + c);
          *reinterpret_cast<float4 *>(o + gr * MO_STRIDE + d) =
              make_float4(On[0][c] * c0, On[1][c] * c0, On[2][c] * c0, On[3][c] * c0);
          *reinterpret_cast<float4 *>(o + (gr + 8) * MO_STRIDE + d) =
              make_float4(On[0][2 + c] * c1, On[1][2 + c] * c1, On[2][2 + c] * c1, On[3][2 + c] * c1);
        }
    } else {
      // a head's column: this lane has heads 2t and 2t + 1
      const float crow0 = *reinterpret_cast<const float *>(smem + K8_OFF_ROW + 8 * t);
      const float crow1 = *reinterpret_cast<const float *>(smem + K8_OFF_ROW + 8 * t + 4);
      uint2 qb[12];
#pragma unroll
      for (int j = 0; j < 12; ++j) qb[j] = make_uint2(lds32(smem + j * 512 + lane * 16), lds32(smem + j * 512 + lane * 16 + 8));
      float O[8][4];  // O[2g + j]: dims 32 g + 4 gr + 2 j (rows gr) and + 1 (rows gr + 8)
#pragma unroll
      for (int n = 0; n < 8; ++n) O[n][0] = O[n][1] = O[n][2] = O[n][3] = 0.f;
      for (int i = 0; i < run_n; ++i) {
        const uint8_t *sT = next_tile(i);
        if (!sT) {
          if (gave_up) break;
          continue;
        }
        any = true;
        // scores: rows keys gr and gr + 8, columns heads 2t, 2t + 1; two sums, as one chain of products waits for itself
        float S[4] = {0.f, 0.f, 0.f, 0.f}, S2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < 3; ++g) {
          const uint4 ka = lds128(sT + g * 1024 + lane * 16), kb = lds128(sT + g * 1024 + 512 + lane * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f16(j & 1 ? S2 : S, kv8_pair<0>(word(ka, j)), kv8_pair<0>(word(kb, j)), kv8_pair<1>(word(ka, j)),
                    kv8_pair<1>(word(kb, j)), qb[4 * g + j].x, qb[4 * g + j].y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) S[e] += S2[e];
        const uint4 tail = lds128(sT + KV8_OFF_TAIL);
        const int left = key_hi - (key_lo + K8_UNIT * (warp + i * K8_WARPS));
        if (left < 16 || tail.z != 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = gr + 8 * e;
            if (k >= left) S[2 * e] = S[2 * e + 1] = NEG_INF;
            else if (tail.z >> k & 1) S[2 * e] = S[2 * e + 1] = __uint_as_float(0x7fffffffu);
          }
        }
        const float ks = __uint_as_float(tail.x), f0 = fmaf(ks, crow0, 0x1p-126f), f1 = fmaf(ks, crow1, 0x1p-126f);
        const float lv = lg2(__uint_as_float(tail.y));
        const float top0 = fmaxf(S[0], S[2]) * f0, top1 = fmaxf(S[1], S[3]) * f1;
        const bool move = fmaxf(top0 - r0, top1 - r1) > K8_SLACK || lv + fmaxf(top0 - R0, top1 - R1) > K8_SLACK + K8_PBIAS;
        if (__any_sync(FULLW, move)) {
          float t0 = top0, t1 = top1;
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(FULLW, t0, o));
            t1 = fmaxf(t1, __shfl_xor_sync(FULLW, t1, o));
          }
          const float n0 = fmaxf(r0, t0), n1 = fmaxf(r1, t1);
          l0 *= ex2(r0 - n0);
          l1 *= ex2(r1 - n1);
          r0 = n0;
          r1 = n1;
          const float N0 = fmaxf(R0, t0 + lv - K8_PBIAS), N1 = fmaxf(R1, t1 + lv - K8_PBIAS);
          const float c0 = ex2(R0 - N0), c1 = ex2(R1 - N1);
          R0 = N0;
          R1 = N1;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            O[n][0] *= c0;
            O[n][1] *= c1;
            O[n][2] *= c0;
            O[n][3] *= c1;
          }
        }
        uint32_t P[2];  // weights: row head gr, columns keys 2t, 2t + 1 and + 8
        const float g0 = lv - R0, g1 = lv - R1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l0 += ex2(fmaf(S[2 * e], f0, -r0));
          l1 += ex2(fmaf(S[2 * e + 1], f1, -r1));
          uint32_t pw = pack_h2(ex2(fmaf(S[2 * e], f0, g0)), ex2(fmaf(S[2 * e + 1], f1, g1)));
          if (tail.z >> 16 && gr + 8 * e < left && (tail.z >> (16 + gr + 8 * e) & 1)) pw = 0x7fff7fffu;  // a V row that is not finite
          P[e] = transpose8(pw);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint4 v = lds128(sT + KV8_OFF_V + g * 512 + lane * 16);
          mma_f16(O[2 * g], kv8_pair<0>(v.x), kv8_pair<0>(v.y), kv8_pair<1>(v.x), kv8_pair<1>(v.y), P[0], P[1]);
          mma_f16(O[2 * g + 1], kv8_pair<0>(v.z), kv8_pair<0>(v.w), kv8_pair<1>(v.z), kv8_pair<1>(v.w), P[0], P[1]);
        }
        __syncwarp();  // the stage is read: the next copy into it may go out
      }
      __syncthreads();  // all warps done with their stages: reuse them as the merge area
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(FULLW, l0, o);
        l1 += __shfl_xor_sync(FULLW, l1, o);
      }
      const float m0 = r0 == K8_NONE ? 0.f : r0, m1 = r1 == K8_NONE ? 0.f : r1;
      const float c0 = ex2(R0 - m0), c1 = ex2(R1 - m1);
      if (gr == 0)
        *reinterpret_cast<float4 *>(mml + warp * 32 + 4 * t) = make_float4(any ? m0 : NEG_INF, l0, any ? m1 : NEG_INF, l1);
      float *o = mo + warp * 16 * MO_STRIDE + 2 * t * MO_STRIDE + 4 * gr;
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float k = c ? c1 : c0;
          *reinterpret_cast<float4 *>(o + c * MO_STRIDE + 32 * g) =
              make_float4(O[2 * g][c] * k, O[2 * g][2 + c] * k, O[2 * g + 1][c] * k, O[2 * g + 1][2 + c] * k);
        }
    }
    __syncthreads();
    float *fac = mo + K8_WARPS * 16 * MO_STRIDE;  // [4 warps][16 heads]
    float *own_ml = fac + K8_WARPS * 16;          // DIRECT: the CTA's merged part, [16][2] and [16][128]
    float *own_o = own_ml + 32;
    if (tid < G) {
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
      float *pml = DIRECT ? own_ml : A.part_ml + (long long)w * G * 2;
      pml[tid * 2] = M;
      pml[tid * 2 + 1] = L;
    }
    __syncthreads();
    for (int idx = tid; idx < G * (DV / 4); idx += blockDim.x) {
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
      *reinterpret_cast<float4 *>(DIRECT ? own_o + g * DV + d4 : A.part_o + ((long long)w * G + g) * DV + d4) = acc;
    }
    if constexpr (DIRECT) {
      cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
      const int rank = (int)cl.block_rank();
      cl.sync();
      for (int idx = rank * (K8_WARPS * 32) + tid; idx < G * (DV / 4); idx += A.cs * (K8_WARPS * 32)) {
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
  for (; seen != sent; ++seen) tc::mbar_wait(sBar + 8 * (seen % K8_STAGES), (seen / K8_STAGES) & 1u, &never);
}

// Short contexts go by clusters in one launch, up to 2048 keys where the GPU
// holds eight CTAs of every row at once, else up to 1024.
bool one_launch(int B, int hkv, long long max_ctx) {
  const long long R = (long long)K8_CTAS * num_sms(), units = (max_ctx + K8_UNIT - 1) / K8_UNIT;
  return units <= (8LL * B * hkv <= R ? 128 : 64);
}

}  // namespace

size_t kv8_decode_workspace(int B, int hq, int hkv, long long max_ctx) {
  if (one_launch(B, hkv, max_ctx)) return 0;
  return line_workspace<K8Line>(B, hq, hkv, max_ctx);
}

cudaError_t launch_kv8_decode(const uint16_t *q, const int64_t *pos, const int32_t *seq, int B, int hq,
                              const Kv8View &pool, const float *table, int64_t max_pos, float softmax_scale,
                              long long max_ctx, void *ws, uint16_t *out, unsigned *status, cudaStream_t st) {
  const int hkv = pool.hkv, G = hq / hkv, R = K8_CTAS * num_sms();
  const long long rows = (long long)B * hkv, units = (max_ctx + K8_UNIT - 1) / K8_UNIT;
  if (rows > 0x7ffffffLL) return cudaErrorInvalidValue;  // (its queries alone would fill the GPU)
  const bool direct = one_launch(B, hkv, max_ctx);
  static void (*const kernels[2][3])(K8Args) = {
      {kv8_decode_kernel<false, K8_LINE>, kv8_decode_kernel<false, K8_TURNS>, kv8_decode_kernel<false, K8_DIRECT>},
      {kv8_decode_kernel<true, K8_LINE>, kv8_decode_kernel<true, K8_TURNS>, kv8_decode_kernel<true, K8_DIRECT>}};
  const int form = direct ? K8_DIRECT : line_turns<K8Line>(B, hkv, max_ctx) > 1 ? K8_TURNS : K8_LINE;
  void (*const kernel)(K8Args) = kernels[G <= 8][form];
  cudaError_t e = ensure_smem_limit(24 + 3 * (G <= 8) + form, (const void *)kernel, K8_SMEM, true);
  if (e != cudaSuccess) return e;
  K8Args A;
  line_args<K8Line>(A, pos, seq, B, hq, hkv, pool.num_seqs, max_pos, max_ctx, ws, out);
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
    while (A.cs < 8 && A.cs * K8_WARPS < units && 2 * A.cs * rows <= R) A.cs *= 2;
    return launch_pdl_cluster(kernel, dim3((unsigned)(rows * A.cs)), dim3(K8_WARPS * 32), (size_t)K8_SMEM, A.cs, st, A);
  }
  return line_launch<K8Line>(kernel, K8_WARPS * 32, (size_t)K8_SMEM, A, status, st);
}

}  // namespace kvr
