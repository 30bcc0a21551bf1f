// line.cuh -- the work line of the decodes over quantised pools: how a batch of
// contexts of any lengths is cut into equal shares for the CTAs, and the merge
// of the pieces.
//
// Every (sequence, KV head) row is laid end to end, ROW units of set-up and
// then its keys in units of UNIT; share c is units c L .. (c + 1) L - 1 of the
// line, L = total / CTAs (at least MIN units), and CTA c takes it, so all CTAs
// end together whatever the contexts are, and a row is cut only where a share
// ends.  The part of row r in share c is piece c + r (line_at): no two pieces share
// a number, and a row's are consecutive.  A share is at most MOST units: a longer
// line is cut into a multiple of the CTAs' number of shares, and CTA c takes c,
// c + CTAs, ...
//
// Neighbouring batch rows of one sequence (the draft tokens of a verification) may
// go together (LN::SHARE): of every aligned block of `rmax` rows, those that follow
// a row of the same sequence join it, the first one (the leader) has the line's
// part for all of them, as long as the longest needs, and the others have none.
//
// A kernel describes its line by a type LN with UNIT, ROW, MIN, MOST, CTAS (the
// CTAs of an SM) and SHARE.
#pragma once

#include "launch.h"
#include "warp_attn.cuh"

namespace kvr {

constexpr unsigned FULLW = 0xffffffffu;
constexpr int LINE_PLAN = 32;          // int64 words of the plan ahead of the rows' prefix: L
constexpr int LINE_INLINE_MAX = 256;   // batches the split kernel plans itself

// What the plan and the merge know of a call.
struct LineArgs {
  const int64_t *pos;
  const int32_t *seq;
  int B, hq, G, hkv, num_seqs;
  int64_t max_pos;
  long long max_ctx;
  int64_t *plan;
  float *part_ml;
  float *part_o;
  uint16_t *out;
  int rmax;  // rows that may go together: a power of two up to 4; 1 without LN::SHARE
};

// Units of keys of sequence b; 0 (flagged once) where its position or id is
// out of range: such a row has no part of the line, and the merge writes zeros.
template <class LN>
__device__ __forceinline__ int line_units(long long p, int s, int num_seqs, int64_t max_pos, long long max_ctx,
                                         unsigned *status) {
  const bool bp = p < 0 || p >= max_pos || p + 1 > max_ctx, bs = s < 0 || s >= num_seqs;
  if (bp || bs) {
    if (status) flag(status, (bp ? ST_BAD_POS : 0u) | (bs ? ST_BAD_SEQ : 0u));
    return 0;
  }
  return (int)((p + LN::UNIT) / LN::UNIT);
}

// Which of a warp's rows (lane l: row l of 32, those of valid position and id
// `valid`, of sequence s) join the row before them.
__device__ __forceinline__ unsigned line_joined(bool valid, int s, int lane, int rmax) {
  const unsigned ok = __ballot_sync(FULLW, valid);
  const int before = __shfl_up_sync(FULLW, s, 1);
  return __ballot_sync(FULLW, (lane & (rmax - 1)) != 0 && (ok >> lane & 1) && (ok >> (lane - 1) & 1) && s == before);
}
// Whether row lane + k goes with row lane.
__device__ __forceinline__ bool line_follows(unsigned joined, int lane, int k) {
  const unsigned m = ((1u << k) - 1u) << 1;  // (k < 4: rows lane + 1 .. lane + k)
  return (joined >> lane & m) == m;
}
// What the plan says of a row with LN::SHARE: how far ahead of it its leader is, and
// how many rows there are from the leader on.
__device__ __forceinline__ uint8_t line_info(unsigned joined, int lane) {
  const int lead = __clz(~(joined << (31 - lane)));  // ones from the row's bit down
  const int more = __ffs(~(joined >> lane >> 1)) - 1;
  return (uint8_t)(lead | (lead + 1 + more) << 4);
}
__device__ __forceinline__ int line_lead(uint8_t info) { return info & 15; }
__device__ __forceinline__ int line_rows(uint8_t info) { return info >> 4; }

// First partial row (of one query row each) of the piece of batch rows b .. b + rows
// - 1 and KV head kv in share c.  Along the line each next piece lies in the next
// share, `rmax` G further, or is the next row's in the same share, `rows` G
// further: no two overlap, and the pieces of all shares and rows fit in shares
// rmax G + B hkv G.
__device__ __forceinline__ long long line_at(const LineArgs &A, long long c, int b, int kv, int rows) {
  return (c * A.rmax + (long long)b * A.hkv + (long long)kv * rows) * A.G;
}

// Units of a share for a line of `total` units.
template <class LN>
__device__ __forceinline__ long long line_share(long long total, long long ctas) {
  long long L = (total + ctas - 1) / ctas;
  if (L > LN::MOST) {
    const long long turns = (L + LN::MOST - 1) / LN::MOST;
    L = (total + ctas * turns - 1) / (ctas * turns);
  }
  return L < LN::MIN ? LN::MIN : L;
}

// The line's prefix over the sequences (prefix[b]: units ahead of sequence b)
// by NT threads, `get(b, p, s)` giving sequence b's position and id; returns L.
template <class LN, int NT, typename Get>
__device__ __forceinline__ long long line_plan(Get get, int B, int hkv, int num_seqs, int64_t max_pos, long long max_ctx,
                                               int ctas, int64_t *prefix, unsigned *status, int rmax = 1,
                                               uint8_t *info = nullptr) {
  __shared__ long long s_sum[NT / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long base = 0;
  for (int b0 = 0; b0 < B; b0 += NT) {
    const int b = b0 + tid;
    long long x = 0;
    int u = 0, q = 0;
    if (b < B) {
      long long p;
      get(b, p, q);
      u = line_units<LN>(p, q, num_seqs, max_pos, max_ctx, status);
    }
    if (LN::SHARE) {
      const unsigned joined = line_joined(u > 0, q, lane, rmax);
      int most = u;
      for (int k = 1; k < rmax; ++k) {
        const int y = __shfl_down_sync(FULLW, u, k);
        if (line_follows(joined, lane, k)) most = max(most, y);
      }
      u = joined >> lane & 1 ? 0 : most;
      if (b < B) info[b] = line_info(joined, lane);
    }
    x = u ? (long long)hkv * (u + LN::ROW) : 0;
    const long long mine = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(FULLW, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    long long before = base;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
      before += i < warp ? s_sum[i] : 0;
      base += s_sum[i];
    }
    if (b < B) prefix[b] = before + x - mine;
    __syncthreads();  // s_sum is rewritten by the next round
  }
  if (tid == 0) prefix[B] = base;
  __syncthreads();
  return line_share<LN>(base, ctas);
}

// Sequence of unit x of the line: the last b with prefix[b] <= x whose part is not empty (x < prefix[B]).
__device__ __forceinline__ int line_find(const int64_t *prefix, int B, long long x) {
  int lo = 0, hi = B;  // prefix[lo] <= x < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

constexpr int LINE_PLAN_THREADS = 256;

// Batches past LINE_INLINE_MAX rows: the plan by a kernel of its own.
template <class LN>
__global__ void __launch_bounds__(LINE_PLAN_THREADS)
    line_plan_kernel(const int64_t *__restrict__ pos, const int32_t *__restrict__ seq, int B, int hkv, int num_seqs,
                     int64_t max_pos, long long max_ctx, int ctas, int64_t *__restrict__ plan, unsigned *status, int rmax) {
  pdl_wait();
  pdl_trigger();
  const auto get = [&](int b, long long &p, int &s) { p = pos[b], s = seq[b]; };
  const long long L = line_plan<LN, LINE_PLAN_THREADS>(get, B, hkv, num_seqs, max_pos, max_ctx, ctas, plan + LINE_PLAN, status, rmax,
                                                         reinterpret_cast<uint8_t *>(plan + LINE_PLAN + B + 1));
  if (threadIdx.x == 0) plan[0] = L;
}

// CTA's part of the line from unit x on: row (b, kv), units [lo, hi) of its
// keys (none where hi <= lo: set-up alone); x moves behind it.
template <class LN>
__device__ __forceinline__ void line_part(const int64_t *prefix, int B, int hkv, long long line_end, long long &x, int &b,
                                         int &kv, int &lo, int &hi) {
  b = line_find(prefix, B, x);
  const int rowlen = (int)((prefix[b + 1] - prefix[b]) / hkv);
  kv = (int)((x - prefix[b]) / rowlen);
  const int off = (int)(x - prefix[b] - (long long)kv * rowlen);
  const int stop = (int)min((long long)rowlen, off + (line_end - x));
  x += stop - off;
  lo = max(off - LN::ROW, 0);
  hi = stop - LN::ROW;
}

// Merge of a row's pieces by log-sum-exp, and normalisation: NW warps per
// (sequence, KV head, q head) fold interleaved pieces, lane l the value dims
// 4l..4l+3, LINE_MERGE_K pieces' loads in flight at a time; the row's first warp
// joins them.
constexpr int LINE_MERGE_WARPS = 16;
constexpr int LINE_MERGE_K = 8;

template <class LN>
__global__ void __launch_bounds__(LINE_MERGE_WARPS * 32)
    line_merge_kernel(LineArgs A, int ctas, int nw) {
  __shared__ float s_ml[LINE_MERGE_WARPS][2];
  __shared__ float4 s_acc[LINE_MERGE_WARPS][32];
  __shared__ int64_t s_prefix[LINE_INLINE_MAX + 1];
  const int G = A.G, hkv = A.hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % nw;
  const long long row = (long long)blockIdx.x * (LINE_MERGE_WARPS / nw) + warp / nw;  // (b hkv + kv) G + g
  const bool have = row < (long long)A.B * A.hq;
  const int g = have ? (int)(row % G) : 0, pair = have ? (int)(row / G) : 0, b = pair / hkv, kv = pair - b * hkv;
  __shared__ uint8_t s_info[LINE_INLINE_MAX];
  int lead = 0, rows = 1;  // (a row that goes with one ahead of it has its pieces among that one's)
  // The plan, while the split kernel still runs: that kernel let this one start
  // after its own wait, so the batch (and the plan kernel's plan) are there.
  long long L, at, next;
  if (A.B <= LINE_INLINE_MAX) {
    const auto get = [&](int i, long long &p, int &s) { p = ld_early_s64(A.pos + i), s = ld_early_s32(A.seq + i); };
    L = line_plan<LN, LINE_MERGE_WARPS * 32>(get, A.B, hkv, A.num_seqs, A.max_pos, A.max_ctx, ctas, s_prefix, nullptr, A.rmax,
                                             s_info);
    if (LN::SHARE) lead = line_lead(s_info[b]), rows = line_rows(s_info[b]);
    at = s_prefix[b - lead];
    next = s_prefix[b - lead + 1];
  } else {
    L = ld_early_s64(A.plan);
    if (LN::SHARE) {
      const uint8_t info = __ldcg(reinterpret_cast<const uint8_t *>(A.plan + LINE_PLAN + A.B + 1) + b);
      lead = line_lead(info), rows = line_rows(info);
    }
    at = ld_early_s64(A.plan + LINE_PLAN + b - lead);
    next = ld_early_s64(A.plan + LINE_PLAN + b - lead + 1);
  }
  const long long len = have ? (next - at) / hkv : 0;  // 0: nothing to attend to
  long long c0 = 0;
  int n = 0;
  if (len > 0) {
    c0 = (at + kv * len + LN::ROW) / L;
    n = (int)((at + kv * len + len - 1) / L - c0) + 1;
  }
  pdl_wait();
  pdl_trigger();
  float M = NEG_INF, S = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = sub; i0 < n; i0 += LINE_MERGE_K * nw) {
    float2 ml[LINE_MERGE_K];
    float4 o[LINE_MERGE_K];
#pragma unroll
    for (int k = 0; k < LINE_MERGE_K; ++k) {
      const int i = i0 + k * nw;
      ml[k] = make_float2(NEG_INF, 0.f);
      o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const long long r = line_at(A, c0 + i, b - lead, kv, rows) + lead * G + g;
        ml[k] = *reinterpret_cast<const float2 *>(A.part_ml + r * 2);
        o[k] = *reinterpret_cast<const float4 *>(A.part_o + r * DV + 4 * lane);
      }
    }
    float Mn = M;
#pragma unroll
    for (int k = 0; k < LINE_MERGE_K; ++k) Mn = fmaxf(Mn, ml[k].x);
    if (Mn == NEG_INF) continue;  // nothing yet (pieces without a block of the pool)
    const float c = ex2(M - Mn);  // M = -inf gives 0
    S *= c;
    acc.x *= c;
    acc.y *= c;
    acc.z *= c;
    acc.w *= c;
#pragma unroll
    for (int k = 0; k < LINE_MERGE_K; ++k) {
      const float f = ex2(ml[k].x - Mn);
      S += ml[k].y * f;
      acc.x += o[k].x * f;
      acc.y += o[k].y * f;
      acc.z += o[k].z * f;
      acc.w += o[k].w * f;
    }
    M = Mn;
  }
  if (nw > 1) {
    if (lane == 0) {
      s_ml[warp][0] = M;
      s_ml[warp][1] = S;
    }
    s_acc[warp][lane] = acc;
    __syncthreads();
    if (sub == 0) {
      float Mt = NEG_INF;
      for (int u = 0; u < nw; ++u) Mt = fmaxf(Mt, s_ml[warp + u][0]);
      S = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (Mt != NEG_INF) {
        for (int u = 0; u < nw; ++u) {
          const float mu = s_ml[warp + u][0];
          if (mu == NEG_INF) continue;
          const float f = ex2(mu - Mt);
          const float4 o = s_acc[warp + u][lane];
          S += s_ml[warp + u][1] * f;
          acc.x += o.x * f;
          acc.y += o.y * f;
          acc.z += o.z * f;
          acc.w += o.w * f;
        }
      }
    }
  }
  if (!have || sub != 0) return;
  const float inv = S == 0.f ? 0.f : 1.f / S;  // (a NaN sum stays one)
  *reinterpret_cast<uint2 *>(A.out + ((long long)b * A.hq + (long long)kv * G + g) * DV + 4 * lane) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }
template <class LN>
size_t line_plan_bytes(int B) {
  return align256(((size_t)LINE_PLAN + B + 1) * 8 + (LN::SHARE ? B : 0));
}

// CTAs: as many as the GPU holds at once and as can have a share (of LN::MIN units at least).
template <class LN>
int line_ctas(int B, int hkv, long long max_ctx) {
  const long long units = (long long)B * hkv * ((max_ctx + LN::UNIT - 1) / LN::UNIT + LN::ROW);
  const long long R = (long long)LN::CTAS * num_sms(), most = (units + LN::MIN - 1) / LN::MIN;
  return (int)(most < R ? most : R);
}
// Shares of a CTA on the longest line.
template <class LN>
long long line_turns(int B, int hkv, long long max_ctx) {
  const long long units = (long long)B * hkv * ((max_ctx + LN::UNIT - 1) / LN::UNIT + LN::ROW);
  const long long most = (long long)line_ctas<LN>(B, hkv, max_ctx) * LN::MOST;
  return (units + most - 1) / most;
}
// Partial rows of all pieces (line_at), on the longest line.
template <class LN>
size_t line_partials(int B, int hkv, int G, long long max_ctx, int rmax) {
  return (size_t)((long long)B * hkv + line_ctas<LN>(B, hkv, max_ctx) * line_turns<LN>(B, hkv, max_ctx) * rmax) * G;
}

// Workspace of a call on the line, and its parts.
template <class LN>
size_t line_workspace(int B, int hq, int hkv, long long max_ctx, int rmax = 1) {
  const size_t n = line_partials<LN>(B, hkv, hq / hkv, max_ctx, rmax);
  return line_plan_bytes<LN>(B) + align256(n * 2 * sizeof(float)) + align256(n * DV * sizeof(float));
}
template <class LN>
void line_args(LineArgs &A, const int64_t *pos, const int32_t *seq, int B, int hq, int hkv, int num_seqs, int64_t max_pos,
               long long max_ctx, void *ws, uint16_t *out, int rmax = 1) {
  A.pos = pos;
  A.seq = seq;
  A.B = B;
  A.hq = hq;
  A.G = hq / hkv;
  A.hkv = hkv;
  A.num_seqs = num_seqs;
  A.max_pos = max_pos;
  A.max_ctx = max_ctx;
  A.plan = reinterpret_cast<int64_t *>(ws);
  uint8_t *w8 = reinterpret_cast<uint8_t *>(ws) + line_plan_bytes<LN>(B);
  A.part_ml = reinterpret_cast<float *>(w8);
  A.part_o = reinterpret_cast<float *>(w8 + align256(line_partials<LN>(B, hkv, A.G, max_ctx, rmax) * 2 * sizeof(float)));
  A.out = out;
  A.rmax = rmax;
}

// The launches of a call on the line: the plan where the CTAs do not make it
// themselves, the split kernel, the merge.
template <class LN, class Args>
cudaError_t line_launch(void (*kernel)(Args), int threads, size_t smem, const Args &A, unsigned *status, cudaStream_t st) {
  const int ctas = line_ctas<LN>(A.B, A.hkv, A.max_ctx);  // (a CTA whose share would lie past the line has nothing to do)
  cudaError_t e;
  if (A.B > LINE_INLINE_MAX) {
    e = launch_pdl(line_plan_kernel<LN>, dim3(1), dim3(LINE_PLAN_THREADS), 0, st, A.pos, A.seq, A.B, A.hkv, A.num_seqs,
                   A.max_pos, A.max_ctx, ctas, A.plan, status, A.rmax);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(kernel, dim3((unsigned)ctas), dim3((unsigned)threads), smem, st, A);
  if (e != cudaSuccess) return e;
  // warps per merged row: about four pieces each
  const int est = (int)(LN::CTAS * num_sms() / ((long long)A.B * A.hkv)) + 1;
  int nw = 1;
  while (nw < LINE_MERGE_WARPS && nw * 4 < est) nw *= 2;
  const long long blocks = ((long long)A.B * A.hq + LINE_MERGE_WARPS / nw - 1) / (LINE_MERGE_WARPS / nw);
  return launch_pdl(line_merge_kernel<LN>, dim3((unsigned)blocks), dim3(LINE_MERGE_WARPS * 32), 0, st,
                    static_cast<const LineArgs &>(A), ctas, nw);
}

}  // namespace kvr
