// kv4_decode.cu -- one-token decode over a full-attention layer kept in 4
// bits.
//
// A key's score takes its scales out of the product,
//   s = scale * sum_g (s_g (q_g . u_g) + m_g sum(q_g)),
// and the values theirs: o = sum_j p_j (s_j u_j + m_j) / sum_j p_j.
//
// First form: one CTA per (sequence, KV head) walks the tiles of 16
// positions; each tile's values go to shared memory in fp32, then scores,
// online softmax and the weighted sum run on the fp32 units.
#include "kv4.cuh"
#include "launch.h"

namespace kvr {
namespace {

constexpr int K4D_THREADS = 128;

__global__ void __launch_bounds__(K4D_THREADS)
    kv4_decode_kernel(const uint16_t *__restrict__ q, const int64_t *__restrict__ pos, const int32_t *__restrict__ seq,
                      int hq, int G, Kv4View pool, const float *__restrict__ table, int64_t max_pos, float scale_log2,
                      long long max_ctx, uint16_t *__restrict__ out, unsigned *status) {
  __shared__ float sQ[16][DQK];
  __shared__ float sK[16][DQK + 1];
  __shared__ float sV[16][DV];
  __shared__ float sS[16][17];
  __shared__ float sM[16], sL[16], sC[16];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int b = blockIdx.x / pool.hkv, kv = blockIdx.x % pool.hkv;
  uint16_t *o = out + ((long long)b * hq + (long long)kv * G) * DV;
  const long long p = pos[b];
  const int s = seq[b];
  const bool bad_pos = p < 0 || p >= max_pos || p + 1 > max_ctx, bad_seq = s < 0 || s >= pool.num_seqs;
  if (bad_pos || bad_seq) {
    if (kv == 0 && tid == 0) flag(status, (bad_pos ? ST_BAD_POS : 0u) | (bad_seq ? ST_BAD_SEQ : 0u));
    for (int e = tid; e < G * DV; e += K4D_THREADS) o[e] = 0;
    return;
  }
  for (int e = tid; e < 16 * DQK; e += K4D_THREADS) {
    const int g = e / DQK, d = e % DQK;
    float x = 0.f;
    if (g < G) {
      const uint16_t *qr = q + ((long long)b * hq + (long long)kv * G + g) * DQK;
      x = bf2f(qr[d]);
      if (d < DROT) {
        const float c = table[p * 64 + 2 * (d & 31)], sn = table[p * 64 + 2 * (d & 31) + 1];
        x = d < HALF ? x * c - bf2f(qr[d + HALF]) * sn : x * c + bf2f(qr[d - HALF]) * sn;
      }
    }
    sQ[g][d] = x * scale_log2;
  }
  if (tid < 16) {
    sM[tid] = -INFINITY;
    sL[tid] = 0.f;
  }
  float O[16];
#pragma unroll
  for (int g = 0; g < 16; ++g) O[g] = 0.f;
  for (long long p0 = 0; p0 <= p; p0 += 16) {
    const int blk = pool.block_table[(long long)s * pool.max_blocks + p0 / pool.block_size];
    if (blk < 0 || blk >= pool.num_blocks) {
      if (tid == 0) flag(status, ST_BAD_BLOCK);
      continue;
    }
    const uint8_t *tile = pool.data + kv4_tile(pool, blk, kv, (int)(p0 % pool.block_size));
    auto half_at = [&](int off) -> float {
      return __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t *>(tile + off)));
    };
    __syncthreads();
    for (int e = tid; e < 16 * DQK; e += K4D_THREADS) {
      const int r = e / DQK, d = e % DQK, g = d / 64, i = d % 64;
      const int u = tile[kv4_k_at(g, r, i / 16) + (i % 16) / 2] >> (4 * (i & 1)) & 15;
      sK[r][d] = fmaf((float)u, half_at(KV4_OFF_KS + (g * 16 + kv4_quad(r)) * 2), half_at(KV4_OFF_KM + r * 8 + g * 2));
    }
    for (int e = tid; e < 16 * DV; e += K4D_THREADS) {
      const int r = e / DV, d = e % DV, g = d / 64, i = d % 64;
      const int u = tile[kv4_v_at(g, r, i / 8, i % 8 / 4) + (i % 4) / 2] >> (4 * (i & 1)) & 15;
      const float x = fmaf((float)u, half_at(KV4_OFF_VS + (g * 16 + kv4_quad(r)) * 2),
                           half_at(KV4_OFF_VM + (g * 16 + kv4_quad(r)) * 2));
      sV[r][d] = p0 + r <= p ? x : 0.f;
    }
    __syncthreads();
    for (int e = tid; e < 256; e += K4D_THREADS) {
      const int g = e >> 4, r = e & 15;
      float x = 0.f;
      for (int d = 0; d < DQK; ++d) x = fmaf(sQ[g][d], sK[r][d], x);
      sS[g][r] = p0 + r <= p ? x : -INFINITY;
    }
    __syncthreads();
    if (tid < 16) {
      float m = sM[tid];
      for (int r = 0; r < 16; ++r) m = fmaxf(m, sS[tid][r]);
      const float base = m == -INFINITY ? 0.f : m;
      const float c = ex2(sM[tid] - base);
      float l = sL[tid] * c;
      for (int r = 0; r < 16; ++r) {
        const float w = ex2(sS[tid][r] - base);
        sS[tid][r] = w;
        l += w;
      }
      sM[tid] = m;
      sL[tid] = l;
      sC[tid] = c;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < 16; ++g) {
      float x = O[g] * sC[g];
      for (int r = 0; r < 16; ++r) x = fmaf(sS[g][r], sV[r][tid], x);
      O[g] = x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 16; ++g)
    if (g < G) o[g * DV + tid] = f2bf(sL[g] == 0.f ? 0.f : O[g] / sL[g]);
}

}  // namespace

size_t kv4_decode_workspace(int B, int hq, int hkv, long long max_ctx) { return full_decode_workspace(B, hq, hkv, max_ctx); }

cudaError_t launch_kv4_decode(const uint16_t *q, const int64_t *pos, const int32_t *seq, int B, int hq,
                              const Kv4View &pool, const float *table, int64_t max_pos, float softmax_scale,
                              long long max_ctx, void *, uint16_t *out, unsigned *status, cudaStream_t st) {
  return launch_pdl(kv4_decode_kernel, dim3((unsigned)(B * pool.hkv)), dim3(K4D_THREADS), 0, st, q, pos, seq, hq,
                    hq / pool.hkv, pool, table, max_pos, softmax_scale * LOG2E, max_ctx, out, status);
}

}  // namespace kvr
