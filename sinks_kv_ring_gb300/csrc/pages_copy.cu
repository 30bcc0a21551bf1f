// pages_copy.cu -- whole blocks of one or more pools copied, by a list of
// (source, destination) ids that a fork or a compaction made on the device: what
// follows kv_pages_fork and kv_pages_compact in every layer that shares their
// block table.
//
// A plane is one array of equal blocks (the K or the V of a bf16 pool, the data of
// a quantised one).  Pairs x planes x pieces of PC_PIECE bytes are laid on one
// line, which the CTAs take in strides, so all layers go in one launch whatever
// the count is (the host does not know it).
//
// What bounds it: HBM.  1440 blocks of 82 KB in each of three layers (710 MB read
// and written) take 112 to 116 us, 0.90 to 0.93 of the copy rate; 4 loads in flight
// a thread 123, four CTAs an SM 123, 32-byte loads 111 but 5% more on what L2 holds.
#include "launch.h"

namespace kvr {
namespace {

constexpr int PC_THREADS = 256;
constexpr int PC_EACH = 8;  // 16-byte loads of a thread in flight
constexpr int PC_PIECE = PC_THREADS * PC_EACH * 16;
constexpr int PC_CTAS = 8;  // per SM

struct CopyArgs {
  uint8_t *data[PAGES_COPY_PLANES];
  long long bytes[PAGES_COPY_PLANES];       // of a block
  int first[PAGES_COPY_PLANES + 1];         // pieces of a pair ahead of the plane
  int planes, num_blocks, n;
  const int32_t *src, *dst, *count;
  unsigned *status;
};

__global__ void __launch_bounds__(PC_THREADS) pages_copy_kernel(const __grid_constant__ CopyArgs A) {
  pdl_wait();
  pdl_trigger();
  const int count = min(*A.count, A.n), per = A.first[A.planes];
  const long long all = (long long)max(count, 0) * per;
  for (long long u = blockIdx.x; u < all; u += gridDim.x) {
    const int k = (int)(u / per), piece = (int)(u - (long long)k * per);
    const int s = A.src[k], d = A.dst[k];
    if (s < 0 || s >= A.num_blocks || d < 0 || d >= A.num_blocks) {
      if (piece == 0 && threadIdx.x == 0) flag(A.status, ST_BAD_BLOCK);
      continue;
    }
    int p = 0;
    while (piece >= A.first[p + 1]) ++p;
    const long long bytes = A.bytes[p], off = (long long)(piece - A.first[p]) * PC_PIECE;
    const int left = (int)min((bytes - off) >> 4, (long long)PC_THREADS * PC_EACH);  // 16-byte words
    const uint4 *from = reinterpret_cast<const uint4 *>(A.data[p] + s * bytes + off);
    uint4 *to = reinterpret_cast<uint4 *>(A.data[p] + d * bytes + off);
    uint4 x[PC_EACH];
#pragma unroll
    for (int i = 0; i < PC_EACH; ++i) {
      const int at = i * PC_THREADS + (int)threadIdx.x;
      if (at < left) x[i] = from[at];
    }
#pragma unroll
    for (int i = 0; i < PC_EACH; ++i) {
      const int at = i * PC_THREADS + (int)threadIdx.x;
      if (at < left) to[at] = x[i];
    }
  }
}

}  // namespace

cudaError_t launch_pages_copy(uint8_t *const *data, const long long *bytes, int planes, int num_blocks,
                              const int32_t *src, const int32_t *dst, const int32_t *count, int n, unsigned *status,
                              cudaStream_t st) {
  for (int p0 = 0; p0 < planes; p0 += PAGES_COPY_PLANES) {
    CopyArgs A;
    A.planes = planes - p0 < PAGES_COPY_PLANES ? planes - p0 : PAGES_COPY_PLANES;
    long long per = 0;
    for (int p = 0; p < A.planes; ++p) {
      A.data[p] = data[p0 + p];
      A.bytes[p] = bytes[p0 + p];
      A.first[p] = (int)per;
      per += (bytes[p0 + p] + PC_PIECE - 1) / PC_PIECE;
    }
    if (per > 0x7fffffffLL) return cudaErrorInvalidValue;  // (a block of 2^46 bytes)
    A.first[A.planes] = (int)per;
    A.num_blocks = num_blocks;
    A.n = n;
    A.src = src;
    A.dst = dst;
    A.count = count;
    A.status = status;
    const long long all = per * n, most = (long long)PC_CTAS * num_sms();
    const cudaError_t e = launch_pdl(pages_copy_kernel, dim3((unsigned)(all < most ? all : most)), dim3(PC_THREADS), 0, st, A);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kvr
