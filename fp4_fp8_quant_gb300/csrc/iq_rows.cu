// K19: the FP8 1x128 quantizer over a list of rows (include/iq.h, section 5):
// output row s holds the codes and scales of row rows[s] of x, or of a row of zeros
// where that is outside [0, num_src).
//
// The arithmetic of a unit (a row's four 128-blocks, by a warp) is the quantizer's
// own (iq_fp8.cuh).  The columns of all rows come one after the other, so that a
// row named several times is read again while it is in L2.  37056 rows naming each of
// 4632 eight times, 7168 columns: 82 us, of which writing alone takes 72 (266 MB; this
// memory is written at 3.7 TB/s); rows first 10 us more.  Blocks of 128 threads, a
// row's place from the grid: 64 x 8 rows 3.1 us, with a division by the number of rows
// 4.1.

#include <cuda_runtime.h>

#include <cstdint>

#include "iq_fp8.cuh"
#include "iq_internal.h"
#include "iq_kv.h"
#include "iq_moe.h"
#include "iq_ptx.cuh"

namespace iq {

namespace {

constexpr int kThreads = 128;

// Units of a warp.  The list's entry is one load ahead of the row's, so a warp
// takes several units side by side, all their loads in flight (37056 rows of 7168
// columns: one 132 us, two 84, four 82, but 64 x 8 rows 4.2 instead of 3.1).
constexpr int kListed = 2;
constexpr int kMaxGridY = 65535;                 // of a launch; columns past 67 million go into the third dimension

// Through L1, where a lane's second half finds the line of its first and rows that
// all name one another's (a list of zeros: 79 us, past L1 303).  (Keeping x's lines in
// L2 before others: 84.)  Ordinary loads: the kernel before this one, which may write
// x, is still running when this one starts, and the read-only path has no duty to see it.
__device__ __forceinline__ uint4 ld_cached_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

__global__ void __launch_bounds__(kThreads)
    quant_1x128_listed_kernel(const uint16_t* __restrict__ x, int num_src, const int32_t* __restrict__ rows, int M, int K,
                              long long ldx, uint8_t* __restrict__ y, long long ldy, int32_t* __restrict__ sf, int m_al,
                              int groups) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, g0 = (blockIdx.y + blockIdx.z * kMaxGridY) * kListed;
  const long long row = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= m_al || g0 >= groups) return;
  const int from = row < M ? static_cast<int>(ld_dependent_u32(rows + row)) : -1;
  const bool there = static_cast<unsigned>(from) < static_cast<unsigned>(num_src);
  uint4 a[kListed], b[kListed];
#pragma unroll
  for (int i = 0; i < kListed; ++i) {
    const int col = (g0 + i) * 512 + lane * 16;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (there && col < K) {
      a[i] = ld_cached_v4(x + from * ldx + col);
      b[i] = ld_cached_v4(x + from * ldx + col + 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kListed; ++i) {
    const int g = g0 + i, col = g * 512 + lane * 16;
    if (g >= groups) break;
    const bool active = row < M && col < K;
    uint4 out;
    const uint32_t word = fp8_quant_unit(a[i], b[i], active, out);
    if (active) *reinterpret_cast<uint4*>(y + row * ldy + col) = out;
    if (lane == 0) sf[static_cast<long long>(g) * m_al + row] = static_cast<int32_t>(word);
  }
}

}  // namespace

cudaError_t launch_quant_1x128_listed(const void* x, int num_src, const int32_t* rows, int M, int K, long long ldx, void* y,
                                      long long ldy, int32_t* sf, cudaStream_t stream) {
  const int m_al = (M + 3) / 4 * 4, groups = (K + 511) / 512, pieces = (groups + kListed - 1) / kListed;
  const dim3 grid((static_cast<unsigned>(m_al) + kThreads / 32 - 1) / (kThreads / 32), pieces < kMaxGridY ? pieces : kMaxGridY,
                  (pieces + kMaxGridY - 1) / kMaxGridY);
  return launch_dependent(quant_1x128_listed_kernel, grid, kThreads, 0, stream,
                          static_cast<const uint16_t*>(x), num_src, rows, M, K, ldx, static_cast<uint8_t*>(y), ldy, sf, m_al,
                          groups);
}

}  // namespace iq
