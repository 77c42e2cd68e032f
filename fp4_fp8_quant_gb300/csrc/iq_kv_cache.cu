// Writing and reading the paged 8-bit KV cache (include/iq.h, section 4).
//
// K7 kv_write_kernel.  A page's scale is one power of two for all its tokens
// of one head, so the unit of work is a run of new rows inside one page, per
// KV head, K and V apart: largest magnitude over the run, exponent, codes.
// Where the run starts inside a page that already holds tokens, the exponent
// may only grow, and only if it grows are the older codes read and rounded
// again (an E4M3 code times 2^-d).  One CTA of 128 threads takes the units
// that begin in a window of consecutive rows; the rows of a unit are read
// once, kept in registers between the maximum and the conversion (16 bytes
// per thread and pass), and its codes leave as one contiguous block.  Bound by
// memory: 8 prompts of 1157 to 8192 tokens (230 MB) 40.3 us = 5.7 TB/s; one
// token per sequence by the latency of its lookups, 64 sequences 4.5 us.
//
// K8 kv_read_kernel.  code * 2^e for every row and head in BF16: 16 codes
// in, 32 bytes out per thread for K and for V.  Bound by memory: 16 ragged
// prompts (403 MB) 67.8 us = 5.9 TB/s.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "iq_fp8.cuh"
#include "iq_internal.h"
#include "iq_kv.h"
#include "iq_ptx.cuh"

namespace iq {

namespace {

constexpr int kWriteThreads = 128;
constexpr int kReadThreads = 256;
constexpr int kReadMaxRows = 64;   // rows of one read CTA
constexpr int kReadAtOnce = 2;     // loads in flight per thread, of K and of V (16 ragged prompts, before rounding: 1 73.6 us, 2 66.5, 4 69.1)

// Four E4M3 codes times f, rounded to E4M3 again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t c, float f) {
  const uint32_t lo = cvt_e4m3x2(e4m3_to_float(c) * f, e4m3_to_float(c >> 8) * f);
  const uint32_t hi = cvt_e4m3x2(e4m3_to_float(c >> 16) * f, e4m3_to_float(c >> 24) * f);
  return lo | hi << 16;
}

template <int kDim, int kPage>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(KvArgs a, KvRows x, int window) {
  constexpr int kLanes = kDim / 8;                   // threads per row
  constexpr int kRows = kWriteThreads / kLanes;      // rows per pass
  constexpr int kPasses = (kPage + kRows - 1) / kRows;
  __shared__ uint32_t s_max[2][kWriteThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int h = blockIdx.y, which = blockIdx.z;
  const int row_in_pass = threadIdx.x / kLanes, col = threadIdx.x % kLanes * 8;
  const long long t_begin = static_cast<long long>(blockIdx.x) * window;
  const int t_end = static_cast<int>(min(t_begin + window, static_cast<long long>(a.num_rows)));
  int t = static_cast<int>(t_begin);
  int b = kv_find_seq(a, t);
  int turn = 0;
  while (t < t_end && b < a.num_seqs) {
    const int row_end = min(a.row_start[b + 1], a.num_rows);
    if (t >= row_end) {
      ++b;
      continue;
    }
    const int base = a.kv_len[b] - a.row_start[b + 1];   // position of row t: base + t
    const int row_first = max(a.row_start[b], 0);
    int pos = base + t;
    // The next unit begins at the sequence's first row with a position, or at
    // a page boundary.
    const bool begins = pos >= 0 && ((pos & (kPage - 1)) == 0 || t == row_first || pos == 0);
    if (!begins) {
      t = pos < 0 ? static_cast<int>(min(static_cast<long long>(row_end), static_cast<long long>(t) - pos))
                  : min(row_end, t + kPage - (pos & (kPage - 1)));
      continue;
    }
    const int off = pos & (kPage - 1);
    const int n = min(row_end - t, kPage - off);
    const int pid = kv_page_of(a, b, pos);
    if (pid >= 0) {
      const long long tile = static_cast<long long>(pid) * a.heads + h;
      uint8_t* codes = a.codes[which] + tile * (kPage * kDim);
      uint8_t* sf = a.sf[which] + tile;
      const uint32_t sf_old = off > 0 ? *sf : 0u;
      const uint16_t* src = x.ptr[which] + t * x.ld[which] + h * kDim + col;
      uint4 r[kPasses];
      uint32_t m2 = 0;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int i = p * kRows + row_in_pass;
        r[p] = make_uint4(0, 0, 0, 0);
        if (i < n) r[p] = ld_stream_v4(src + static_cast<long long>(i) * x.ld[which]);
      }
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        m2 = abs_max_bf16x2(m2, r[p].x);
        m2 = abs_max_bf16x2(m2, r[p].y);
        m2 = abs_max_bf16x2(m2, r[p].z);
        m2 = abs_max_bf16x2(m2, r[p].w);
      }
      const uint32_t wmax = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
      if ((threadIdx.x & 31) == 0) s_max[turn][threadIdx.x >> 5] = wmax;
      __syncthreads();                                  // also: every thread has read *sf
      uint32_t m1 = s_max[turn][0];
#pragma unroll
      for (int w = 1; w < kWriteThreads / 32; ++w) m1 = max(m1, s_max[turn][w]);
      turn ^= 1;
      int e = fp8_scale_exponent(__uint_as_float(m1 << 16));
      if (off > 0) {
        const int e_old = static_cast<int>(sf_old) - 127;
        if (e > e_old) {
          // 2^-d is a normal float for d <= 126; a code times less rounds to zero all the same.
          const float f = __uint_as_float(static_cast<uint32_t>(127 - min(e - e_old, 126)) << 23);
          for (int i = threadIdx.x; i < off * kDim / 16; i += kWriteThreads) {
            uint4 c = reinterpret_cast<const uint4*>(codes)[i];
            c.x = rescale_e4m3x4(c.x, f);
            c.y = rescale_e4m3x4(c.y, f);
            c.z = rescale_e4m3x4(c.z, f);
            c.w = rescale_e4m3x4(c.w, f);
            reinterpret_cast<uint4*>(codes)[i] = c;
          }
        } else {
          e = e_old;
        }
      }
      if (threadIdx.x == 0) *sf = static_cast<uint8_t>(e + 127);
      const float inv = fp8_inv_scale(e);
      uint8_t* dst = codes + off * kDim + col;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int i = p * kRows + row_in_pass;
        if (i < n) {
          *reinterpret_cast<uint2*>(dst + i * kDim) =
              make_uint2(quant_quad(r[p].x, r[p].y, inv), quant_quad(r[p].z, r[p].w, inv));
        }
      }
    }
    t += n;
  }
}

// Two E4M3 codes (low 16 bits) times f, as packed BF16.  Exact (four significant
// bits and a power of two) but at the ends of BF16's range, where it rounds.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t c, float f) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(e4m3_to_float(c) * f, e4m3_to_float(c >> 8) * f);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int kDim>
__global__ void __launch_bounds__(kReadThreads, 5) kv_read_kernel(KvArgs a, KvRows out, int rows_per_cta) {
  constexpr int kLanes = kDim / 16;                  // threads per (row, head)
  __shared__ int s_pid[kReadMaxRows], s_off[kReadMaxRows];
  grid_launch_dependents();
  grid_dependency_wait();
  const int t0 = blockIdx.x * rows_per_cta;
  const int rows = min(rows_per_cta, a.num_rows - t0);
  // One thread per row finds its sequence (bisection), page and slot.
  if (threadIdx.x < rows) {
    const int t = t0 + threadIdx.x;
    const int b = kv_find_seq_thread(a, t);
    int pid = -1, off = 0;
    if (b < a.num_seqs) {
      const int pos = a.kv_len[b] - a.row_start[b + 1] + t;
      pid = kv_page_of(a, b, pos);
      off = pos & (a.page - 1);
    }
    s_pid[threadIdx.x] = pid;
    s_off[threadIdx.x] = off;
  }
  __syncthreads();
  const int per_row = a.heads * kLanes, units = rows * per_row;
  const int step_i = kReadThreads / per_row, step_j = kReadThreads - step_i * per_row;
  int i = threadIdx.x / per_row, j = threadIdx.x - i * per_row;   // row, 16 values of it
  for (int u0 = threadIdx.x; u0 < units; u0 += kReadAtOnce * kReadThreads) {
    // All loads before the first store.
    uint4 c[kReadAtOnce][2];
    float f[kReadAtOnce][2];
    int to_i[kReadAtOnce], to_j[kReadAtOnce];
#pragma unroll
    for (int n = 0; n < kReadAtOnce; ++n) {
      to_i[n] = i;
      to_j[n] = j;
      const int pid = u0 + n * kReadThreads < units ? s_pid[i] : -1;
      const int h = j / kLanes, col = j % kLanes * 16;
      const long long tile = static_cast<long long>(pid) * a.heads + h;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        c[n][w] = make_uint4(0, 0, 0, 0);
        f[n][w] = 0.f;
        if (pid >= 0) {
          c[n][w] = ld_stream_v4(a.codes[w] + (tile * a.page + s_off[i]) * kDim + col);
          const uint32_t b = a.sf[w][tile];
          f[n][w] = __uint_as_float(__float_as_uint(ue8m0_to_float(b)) + ((b + 1) >> 8 << 22));   // 255 is NaN
        }
      }
      i += step_i;
      j += step_j;
      if (j >= per_row) {
        j -= per_row;
        ++i;
      }
    }
#pragma unroll
    for (int n = 0; n < kReadAtOnce; ++n) {
      if (u0 + n * kReadThreads >= units) break;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint16_t* dst = out.ptr[w] + (t0 + to_i[n]) * out.ld[w] + to_j[n] * 16;
        uint4 lo, hi;
        lo.x = e4m3x2_to_bf16x2(c[n][w].x, f[n][w]);
        lo.y = e4m3x2_to_bf16x2(c[n][w].x >> 16, f[n][w]);
        lo.z = e4m3x2_to_bf16x2(c[n][w].y, f[n][w]);
        lo.w = e4m3x2_to_bf16x2(c[n][w].y >> 16, f[n][w]);
        hi.x = e4m3x2_to_bf16x2(c[n][w].z, f[n][w]);
        hi.y = e4m3x2_to_bf16x2(c[n][w].z >> 16, f[n][w]);
        hi.z = e4m3x2_to_bf16x2(c[n][w].w, f[n][w]);
        hi.w = e4m3x2_to_bf16x2(c[n][w].w >> 16, f[n][w]);
        *reinterpret_cast<uint4*>(dst) = lo;
        *reinterpret_cast<uint4*>(dst + 8) = hi;
      }
    }
  }
}

template <int kDim>
void (*write_kernel(int page))(KvArgs, KvRows, int) {
  switch (page) {
    case 16: return kv_write_kernel<kDim, 16>;
    case 32: return kv_write_kernel<kDim, 32>;
    case 64: return kv_write_kernel<kDim, 64>;
    default: return kv_write_kernel<kDim, 128>;
  }
}

}  // namespace

cudaError_t launch_kv_cache_write(const KvArgs& a, const KvRows& rows, cudaStream_t stream) {
  // Window: the largest power of two up to the mean number of rows per
  // sequence and the page.  Sequences of one row (decode) then get one CTA
  // each; long ones about one page-sized unit per CTA.  (64 sequences of one
  // row: window 1 4.5 us, a page 69 us; 8 prompts: a page 40 us, 1 1166 us.)
  int window = 1;
  while (window * 2 <= a.page && window * 2 <= a.num_rows / a.num_seqs) window *= 2;
  return launch_dependent(a.dim == 64 ? write_kernel<64>(a.page) : write_kernel<128>(a.page),
                          dim3((a.num_rows + window - 1) / window, a.heads, 2), kWriteThreads, 0, stream, a, rows, window);
}

cudaError_t launch_kv_cache_read(const KvArgs& a, const KvRows& rows, cudaStream_t stream) {
  // Rows per CTA: up to 32768 values of K, fewer where there would not be two
  // CTAs per SM.  (16 ragged prompts, 1024 values per row: 32 rows 66.6 us, 8
  // 67.1, 64 76.5, one 135; 137 rows of 256 values: one row 2.1 us, 64 3.9.)
  int per_cta = kReadMaxRows;
  while (per_cta > 1 && static_cast<long long>(per_cta) * a.heads * a.dim > 32768) per_cta /= 2;
  while (per_cta > 1 && (a.num_rows + per_cta - 1) / per_cta < 304) per_cta /= 2;
  return launch_dependent(a.dim == 64 ? kv_read_kernel<64> : kv_read_kernel<128>,
                          dim3((a.num_rows + per_cta - 1) / per_cta, 1, 1), kReadThreads, 0, stream, a, rows, per_cta);
}

}  // namespace iq
