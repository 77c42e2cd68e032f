// The paged 8-bit KV cache as the kernels see it, shared by the cache
// kernels, the attention kernels and the C-ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace iq {

// One batch over one cache (include/iq.h, iq_kv_cache and iq_kv_batch).
struct KvArgs {
  uint8_t* codes[2];        // K, V: [num_pages][heads][page][dim]
  uint8_t* sf[2];           // K, V: [num_pages][heads]
  const int32_t* table;     // [num_seqs][table_ld]
  const int32_t* row_start; // [num_seqs + 1]
  const int32_t* kv_len;    // [num_seqs]
  long long table_ld;
  int num_pages;
  int heads;
  int page;
  int page_log2;
  int dim;
  int max_pages;
  int num_seqs;
  int num_rows;
};

// BF16 rows of K and V: row t at ptr + t * ld elements.
struct KvRows {
  uint16_t* ptr[2];
  long long ld[2];
};

cudaError_t launch_kv_cache_write(const KvArgs& a, const KvRows& rows, cudaStream_t stream);
cudaError_t launch_kv_cache_read(const KvArgs& a, const KvRows& rows, cudaStream_t stream);

struct AttnArgs {
  KvArgs kv;
  const uint16_t* q;        // row t at q + t * ldq, [q_heads][dim]
  long long ldq;
  uint16_t* out;            // row t at out + t * ldo
  long long ldo;
  const int32_t* indices;   // [num_rows][ld_idx] or nullptr: all visible keys
  long long ld_idx;
  int topk;
  int q_heads;
  int group;                // query heads per KV head
  float scale_log2;         // softmax scale * log2(e)
};

// tm_k, tm_v: the codes as matrices [num_pages * heads * page][dim]; boxes of
// one page (all visible keys) or of one row (selected keys), 128-byte swizzle
// (64-byte with dim 64).
cudaError_t kv_attention_setup_device();
size_t kv_attention_workspace(int num_rows, int q_heads, int kv_heads, int dim);
cudaError_t launch_kv_attention(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a, void* ws,
                                int sm_count, unsigned long long timeout_ns, cudaStream_t stream);
cudaError_t read_kv_status(uint32_t* flags, bool reset);

#ifdef __CUDACC__

// Launches a kernel that may start before the one ahead of it has completed
// (and waits for that itself).
template <typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The sequence row t belongs to: the number of sequences that end at or
// before t (num_seqs when t is past the last row).  Called by a whole warp,
// every lane gets the result: the ends of 32 equal blocks of sequences at a
// time, so up to 32 sequences take one load's latency and 1024 two.
__device__ __forceinline__ int kv_find_seq(const KvArgs& a, int t) {
  int lo = 0, n = a.num_seqs;                        // it lies in [lo, lo + n]
  while (n > 0) {
    const int block = (n + 31) >> 5, last = (static_cast<int>(threadIdx.x & 31) + 1) * block - 1;
    const bool past = last < n && a.row_start[lo + last + 1] <= t;
    const int skip = __popc(__ballot_sync(0xFFFFFFFFu, past)) * block;
    lo += skip;
    n = min(block - 1, n - skip);
  }
  return lo;
}

// The same by one thread alone: bisection over the sequences' ends.
__device__ __forceinline__ int kv_find_seq_thread(const KvArgs& a, int t) {
  int lo = 0, hi = a.num_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.row_start[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Page of a position of sequence b, or -1 when there is none.
__device__ __forceinline__ int kv_page_of(const KvArgs& a, int b, int pos) {
  const int j = pos >> a.page_log2;
  if (pos < 0 || j >= a.max_pages) return -1;
  const int pid = a.table[static_cast<long long>(b) * a.table_ld + j];
  return static_cast<unsigned>(pid) < static_cast<unsigned>(a.num_pages) ? pid : -1;
}

// 2^(b - 127) of a UE8M0 byte; b = 0 is the float32 subnormal 2^-127, and 255,
// which stands for NaN, gives an infinity.  (NaN itself would cost the prompt
// kernel 2 % and chunks 8 %, for keys and values that no call has to take.)
__device__ __forceinline__ float ue8m0_to_float(uint32_t b) {
  return __uint_as_float(max(b << 23, 0x400000u));
}

#endif

}  // namespace iq
