// The experts' feed-forward block (routing, grouped products, combination) and
// the per-request adapters, as the kernels see them; shared by the kernels and
// the C-ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace iq {

constexpr int kMaxGroups = 1024;   // groups of one grouped product (their row bounds are kept in shared memory)

// The FP8 1x128 quantizer (iq_internal.h, launch_quant_1x128) over a list of M rows
// of x (num_src rows); a row outside is zeros.
cudaError_t launch_quant_1x128_listed(const void* x, int num_src, const int32_t* rows, int M, int K, long long ldx, void* y,
                                      long long ldy, int32_t* sf, cudaStream_t stream);

struct RouteArgs {
  const void* logits;        // [tokens][ld] float32 or BF16
  long long ld;
  int tokens;
  int experts;
  int k;
  bool bf16;
  bool sigmoid;
  bool normalize;
  float scale;
  float* weights;            // [tokens][k]
  int32_t* out_experts;      // [tokens][k]
  int32_t* slots;            // [tokens][k]
  int32_t* rows;             // [tokens * k]
  int32_t* row_start;        // [experts + 1]
  int* counts;               // workspace: [blocks + 1][experts]
  int block_tokens;          // tokens of a block; found at the launch
};

constexpr int kMaxChosen = 32;     // experts of one token (a lane each)

size_t route_workspace(int tokens, int experts);
cudaError_t route_setup_device();
cudaError_t launch_route(RouteArgs a, int sm_count, cudaStream_t stream);

struct CombineArgs {
  const uint16_t* y;         // row s at y + s * ldy
  long long ldy;
  int rows;                  // of y
  const int32_t* slots;      // [tokens][k]
  const float* weights;      // [tokens][k]
  const uint16_t* add;       // row t at add + t * ld_add, or nullptr
  long long ld_add;
  uint16_t* out;             // row t at out + t * ld_out
  long long ld_out;
  int tokens;
  int k;
  int cols;
};

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream);

// K of a grouped product: the units of two tiles per pair fit 32 bits.
constexpr int kMaxGroupedK = 1 << 20;

struct GroupedArgs {
  const int32_t* x_sf;       // [ceil(K / 512)][m_al] packed UE8M0 words
  const uint8_t* w_sf;       // [groups][n_blocks][k_blocks]
  const int32_t* row_start;  // [groups + 1]
  uint16_t* y;               // row m at y + m * ldy
  long long ldy;
  int M;
  int m_al;
  int groups;
  int n;                     // weight rows per group
  int n_out;                 // output columns: n, or n / 2 gated
  int n_blocks;
  int k_blocks;
  int f_tiles;               // feature tiles of a pair
  int widest;                // token columns of the widest tile
  int short_rows;            // rows of a box of tm_x
  int tall_rows;             // and of tm_tall
  int pairs;                 // CTA pairs launched
  float* part;               // [2 * pairs][2 CTAs][widest][128] partial sums of cut tiles; nullptr: none is cut
  int4* heads;               // [2 * pairs] header of the tile cut at the end of each pair's run
  unsigned long long timeout_ns;
};

// Boxes are of 128 bytes of K, two K-blocks at a time, the K-blocks outermost:
// tm_x, tm_tall: [K / 128][M][128], boxes of grouped_short_rows(M) and of
// grouped_widest(M) / 2 rows; tm_w plain: [groups][K / 128][n][128], boxes of 128
// rows; gated [K / 128][groups * n / 16][2][16][128], 16 gate rows and the same 16
// up rows in turn, boxes of 128 rows.  128-byte swizzle.
int grouped_widest(int M);
int grouped_short_rows(int M);
cudaError_t grouped_setup_device();
size_t grouped_workspace(int M, int K);     // enough for all calls of up to M rows
size_t grouped_need(int M, int K);          // what a call of M rows uses, possibly nothing
cudaError_t launch_grouped(const CUtensorMap& tm_x, const CUtensorMap& tm_tall, const CUtensorMap& tm_w, GroupedArgs a, bool gated,
                           void* ws, int max_pairs, cudaStream_t stream);
cudaError_t read_grouped_status(uint32_t* flags, bool reset);

constexpr int kMaxRequests = 1024;   // of one adapter call (their rows are kept in shared memory)
constexpr int kMaxRank = 128;        // rows of A: lanes of the accumulator

struct AdapterArgs {
  const uint16_t* base;      // row t at base + t * ld_base, or nullptr
  long long ld_base;
  uint16_t* out;             // row t at out + t * ld_out
  long long ld_out;
  const float* scale;        // [adapters]
  const int32_t* row_start;  // [requests + 1]
  const int32_t* adapter;    // [requests]
  int tokens;
  int requests;
  int adapters;
  int rank;
  int cols;                  // N
  int k_blocks;              // ceil(K / 64)
  int f_tiles;               // ceil(N / 128)
  bool whole_steps;          // K % 64 == 0: a step's K-blocks come with one load
  int step;                  // K-blocks of a step; the rest is derived at the launch
  int k_steps;
  int tall_rows;
  int stage_bytes;
  int stages;
  int down_ctas;
  int down_least;            // units of the shortest of their runs
  float* part;               // parts of V, see adapters_workspace
  unsigned long long timeout_ns;
};

// BF16, 128-byte swizzle.  With K % 64 == 0 x is [K / 64][tokens][64] and A
// [adapters][K / 64][rank][64], in boxes of adapters_step() K-blocks; else
// [1][tokens][K] and [adapters][1][rank][K], in boxes of one.  Boxes of x have 8, 64
// and adapters_tall_rows() rows, those of A all of the rank's; b: [adapters][N][rank],
// boxes of 128 rows x 64.
struct AdapterMaps {
  CUtensorMap x8, x64, tall, a, b;
};
int adapters_tall_rows(int tokens);
int adapters_step(int tokens, int rank);
bool adapters_countable(int tokens, int requests, int rank, int K, int N);   // units are counted in 32 bits
cudaError_t adapters_setup_device();
size_t adapters_workspace(int tokens, int rank);
cudaError_t launch_adapters(const AdapterMaps& m, AdapterArgs a, void* ws, int sm_count, cudaStream_t stream);
cudaError_t read_adapters_status(uint32_t* flags, bool reset);

#ifdef __CUDACC__

// 16 lanes x 32 columns of tensor memory: thread t receives, for columns 8j ..
// 8j + 7, lane t / 4 columns 2 (t % 4) and + 1 in v[4j], v[4j + 1] and lane
// t / 4 + 8 in v[4j + 2], v[4j + 3]: what stmatrix takes.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Stores four 8x8 matrices of 16-bit values transposed; lane l gives the
// address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

#endif

}  // namespace iq
