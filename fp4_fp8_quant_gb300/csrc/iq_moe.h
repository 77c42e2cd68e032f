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
  int* counts;               // workspace: [blocks][experts]
};

constexpr int kMaxChosen = 32;     // experts of one token (a lane each)

size_t route_workspace(int tokens, int experts);
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);

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
  int join_pairs;            // CTA pairs launched
  float* part;               // [2 * pairs][2 CTAs][widest][128] partial sums of cut tiles
  int4* heads;               // [2 * pairs] header of the tile cut at the end of each pair's run
  unsigned long long timeout_ns;
};

// tm_x: [M][K] codes, boxes of 32 rows x 128 bytes.  tm_w: plain [groups][n][K],
// boxes of 128 rows; gated [groups][2][n / 2][K], boxes of 16 rows of both
// halves; 128-byte swizzle.
cudaError_t grouped_setup_device();
size_t grouped_workspace(int M);
cudaError_t launch_grouped(const CUtensorMap& tm_x, const CUtensorMap& tm_w, GroupedArgs a, bool gated, void* ws,
                           int max_pairs, cudaStream_t stream);
cudaError_t read_grouped_status(uint32_t* flags, bool reset);

}  // namespace iq
