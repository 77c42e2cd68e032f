// Matrix products grouped by expert with ragged sizes (include/iq.h, section 5):
//   y[m, n] = sum_kb 2^(ex[m, kb] + ew[g, n / 128, kb]) sum_{k in kb} x[m, k] w[g, n, k]
// for the rows m of group g, row_start[g] <= m < row_start[g + 1]; gated: the
// weights hold gate rows and then up rows, and silu(gate) * up comes out.
//
// K12 grouped_gemm_kernel.  The weights are the MMA's M side, 256 of them over a
// CTA pair (tcgen05 cta_group::2, kind::mxf8f6f4 with block scales), and the
// group's rows its N side, which takes any multiple of 16 up to 256: rows are
// divided into the fewest equal tiles, so that a group of one row costs little
// more than reading its weights, and no group is padded by more than 15 rows per
// tile.  An MMA of 256 x N x 32 takes some 130 cycles up to N = 224 and 150 at 256:
// loading the weights' side is what it waits for, so wide tiles are what count.
// The scales are powers of two per 128 of K; the MMA takes one per 32, so each is
// used four times (the instruction descriptor picks the byte of the packed word):
// exact.
//
// Gated.  A tensor map of five dimensions loads 16 gate rows and the 16 up rows
// that belong to them in turn, so that a thread that reads accumulator lanes
// l and l + 16 holds gate and up of one feature: silu is taken in registers.
//
// Roles (384 threads, one CTA per SM): warps 0..7 epilogue, 8 producer, 9 MMA
// issuer (leader CTA), 10 and 11 scales.
//   - A stage holds two K-blocks: one wait, two loads and one commit for eight
//     MMAs.  What an issuing warp does between MMAs has to be short: with a K-block
//     per stage, four loads of 32 rows each and issue from one lane, the producer
//     took longer than the MMAs (4632-token prompt, first product 1186 us, second
//     522; 877 and 492 with two loads).
//   - Scales go through shared to tensor memory in groups of four K-blocks, loaded
//     by two warps that are a group ahead of what they publish: their loads'
//     latency was what a group took (877 -> 776 us).
//   - Two accumulators; up to 224 columns each they do not touch, wider ones share
//     at most 64 columns, which the epilogue reads and gives back first.
//   - The epilogue reads the accumulator in the 16x256b shape, whose registers are
//     what stmatrix takes: rounded pairs are stored transposed and leave as rows,
//     64 (gated 32) bytes per row and warp.
//
// Division: see Walker and cut_steps.  Tiles that run at a time lie side by side;
// a run of consecutive tiles per pair instead made every pair read its own group's
// weights from HBM (first product 1737 us against 1186).
//
// Measured (one GB300; in a CUDA graph; the rows' quantiser included): 64 experts,
// 7168 -> 2 x 2048 gated: 4632 tokens x 8 (37056 rows) 833 us, of which the product
// is 750 = 2.9 PFLOP/s at 1.9 GHz (under the power limit, at 1.45 GHz, 850); its
// MMAs alone, without loads or epilogue, 598.  64 tokens x 8 301 us = 6.3 TB/s (92 %
// of the measured copy rate); one token 47.5 us = 5.0 TB/s, of which some 7 us are
// beginning and end.  2048 -> 7168, 37056 rows: 446 us; MMAs alone 338, the
// epilogue's stores (531 MB) and its share of shared memory make the difference.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "iq_internal.h"
#include "iq_kv.h"
#include "iq_moe.h"
#include "iq_ptx.cuh"

namespace iq {

__device__ uint32_t g_iq_status_grouped;

namespace {

constexpr int kPair = 2;
constexpr uint16_t kPairMask = 0x3;
constexpr int kMaxWidth = 256;                   // token columns of a tile
constexpr int kLanes = 128;                      // weight rows of a CTA
constexpr int kWBytes = kLanes * 128;            // of one K-block
constexpr int kStep = 2;                         // K-blocks of a stage
constexpr int kSfStages = 4;                     // groups of four K-blocks whose scales are held
constexpr int kSfBytes = (128 + 256) * 4;        // scales of 128 weight rows and 256 token rows
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = kEpiWarps, kMmaWarp = kProducerWarp + 1, kScaleWarp = kMmaWarp + 1;
constexpr int kThreads = (kEpiWarps + 4) * 32;
constexpr int kWarps = kThreads / 32;
constexpr int kStageBytes = 2048;                // output staging of a warp: 32 rows x 32 features
constexpr uint32_t kTmemCols = 512;
constexpr int kAccCols = 448;                    // of the two accumulators
constexpr int kOverlap = 2 * kMaxWidth - kAccCols;
static_assert(kOverlap == 64, "one turn of the epilogue's warps");
constexpr uint32_t kSfCol = kAccCols;            // + 16 s: weights 4 columns, rows 8 columns at + 8
constexpr int kMaxPairs = 80;

// Units of work: a step of a tile of w columns weighs kUnitBase + w, beginning and
// ending a tile kUnitEnds more.
constexpr int kUnitBase = 512;
constexpr int kUnitEnds = 512;
// What cutting costs in steps: every part's way through the workspace, and the
// join's.  It pays where the steps that pairs would be idle for, per pair, are more.
// us per call in a CUDA graph, whole / cut, by those idle steps (76 pairs):
//   16 columns:   4.4 26.0 / 28.7    5.9 52.2 / 53.9    8.8 44.9 / 47.2   11.8 49.8 / 48.4
//                14.7 49.2 / 45.9   20.6 48.2 / 40.8
//   176 columns: 23.6 26.6 / 18.2
//   256 columns: 13.3 31.2 / 32.1   14.7 58.2 / 64.7   17.9 22.6 / 19.3   20.6 56.9 / 55.9
//                25.1 82.0 / 78.8
// The price is that of the widest tile that M rows can make, which the workspace goes
// by, not of the groups' own: 14 or 15 groups of 16 rows (11.8 and 14.7 above, priced
// at 16) and 64 tokens x 8 over 64 experts (tiles of 16 columns, 14.7 idle steps, priced
// at 17; 300.5 / 296.9) are dealt out whole, which is the slower way.  K13 is launched
// wherever a tile could be cut: 1.2 us of the whole ones up to 16 rows, 5.6 from 256 on.
__host__ __device__ __forceinline__ int cut_steps(int width) { return 9 + width / 32; }

// kNarrow: no tile is wider than kNarrowWidth columns, so a stage holds fewer
// token rows and there are more stages.
constexpr int kNarrowWidth = 64;
template <bool kNarrow>
struct Layout {
  static constexpr int kStages = kNarrow ? 4 : 3;
  static constexpr int kXBytes = (kNarrow ? kNarrowWidth : kMaxWidth) / 2 * 128;   // of one K-block
  static constexpr int kOffX = kStages * kStep * kWBytes;
  static constexpr int kOffSf = kOffX + kStages * kStep * kXBytes;
  static constexpr int kOffOut = kOffSf + kSfStages * kSfBytes;
  static constexpr int kOffWork = kOffOut + kEpiWarps * kStageBytes;          // Work: int [3][kMaxGroups + 1]
  static constexpr int kNumBars = 2 * kStages + 2 * kSfStages + 6 + 1;
  static constexpr int kOffBar = (kOffWork + 3 * (kMaxGroups + 1) * 4 + 7) & ~7;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;                     // tensor-memory address, abort flag, warps' sums
  static constexpr int kSmemBytes = kOffMisc + 16 + kWarps * 4;
  static_assert(kOffX % 1024 == 0 && kXBytes % 1024 == 0 && kOffSf % 128 == 0 && kOffOut % 16 == 0 && kOffBar % 8 == 0,
                "alignment");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};
static_assert(kSfCol + 16 * kSfStages <= kTmemCols, "tensor memory");

__device__ __forceinline__ void fail(volatile uint32_t* abort_flag, uint32_t bit) {
  atomicOr(&g_iq_status_grouped, bit);
  *abort_flag = 1u;
}

// ---- instruction pieces: the CTA-pair forms, issued by a whole warp, which
// elects a lane.  Operands are known to be the same in all lanes (`uniform`).

// The same value in every lane, known as such to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// The four MMAs of a K-block: 32 bytes along K of both operands at a time, inside
// the 128-byte swizzle atom.  a, b: low words of the operands' descriptors, whose
// high words are those of smem_desc_sw128.
__device__ __forceinline__ void mma_k_block(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
  constexpr uint32_t kHi = (1024u >> 4) | 1u << 14 | 2u << 29;
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %12, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 a0, {%1, %14};\n\tmov.b64 a1, {%2, %14};\n\tmov.b64 a2, {%3, %14};\n\tmov.b64 a3, {%4, %14};\n\t"
      "mov.b64 b0, {%5, %14};\n\tmov.b64 b1, {%6, %14};\n\tmov.b64 b2, {%7, %14};\n\tmov.b64 b3, {%8, %14};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a0, b0, %9, [%10], [%11], p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, %9, [%10], [%11], t;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, %9, [%10], [%11], t;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, %9, [%10], [%11], t;\n\t}" ::"r"(d),
      "r"(a), "r"(a + 2), "r"(a + 4), "r"(a + 6), "r"(b), "r"(b + 2), "r"(b + 4), "r"(b + 6), "r"(idesc), "r"(sfa), "r"(sfb),
      "r"(accumulate), "r"(0), "r"(kHi)
      : "memory");
}

// Two tcgen05.cp 32x128b (each CTA's shared memory to its own tensor memory), and
// a third one if `more`.  sf: low word of the first tile's descriptor; the tiles
// are 512 bytes apart.
__device__ __forceinline__ void cp_scales(uint32_t cols, uint32_t sf, uint32_t more) {
  constexpr uint32_t kHi = (128u >> 4) | 1u << 14;      // of smem_desc_sf
  asm volatile(
      "{\n\t.reg .pred e, m;\n\t.reg .b64 s0, s1, s2;\n\tsetp.ne.b32 m, %6, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 s0, {%3, %7};\n\tmov.b64 s1, {%4, %7};\n\tmov.b64 s2, {%5, %7};\n\tand.pred m, m, e;\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], s0;\n\t@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%1], s1;\n\t"
      "@m tcgen05.cp.cta_group::2.32x128b.warpx4 [%2], s2;\n\t}" ::"r"(cols),
      "r"(cols + 8), "r"(cols + 12), "r"(sf), "r"(sf + 32), "r"(sf + 64), "r"(more), "r"(kHi)
      : "memory");
}

// Arrives in both CTAs once everything the elected lane issued has completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(kPairMask)
      : "memory");
}

__device__ __forceinline__ void expect_tx_elected(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

// Loads into this CTA's shared memory, completed on a barrier that may be the
// other CTA's.
__device__ __forceinline__ void load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t x, uint32_t y, uint32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void load_4d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t x, uint32_t y, uint32_t z, uint32_t u) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u)
      : "memory");
}

__device__ __forceinline__ void load_5d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t x, uint32_t y, uint32_t z, uint32_t u, uint32_t v) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v)
      : "memory");
}

// Where the accumulator of a run's segment seg begins: the even ones at the
// first column, the odd ones end at the last.  Two neighbours that are wider than
// kAccCols together overlap, by at most kOverlap columns: an even one's last, an
// odd one's first.  These are read first and given back by themselves.
__device__ __forceinline__ uint32_t acc_column(uint32_t seg, uint32_t width) { return (seg & 1u) != 0u ? kAccCols - width : 0u; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// silu(g) * u by exp(-|g|), which is at most 1: the divisor is between 1 and 2, and
// nothing overflows on the way to a product that does not, however large u is.
__device__ __forceinline__ float gate(float g, float u) {
  const float e = __expf(-fabsf(g));
  return __fdividef(g < 0.f ? g * e : g, 1.f + e) * u;
}

// ---- division of the work

// A group's rows in the fewest tiles of at most kMaxWidth columns, all equally
// wide (a multiple of 16; the last may have fewer rows, never none).
struct Tiling {
  int tiles, width;
};
__device__ __forceinline__ Tiling tiling(int rows) {
  if (rows <= 0) return {0, 16};
  const int tiles = (rows + kMaxWidth - 1) / kMaxWidth;
  return {tiles, ((rows + tiles - 1) / tiles + 15) & ~15};
}

// K-blocks [kb0, kb1) of one tile.
struct Segment {
  int e, f;          // group, feature tile
  int m0, n;         // rows [m0, m0 + n)
  int width;         // n rounded up to 16
  int kb0, kb1;
  int end;           // cut tiles: unit at which the tile ends
};

// The division, found by every CTA for itself and kept in shared memory.
struct Work {
  int* tile;         // [groups + 1] tiles of the groups before
  int* cost;         // [groups + 1] units of their cut tiles
  int* row;          // [groups + 1] first rows, rising
  int waves;         // turns in which whole tiles are dealt out
  int whole;         // and their number
  int per;           // units of a pair's run of cut tiles
};

__device__ __forceinline__ int tile_units(int k_blocks, int width) {
  return (k_blocks + kStep - 1) / kStep * (kUnitBase + width) + kUnitEnds;
}

// The tiles of all groups stand in one row, the feature tiles of one token tile
// side by side.  They are dealt out whole, so that what runs at a time lies side by
// side and shares its rows and its group's weights in L2.  Where the last turn
// would leave many pairs idle, the last one to two per pair (all, where there are
// few) are laid end to end in units instead and cut into one equal run per pair,
// between steps.
struct Walker {
  const Work& w;
  const GroupedArgs& a;
  int pair, wave, u, u1, e, rows;
  Tiling t;

  __device__ Walker(const Work& work, const GroupedArgs& args, int p) : w(work), a(args), pair(p), wave(0), e(-1), rows(0), t{0, 16} {
    const int total = w.cost[a.groups];
    u = min(static_cast<long long>(w.per) * pair, static_cast<long long>(total));
    u1 = min(static_cast<long long>(u) + w.per, static_cast<long long>(total));
  }

  // Moves on to the last group that begins at or before x in `from`.
  __device__ __forceinline__ void seek(const int* from, int x) {
    if (e >= 0 && from[e + 1] > x) return;
    int lo = max(e, 0), hi = a.groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (from[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    e = lo;
    rows = w.row[e + 1] - w.row[e];
    t = tiling(rows);
  }

  __device__ __forceinline__ void place(Segment& s, int j) const {
    const int tt = j / a.f_tiles;
    s.e = e;
    s.f = j - tt * a.f_tiles;
    s.m0 = w.row[e] + tt * t.width;
    s.n = min(t.width, rows - tt * t.width);
    s.width = (s.n + 15) & ~15;
  }

  __device__ __forceinline__ bool next(Segment& s) {
    if (wave < w.waves) {
      const int i = wave++ * a.pairs + pair;
      if (i >= w.whole) return false;                // only in the last turn, and none is cut then
      seek(w.tile, i);
      place(s, i - w.tile[e]);
      s.kb0 = 0;
      s.kb1 = a.k_blocks;
      s.end = 0;
      return true;
    }
    while (u < u1) {
      seek(w.cost, u);
      const int c = kUnitBase + t.width, whole = tile_units(a.k_blocks, t.width);
      const int j = (u - w.cost[e]) / whole, begin = w.cost[e] + j * whole;
      const int from = u - begin - kUnitEnds, to = min(whole, u1 - begin) - kUnitEnds;
      place(s, max(0, w.whole - w.tile[e]) + j);
      s.kb0 = from > 0 ? from / c * kStep : 0;
      s.kb1 = min(to > 0 ? to / c * kStep : 0, a.k_blocks);
      s.end = u = begin + whole;
      if (s.kb1 > s.kb0) return true;
    }
    return false;
  }
};

__device__ __forceinline__ int warp_prefix(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, v, w);
    if (lane >= w) v += o;
  }
  return v;
}

// to[g + 1] = sum of value(g') over g' <= g, by the whole block: every warp adds
// up some pieces of 32 groups, then the warps' totals are added.
template <typename Value>
__device__ __forceinline__ void prefix_groups(int groups, int* to, int* s_sums, Value value) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pieces = (groups + 31) / 32, per_warp = (pieces + kWarps - 1) / kWarps;
  const int p0 = warp * per_warp, p1 = min(pieces, p0 + per_warp);
  int sum = 0;
  for (int p = p0; p < p1; ++p) {
    const int e = p * 32 + lane;
    const int upto = warp_prefix(e < groups ? value(e) : 0);
    if (e < groups) to[e + 1] = sum + upto;
    sum += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  if (lane == 0) s_sums[warp] = sum;
  if (threadIdx.x == 0) to[0] = 0;
  __syncthreads();
  if (warp > 0 && p0 < p1) {
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s_sums[w];
    for (int p = p0; p < p1; ++p) {
      if (p * 32 + lane < groups) to[p * 32 + lane + 1] += before;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void divide(const GroupedArgs& a, Work& w, int* s_sums) {
  prefix_groups(a.groups, w.tile, s_sums, [&](int e) {
    // Whatever row_start holds, rows lie in [0, M).
    const int r0 = min(max(a.row_start[e], 0), a.M), r1 = min(max(a.row_start[e + 1], r0), a.M);
    w.row[e] = r0;
    if (e == a.groups - 1) w.row[e + 1] = r1;
    return tiling(r1 - r0).tiles * a.f_tiles;
  });
  // Dealt out whole, the tiles take as many turns as the pair with most of them
  // has; cut, the last ones take the mean, and the parts' way through the
  // workspace.
  const int tiles = w.tile[a.groups], turns = (tiles + a.pairs - 1) / a.pairs;
  const int steps = (a.k_blocks + kStep - 1) / kStep;
  const bool cut = a.part != nullptr && (static_cast<long long>(turns) * a.pairs - tiles) * steps >
                                            static_cast<long long>(cut_steps(a.widest)) * a.pairs;
  w.waves = !cut ? turns : max(0, tiles / a.pairs - 1);
  const int whole = min(tiles, w.waves * a.pairs);
  w.whole = whole;
  w.cost[0] = w.cost[a.groups] = 0;
  w.per = 1;
  if (!cut) {
    __syncthreads();
    return;
  }
  __syncthreads();
  prefix_groups(a.groups, w.cost, s_sums, [&](int e) {
    const int left = w.tile[e + 1] - max(w.tile[e], whole);
    return left > 0 ? left * tile_units(a.k_blocks, tiling(w.row[e + 1] - w.row[e]).width) : 0;
  });
  // At least three steps: a run inside one tile has some.
  w.per = max((w.cost[a.groups] + a.pairs - 1) / a.pairs, kUnitEnds + 3 * (kUnitBase + a.widest));
}

template <bool kGated, bool kNarrow>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_tall,
                        const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ GroupedArgs a) {
  using L = Layout<kNarrow>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);   // leader: both CTAs' loads of a stage landed
  uint64_t* empty = full + kStages;                               // both: the pair's MMAs released a stage
  uint64_t* sf_full = empty + kStages;                            // leader: both CTAs staged a group's scales
  uint64_t* sf_empty = sf_full + kSfStages;                       // both: the MMAs that use them are done
  uint64_t* tmem_full = sf_empty + kSfStages;                     // both: accumulator b holds a segment
  uint64_t* tmem_empty = tmem_full + 2;                           // leader: both CTAs have read accumulator b
  uint64_t* tmem_part = tmem_empty + 2;                           // leader: the columns that may overlap the next one's
  uint64_t* final_bar = tmem_part + 2;                            // both: every MMA has completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc + 4);
  int* s_sums = reinterpret_cast<int*>(smem + L::kOffMisc + 16);

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint64_t timeout = a.timeout_ns;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(cluster_id_x());

  grid_launch_dependents();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kSfStages; ++i) {
      mbar_init(&sf_full[i], kPair);
      mbar_init(&sf_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], kPair * kEpiWarps);
      mbar_init(&tmem_part[i], kPair * kEpiWarps);
    }
    mbar_init(final_bar, 1);
    *abort_flag = (smem_u32(smem) & 1023u) != 0 ? 1u : 0u;   // the swizzles would not match; never seen
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  // Barriers and tensor memory must be ready in both CTAs before either issues
  // anything that touches the other.
  tc_fence_before_sync();
  __syncthreads();
  cluster_arrive_release();
  grid_dependency_wait();

  int* s_work = reinterpret_cast<int*>(smem + L::kOffWork);
  Work work = {s_work, s_work + kMaxGroups + 1, s_work + 2 * (kMaxGroups + 1), 0, 0, 1};
  divide(a, work, s_sums);
  cluster_wait();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Walker walk(work, a, pair);
  Segment g;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------- producer
    const uint32_t base = uniform(smem_u32(smem)), full0 = uniform(mapa_shared(smem_u32(&full[0]), 0));
    const uint32_t full_here = uniform(smem_u32(&full[0]));
    uint32_t count = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const int half = g.width / 2;                    // rows of this CTA
      const bool tall = !kNarrow && half > a.short_rows;
      const uint32_t rows = uniform(tall || kNarrow ? a.tall_rows : a.short_rows);
      const uint32_t m = uniform(g.m0 + static_cast<int>(rank) * half), e = uniform(g.e), kb1 = uniform(g.kb1);
      const uint32_t f = uniform(kGated ? g.e * (a.n / 16) + g.f * (kLanes / 16) + rank * (kLanes / 32)
                                        : g.f * 2 * kLanes + rank * kLanes);
      const uint32_t is_tall = uniform(tall ? 1u : 0u);
      ok = __all_sync(0xFFFFFFFFu, *abort_flag == 0u);
      for (uint32_t kb = uniform(g.kb0); ok && kb < kb1; kb += kStep) {
        const uint32_t stage = uniform(count % kStages);
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], (count / kStages & 1u) ^ 1u, timeout));
        if (!ok) break;
        if (leader) expect_tx_elected(full_here + 8u * stage, kPair * kStep * (kWBytes + rows * 128));
        const uint32_t bar = full0 + 8u * stage, w = base + stage * kStep * kWBytes, x = base + L::kOffX + stage * kStep * L::kXBytes;
        if constexpr (kGated) {
          load_5d_pair(w, &tm_w, bar, 0, 0, 0, f, kb);
        } else {
          load_4d_pair(w, &tm_w, bar, 0, f, kb, e);
        }
        if (kNarrow || is_tall != 0u) {
          load_3d_pair(x, &tm_tall, bar, 0, m, kb);
        } else {
          load_3d_pair(x, &tm_x, bar, 0, m, kb);
        }
        ++count;
      }
    }
    if (!ok) fail(abort_flag, kStatusProducerWait);
    // This CTA's loads have landed once the pair's MMAs, which consumed them,
    // have released the stages.
    for (uint32_t i = count > kStages ? count - kStages : 0; i < count; ++i) {
      if (!mbar_wait(&empty[i % kStages], i / kStages & 1u, 2 * timeout)) fail(abort_flag, kStatusTeardownWait);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA issuer
    if (leader) {
      const uint32_t base = uniform(smem_u32(smem)), acc0 = uniform(tmem);
      const uint32_t w_desc = base >> 4 | 1u << 16, x_desc = (base + L::kOffX) >> 4 | 1u << 16, sf_desc = (base + L::kOffSf) >> 4;
      const uint32_t empty0 = uniform(smem_u32(&empty[0])), sf_empty0 = uniform(smem_u32(&sf_empty[0]));
      uint32_t count = 0, sf = 0, seg = 0, before = 0;
      bool ok = true;
      while (ok && walk.next(g)) {
        const uint32_t acc = uniform(seg & 1u), width = uniform(g.width), kb0 = uniform(g.kb0), kb1 = uniform(g.kb1);
        ok = mbar_wait(&tmem_empty[acc], (seg >> 1 & 1u) ^ 1u, timeout) && *abort_flag == 0u;
        if (before + width > kAccCols) ok = ok && mbar_wait(&tmem_part[acc ^ 1u], (seg - 1) >> 1 & 1u, timeout);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        before = width;
        tc_fence_after_sync();
        const uint32_t d = uniform(acc0 + acc_column(seg, width));
        const uint32_t idesc0 = idesc_mxf8_e4m3(kPair * kLanes, width, 0, 0);
        const uint32_t rows = uniform(kNarrow || static_cast<int>(width) / 2 > a.short_rows ? a.tall_rows : a.short_rows);
        for (uint32_t kb = kb0; kb < kb1; kb += kStep) {
          const uint32_t slot = uniform(sf % kSfStages), cols = acc0 + kSfCol + 16 * slot, stage = uniform(count % kStages);
          const bool fresh = kb == kb0 || (kb & 3u) == 0u;
          bool landed = true;
          if (fresh) landed = mbar_wait(&sf_full[slot], sf / kSfStages & 1u, timeout);
          landed = landed && mbar_wait(&full[stage], count / kStages & 1u, timeout);
          ok = __all_sync(0xFFFFFFFFu, landed);
          if (!ok) break;
          if (fresh) {
            tc_fence_after_sync();
            cp_scales(cols, sf_desc + slot * (kSfBytes >> 4), width > 128u ? 1u : 0u);
          }
          const uint32_t w = w_desc + stage * (kStep * kWBytes >> 4), x = x_desc + stage * (kStep * L::kXBytes >> 4);
          const uint32_t id = kb & 3u, idesc = idesc0 | (id << 4) | (id << 29);
          mma_k_block(d, w, x, idesc, cols, cols + 8, kb != kb0 ? 1u : 0u);
          if (kb + 1 < kb1) mma_k_block(d, w + (kWBytes >> 4), x + rows * 8, idesc + (1u << 4) + (1u << 29), cols, cols + 8, 1u);
          commit_pair(empty0 + 8u * stage);
          if (kb + kStep >= kb1 || id == 2u) {
            commit_pair(sf_empty0 + 8u * slot);
            ++sf;
          }
          ++count;
        }
        if (ok) commit_pair(uniform(smem_u32(&tmem_full[acc])));
        ++seg;
      }
      if (!ok) fail(abort_flag, kStatusMmaWait);
      commit_pair(uniform(smem_u32(final_bar)));
    }
    // Every MMA that writes this CTA's tensor memory or reads its shared memory
    // has completed.  (The other CTA's issuer reaches its last commit only
    // after its own waits: some for each segment.)
    bool done = false;
    do {
      done = mbar_wait(final_bar, 0, 2 * timeout);
    } while (!done && *abort_flag == 0u && walk.next(g));
    if (!done) fail(abort_flag, kStatusTeardownWait);
    __syncwarp();
  } else if (warp >= kScaleWarp) {
    // --------------------------------------------------------------- scales
    // In the layout tcgen05.cp 32x128b expects, word [4 r + c] of 128 rows is
    // row 32 c + r.  A word holds the scales of four K-blocks.  Two warps take
    // alternate groups of four, and each has the loads of its next one under way
    // while it waits for the place of the present one.
    const uint32_t sf_full0 = mapa_shared(smem_u32(&sf_full[0]), 0);
    const uint8_t* ws[2] = {};
    int grp = 0, last = 0;                           // group of four K-blocks, the segment's last one
    bool more = true;
    auto step = [&] {                                // to the run's next group
      if (!more || grp++ < last) return;
      more = walk.next(g);
      if (!more) return;
      grp = g.kb0 >> 2;
      last = (g.kb1 - 1) >> 2;
      const int block = kGated ? g.f : 2 * g.f + static_cast<int>(rank);
      const uint8_t* base = a.w_sf + static_cast<long long>(g.e) * a.n_blocks * a.k_blocks;
      ws[0] = base + static_cast<long long>(min(block, a.n_blocks - 1)) * a.k_blocks;
      ws[1] = kGated ? base + static_cast<long long>(a.n_blocks / 2 + block) * a.k_blocks : ws[0];
    };
    auto fetch = [&](uint32_t (&rows)[8], uint32_t& w) {
      const int32_t* from = a.x_sf + static_cast<long long>(grp) * a.m_al + g.m0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int i = 32 * c + lane;
        rows[c] = i < g.n ? static_cast<uint32_t>(from[i]) : 0u;
      }
      const uint8_t* of = kGated && lane >= 16 ? ws[1] : ws[0];   // gated: 16 gate rows, 16 up rows, and so on
      w = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (4 * grp + b < a.k_blocks) w |= static_cast<uint32_t>(of[4 * grp + b]) << (8 * b);
      }
    };
    uint32_t sf = warp - kScaleWarp;
    bool ok = true;
    auto publish = [&](const uint32_t (&rows)[8], uint32_t w) {
      const uint32_t slot = sf % kSfStages;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sf_empty[slot], (sf / kSfStages & 1u) ^ 1u, timeout) && *abort_flag == 0u);
      if (!ok) return;
      uint4* to = reinterpret_cast<uint4*>(smem + L::kOffSf + slot * kSfBytes) + lane;
      to[0] = make_uint4(w, w, w, w);
      to[32] = make_uint4(rows[0], rows[1], rows[2], rows[3]);
      to[64] = make_uint4(rows[4], rows[5], rows[6], rows[7]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(sf_full0 + 8u * slot);
      sf += 2;
    };
    uint32_t rows0[8], rows1[8], w0 = 0, w1 = 0;
    step();
    if (warp != kScaleWarp) step();
    if (more) fetch(rows0, w0);
    while (ok && more) {
      step();
      step();
      const bool then = more;
      if (then) fetch(rows1, w1);
      publish(rows0, w0);
      if (!ok || !then) break;
      step();
      step();
      if (more) fetch(rows0, w0);
      publish(rows1, w1);
    }
    if (!ok) fail(abort_flag, kStatusProducerWait);
  } else if (warp < kEpiWarps) {
    // ------------------------------------------------------------- epilogue
    // Warps w and w + 4 share the 32 lanes of quarter w % 4 and take every
    // other 32 columns.
    const uint32_t tmem_empty0 = mapa_shared(smem_u32(&tmem_empty[0]), 0), tmem_part0 = mapa_shared(smem_u32(&tmem_part[0]), 0);
    const int quad = warp & 3, which = warp >> 2;
    uint8_t* stage = smem + L::kOffOut + warp * kStageBytes;
    const uint32_t stage_at = smem_u32(stage);
    uint32_t seg = 0;
    bool ok = true, open = false;
    while (walk.next(g)) {
      const uint32_t acc = seg & 1u;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&tmem_full[acc], seg >> 1 & 1u, timeout) && *abort_flag == 0u);
      if (!ok) break;
      tc_fence_after_sync();
      const bool whole = g.kb0 == 0 && g.kb1 == a.k_blocks;
      const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc_column(seg, g.width);
      auto release = [&](uint32_t bar0) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(bar0 + 8u * acc);
      };
      if (whole) {
        // All of this warp's values leave the accumulator, rounded, before any is
        // stored.
        constexpr int kChunks = kMaxWidth / 64, kPacked = kGated ? 8 : 16;
        uint32_t packed[kChunks][kPacked];
        auto chunk_at = [&](int i) { return 32 * which + 64 * (acc != 0u ? i : kChunks - 1 - i); };
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c0 = chunk_at(i);
          if (c0 < g.n) {
            float lo[16], hi[16];                     // lanes 0 .. 15 and 16 .. 31 of the quarter
            tmem_ld_16x256b_x4(from + c0, lo);
            tmem_ld_16x256b_x4(from + (16u << 16) + c0, hi);
            tmem_ld_wait16(lo);
            tmem_ld_wait16(hi);
            if constexpr (kGated) {                   // gate and up of a feature are in one thread
#pragma unroll
              for (int k = 0; k < 16; ++k) lo[k] = gate(lo[k], hi[k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              packed[i][k] = pack_bf16(lo[2 * k], lo[2 * k + 1]);
              if constexpr (!kGated) packed[i][8 + k] = pack_bf16(hi[2 * k], hi[2 * k + 1]);
            }
          }
          if (i == 0) release(tmem_part0);
        }
        release(tmem_empty0);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c0 = chunk_at(i);
          if (c0 < g.n) {
            const uint32_t* p = packed[i];
            if constexpr (kGated) {
#pragma unroll
              for (int t = 0; t < 4; t += 2) {        // 16 rows at a time; rows of 16 features, 32 bytes
                const int r = 8 * (t + (lane >> 4)) + (lane & 7), chunk = lane >> 3 & 1;
                stmatrix_x4_trans(stage_at + r * 32 + ((chunk ^ (r >> 2 & 1)) << 4), p[2 * t], p[2 * t + 1], p[2 * t + 2],
                                  p[2 * t + 3]);
              }
            } else {
#pragma unroll
              for (int t = 0; t < 4; ++t) {           // 8 rows at a time; rows of 32 features, 64 bytes
                const int r = 8 * t + (lane & 7), chunk = lane >> 3;
                stmatrix_x4_trans(stage_at + r * 64 + ((chunk ^ (r >> 1 & 3)) << 4), p[2 * t], p[2 * t + 1], p[8 + 2 * t],
                                  p[8 + 2 * t + 1]);
              }
            }
            __syncwarp();
            constexpr int kPieces = kGated ? 2 : 4, kRows = 32 / kPieces;
            const int piece = lane % kPieces;
            const int col = kGated ? g.f * kLanes + static_cast<int>(rank) * 64 + quad * 16 + piece * 8
                                   : (2 * g.f + static_cast<int>(rank)) * kLanes + quad * 32 + piece * 8;
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
              const int r = k * kRows + lane / kPieces;
              const int swz = kGated ? r >> 2 & 1 : r >> 1 & 3;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + r * (16 * kPieces) + ((piece ^ swz) << 4));
              if (c0 + r < g.n && col < a.n_out) {
                *reinterpret_cast<uint4*>(a.y + static_cast<long long>(g.m0 + c0 + r) * a.ldy + col) = v;
              }
            }
            __syncwarp();
          }
        }
      } else {
        const int part = 2 * pair + (g.kb0 > 0 ? 0 : 1);
        float* part_at = a.part + ((static_cast<long long>(part) * kPair + rank) * a.widest) * kLanes + quad * 32 + lane;
        for (int c0 = 32 * which; c0 < g.n; c0 += 64) {
          float v[32];
          tmem_ld_32x32b_x32(from + c0, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (c0 + i < g.n) part_at[static_cast<long long>(c0 + i) * kLanes] = v[i];
          }
        }
        release(tmem_part0);
        release(tmem_empty0);
      }
      // Header of a tile that begins here and goes on in the next pair.
      open = !whole && g.kb0 == 0;
      if (threadIdx.x == 0 && leader && open) {
        a.heads[2 * pair] = make_int4(1, (g.end - 1) / work.per, g.f, 0);
        a.heads[2 * pair + 1] = make_int4(g.m0, g.n, 0, 0);
      }
      ++seg;
    }
    if (!ok) fail(abort_flag, kStatusEpilogueWait);
    if (threadIdx.x == 0 && leader && a.part != nullptr && (!ok || !open)) a.heads[2 * pair] = make_int4(0, 0, 0, 0);
  }

  // Neither CTA leaves or frees tensor memory while the pair may still use its
  // shared memory, barriers or tensor memory.
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// K13: adds up the partial sums of the tiles cut between pairs, in the order of
// the pairs.  Pair c of K12 left a header if a tile begins in its run and ends
// in that of pair c1.  A block takes kJoinRows of the tile's rows, a thread one
// weight row.
constexpr int kJoinRows = 4;

template <bool kGated>
__global__ void __launch_bounds__(256) grouped_join_kernel(const __grid_constant__ GroupedArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int c = blockIdx.x;
  const int4 head = a.heads[2 * c];
  if (head.x == 0) return;
  const int4 where = a.heads[2 * c + 1];
  const int i0 = blockIdx.y * kJoinRows;
  if (i0 >= where.y) return;
  const int rank = threadIdx.x >> 7, lane = threadIdx.x & 127;
  const long long plane = static_cast<long long>(a.widest) * kLanes;     // of one part and CTA
  const float* from = a.part + rank * plane + static_cast<long long>(i0) * kLanes + lane;
  float sum[kJoinRows];
#pragma unroll
  for (int i = 0; i < kJoinRows; ++i) sum[i] = 0.f;
  for (int j = c; j <= head.y; ++j) {
    const float* p = from + (j == c ? 2 * c + 1 : 2 * j) * kPair * plane;
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
      if (i0 + i < where.y) sum[i] += p[i * kLanes];
    }
  }
#pragma unroll
  for (int i = 0; i < kJoinRows; ++i) {
    float v = sum[i];
    int col = (2 * head.z + rank) * kLanes + lane;
    bool there = true;
    if constexpr (kGated) {
      const float u = __shfl_xor_sync(0xFFFFFFFFu, v, 16);               // 16 gate rows, 16 up rows
      v = gate(v, u);
      col = head.z * kLanes + rank * 64 + (lane >> 5) * 16 + (lane & 15);
      there = (lane & 16) == 0;
    }
    if (there && i0 + i < where.y && col < a.n_out) {
      a.y[static_cast<long long>(where.x + i0 + i) * a.ldy + col] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
  }
}

template <bool kGated, bool kNarrow>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(grouped_gemm_kernel<kGated, kNarrow>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Layout<kNarrow>::kSmemBytes);
}

template <bool kGated, bool kNarrow>
cudaError_t launch_instance(const CUtensorMap& tm_x, const CUtensorMap& tm_tall, const CUtensorMap& tm_w, const GroupedArgs& a,
                            cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPair;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.pairs * kPair, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<kNarrow>::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, grouped_gemm_kernel<kGated, kNarrow>, tm_x, tm_tall, tm_w, a);
  if (err != cudaSuccess || a.part == nullptr) return err;
  return launch_dependent(grouped_join_kernel<kGated>, dim3(a.pairs, (a.widest + kJoinRows - 1) / kJoinRows, 1), 256, 0,
                          stream, a);
}

}  // namespace

int grouped_widest(int M) { return M >= kMaxWidth ? kMaxWidth : (M + 15) / 16 * 16; }

int grouped_short_rows(int M) { return grouped_widest(M) < 128 ? grouped_widest(M) / 2 : 64; }

cudaError_t grouped_setup_device() {
  for (cudaError_t err : {set_smem<false, false>(), set_smem<true, false>(), set_smem<false, true>(), set_smem<true, true>()}) {
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

namespace {

// Fewer than one turn's tiles idle: a tile that takes no longer than cutting does
// is never cut (see divide()).
bool cuts(int widest, int K) { return (K / 128 + kStep - 1) / kStep > cut_steps(widest); }

size_t parts_bytes(int widest) {
  return 2 * static_cast<size_t>(kMaxPairs) * (kPair * static_cast<size_t>(widest) * kLanes * sizeof(float) + sizeof(int4));
}

}  // namespace

size_t grouped_need(int M, int K) { return cuts(grouped_widest(M), K) ? parts_bytes(grouped_widest(M)) : 0; }

// Wider tiles are dearer to cut, so a call of many rows may need none where one of
// fewer rows does: the size is that of the widest tiles up to M rows that are cut.
size_t grouped_workspace(int M, int K) {
  int widest = grouped_widest(M);
  while (widest > 0 && !cuts(widest, K)) widest -= 16;
  return widest > 0 ? parts_bytes(widest) : 0;
}

cudaError_t launch_grouped(const CUtensorMap& tm_x, const CUtensorMap& tm_tall, const CUtensorMap& tm_w, GroupedArgs a, bool gated,
                           void* ws, int max_pairs, cudaStream_t stream) {
  a.widest = grouped_widest(a.M);
  a.tall_rows = a.widest / 2;
  a.short_rows = grouped_short_rows(a.M);
  a.pairs = max_pairs < kMaxPairs ? max_pairs : kMaxPairs;
  a.part = cuts(a.widest, a.k_blocks * 128) ? static_cast<float*>(ws) : nullptr;
  a.heads = reinterpret_cast<int4*>(a.part + 2 * static_cast<size_t>(kMaxPairs) * kPair * a.widest * kLanes);
  if (a.widest <= kNarrowWidth) {
    return gated ? launch_instance<true, true>(tm_x, tm_tall, tm_w, a, stream) : launch_instance<false, true>(tm_x, tm_tall, tm_w, a, stream);
  }
  return gated ? launch_instance<true, false>(tm_x, tm_tall, tm_w, a, stream) : launch_instance<false, false>(tm_x, tm_tall, tm_w, a, stream);
}

cudaError_t read_grouped_status(uint32_t* flags, bool reset) {
  uint32_t v = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_iq_status_grouped, sizeof(v));
  if (err != cudaSuccess) return err;
  if (flags) *flags = v;
  if (reset) {
    const uint32_t zero = 0;
    err = cudaMemcpyToSymbol(g_iq_status_grouped, &zero, sizeof(zero));
  }
  return err;
}

}  // namespace iq
