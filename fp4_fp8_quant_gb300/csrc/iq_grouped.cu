// Matrix products grouped by expert with ragged sizes (include/iq.h, section 5):
//   y[m, n] = sum_kb 2^(ex[m, kb] + ew[g, n / 128, kb]) sum_{k in kb} x[m, k] w[g, n, k]
// for the rows m of group g, row_start[g] <= m < row_start[g + 1].
//
// K12 grouped_gemm_kernel.  The weights are the MMA's M side (256 of them over
// a CTA pair) and the rows its N side, which takes any multiple of 16 up to
// 224: a group's rows are divided into the fewest equal tiles, so a group of one
// row costs little more than reading its weights and no group is padded by more
// than 15 rows.

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
constexpr int kMaxWidth = 224;                   // token columns of a tile
constexpr int kLanes = 128;                      // weight rows of a CTA
constexpr int kWBytes = kLanes * 128;            // of one K-block
constexpr int kBoxRows = 32;                     // token rows of one load
constexpr int kSfStages = 4;                     // groups of four K-blocks whose scales are held
constexpr int kSfBytes = (128 + 256) * 4;        // scales of 128 weight rows and 256 token rows
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = kEpiWarps, kMmaWarp = kProducerWarp + 1, kScaleWarp = kMmaWarp + 1;
constexpr int kThreads = (kEpiWarps + 4) * 32;
constexpr int kWarps = kThreads / 32;
constexpr int kStageBytes = 2048;                // output staging of a warp: 32 rows x 32 features
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol = 2 * kMaxWidth;       // + 16 s: weights 4 columns, rows 8 columns at + 8
constexpr int kMaxPairs = 80;

// Units of work: a K-block of a tile of w columns weighs kUnitBase + w, beginning
// and ending a tile kUnitEnds more.
constexpr int kUnitBase = 96;
constexpr int kUnitEnds = 256;

// kNarrow: no tile is wider than 64 columns, so a stage holds 32 rows of each
// CTA's half and there are more stages.
template <bool kNarrow>
struct Layout {
  static constexpr int kStages = kNarrow ? 9 : 6;
  static constexpr int kXBytes = (kNarrow ? kBoxRows : 128) * 128;
  static constexpr int kOffX = kStages * kWBytes;
  static constexpr int kOffSf = kOffX + kStages * kXBytes;
  static constexpr int kOffOut = kOffSf + kSfStages * kSfBytes;
  static constexpr int kOffWork = kOffOut + kEpiWarps * kStageBytes;          // Work: int [3][kMaxGroups + 1]
  static constexpr int kNumBars = 2 * kStages + 2 * kSfStages + 4 + 1;
  static constexpr int kOffBar = (kOffWork + 3 * (kMaxGroups + 1) * 4 + 7) & ~7;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;                     // tensor-memory address, abort flag, warps' sums
  static constexpr int kSmemBytes = kOffMisc + 16 + kWarps * 4;
  static_assert(kOffX % 1024 == 0 && kOffSf % 128 == 0 && kOffOut % 16 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};
constexpr int kNarrowWidth = 2 * kBoxRows;
static_assert(kSfCol + 16 * kSfStages <= kTmemCols, "tensor memory");

__device__ __forceinline__ void fail(volatile uint32_t* abort_flag, uint32_t bit) {
  atomicOr(&g_iq_status_grouped, bit);
  *abort_flag = 1u;
}

// ---- instruction pieces: the CTA-pair forms issued by a whole warp, which
// elects a lane (see iq_kv_attention.cuh).

__device__ __forceinline__ void mma_mxf8_pair_elected(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                      uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

__device__ __forceinline__ void cp_32x128b_pair_elected(uint32_t taddr, uint64_t sdesc) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc)
      : "memory");
}

__device__ __forceinline__ void commit_pair_elected(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(mask)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                                 int u, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// silu(g) * u.  (g far below 0: the quotient by infinity is 0.)
__device__ __forceinline__ float gate(float g, float u) { return __fdividef(g * u, 1.f + __expf(-g)); }

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
  int waves;         // whole tiles of every pair
  int per;           // units of a pair's run of cut tiles
};

__device__ __forceinline__ int tile_units(int k_blocks, int width) { return k_blocks * (kUnitBase + width) + kUnitEnds; }

// The tiles of all groups stand in one row, the feature tiles of one token tile
// side by side.  All but the last one to two per pair are dealt out whole, so
// that what runs at a time lies side by side and shares its rows and its
// group's weights in L2; the last ones (all, where there are few) are laid end to
// end in units and cut into one equal run per pair, at K-blocks.
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
      place(s, max(0, w.waves * a.pairs - w.tile[e]) + j);
      s.kb0 = from > 0 ? from / c : 0;
      s.kb1 = to > 0 ? to / c : 0;
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
  const int tiles = w.tile[a.groups];
  w.waves = tiles >= 2 * a.pairs ? tiles / a.pairs - 1 : 0;
  const int whole = w.waves * a.pairs;
  prefix_groups(a.groups, w.cost, s_sums, [&](int e) {
    const int left = w.tile[e + 1] - max(w.tile[e], whole);
    return left > 0 ? left * tile_units(a.k_blocks, tiling(w.row[e + 1] - w.row[e]).width) : 0;
  });
  // At least four K-blocks: a run inside one tile has some.
  w.per = max((w.cost[a.groups] + a.pairs - 1) / a.pairs, kUnitEnds + 4 * (kUnitBase + a.widest));
}

template <bool kGated, bool kNarrow>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_tall,
                        const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ GroupedArgs a) {
  using L = Layout<kNarrow>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* s_w = smem;
  uint8_t* s_x = smem + L::kOffX;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);   // leader: both CTAs' loads of a stage landed
  uint64_t* empty = full + kStages;                               // both: the pair's MMAs released a stage
  uint64_t* sf_full = empty + kStages;                            // leader: both CTAs staged a group's scales
  uint64_t* sf_empty = sf_full + kSfStages;                       // both: the MMAs that use them are done
  uint64_t* tmem_full = sf_empty + kSfStages;                     // both: accumulator b holds a segment
  uint64_t* tmem_empty = tmem_full + 2;                           // leader: both CTAs have read accumulator b
  uint64_t* final_bar = tmem_empty + 2;                           // both: every MMA has completed
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
    }
    mbar_init(final_bar, 1);
    *abort_flag = (smem_u32(smem) & 1023u) != 0 ? 1u : 0u;   // the swizzles would not match; never seen
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  grid_dependency_wait();

  int* s_work = reinterpret_cast<int*>(smem + L::kOffWork);
  Work work = {s_work, s_work + kMaxGroups + 1, s_work + 2 * (kMaxGroups + 1), 0, 0};
  divide(a, work, s_sums);
  // Barriers and tensor memory must be ready in both CTAs before either
  // issues anything that touches the other.
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Walker walk(work, a, pair);
  Segment g;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------- producer
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);
      uint32_t stage = 0, phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      while (ok && walk.next(g)) {
        // The rows of this CTA's half: up to 64 in boxes of 32, more in one.
        const int half = g.width / 2;
        const bool tall = !kNarrow && half > 2 * kBoxRows;
        const int boxes = tall ? 1 : (half + kBoxRows - 1) / kBoxRows;
        const uint32_t bytes = kPair * (kWBytes + (tall ? a.tall_rows : boxes * kBoxRows) * 128);
        const CUtensorMap* map_x = tall ? &tm_tall : &tm_x;
        const int m = g.m0 + static_cast<int>(rank) * half;
        for (int kb = g.kb0; kb < g.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, timeout) || *abort_flag != 0u) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const uint32_t bar = full0 + 8u * stage;
          uint8_t* w = s_w + stage * kWBytes;
          if constexpr (kGated) {
            tma_load_5d_pair(w, &tm_w, bar, kb * 128, 0, 0, g.f * (kLanes / 16) + static_cast<int>(rank) * (kLanes / 32), g.e);
          } else {
            tma_load_3d_pair(w, &tm_w, bar, kb * 128, g.f * 2 * kLanes + static_cast<int>(rank) * kLanes, g.e);
          }
          uint8_t* x = s_x + stage * L::kXBytes;
          tma_load_2d_pair(x, map_x, bar, kb * 128, m);
          if (boxes > 1) tma_load_2d_pair(x + kBoxRows * 128, map_x, bar, kb * 128, m + kBoxRows);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) fail(abort_flag, kStatusProducerWait);
      // This CTA's loads have landed once the pair's MMAs, which consumed
      // them, have released the stages.
      for (int s = 0; s < kStages; ++s) {
        if ((issued >> s & 1u) != 0u && !mbar_wait(&empty[s], issued_phase >> s & 1u, 2 * timeout)) {
          fail(abort_flag, kStatusTeardownWait);
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA issuer
    if (leader) {
      const uint64_t w_desc = smem_desc_sw128(smem_u32(s_w)), x_desc = smem_desc_sw128(smem_u32(s_x));
      const uint64_t sf_desc = smem_desc_sf(smem_u32(smem + L::kOffSf));
      uint32_t stage = 0, phase = 0, sf = 0, seg = 0;
      bool ok = true;
      while (ok && walk.next(g)) {
        const uint32_t acc = seg & 1u;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&tmem_empty[acc], (seg >> 1 & 1u) ^ 1u, timeout) && *abort_flag == 0u);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t d = tmem + acc * kMaxWidth;
        const uint32_t idesc0 = idesc_mxf8_e4m3(kPair * kLanes, g.width, 0, 0);
        for (int kb = g.kb0; kb < g.kb1; ++kb) {
          const uint32_t slot = sf % kSfStages, cols = tmem + kSfCol + 16 * slot;
          bool landed = true;
          if (kb == g.kb0 || (kb & 3) == 0) {
            landed = mbar_wait(&sf_full[slot], sf / kSfStages & 1u, timeout);
            if (!__all_sync(0xFFFFFFFFu, landed)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint64_t from = sf_desc + slot * (kSfBytes >> 4);
            cp_32x128b_pair_elected(cols, from);
            cp_32x128b_pair_elected(cols + 8, from + (512 >> 4));
            if (g.width > 128) cp_32x128b_pair_elected(cols + 12, from + (1024 >> 4));
          }
          landed = mbar_wait(&full[stage], phase, timeout);
          if (!__all_sync(0xFFFFFFFFu, landed)) {
            ok = false;
            break;
          }
          const uint32_t id = static_cast<uint32_t>(kb) & 3u, idesc = idesc0 | (id << 4) | (id << 29);
          const uint64_t wd = w_desc + stage * (kWBytes >> 4), xd = x_desc + stage * (L::kXBytes >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {               // 32 bytes along K inside the swizzle atom
            mma_mxf8_pair_elected(d, wd + 2 * k, xd + 2 * k, idesc, cols, cols + 8, (kb != g.kb0 || k != 0) ? 1u : 0u);
          }
          commit_pair_elected(&empty[stage], kPairMask);
          if (kb + 1 == g.kb1 || (kb & 3) == 3) {
            commit_pair_elected(&sf_empty[slot], kPairMask);
            ++sf;
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) commit_pair_elected(&tmem_full[acc], kPairMask);
        ++seg;
      }
      if (!ok) fail(abort_flag, kStatusMmaWait);
      commit_pair_elected(final_bar, kPairMask);
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
  } else if (warp == kScaleWarp) {
    // --------------------------------------------------------------- scales
    // In the layout tcgen05.cp 32x128b expects, word [4 r + c] of 128 rows is
    // row 32 c + r.  A word holds the scales of four K-blocks.
    const uint32_t sf_full0 = mapa_shared(smem_u32(&sf_full[0]), 0);
    uint32_t sf = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const uint8_t* ws[2];
      {
        const int block = kGated ? g.f : 2 * g.f + static_cast<int>(rank);
        const uint8_t* base = a.w_sf + static_cast<long long>(g.e) * a.n_blocks * a.k_blocks;
        ws[0] = base + static_cast<long long>(min(block, a.n_blocks - 1)) * a.k_blocks;
        ws[1] = kGated ? base + static_cast<long long>(a.n_blocks / 2 + block) * a.k_blocks : ws[0];
      }
      uint32_t ra[8], rw[2];
      auto fetch = [&](int grp) {
        const int32_t* from = a.x_sf + static_cast<long long>(grp) * a.m_al + g.m0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int i = 32 * c + lane;
          ra[c] = i < g.n ? static_cast<uint32_t>(from[i]) : 0u;
        }
#pragma unroll
        for (int h = 0; h < (kGated ? 2 : 1); ++h) {
          rw[h] = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            if (4 * grp + b < a.k_blocks) rw[h] |= static_cast<uint32_t>(ws[h][4 * grp + b]) << (8 * b);
          }
        }
        if constexpr (!kGated) rw[1] = rw[0];
      };
      const int g0 = g.kb0 >> 2, g1 = (g.kb1 + 3) >> 2;
      fetch(g0);
      for (int grp = g0; grp < g1; ++grp, ++sf) {
        const uint32_t slot = sf % kSfStages;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sf_empty[slot], (sf / kSfStages & 1u) ^ 1u, timeout) && *abort_flag == 0u);
        if (!ok) break;
        uint4* to = reinterpret_cast<uint4*>(smem + L::kOffSf + slot * kSfBytes) + lane;
        // Gated: 16 gate rows, 16 up rows, and so on.
        const uint32_t w = lane < 16 ? rw[0] : rw[1];
        to[0] = make_uint4(w, w, w, w);
        to[32] = make_uint4(ra[0], ra[1], ra[2], ra[3]);
        to[64] = make_uint4(ra[4], ra[5], ra[6], ra[7]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(sf_full0 + 8u * slot);
        if (grp + 1 < g1) fetch(grp + 1);
      }
    }
    if (!ok) fail(abort_flag, kStatusProducerWait);
  } else if (warp < kEpiWarps) {
    // ------------------------------------------------------------- epilogue
    // Warps w and w + 4 share the 32 lanes of quarter w % 4 and take every
    // other 32 columns.
    const uint32_t tmem_empty0 = mapa_shared(smem_u32(&tmem_empty[0]), 0);
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
      const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * kMaxWidth;
      const int part = 2 * pair + (g.kb0 > 0 ? 0 : 1);
      float* part_at = a.part + ((static_cast<long long>(part) * kPair + rank) * a.widest) * kLanes + quad * 32 + lane;
      for (int c0 = 32 * which; c0 < g.n; c0 += 64) {
        if (whole) {
          float lo[16], hi[16];                       // lanes 0 .. 15 and 16 .. 31 of the quarter
          tmem_ld_16x256b_x4(from + c0, lo);
          tmem_ld_16x256b_x4(from + (16u << 16) + c0, hi);
          tmem_ld_wait16(lo);
          tmem_ld_wait16(hi);
          if constexpr (kGated) {
            // Gate and up of a feature are in one thread.
#pragma unroll
            for (int i = 0; i < 16; ++i) lo[i] = gate(lo[i], hi[i]);
#pragma unroll
            for (int t = 0; t < 4; t += 2) {          // 16 rows at a time; rows of 16 features, 32 bytes
              const int r = 8 * (t + (lane >> 4)) + (lane & 7), chunk = lane >> 3 & 1;
              stmatrix_x4_trans(stage_at + r * 32 + ((chunk ^ (r >> 2 & 1)) << 4), pack_bf16(lo[4 * t], lo[4 * t + 1]),
                                pack_bf16(lo[4 * t + 2], lo[4 * t + 3]), pack_bf16(lo[4 * t + 4], lo[4 * t + 5]),
                                pack_bf16(lo[4 * t + 6], lo[4 * t + 7]));
            }
          } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {             // 8 rows at a time; rows of 32 features, 64 bytes
              const int r = 8 * t + (lane & 7), chunk = lane >> 3;
              stmatrix_x4_trans(stage_at + r * 64 + ((chunk ^ (r >> 1 & 3)) << 4), pack_bf16(lo[4 * t], lo[4 * t + 1]),
                                pack_bf16(lo[4 * t + 2], lo[4 * t + 3]), pack_bf16(hi[4 * t], hi[4 * t + 1]),
                                pack_bf16(hi[4 * t + 2], hi[4 * t + 3]));
            }
          }
          __syncwarp();
          constexpr int kChunks = kGated ? 2 : 4, kRows = 32 / kChunks;
          const int chunk = lane % kChunks;
          const int col = kGated ? g.f * kLanes + static_cast<int>(rank) * 64 + quad * 16 + chunk * 8
                                 : (2 * g.f + static_cast<int>(rank)) * kLanes + quad * 32 + chunk * 8;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int r = i * kRows + lane / kChunks;
            const int swz = kGated ? r >> 2 & 1 : r >> 1 & 3;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + r * (16 * kChunks) + ((chunk ^ swz) << 4));
            if (c0 + r < g.n && col < a.n_out) {
              *reinterpret_cast<uint4*>(a.y + static_cast<long long>(g.m0 + c0 + r) * a.ldy + col) = v;
            }
          }
          __syncwarp();
        } else {
          float v[32];
          tmem_ld_32x32b_x32(from + c0, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (c0 + i < g.n) part_at[static_cast<long long>(c0 + i) * kLanes] = v[i];
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tmem_empty0 + 8u * acc);
      // Header of a tile that begins here and goes on in the next pair.
      open = !whole && g.kb0 == 0;
      if (threadIdx.x == 0 && leader && open) {
        a.heads[2 * pair] = make_int4(1, (g.end - 1) / work.per, g.f, 0);
        a.heads[2 * pair + 1] = make_int4(g.m0, g.n, 0, 0);
      }
      ++seg;
    }
    if (!ok) fail(abort_flag, kStatusEpilogueWait);
    if (threadIdx.x == 0 && leader && (!ok || !open)) a.heads[2 * pair] = make_int4(0, 0, 0, 0);
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
  if (err != cudaSuccess) return err;
  return launch_dependent(grouped_join_kernel<kGated>, dim3(a.pairs, (a.widest + kJoinRows - 1) / kJoinRows, 1), 256, 0,
                          stream, a);
}

}  // namespace

int grouped_widest(int M) { return M >= kMaxWidth ? kMaxWidth : (M + 15) / 16 * 16; }

cudaError_t grouped_setup_device() {
  for (cudaError_t err : {set_smem<false, false>(), set_smem<true, false>(), set_smem<false, true>(), set_smem<true, true>()}) {
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

size_t grouped_workspace(int M) {
  return 2 * static_cast<size_t>(kMaxPairs) * (kPair * static_cast<size_t>(grouped_widest(M)) * kLanes * sizeof(float) + sizeof(int4));
}

cudaError_t launch_grouped(const CUtensorMap& tm_x, const CUtensorMap& tm_tall, const CUtensorMap& tm_w, GroupedArgs a, bool gated,
                           void* ws, int max_pairs, cudaStream_t stream) {
  a.widest = grouped_widest(a.M);
  a.tall_rows = a.widest / 2;
  a.pairs = max_pairs < kMaxPairs ? max_pairs : kMaxPairs;
  a.part = static_cast<float*>(ws);
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
