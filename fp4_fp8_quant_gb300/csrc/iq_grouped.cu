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
constexpr int kStages = 6;
constexpr int kMaxWidth = 224;                   // token columns of a tile
constexpr int kLanes = 128;                      // weight rows of a CTA
constexpr int kWBytes = kLanes * 128;            // of one K-block
constexpr int kXBytes = 128 * 128;
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

constexpr int kOffW = 0;
constexpr int kOffX = kOffW + kStages * kWBytes;
constexpr int kOffSf = kOffX + kStages * kXBytes;
constexpr int kOffOut = kOffSf + kSfStages * kSfBytes;
constexpr int kOffCost = kOffOut + kEpiWarps * kStageBytes;          // long long [kMaxGroups + 1]
constexpr int kOffRow = kOffCost + (kMaxGroups + 1) * 8;             // int2 would not fit: int [kMaxGroups + 1]
constexpr int kNumBars = 2 * kStages + 2 * kSfStages + 4 + 1;
constexpr int kOffBar = kOffRow + (kMaxGroups + 2) * 4;
constexpr int kOffMisc = kOffBar + kNumBars * 8;                     // tensor-memory address, abort flag, warps' sums
constexpr int kSmemBytes = kOffMisc + 16 + kWarps * 8;
static_assert(kOffX % 1024 == 0 && kOffSf % 128 == 0 && kOffOut % 16 == 0 && kOffCost % 8 == 0 && kOffBar % 8 == 0, "alignment");
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
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

__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                                 int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// silu(g) * u.  (g far below 0: the quotient by infinity is 0.)
__device__ __forceinline__ float gate(float g, float u) { return __fdividef(g * u, 1.f + __expf(-g)); }

// a / b for a >= 0, b > 0.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 31 == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
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
  long long end;     // unit at which the tile ends
};

// All tiles of all groups are laid end to end in units (feature tiles of one
// token tile side by side, so that what runs at a time shares its rows and its
// group's weights in L2) and cut into one equal run per CTA pair.
struct Walker {
  const long long* cost;     // [groups + 1] units before each group
  const int* row;            // [groups + 1] first rows, rising
  int k_blocks, f_tiles;
  long long u, u1;
  int e;
  Tiling t;
  int rows;

  __device__ Walker(const long long* c, const int* r, const GroupedArgs& a, long long per, int pair)
      : cost(c), row(r), k_blocks(a.k_blocks), f_tiles(a.f_tiles), u(per * pair), e(-1) {
    const long long total = c[a.groups];
    u1 = min(u + per, total);
    if (u >= u1) return;
    int lo = 0, hi = a.groups - 1;         // the last group that begins at or before u and is not empty
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (c[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    enter(lo);
  }

  __device__ __forceinline__ void enter(int group) {
    e = group;
    rows = row[e + 1] - row[e];
    t = tiling(rows);
  }

  __device__ __forceinline__ bool next(Segment& s) {
    while (u < u1) {
      while (cost[e + 1] <= u) enter(e + 1);
      const int c = kUnitBase + t.width;
      const long long whole = static_cast<long long>(k_blocks) * c + kUnitEnds;
      const long long j = quotient(u - cost[e], whole), begin = cost[e] + j * whole;
      const long long from = u - begin - kUnitEnds, to = min(whole, u1 - begin) - kUnitEnds;
      const int tt = static_cast<int>(quotient(j, f_tiles));
      s.e = e;
      s.f = static_cast<int>(j - static_cast<long long>(tt) * f_tiles);
      s.m0 = row[e] + tt * t.width;
      s.n = min(t.width, rows - tt * t.width);
      s.width = (s.n + 15) & ~15;
      s.kb0 = from > 0 ? static_cast<int>(quotient(from, c)) : 0;
      s.kb1 = to > 0 ? static_cast<int>(quotient(to, c)) : 0;
      s.end = u = begin + whole;
      if (s.kb1 > s.kb0) return true;
    }
    return false;
  }
};

__device__ __forceinline__ long long warp_prefix(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, v, w);
    if (lane >= w) v += o;
  }
  return v;
}

// Units a run has at least: a run inside one tile has a K-block.
__device__ __forceinline__ long long run_units(long long total, const GroupedArgs& a) {
  const long long per = quotient(total + a.join_pairs - 1, a.join_pairs);
  return max(per, static_cast<long long>(kUnitEnds + 4 * (kUnitBase + a.widest)));
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                        const __grid_constant__ GroupedArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* s_w = smem + kOffW;
  uint8_t* s_x = smem + kOffX;
  long long* s_cost = reinterpret_cast<long long*>(smem + kOffCost);
  int* s_row = reinterpret_cast<int*>(smem + kOffRow);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);   // leader: both CTAs' loads of a stage landed
  uint64_t* empty = full + kStages;                               // both: the pair's MMAs released a stage
  uint64_t* sf_full = empty + kStages;                            // leader: both CTAs staged a group's scales
  uint64_t* sf_empty = sf_full + kSfStages;                       // both: the MMAs that use them are done
  uint64_t* tmem_full = sf_empty + kSfStages;                     // both: accumulator b holds a segment
  uint64_t* tmem_empty = tmem_full + 2;                           // leader: both CTAs have read accumulator b
  uint64_t* final_bar = tmem_empty + 2;                           // both: every MMA has completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc + 4);
  long long* s_sums = reinterpret_cast<long long*>(smem + kOffMisc + 16);

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

  // Units before each group: every warp adds up a block of 32-group pieces,
  // then the warps' totals are added.
  {
    const int pieces = (a.groups + 31) / 32, per_warp = (pieces + kWarps - 1) / kWarps;
    long long sum = 0;
    for (int p = warp * per_warp; p < min(pieces, (warp + 1) * per_warp); ++p) {
      const int e = p * 32 + lane;
      int r0 = 0, r1 = 0;
      if (e < a.groups) {                              // whatever row_start holds, rows lie in [0, M) and rise
        r0 = min(max(a.row_start[e], 0), a.M);
        r1 = min(max(a.row_start[e + 1], r0), a.M);
      }
      const Tiling t = tiling(r1 - r0);
      const long long own = static_cast<long long>(t.tiles) * a.f_tiles *
                            (static_cast<long long>(a.k_blocks) * (kUnitBase + t.width) + kUnitEnds);
      const long long upto = warp_prefix(own);
      if (e < a.groups) {
        s_cost[e + 1] = sum + upto;
        s_row[e] = r0;
        if (e == a.groups - 1) s_row[e + 1] = r1;
      }
      sum += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    if (lane == 0) s_sums[warp] = sum;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += s_sums[w];
    for (int p = warp * per_warp; p < min(pieces, (warp + 1) * per_warp); ++p) {
      if (p * 32 + lane < a.groups) s_cost[p * 32 + lane + 1] += before;
    }
    if (threadIdx.x == 0) s_cost[0] = 0;
  }
  // Barriers and tensor memory must be ready in both CTAs before either
  // issues anything that touches the other.
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const long long per = run_units(s_cost[a.groups], a);
  Walker walk(s_cost, s_row, a, per, pair);
  Segment g;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------- producer
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);
      uint32_t stage = 0, phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      while (ok && walk.next(g)) {
        const int half = g.width / 2, boxes = (half + kBoxRows - 1) / kBoxRows;
        const uint32_t bytes = kPair * (kWBytes + boxes * kBoxRows * 128);
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
            const int f0 = g.f * kLanes + static_cast<int>(rank) * (kLanes / 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) tma_load_4d_pair(w + i * 4096, &tm_w, bar, kb * 128, f0 + 16 * i, 0, g.e);
          } else {
            tma_load_3d_pair(w, &tm_w, bar, kb * 128, g.f * 2 * kLanes + static_cast<int>(rank) * kLanes, g.e);
          }
          uint8_t* x = s_x + stage * kXBytes;
          for (int i = 0; i < boxes; ++i) tma_load_2d_pair(x + i * kBoxRows * 128, &tm_x, bar, kb * 128, m + i * kBoxRows);
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
      const uint64_t sf_desc = smem_desc_sf(smem_u32(smem + kOffSf));
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
          const uint64_t wd = w_desc + stage * (kWBytes >> 4), xd = x_desc + stage * (kXBytes >> 4);
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
        uint4* to = reinterpret_cast<uint4*>(smem + kOffSf + slot * kSfBytes) + lane;
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
    uint8_t* stage = smem + kOffOut + warp * kStageBytes;
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
        a.heads[2 * pair] = make_int4(1, static_cast<int>(quotient(g.end - 1, per)), g.f, 0);
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

int widest_tile(int M) { return M >= kMaxWidth ? kMaxWidth : (M + 15) / 16 * 16; }

template <bool kGated>
cudaError_t launch_instance(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const GroupedArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPair;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.join_pairs * kPair, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, grouped_gemm_kernel<kGated>, tm_x, tm_w, a);
  if (err != cudaSuccess) return err;
  return launch_dependent(grouped_join_kernel<kGated>, dim3(a.join_pairs, (a.widest + kJoinRows - 1) / kJoinRows, 1), 256, 0,
                          stream, a);
}

}  // namespace

cudaError_t grouped_setup_device() {
  const cudaError_t err =
      cudaFuncSetAttribute(grouped_gemm_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (err != cudaSuccess) return err;
  return cudaFuncSetAttribute(grouped_gemm_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

size_t grouped_workspace(int M) {
  return 2 * static_cast<size_t>(kMaxPairs) * (kPair * static_cast<size_t>(widest_tile(M)) * kLanes * sizeof(float) + sizeof(int4));
}

cudaError_t launch_grouped(const CUtensorMap& tm_x, const CUtensorMap& tm_w, GroupedArgs a, bool gated, void* ws,
                           int max_pairs, cudaStream_t stream) {
  a.widest = widest_tile(a.M);
  a.join_pairs = max_pairs < kMaxPairs ? max_pairs : kMaxPairs;
  a.part = static_cast<float*>(ws);
  a.heads = reinterpret_cast<int4*>(a.part + 2 * static_cast<size_t>(kMaxPairs) * kPair * a.widest * kLanes);
  return gated ? launch_instance<true>(tm_x, tm_w, a, stream) : launch_instance<false>(tm_x, tm_w, a, stream);
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
