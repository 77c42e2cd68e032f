// Low-rank adapters of many requests beside a shared projection (include/iq.h,
// section 6):   out[t] = base[t] + scale[a] B[a] (A[a] x[t]),  a the adapter of
// t's request.
//
// Requests of one adapter that follow one another are taken together; their rows
// are divided into the fewest equal tiles of at most 128.  In both products
// (tcgen05 kind::f16, BF16) the adapter's matrix is the MMA's M side and the rows its
// N side (a multiple of 16), so a request of one row costs little more than
// reading its adapter.
//
// K17 adapter_down_kernel, V = A x.  The steps of all tiles along K, laid end to
// end, are cut into one equal run per CTA, whatever the requests' lengths, so that
// few rows load many SMs too (runs are not shorter than an eighth of a tile); each run
// leaves its part of a tile's V in the workspace (float32).
//
// K18 adapter_up_kernel, out = base + B (scale V).  The parts are added up in
// the order of the runs and split into three BF16 terms, which hold all 24 bits
// of a float32 (with two terms, 16 bits, results where base and the adapter's part
// nearly cancel were off by whole units of what is left).  The features of a row tile are
// taken one after the other by a CTA (128 at a time, 256 where there are few rows);
// base rows are loaded ahead of the product, meet it in registers in the
// accumulator's own layout (ldmatrix, transposed) and leave as rows again.  A CTA of
// K18 may start as soon as a CTA of K17 leaves its SM: it finds its work and loads B
// and base while others still run, and waits for V alone.
//
// Both are bound by memory and by the latencies around it.  Measured (per call in a
// CUDA graph): 64 requests of one row over 48 adapters of rank 64, 7168 -> 8192,
// 31.2 us for 97 MB (14.3 us at the measured copy rate).  Five prompts of 4632 rows
// together, rank 32, 7168 -> 1536: 26.0 us for 77 MB.  One request 8.8 us.  (Of these,
// V's third term takes 1.8, 0.7 and 0.2 us: half as many MMAs again.)  Of 64 requests,
// with two terms: K17 2.2 us to find its runs, 10.5 for 58 MB (an adapter used twice is
// read twice, from L2); K18 6 until its first product (start, runs, the wait for all of
// K17, V), 9 for 66 MB of B.
// What did not help (with two terms, 29.4 and 25.4 us): all of the SM's memory as
// shared memory, so that K18's CTAs do run beside K17's from its beginning (64 requests
// 30.4 us, five prompts 28.9 -> 31.9); what is left of B asked for into L2 as K17's loads
// end (64 requests 33.8).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "iq_internal.h"
#include "iq_kv.h"
#include "iq_kv_attention.cuh"
#include "iq_moe.h"
#include "iq_ptx.cuh"

namespace iq {

__device__ uint32_t g_iq_status_adapters;

namespace {

constexpr int kMaxWidth = 128;                    // rows of a tile

// ---- instruction pieces

// Issued by a whole warp, which elects a lane; operands are the same in all lanes.
__device__ __forceinline__ void expect_tx_elected(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t x, uint32_t y, uint32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t x, uint32_t y, uint32_t z,
                                        uint32_t u) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u)
      : "memory");
}

__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// Four 8x8 matrices of 16-bit values, transposed (see stmatrix_x4_trans).
__device__ __forceinline__ uint4 ldmatrix_x4_trans(uint32_t addr) {
  uint4 r;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// ---- division of the work

// Runs of neighbouring requests that have one adapter, in shared memory: arrays of
// requests + 1 entries.
struct Runs {
  int* first;        // first row
  int* end;          // row behind the last
  int* id;           // adapter, or -1
  int* rows;         // rows with an adapter in the runs before, [count] of all
  int* down;         // K17's units of the runs before, [count] of all
  int* up;           // K18's
  int count;
};
constexpr int kRunArrays = 6;

__device__ __forceinline__ Runs runs_at(int* area, int requests) {
  const int n = requests + 1;
  return {area, area + n, area + 2 * n, area + 3 * n, area + 4 * n, area + 5 * n, 0};
}

struct Tiling {
  int tiles, width;
};
__device__ __forceinline__ Tiling tiling(int rows) {
  if (rows <= 0) return {0, 16};
  const int tiles = (rows + kMaxWidth - 1) / kMaxWidth;
  return {tiles, ((rows + tiles - 1) / tiles + 15) & ~15};
}

// Units of a step of K17: rows that are read, and what a step costs however few
// they are (with 16 instead of 64 the CTA with the tile of one row, of five
// prompts, took 15.6 us and the others 11).
constexpr int kStepUnits = 64;
__device__ __forceinline__ int down_unit(const AdapterArgs& a, int id, int width) { return id < 0 ? 0 : kStepUnits + a.rank + width; }

// K18 takes a row tile in the fewest equal pieces of at most kUpWidth rows.  (With
// 128 rows at a time five prompts of 4632 tokens, 1536 features, leave a CTA one
// or two units: 38 us for both kernels, with 64 34.)
constexpr int kUpWidth = 64;
__device__ __forceinline__ Tiling up_pieces(int width) {
  const int pieces = (width + kUpWidth - 1) / kUpWidth;
  return {pieces, ((width + pieces - 1) / pieces + 15) & ~15};
}
// Pieces of up to kNarrow rows are multiplied with 256 features at a time, which
// keeps all warps busy, the others with 128.
constexpr int kNarrow = 32;
__device__ __forceinline__ int up_halves(int width) { return width <= kNarrow ? 2 : 1; }
__device__ __forceinline__ int up_tiles(const AdapterArgs& a, int width) { return (a.f_tiles + up_halves(width) - 1) / up_halves(width); }
// What such a unit of K18 costs: mostly its latencies.
__device__ __forceinline__ int up_unit(int id, int width) { return (id < 0 ? 64 : 96) + width; }

// Scratch of find_runs: a word of each warp, three times.
constexpr int kScratchBytes = 3 * 16 * 4;

template <int kWarps>
__device__ __forceinline__ void sync_warps() {
  if constexpr (kWarps == 1) __syncwarp();
  else __syncthreads();
}

// join(sum so far, this warp's) over the warps before this one and over all of them;
// own: the same in all lanes.
template <int kWarps, typename Join>
__device__ __forceinline__ int over_warps(int* scratch, int own, int& so_far, Join join) {
  int before = so_far;
  if constexpr (kWarps == 1) {
    so_far = join(so_far, own);
  } else {
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = own;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == static_cast<int>(threadIdx.x >> 5)) before = so_far;
      so_far = join(so_far, scratch[w]);
    }
  }
  return before;
}

// Finds the runs and returns their number; by the block's first kWarps warps, which
// are one or all of it, a request per thread and turn.
template <int kWarps>
__device__ __forceinline__ int find_runs(const AdapterArgs& a, Runs& s, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int *s0 = scratch, *s1 = scratch + 16, *s2 = scratch + 32;
  int *ends = s.down, *ids = s.up;                     // of the requests, until the runs' units go there
  for (int i = threadIdx.x; i < a.requests; i += 32 * kWarps) s.end[i] = 0;
  int count = 0, last = -1, covered = 0;               // runs, the last request with rows, rows of earlier requests: so far
#pragma unroll 1
  for (int i0 = 0; i0 < a.requests; i0 += 32 * kWarps) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    int start = 0, to = 0, id = -1;
    if (i < a.requests) {
      start = static_cast<int>(ld_dependent_u32(a.row_start + i));
      to = static_cast<int>(ld_dependent_u32(a.row_start + i + 1));
      id = static_cast<int>(ld_dependent_u32(a.adapter + i));
    }
    // Whatever row_start holds, rows lie in [0, T) and belong to one request.
    to = min(max(to, 0), a.tokens);
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.adapters)) id = -1;
    int upto = to;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, upto, w);
      if (lane >= w) upto = max(upto, o);
    }
    int before = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
    if (lane == 0) before = 0;
    before = max(before, over_warps<kWarps>(s0, __shfl_sync(0xFFFFFFFFu, upto, 31), covered, [](int x, int y) { return max(x, y); }));
    const int r0 = max(min(max(start, 0), a.tokens), before), r1 = max(to, r0);
    const bool some = i < a.requests && r1 > r0;
    if (some) {
      ends[i] = r1;
      ids[i] = id;
    }
    const uint32_t with = __ballot_sync(0xFFFFFFFFu, some), below = with & ((1u << lane) - 1u);
    const int warp0 = i0 + 32 * warp;
    if constexpr (kWarps == 1) __syncwarp();
    int prev = over_warps<kWarps>(s1, with != 0u ? warp0 + 31 - __clz(with) : -1, last, [](int x, int y) { return max(x, y); });
    if (below != 0u) prev = warp0 + 31 - __clz(below);
    const bool begins = some && !(prev >= 0 && ids[prev] == id && ends[prev] == r0);
    const uint32_t heads = __ballot_sync(0xFFFFFFFFu, begins);
    const auto add = [](int x, int y) { return x + y; };
    const int run = __popc(heads & ((2u << lane) - 1u)) - 1 + over_warps<kWarps>(s2, __popc(heads), count, add);
    if (begins) {
      s.first[run] = r0;
      s.id[run] = id;
    }
    if (some) atomicMax(&s.end[run], r1);
  }
  sync_warps<kWarps>();
  int up = 0, down = 0, rows = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += 32 * kWarps) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    const bool there = i < count;
    const int n = there ? s.end[i] - s.first[i] : 0, id = there ? s.id[i] : -1;
    const Tiling t = tiling(n);
    const Tiling p = up_pieces(t.width);
    const int own_d = t.tiles * a.k_steps * down_unit(a, id, t.width);
    const int own_u = t.tiles * p.tiles * up_tiles(a, p.width) * up_unit(id, p.width);
    const int own_r = id >= 0 ? n : 0;
    int d = own_d, u = own_u, r = own_r;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int od = __shfl_up_sync(0xFFFFFFFFu, d, w), ou = __shfl_up_sync(0xFFFFFFFFu, u, w);
      const int o = __shfl_up_sync(0xFFFFFFFFu, r, w);
      if (lane >= w) {
        d += od;
        u += ou;
        r += o;
      }
    }
    const auto add = [](int x, int y) { return x + y; };
    d += over_warps<kWarps>(s0, __shfl_sync(0xFFFFFFFFu, d, 31), down, add) - own_d;
    u += over_warps<kWarps>(s1, __shfl_sync(0xFFFFFFFFu, u, 31), up, add) - own_u;
    r += over_warps<kWarps>(s2, __shfl_sync(0xFFFFFFFFu, r, 31), rows, add) - own_r;
    if (there) {
      s.down[i] = d;
      s.up[i] = u;
      s.rows[i] = r;
    }
    sync_warps<kWarps>();
  }
  if (threadIdx.x == 0) {
    s.down[count] = down;
    s.up[count] = up;
    s.rows[count] = rows;
  }
  return count;
}

// The last run that begins at or before u in `from`.
__device__ __forceinline__ int find_run(const Runs& s, const int* from, int u) {
  int lo = 0, hi = s.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (from[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A tile's V comes in about so many parts at most, which every unit of K18 has to add
// up (94 rows of one adapter of rank 104, 6584 -> 200: a part per step 34 us, six 14.9,
// eight 13.5, ten 14.5; 1106 rows, rank 120, 4040 -> 5800: 48, 38, 37, 41).
constexpr int kMaxParts = 8;

// Units of a run of K17.
__device__ __forceinline__ int down_per(const AdapterArgs& a, int total) {
  return max((total + a.down_ctas - 1) / a.down_ctas, a.down_least);
}

// The first run that holds steps of the tile at units [begin, begin + steps * c).
__device__ __forceinline__ int first_part(int begin, int c, int per) {
  const int p = begin / per;
  return (p + 1) * per - begin < c ? p + 1 : p;
}

// ---- K17

constexpr int kDownThreads = 192;
constexpr int kMaxDownStages = 8;
constexpr int kDownStageBytes = 128 * 1024;       // of all stages
constexpr int kDownOffBar = kDownStageBytes;
constexpr int kDownBars = 2 * kMaxDownStages + 4 + 1;
constexpr int kDownOffMisc = kDownOffBar + kDownBars * 8;
constexpr int kDownOffRuns = kDownOffMisc + 16 + kScratchBytes;

struct DownSegment {
  int id, m0, n, width, row, k0, k1, part;         // steps [k0, k1)
};

struct DownWalker {
  const AdapterArgs& a;
  const Runs& s;
  int per, u, u1, run;
  __device__ __forceinline__ DownWalker(const AdapterArgs& args, const Runs& runs)
      : a(args), s(runs), per(down_per(args, runs.down[runs.count])), run(0) {
    const long long total = s.down[s.count], from = static_cast<long long>(per) * blockIdx.x;
    u = static_cast<int>(min(from, total));
    u1 = static_cast<int>(min(from + per, total));
    if (u < u1) run = find_run(s, s.down, u);
  }
  __device__ __forceinline__ bool next(DownSegment& g) {
    while (u < u1) {
      while (s.down[run + 1] <= u) ++run;
      const int rows = s.end[run] - s.first[run];
      const Tiling t = tiling(rows);
      const int c = down_unit(a, s.id[run], t.width), whole = a.k_steps * c;
      const int j = (u - s.down[run]) / whole, begin = s.down[run] + j * whole;
      g.id = s.id[run];
      g.m0 = s.first[run] + j * t.width;
      g.n = min(t.width, rows - j * t.width);
      g.width = (g.n + 15) & ~15;
      g.row = s.rows[run] + j * t.width;
      g.k0 = (u - begin) / c;
      g.k1 = min(whole, u1 - begin) / c;
      g.part = static_cast<int>(blockIdx.x) - first_part(begin, c, per);
      u = begin + whole;
      if (g.k1 > g.k0) return true;
    }
    return false;
  }
};

// An MMA adds to its accumulator by truncating, so a long chain is off to one side
// (64 tiles of one row, 192 MMAs per part of V: 4.7e-6 of a sum of positive numbers;
// now below 1.5e-6).  Tiles that leave columns of the accumulator free are
// summed in as many chains as fit, the four MMAs of a K-block dealt out to them, and
// these are added up in registers.
__device__ __forceinline__ uint32_t chains(int width) { return width <= 32 ? 4u : (width <= 64 ? 2u : 1u); }

// Rows of x that a tile of n rows loads: the lowest box that holds them.  (What
// stands behind them in shared memory reaches only columns of the product that
// nobody reads.)
__device__ __forceinline__ uint32_t x_rows(const AdapterArgs& a, int n) {
  return n <= 8 ? 8u : (n <= 64 && a.tall_rows > 64 ? 64u : static_cast<uint32_t>(a.tall_rows));
}

template <bool kMany>
__global__ void __launch_bounds__(kDownThreads, 1)
    adapter_down_kernel(const __grid_constant__ CUtensorMap tm_x8, const __grid_constant__ CUtensorMap tm_x64,
                        const __grid_constant__ CUtensorMap tm_tall, const __grid_constant__ CUtensorMap tm_a,
                        const __grid_constant__ AdapterArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Runs runs = runs_at(reinterpret_cast<int*>(smem + kDownOffRuns), a.requests);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kDownOffBar);
  uint64_t* empty = full + kMaxDownStages;
  uint64_t* tmem_full = empty + kMaxDownStages;   // [2]
  uint64_t* tmem_empty = tmem_full + 2;           // [2]
  uint64_t* drained = tmem_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kDownOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + kDownOffMisc + 4);
  int* s_count = reinterpret_cast<int*>(smem + kDownOffMisc + 8);
  int* scratch = reinterpret_cast<int*>(smem + kDownOffMisc + 16);
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint64_t timeout = a.timeout_ns;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_tall);
    tma_prefetch_desc(&tm_x8);
    tma_prefetch_desc(&tm_a);
    for (int i = 0; i < kMaxDownStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], 4);
    }
    mbar_init(drained, 1);
    *abort_flag = (smem_u32(smem) & 1023u) != 0 ? 1u : 0u;   // the swizzles would not match; never seen
    fence_mbar_init();
  }
  // Tensor memory is taken by kernels that wait for nothing but others that have
  // theirs: after the wait, and before the next kernel may start.
  grid_dependency_wait();
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  __syncthreads();
  // (Only now: K18 reads its inputs, which the kernels before this one may have
  // written, while this one runs.)
  grid_launch_dependents();
  if constexpr (kMany) {
    runs.count = find_runs<kDownThreads / 32>(a, runs, scratch);
  } else if (warp == 0) {
    const int count = find_runs<1>(a, runs, scratch);
    if (lane == 0) *s_count = count;
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (!kMany) runs.count = *s_count;
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  DownWalker walk(a, runs);
  DownSegment g;

  if (warp == 0) {
    // ------------------------------------------------------------- producer
    // A stage: a step's K-blocks of A, then those of x.
    const uint32_t base = uniform(smem_u32(smem)), full0 = uniform(smem_u32(&full[0]));
    const uint32_t step = a.step, a_bytes = a.rank * 128, loads = a.whole_steps ? 1 : step;
    uint32_t count = 0, stage = 0, phase = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const uint32_t rows = uniform(x_rows(a, g.n)), m = uniform(g.m0), id = uniform(g.id), k1 = uniform(g.k1);
      ok = __all_sync(0xFFFFFFFFu, *abort_flag == 0u);
      for (uint32_t k = uniform(g.k0); ok && k < k1; ++k) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, timeout));
        if (!ok) break;
        const uint32_t bar = full0 + 8u * stage, at = uniform(base + stage * a.stage_bytes);
        expect_tx_elected(bar, (a_bytes + rows * 128) * step);
        for (uint32_t i = 0; i < loads; ++i) {
          const uint32_t kb = k * step + i, x = a.whole_steps ? 0u : kb * 64u, z = a.whole_steps ? kb : 0u;
          const uint32_t to = at + a_bytes * step + i * rows * 128;
          load_4d(at + i * a_bytes, &tm_a, bar, x, 0, z, id);
          if (rows == 8u) {
            load_3d(to, &tm_x8, bar, x, m, z);
          } else if (rows == static_cast<uint32_t>(a.tall_rows)) {
            load_3d(to, &tm_tall, bar, x, m, z);
          } else {
            load_3d(to, &tm_x64, bar, x, m, z);
          }
        }
        ++count;
        if (++stage == static_cast<uint32_t>(a.stages)) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) fail(&g_iq_status_adapters, abort_flag, kStatusProducerWait);
    // Every copy has landed before the CTA ends, also when a wait gave up.
    const uint32_t n = a.stages;
    for (uint32_t i = count > n ? count - n : 0; i < count; ++i) {
      if (!mbar_wait(&full[i % n], i / n & 1u, timeout)) fail(&g_iq_status_adapters, abort_flag, kStatusTeardownWait);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    const uint32_t base = uniform(smem_u32(smem)), acc0 = uniform(tmem), empty0 = uniform(smem_u32(&empty[0]));
    const uint32_t step = a.step, a_bytes = a.rank * 128;
    uint32_t stage = 0, phase = 0, seg = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const uint32_t acc = uniform(seg & 1u), rows = uniform(x_rows(a, g.n)), k0 = uniform(g.k0), k1 = uniform(g.k1);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&tmem_empty[acc], (seg >> 1 & 1u) ^ 1u, timeout) && *abort_flag == 0u);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t idesc = uniform(idesc_f32(128, g.width, 0, 0) | kBf16Operands);
      const uint32_t last = uniform(chains(g.width) - 1u), apart = uniform(kMaxWidth / chains(g.width));
      for (uint32_t k = k0; k < k1; ++k) {
        ok = __all_sync(0xFFFFFFFFu, 0 != mbar_wait(&full[stage], phase, timeout));
        if (!ok) break;
        const uint32_t at = uniform(base + stage * a.stage_bytes);
        const Desc a_desc = smem_desc(at, 16, 1024, 2), x_desc = smem_desc(at + a_bytes * step, 16, 1024, 2);
        const uint32_t n = min(step, a.k_blocks - k * step);
        for (uint32_t i = 0; i < n; ++i) {
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) {
            tc_mma_f16(acc0 + acc * kMaxWidth + (q & last) * apart, a_desc.at(i * a_bytes + 32 * q), x_desc.at(i * rows * 128 + 32 * q),
                       idesc, k != k0 || i != 0 || q > last ? 1u : 0u);
          }
        }
        commit_elected(empty0 + 8u * stage);
        if (++stage == static_cast<uint32_t>(a.stages)) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) commit_elected(uniform(smem_u32(&tmem_full[acc])));
      ++seg;
    }
    if (!ok) fail(&g_iq_status_adapters, abort_flag, kStatusMmaWait);
    commit_elected(uniform(smem_u32(drained)));
  } else {
    // ----------------------------------------------- a part of V, per segment
    const int quad = warp & 3, r = quad * 32 + lane;
    uint32_t seg = 0;
    bool ok = true;
    const long long plane = runs.rows[runs.count];
    while (walk.next(g)) {
      const uint32_t acc = seg & 1u;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&tmem_full[acc], seg >> 1 & 1u, timeout) && *abort_flag == 0u);
      if (!ok) break;
      tc_fence_after_sync();
      if (quad * 32 < a.rank) {
        // 32 columns at a time: with 16 the last tile's way out took 2.5 us (five
        // prompts, both kernels: 28.7 us, with 32 26.1).
        float* to = a.part + (g.part * plane + g.row) * a.rank + r;
        const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * kMaxWidth;
        for (int c0 = 0; c0 < g.n; c0 += 32, to += 32ll * a.rank) {
          float v[32];
          tmem_ld_32x32b_x32(from + c0, v);
          tmem_ld_wait(v);
          for (uint32_t chain = 1; chain < chains(g.width); ++chain) {
            float w[32];
            tmem_ld_32x32b_x32(from + chain * (kMaxWidth / chains(g.width)) + c0, w);
            tmem_ld_wait(w);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += w[i];
          }
          if (r < a.rank) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (c0 + i < g.n) to[i * a.rank] = v[i];
            }
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tmem_empty[acc]);
      ++seg;
    }
    if (!ok) fail(&g_iq_status_adapters, abort_flag, kStatusEpilogueWait);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    if (!mbar_wait(drained, 0, 2 * timeout)) fail(&g_iq_status_adapters, abort_flag, kStatusTeardownWait);
    tc_fence_after_sync();
    tmem_dealloc(tmem, 256);
  }
}

// ---- K18

constexpr int kUpThreads = 320;
constexpr int kUpWarps = 8;                       // 2 .. 9: V, base, output
constexpr int kTerms = 3;                         // BF16 terms of scale V
// kAtoms: 64-wide pieces of the rank.
template <int kAtoms>
struct UpLayout {
  static constexpr int kStages = 3;
  static constexpr int kCtasPerSm = kAtoms == 1 ? 2 : 1;
  static constexpr int kBBytes = 128 * 128 * kAtoms;
  static constexpr int kTermBytes = kUpWidth * 128 * kAtoms;
  static constexpr int kOffV = kStages * kBBytes;
  static constexpr int kOffOut = kOffV + kTerms * kTermBytes;
  static constexpr int kOffBar = kOffOut + kUpWarps * 2048;
  static constexpr int kNumBars = 2 * kStages + 4 + 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffRuns = kOffMisc + 16 + kScratchBytes;
  static_assert(kOffRuns + kRunArrays * (kMaxRequests + 1) * 4 <= 227 * 1024, "shared memory");
};

// The features of a tile of rows that are multiplied at a time: one or two tiles
// of 128.
struct UpUnit {
  int id, m0, n, width, row;
  int f, halves;            // first tile of 128 features, and how many
  int begin;                // where the row tile begins in K17's units
  int c;                    // K17's units of one step
  bool narrow;              // two at a time
  bool same;                // the rows of the unit before
};

struct UpWalker {
  const AdapterArgs& a;
  const Runs& s;
  int u, u1;                // where the next unit begins, and the CTA's run ends
  int run, tt, piece, f, each, c, f_units;
  Tiling t, p;
  bool same;
  __device__ __forceinline__ UpWalker(const AdapterArgs& args, const Runs& runs)
      : a(args), s(runs), run(0), tt(0), piece(0), f(0), same(false) {
    const int total = s.up[s.count], per = (total + gridDim.x - 1) / static_cast<int>(gridDim.x);
    u = static_cast<int>(min(static_cast<long long>(per) * blockIdx.x, static_cast<long long>(total)));
    u1 = static_cast<int>(min(static_cast<long long>(u) + per, static_cast<long long>(total)));
    if (u >= u1) return;
    run = find_run(s, s.up, u);
    enter();
    // A unit belongs to the CTA in whose run it begins.
    const int j = (u - s.up[run] + each - 1) / each, pieces = j / f_units;
    u = s.up[run] + j * each;
    f = j - pieces * f_units;
    tt = pieces / p.tiles;
    piece = pieces - tt * p.tiles;
    if (tt == t.tiles) {                               // behind the run's last unit
      --tt;
      piece = p.tiles;
    }
  }
  __device__ __forceinline__ void enter() {
    t = tiling(s.end[run] - s.first[run]);
    p = up_pieces(t.width);
    each = up_unit(s.id[run], p.width);
    c = down_unit(a, s.id[run], t.width);
    f_units = up_tiles(a, p.width);
  }
  __device__ __forceinline__ bool next(UpUnit& g) {
    while (u < u1) {
      if (piece == p.tiles) {
        piece = 0;
        if (++tt == t.tiles) {
          tt = 0;
          ++run;
          enter();
        }
      }
      const int first = tt * t.width + piece * p.width;
      const int rows = min(min(t.width * (tt + 1), s.end[run] - s.first[run]) - first, p.width);
      if (rows <= 0) {                                 // a run's last tile may have fewer pieces
        u += (f_units - f) * each;
        f = 0;
        ++piece;
        continue;
      }
      g.id = s.id[run];
      g.m0 = s.first[run] + first;
      g.n = rows;
      g.width = (rows + 15) & ~15;
      g.row = s.rows[run] + first;
      const int halves = up_halves(p.width);
      g.f = f * halves;
      g.halves = min(halves, a.f_tiles - g.f);
      g.narrow = halves == 2;
      g.c = c;
      g.begin = s.down[run] + tt * a.k_steps * c;
      g.same = same;
      same = true;
      u += each;
      if (++f == f_units) {
        f = 0;
        ++piece;
        same = false;
      }
      return true;
    }
    return false;
  }
};

template <int kAtoms, bool kMany>
__global__ void __launch_bounds__(kUpThreads, UpLayout<kAtoms>::kCtasPerSm)
    adapter_up_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ AdapterArgs a) {
  using L = UpLayout<kAtoms>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Runs runs = runs_at(reinterpret_cast<int*>(smem + L::kOffRuns), a.requests);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty = full + L::kStages;
  uint64_t* tmem_full = empty + L::kStages;       // [2]
  uint64_t* tmem_empty = tmem_full + 2;           // [2]
  uint64_t* v_full = tmem_empty + 2;              // V of a row tile is staged
  uint64_t* drained = v_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc + 4);
  int* s_count = reinterpret_cast<int*>(smem + L::kOffMisc + 8);
  int* scratch = reinterpret_cast<int*>(smem + L::kOffMisc + 16);
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint64_t timeout = a.timeout_ns;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_b);
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], kUpWarps);
    }
    mbar_init(v_full, kUpWarps);
    mbar_init(drained, 1);
    *abort_flag = (smem_u32(smem) & 1023u) != 0 ? 1u : 0u;   // the swizzles would not match; never seen
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * kUpWidth);
    tmem_relinquish();
  }
  // K17 lets this kernel start when all kernels before it have completed, so what
  // K17 does not write may be read while it runs: the runs are found, B and base
  // are loaded ahead, and only V waits for it.
  if constexpr (kMany) {
    runs.count = find_runs<kUpThreads / 32>(a, runs, scratch);
  } else if (warp == 0) {
    const int count = find_runs<1>(a, runs, scratch);
    if (lane == 0) *s_count = count;
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (!kMany) runs.count = *s_count;
  grid_launch_dependents();                         // this CTA has its tensor memory
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  UpWalker walk(a, runs);
  UpUnit g;

  if (warp == 0) {
    // ------------------------------------------------------------- producer
    const uint32_t base = uniform(smem_u32(smem)), full0 = uniform(smem_u32(&full[0]));
    uint32_t count = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      if (g.id < 0) continue;
      const uint32_t id = uniform(g.id), f1 = uniform(g.f + g.halves);
      for (uint32_t f = uniform(g.f); f < f1; ++f) {
        const uint32_t stage = uniform(count % L::kStages), bar = full0 + 8u * stage;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], (count / L::kStages & 1u) ^ 1u, timeout) && *abort_flag == 0u);
        if (!ok) break;
        expect_tx_elected(bar, L::kBBytes);
#pragma unroll
        for (int i = 0; i < kAtoms; ++i) load_3d(base + stage * L::kBBytes + i * 128 * 128, &tm_b, bar, 64 * i, f * 128, id);
        ++count;
      }
    }
    if (!ok) fail(&g_iq_status_adapters, abort_flag, kStatusProducerWait);
    for (uint32_t i = count > L::kStages ? count - L::kStages : 0; i < count; ++i) {
      if (!mbar_wait(&full[i % L::kStages], i / L::kStages & 1u, timeout)) {
        fail(&g_iq_status_adapters, abort_flag, kStatusTeardownWait);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    const uint32_t base = uniform(smem_u32(smem)), acc0 = uniform(tmem);
    const uint32_t empty0 = uniform(smem_u32(&empty[0])), tmem_full0 = uniform(smem_u32(&tmem_full[0]));
    const Desc b_desc = smem_desc(base, 16, 1024, 2), v_desc = smem_desc(base + L::kOffV, 16, 1024, 2);
    const uint32_t steps = (a.rank + 15) / 16;
    uint32_t count = 0, tiles = 0, units = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      if (g.id < 0) continue;
      const uint32_t acc = uniform(units & 1u), halves = uniform(g.halves);
      if (!g.same) {
        ok = mbar_wait(v_full, tiles & 1u, timeout);
        ++tiles;
      }
      ok = ok && mbar_wait(&tmem_empty[acc], (units >> 1 & 1u) ^ 1u, timeout) && *abort_flag == 0u;
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t idesc = uniform(idesc_f32(128, g.width, 0, 0) | kBf16Operands);
      for (uint32_t h = 0; h < halves; ++h, ++count) {
        const uint32_t stage = uniform(count % L::kStages);
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], count / L::kStages & 1u, timeout));
        if (!ok) break;
        for (uint32_t term = 0; term < kTerms; ++term) {
          for (uint32_t k = 0; k < steps; ++k) {
            const uint32_t in = 32 * (k & 3), atom = k >> 2;
            tc_mma_f16(acc0 + acc * kUpWidth + h * kNarrow, b_desc.at(stage * L::kBBytes + atom * (128 * 128) + in),
                       v_desc.at(term * L::kTermBytes + atom * (kUpWidth * 128) + in), idesc, (term | k) != 0 ? 1u : 0u);
          }
        }
        commit_elected(empty0 + 8u * stage);
      }
      if (ok) commit_elected(tmem_full0 + 8u * acc);
      ++units;
    }
    if (!ok) fail(&g_iq_status_adapters, abort_flag, kStatusMmaWait);
    commit_elected(uniform(smem_u32(drained)));
  } else {
    // ------------------------------------------------- V, base and the output
    // Warps w and w + 4 share the 32 features of quarter w % 4 and take every
    // other 32 rows.
    const int quad = warp & 3, which = (warp - 2) >> 2, tid = threadIdx.x - 64;
    uint8_t* stage = smem + L::kOffOut + (warp - 2) * 2048;
    const uint32_t stage_at = smem_u32(stage);
    const int chunk = lane & 3, row8 = lane >> 2;           // of a row-wise access: 4 pieces of 8 rows
    uint32_t count = 0;
    bool ok = true;
    const int per = down_per(a, runs.down[runs.count]);
    const long long plane = runs.rows[runs.count];
    // This warp's features and rows of a unit: warps w and w + 4 take a tile of
    // features each, or 32 rows each.
    auto column = [&](const UpUnit& of) { return (of.f + (of.narrow ? which : 0)) * 128 + quad * 32 + chunk * 8; };
    auto first_row = [&](const UpUnit& of) { return of.narrow ? (which < of.halves ? 0 : kUpWidth) : 32 * which; };
    // Those rows of base, in this lane's pieces.
    auto load_base = [&](const UpUnit& of, uint4 (&held)[4]) {
      const int col = column(of), c0 = first_row(of);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = c0 + 8 * i + row8;
        held[i] = make_uint4(0, 0, 0, 0);
        if (a.base != nullptr && r < of.n && col < a.cols) {
          held[i] = ld_dependent_v4(a.base + (of.m0 + r) * a.ld_base + col);
        }
      }
    };
    // V of a row tile: the parts in order, times scale, as three BF16 terms under the
    // 128-byte swizzle.  (The products with the V before are done: this warp has
    // waited for the last of them.)
    bool waited = false;
    auto stage_v = [&](const UpUnit& of) {
      if (!waited) grid_dependency_wait();
      waited = true;
      const int first = first_part(of.begin, of.c, per);
      const int parts = (of.begin + a.k_steps * of.c - 1) / per - first + 1;
      const float scale = a.scale[of.id];
      const int chunks = (a.rank + 15) / 16 * 2;            // the products read the rank rounded up to 16
      for (int i = tid; i < of.width * chunks; i += kUpWarps * 32) {
        const int r = i / chunks, c = i - r * chunks;          // eight values of one row
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
        if (r < of.n && 8 * c < a.rank) {
          const float* from = a.part + static_cast<long long>(of.row + r) * a.rank + 8 * c;
#pragma unroll 4
          for (int p = 0; p < parts; ++p) {
            const float4 x = *reinterpret_cast<const float4*>(from + p * plane * a.rank);
            const float4 y = *reinterpret_cast<const float4*>(from + p * plane * a.rank + 4);
            v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
            v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] *= scale;
        }
        uint8_t* to = smem + L::kOffV + (c >> 3) * (kUpWidth * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
#pragma unroll
        for (int term = 0; term < kTerms; ++term, to += L::kTermBytes) {
          // The upper eight bits of what is left, cut off, not rounded: the largest
          // floats would round to an infinity.  Of an infinity or NaN (that of a
          // product: all its bits are set) the first term is all there is.
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] = __byte_perm(__float_as_uint(v[2 * k]), __float_as_uint(v[2 * k + 1]), 0x7632);
            v[2 * k] = fabsf(v[2 * k]) < INFINITY ? v[2 * k] - bf16_lo(w[k]) : 0.f;
            v[2 * k + 1] = fabsf(v[2 * k + 1]) < INFINITY ? v[2 * k + 1] - bf16_hi(w[k]) : 0.f;
          }
          *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full);
    };
    // The next unit's base rows are asked for as soon as this one's have left the
    // registers.  (One body for all of it: the loop unrolled twice, with two sets of
    // registers, waits for instructions.)
    uint4 held[4];
    UpUnit then;
    bool more = walk.next(g);
    if (more) load_base(g, held);
    while (more) {
      const bool adapts = g.id >= 0;
      if (adapts && !g.same) stage_v(g);
      more = walk.next(then);
      const uint32_t acc = count & 1u;
      if (adapts) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&tmem_full[acc], count >> 1 & 1u, timeout) && *abort_flag == 0u);
        if (!ok) break;
        tc_fence_after_sync();
      }
      const int col = column(g), c0 = first_row(g);
      const bool rows = c0 < g.n;                      // the same in all lanes
      if (rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + row8;
          *reinterpret_cast<uint4*>(stage + r * 64 + ((chunk ^ (r >> 1 & 3)) << 4)) = held[i];
        }
      }
      if (more) load_base(then, held);
      __syncwarp();
      if (rows && adapts) {
        const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * kUpWidth + which * kNarrow;
        float lo[16], hi[16];                         // features 0 .. 15 and 16 .. 31 of the quarter
        tmem_ld_16x256b_x4(from, lo);
        tmem_ld_16x256b_x4(from + (16u << 16), hi);
        tmem_ld_wait16(lo);
        tmem_ld_wait16(hi);
#pragma unroll
        for (int t = 0; t < 4; ++t) {                 // 8 rows at a time
          if (c0 + 8 * t >= g.n) break;
          const int r = 8 * t + (lane & 7), at = r * 64 + (((lane >> 3) ^ (r >> 1 & 3)) << 4);
          const uint4 b = ldmatrix_x4_trans(stage_at + at);
          stmatrix_x4_trans(stage_at + at, cvt_bf16x2(lo[4 * t] + bf16_lo(b.x), lo[4 * t + 1] + bf16_hi(b.x)),
                            cvt_bf16x2(lo[4 * t + 2] + bf16_lo(b.y), lo[4 * t + 3] + bf16_hi(b.y)),
                            cvt_bf16x2(hi[4 * t] + bf16_lo(b.z), hi[4 * t + 1] + bf16_hi(b.z)),
                            cvt_bf16x2(hi[4 * t + 2] + bf16_lo(b.w), hi[4 * t + 3] + bf16_hi(b.w)));
        }
      }
      if (adapts) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tmem_empty[acc]);
        ++count;
      }
      if (rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + row8;
          if (c0 + r < g.n && col < a.cols) {
            *reinterpret_cast<uint4*>(a.out + (g.m0 + c0 + r) * a.ld_out + col) =
                *reinterpret_cast<const uint4*>(stage + r * 64 + ((chunk ^ (r >> 1 & 3)) << 4));
          }
        }
      }
      __syncwarp();
      g = then;
    }
    if (!waited) grid_dependency_wait();
    if (!ok) fail(&g_iq_status_adapters, abort_flag, kStatusEpilogueWait);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    if (!mbar_wait(drained, 0, 2 * timeout)) fail(&g_iq_status_adapters, abort_flag, kStatusTeardownWait);
    tc_fence_after_sync();
    tmem_dealloc(tmem, 2 * kUpWidth);
  }
}

constexpr int kMaxDownCtas = 160;

// kMany: more requests than this, whose runs all of a block's warps find; up to here
// one warp does it without waiting for others (one request: both kernels 8.8 us, by
// all warps 9.9; 64 requests 29.8 by all and 30.3 by one, 1024 requests 30 and 41).
constexpr int kFewRequests = 32;

size_t runs_bytes(const AdapterArgs& a) { return kRunArrays * (static_cast<size_t>(a.requests) + 1) * sizeof(int); }

template <int kAtoms, bool kMany>
cudaError_t launch_up(const CUtensorMap& tm_b, const AdapterArgs& a, int sm_count, cudaStream_t stream) {
  using L = UpLayout<kAtoms>;
  return launch_dependent(adapter_up_kernel<kAtoms, kMany>, dim3(sm_count * L::kCtasPerSm), kUpThreads, L::kOffRuns + runs_bytes(a), stream,
                          tm_b, a);
}

}  // namespace

cudaError_t adapters_setup_device() {
  for (const void* f : {reinterpret_cast<const void*>(adapter_down_kernel<false>), reinterpret_cast<const void*>(adapter_down_kernel<true>),
                        reinterpret_cast<const void*>(adapter_up_kernel<1, false>), reinterpret_cast<const void*>(adapter_up_kernel<1, true>),
                        reinterpret_cast<const void*>(adapter_up_kernel<2, false>), reinterpret_cast<const void*>(adapter_up_kernel<2, true>)}) {
    const cudaError_t err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// Part p of row i is row p * R + i of the workspace, R the rows with an adapter.  A
// tile lies in at most kMaxParts + 1 runs, as a run is not shorter than a kMaxParts-th
// of it.  It also lies in at most ctas / tiles + 2, and there are at least R / kMaxWidth
// tiles: fewer than ctas * kMaxWidth + 2 R rows.
size_t adapters_workspace(int tokens, int rank) {
  const size_t t = static_cast<size_t>(tokens), few = (kMaxParts + 1) * t, many = 3 * t + static_cast<size_t>(kMaxDownCtas) * kMaxWidth;
  return (few < many ? few : many) * static_cast<size_t>(rank) * sizeof(float);
}

// K-blocks of a stage of K17: as many as leave room for three stages.
int adapters_step(int tokens, int rank) {
  const int rows = rank + adapters_tall_rows(tokens);
  return rows <= 64 ? 4 : (rows <= 128 ? 2 : 1);
}

bool adapters_countable(int tokens, int requests, int rank, int K, int N) {
  const long long tiles = tokens / kMaxWidth + 1ll + (requests < tokens ? requests : tokens);
  const long long down = ((K + 63ll) / 64) * (kStepUnits + rank + kMaxWidth), up = ((N + 127ll) / 128) * 2 * (96 + kUpWidth);
  return tiles * (down > up ? down : up) < 1ll << 30;
}

// The highest box of rows of x.
int adapters_tall_rows(int tokens) { return tokens >= kMaxWidth ? kMaxWidth : (tokens + 15) / 16 * 16; }

cudaError_t launch_adapters(const AdapterMaps& m, AdapterArgs a, void* ws, int sm_count, cudaStream_t stream) {
  a.part = static_cast<float*>(ws);
  a.down_ctas = sm_count < kMaxDownCtas ? sm_count : kMaxDownCtas;
  a.tall_rows = adapters_tall_rows(a.tokens);
  a.step = adapters_step(a.tokens, a.rank);
  a.k_steps = (a.k_blocks + a.step - 1) / a.step;
  a.stage_bytes = (a.rank + a.tall_rows) * 128 * a.step;
  a.stages = kDownStageBytes / a.stage_bytes < kMaxDownStages ? kDownStageBytes / a.stage_bytes : kMaxDownStages;
  // At least one step, so that every run inside a tile has some.
  const int least = (a.k_steps * (kStepUnits + a.rank + a.tall_rows) + kMaxParts - 1) / kMaxParts, step = kStepUnits + a.rank + kMaxWidth;
  a.down_least = least > step ? least : step;
  // Rows of A past the rank are read from what follows them.
  const size_t runs = kDownOffRuns + runs_bytes(a), read = static_cast<size_t>(a.stages - 1) * a.stage_bytes + ((a.step - 1) * a.rank + 128) * 128;
  const size_t smem = runs > read ? runs : read;
  const bool many = a.requests > kFewRequests;
  const cudaError_t err = many ? launch_dependent(adapter_down_kernel<true>, dim3(a.down_ctas), kDownThreads, smem, stream, m.x8, m.x64,
                                                  m.tall, m.a, a)
                               : launch_dependent(adapter_down_kernel<false>, dim3(a.down_ctas), kDownThreads, smem, stream, m.x8, m.x64,
                                                  m.tall, m.a, a);
  if (err != cudaSuccess) return err;
  if (a.rank <= 64) return many ? launch_up<1, true>(m.b, a, sm_count, stream) : launch_up<1, false>(m.b, a, sm_count, stream);
  return many ? launch_up<2, true>(m.b, a, sm_count, stream) : launch_up<2, false>(m.b, a, sm_count, stream);
}

cudaError_t read_adapters_status(uint32_t* flags, bool reset) {
  uint32_t v = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_iq_status_adapters, sizeof(v));
  if (err != cudaSuccess) return err;
  if (flags) *flags = v;
  if (reset) {
    const uint32_t zero = 0;
    err = cudaMemcpyToSymbol(g_iq_status_adapters, &zero, sizeof(zero));
  }
  return err;
}

}  // namespace iq
