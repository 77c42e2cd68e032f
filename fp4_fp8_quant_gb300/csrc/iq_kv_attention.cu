// Attention over the paged 8-bit KV cache (include/iq.h, section 4):
//   out = sum_s p_s v_s / sum_s p_s,  p_s = 2^(x_s),  x_s = scale log2(e) q . k_s.
//
// K9 kv_attention_kernel, for items of up to 32 rows (decode; a row is one
// (token, query head), an item the rows of one KV head, N at a time).  The keys
// are the MMA's M side in the first product and its K side in the second, the
// rows its N side in both:
//   S^T [128 keys, N rows]  = K [128, D]  x  Q^T [D, N]
//   O^T [D, N rows]        += V^T [D, 128]  x  P [128, N]   (two terms of P)
// so a tile costs the tensor cores little although the rows are few, and what
// bounds the kernel is the cache's bytes: every one is moved once, by TMA.
//
// BF16 times E4M3 without loss.  The first product multiplies E4M3 by E4M3, and
// a BF16 value is the sum of two: with a row scaled by a power of two to at
// most 448, q1 = E4M3(q) leaves a remainder of at most four significant bits,
// which q2 = E4M3(q - q1) holds exactly (down to 2^-19 of the row's largest
// value).  The two products add up in one float32 accumulator.  The second
// product is in BF16, which has float32's exponents: a value's code is exact in
// it, and a weight is the sum of two terms with 16 significant bits, however far
// it lies below the row's largest (8 bits from some 2^-47 of it on).  The terms are columns of one MMA, which reads
// V once (a second MMA for the second term: 64 ragged sequences 172 -> 205 us).
//
// Scales.  A key's scale 2^eK multiplies its scores, one factor per lane of
// the accumulator; a value's scale 2^eV multiplies its key's weights, so values
// stay codes.
//
// The running maximum is lazy: m moves, and the accumulator is scaled, only
// when some weight 2^(x - m) would pass 2^kMost.  Maximum and exponents come from the same rounded x:
// one step settles a tile however large the scores are.
//
// Work is divided by key tiles: the tiles of all items, laid end to end, are
// cut into one equal run per CTA (two CTAs per SM), so ragged lengths, one long
// sequence and many short ones load the SMs alike; an item counts kItemTiles
// tiles more for its beginning and end.  An item cut between CTAs leaves its
// partial sums (float32, with m and the sum) in the workspace, and K10 joins
// them in a fixed order, so the same call gives the same bits.
//
// Warps: 0..3 softmax (one key per thread; the same threads split Q, convert V
// and store O, one dimension per thread), 4 producer (page lookups, TMA), 5 MMA
// issuer.  K and V have a ring of slots each; the scores are double buffered, so
// S of the next tile is computed while the softmax works on this one.  Every
// wait is bounded.
//
// Where keys are selected, K's rows are gathered by TMA, four at a time, and
// V's are copied by the threads that convert them.  Gathering takes 13 cycles
// per row: with V gathered too, 2048 keys for each of 4632 tokens under 8 query
// heads took 823 us, with them copied 470 (498 with two terms of P); copying a part of K as well gained nothing.
//
// Measured: 64 sequences of up to 16384 keys, 8 KV heads (1.08 GB of cache)
// 172 us; one row over 262144 keys, 4 KV heads (268 MB) 53.0 us with the join;
// over 4632 keys 12.9 us, of which 2 us find the CTA's place, 2 us are the first
// page's lookup, 4 us the tile itself and 4 us the join.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "iq_internal.h"
#include "iq_kv.h"
#include "iq_kv_attention.cuh"
#include "iq_ptx.cuh"

namespace iq {

__device__ uint32_t g_iq_status_kv;

namespace {

constexpr int kSoftmax = 128;              // softmax threads, one key each
constexpr float kMost = 40.f;              // log2 of the largest weight
static_assert(kUp == 0x1p40f, "kMost");

template <int N, int D>
struct Layout {
  static constexpr int kThreads = kSoftmax + 64;
  static constexpr int kCtasPerSm = 2;
  static constexpr int kSlotBytes = kTile * D;
  static constexpr int kSlotsK = 2;
  static constexpr int kSlotsV = N <= 16 || D == 64 ? 2 : 1;
  static constexpr int kMetaTiles = 4;           // tiles whose key scales are held
  static constexpr int kQBytes = N * D;          // one term of Q
  static constexpr int kPBytes = kTile * N * 2;  // one term of P
  static constexpr int kVBytes = kTile * D * 2;  // values in BF16
  static constexpr int kOffCodesV = kSlotsK * kSlotBytes;
  static constexpr int kOffV = kOffCodesV + kSlotsV * kSlotBytes;
  static constexpr int kOffQ = kOffV + kVBytes;
  static constexpr int kOffP = kOffQ + 2 * kQBytes;
  static constexpr int kOffMeta = kOffP + 2 * kPBytes;
  static constexpr int kOffOut = kOffMeta + kMetaTiles * kTile * 8;  // long long [N]: where the row's output goes
  static constexpr int kOffRows = kOffOut + N * 8;                   // float m, nm, bq, corr [N], int vis [N]
  static constexpr int kOffRed = kOffRows + 5 * N * 4;               // float [4][N]
  static constexpr int kOffBar = kOffRed + 4 * N * 4;
  static constexpr int kNumBars = 2 * (kSlotsK + kSlotsV) + 2 + 4 + kMetaTiles;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 96;
  // Tensor memory: two score buffers and the output accumulator, N columns for
  // each term of P (a power of two is allocated).
  static constexpr uint32_t kColS = 0, kColO = 2 * N, kTmemCols = 4 * N;
  static_assert(kOffQ % 1024 == 0 && kOffP % 128 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(kSmemBytes <= 226 * 1024 / kCtasPerSm, "shared memory");
  static_assert(kMetaTiles >= kSlotsK + 2, "a tile's key scales stay until its softmax is done");
};

template <int N, int D, bool kSelected>
__global__ void __launch_bounds__(Layout<N, D>::kThreads, Layout<N, D>::kCtasPerSm)
    kv_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ AttnParams p) {
  using L = Layout<N, D>;
  // Two CTAs leave no room for moving to a boundary.  (What is added is 0 below,
  // but known only at run time: the arrays' addresses then are sums of a register
  // and not constants to be made each time, 64 ragged sequences 174 -> 171 us.)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (smem_u32(smem_raw) & 1023u);
  uint8_t* s_q = smem + L::kOffQ;
  uint8_t* s_p = smem + L::kOffP;
  long long* s_out = reinterpret_cast<long long*>(smem + L::kOffOut);
  int2* s_meta = reinterpret_cast<int2*>(smem + L::kOffMeta);        // [L::kMetaTiles][128] row, scale bytes eK | eV << 16
  float* s_m = reinterpret_cast<float*>(smem + L::kOffRows);         // running maximum
  float* s_nm = s_m + N;                                             // its negative
  float* s_bq = s_m + 2 * N;                                         // scale of the query row
  float* s_corr = s_m + 3 * N;
  int* s_vis = reinterpret_cast<int*>(s_m + 4 * N);
  float* s_red = reinterpret_cast<float*>(smem + L::kOffRed);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* k_empty = k_full + L::kSlotsK;
  uint64_t* v_full = k_empty + L::kSlotsK;  // codes of V
  uint64_t* v_empty = v_full + L::kSlotsV;
  uint64_t* s_full = v_empty + L::kSlotsV;  // [2] scores of a tile are there
  uint64_t* q_full = s_full + 2;            // Q of a segment is staged
  uint64_t* p_full = q_full + 1;            // weights and values of a tile are staged, its scores read
  uint64_t* pv_done = q_full + 2;           // second product of a tile is done
  uint64_t* drained = q_full + 3;           // everything the issuer sent is done
  uint64_t* meta_full = q_full + 4;         // [L::kMetaTiles]
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + 4);
  Start* s_start = reinterpret_cast<Start*>(smem + L::kOffMisc + 8);
  static_assert(sizeof(Start) <= 88, "start");

  const AttnArgs& a = p.a;
  const uint64_t timeout = p.timeout_ns;
  if ((smem_u32(smem_raw) & 1023u) != 0) {                  // the swizzles would not match; never seen
    if (threadIdx.x == 0) {
      atomicOr(&g_iq_status_kv, kStatusProducerWait);
      p.heads[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kProducerWarp = kSoftmax / 32, kMmaWarp = kProducerWarp + 1;

  grid_launch_dependents();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int i = 0; i < L::kSlotsK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < L::kSlotsV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], kSoftmax);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(q_full, kSoftmax);
    mbar_init(p_full, kSoftmax);
    mbar_init(pv_done, 1);
    mbar_init(drained, 1);
    for (int i = 0; i < L::kMetaTiles; ++i) mbar_init(&meta_full[i], 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  if (warp == kProducerWarp) {
    const Start st = find_start<N>(a);
    if (lane == 0) *s_start = st;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const Start& start = *s_start;
  const int none = a.kv.num_pages * a.kv.heads * a.kv.page;   // a row past the end: TMA fills zeros

  if (warp == kProducerWarp) {
    // -------------------------------------------------------------- producer
    Walker<N> walk(start);
    Segment g = {};
    [[maybe_unused]] const bool leader = ((4 * lane) & (a.kv.page - 1)) == 0;
    int pushed = 0, pushed_v = 0;                     // tiles whose K / V is on its way
    bool ok = true;                                   // the same in every lane

    // Loads the tile's codes into the next slot of a ring.
    auto push = [&](const CUtensorMap* map, uint64_t* full, uint64_t* empty, uint8_t* ring, int slots, int& count,
                    const int* rows) {
      const int slot = count % slots;
      const bool free = mbar_wait(&empty[slot], (count / slots & 1) ^ 1, timeout) && *abort_flag == 0u;
      if (!__all_sync(0xFFFFFFFFu, free)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], L::kSlotBytes);
      __syncwarp();
      uint8_t* dst = ring + slot * L::kSlotBytes + 4 * lane * D;
      if constexpr (kSelected) {
        tma_gather4(dst, map, &full[slot], make_int4(rows[0], rows[1], rows[2], rows[3]));
      } else if (leader) {
        tma_load_2d(dst, map, &full[slot], 0, rows[0]);
      }
      ++count;
      return true;
    };
    auto push_v = [&](const int* rows) {
      return push(&tm_v, v_full, v_empty, smem + L::kOffCodesV, L::kSlotsV, pushed_v, rows);
    };

    auto push_k = [&](const int* rows) { return push(&tm_k, k_full, k_empty, smem, L::kSlotsK, pushed, rows); };
    // What the others need of the keys of the tile pushed last: rows and scales.
    auto publish = [&](const int* rows, const uint32_t* sf) {
      const int mslot = (pushed - 1) % L::kMetaTiles;
      int4* dst = reinterpret_cast<int4*>(s_meta + mslot * kTile + 4 * lane);
      dst[0] = make_int4(rows[0], sf[0], rows[1], sf[1]);
      dst[1] = make_int4(rows[2], sf[2], rows[3], sf[3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&meta_full[mslot]);
    };

    if constexpr (!kSelected) {
      // Pages in order: lane l looks up page l of a batch of 32, one batch
      // ahead, pages while the batch begins and their scales a tile later.
      const int per_tile = kTile >> a.kv.page_log2;
      while (ok && walk.next(a, g)) {
        const int page0 = (g.kt0 * kTile) >> a.kv.page_log2;
        const int my_page = (4 * lane) >> a.kv.page_log2;          // of a tile
        int pid, next_pid;
        uint32_t ek = 0, ev = 0, next_ek = 0, next_ev = 0;
        auto find_page = [&](int j) {
          const long long pos = static_cast<long long>(page0 + j + lane) << a.kv.page_log2;
          return pos < g.keys ? kv_page_of(a.kv, g.b, static_cast<int>(pos)) : -1;
        };
        auto find_scales = [&](int id, uint32_t& k, uint32_t& v) {
          if (id >= 0) {
            const long long at = static_cast<long long>(id) * a.kv.heads + g.h;
            k = a.kv.sf[0][at];
            v = a.kv.sf[1][at];
          }
        };
        pid = find_page(0);
        next_pid = find_page(32);
        find_scales(pid, ek, ev);
        int last_row = none;
        for (int i = 0; ok && i < g.n; ++i) {
          const int j = (i * per_tile) & 31;
          if (j == 0 && i > 0) {
            pid = next_pid;
            ek = next_ek;
            ev = next_ev;
            next_pid = find_page(i * per_tile + 32);
          }
          const int id = __shfl_sync(0xFFFFFFFFu, pid, j + my_page);
          const int pos = (g.kt0 + i) * kTile + 4 * lane;
          const int row = id >= 0 ? static_cast<int>((static_cast<long long>(id) * a.kv.heads + g.h) * a.kv.page) : none;
          ok = push_k(&row);
          if (!ok) break;
          const uint32_t k = __shfl_sync(0xFFFFFFFFu, ek, j + my_page), v = __shfl_sync(0xFFFFFFFFu, ev, j + my_page);
          int rows[4];
          const uint32_t sf[4] = {k | v << 16, k | v << 16, k | v << 16, k | v << 16};
#pragma unroll
          for (int c = 0; c < 4; ++c) rows[c] = id >= 0 && pos + c < g.keys ? row + ((pos + c) & (a.kv.page - 1)) : none;
          publish(rows, sf);
          if (i > 0) ok = push_v(&last_row);
          last_row = row;
          if (j == 0) find_scales(next_pid, next_ek, next_ev);
        }
        ok = ok && push_v(&last_row);
      }
    } else {
      // Single rows, four keys per lane.  The three dependent loads (position,
      // page, scales) of a tile are issued two, one and one tiles ahead.  The
      // values are the softmax threads' own copies.
      while (ok && walk.next(a, g)) {
        int pos[4], pos1[4], pid[4], row[4];
        uint32_t sf[4];
        const int32_t* list = a.indices + static_cast<long long>(g.list) * a.ld_idx;
        const int32_t* table = a.kv.table + static_cast<long long>(g.b) * a.kv.table_ld;
        const int left = min(a.topk, (g.kt0 + g.n) * kTile);          // this segment's part of the list ends here
        auto find_pos = [&](int i, int* pos) {
          const int j = (g.kt0 + i) * kTile + 4 * lane;
#pragma unroll
          for (int k = 0; k < 4; ++k) pos[k] = j + k < left ? list[j + k] : -1;
        };
        auto find_pid = [&] {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            pid[k] = static_cast<unsigned>(pos[k]) < static_cast<unsigned>(g.keys) ? table[pos[k] >> a.kv.page_log2] : -1;
          }
        };
        auto find_row = [&] {                                         // (rows fit 31 bits)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            row[k] = static_cast<unsigned>(pid[k]) < static_cast<unsigned>(a.kv.num_pages)
                         ? ((pid[k] * a.kv.heads + g.h) << a.kv.page_log2) + (pos[k] & (a.kv.page - 1))
                         : none;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = row[k] != none ? row[k] >> a.kv.page_log2 : 0;
            sf[k] = a.kv.sf[0][at] | static_cast<uint32_t>(a.kv.sf[1][at]) << 16;
          }
        };
        find_pos(0, pos);
        find_pos(1, pos1);
        find_pid();
        find_row();
        for (int i = 0; ok && i < g.n; ++i) {
#pragma unroll
          for (int k = 0; k < 4; ++k) pos[k] = pos1[k];
          find_pid();
          find_pos(i + 2, pos1);
          ok = push_k(row);
          if (ok) publish(row, sf);
          find_row();
        }
      }
    }
    if (!ok) fail(&g_iq_status_kv, abort_flag, kStatusProducerWait);
    // Every copy has landed before the CTA ends (also when a wait gave up).
    for (int i = max(0, pushed - L::kSlotsK); i < pushed; ++i) {
      if (!mbar_wait(&k_full[i % L::kSlotsK], i / L::kSlotsK & 1, timeout)) fail(&g_iq_status_kv, abort_flag, kStatusTeardownWait);
    }
    for (int i = max(0, pushed_v - L::kSlotsV); i < pushed_v; ++i) {
      if (!mbar_wait(&v_full[i % L::kSlotsV], i / L::kSlotsV & 1, timeout)) fail(&g_iq_status_kv, abort_flag, kStatusTeardownWait);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    Walker<N> walk(start);
    Segment g = {};
    constexpr uint32_t kSwizzle = D == 128 ? 2u : 4u;
    const uint32_t idesc_s = idesc_f32(128, N, 0, 0), idesc_o = idesc_f32(128, 2 * N, 1, 1) | kBf16Operands;
    const uint32_t base = uniform(smem_u32(smem)), acc = uniform(tmem);
    // Q is K-major without swizzle: [16 dims][row][16].  V: 16 keys are two
    // groups of eight rows of 64 dimensions; the next 64 dimensions are 128
    // rows on (with D = 64 the second 64 lanes repeat the first).  P:
    // [8 columns][key][8].
    const Desc k_desc = smem_desc(base, 16, 8 * D, kSwizzle), q_desc = smem_desc(base + L::kOffQ, 16 * N, 128, 0);
    const Desc v_desc = smem_desc(base + L::kOffV, D == 128 ? kTile * 128 : 0, 1024, 2);
    const Desc p_desc = smem_desc(base + L::kOffP, 128, kTile * 16, 0);
    uint32_t tile = 0, seg = 0;
    bool ok = true;                                      // the same in every lane
    auto scores = [&](uint32_t t) {                      // S of tile t
      const uint32_t slot = uniform(t % L::kSlotsK);
      if (!__all_sync(0xFFFFFFFFu, 0 != mbar_wait(&k_full[slot], t / L::kSlotsK & 1u, timeout))) return false;
      tc_fence_after_sync();
      const uint32_t d = acc + L::kColS + uniform(t & 1u) * N;
      const Desc k_tile = k_desc.at(slot * L::kSlotBytes);
#pragma unroll
      for (int term = 0; term < 2; ++term) {
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          tc_mma_f8(d, k_tile.at(32 * k), q_desc.at(term * L::kQBytes + 2 * k * (16 * N)), idesc_s, (term | k) != 0);
        }
      }
      tc_commit_elected(&k_empty[slot]);
      tc_commit_elected(&s_full[t & 1u]);
      return true;
    };
    while (ok && walk.next(a, g)) {
      ok = __all_sync(0xFFFFFFFFu, 0 != mbar_wait(q_full, seg & 1u, timeout));
      ++seg;
      tc_fence_after_sync();
      ok = ok && scores(tile);
      for (int i = 0; ok && i < g.n; ++i, ++tile) {
        if (i + 1 < g.n) ok = scores(tile + 1);
        ok = ok && __all_sync(0xFFFFFFFFu, 0 != mbar_wait(p_full, tile & 1u, timeout)) && __all_sync(0xFFFFFFFFu, *abort_flag == 0u);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t more = uniform(i != 0 ? 1u : 0u);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k) {
          tc_mma_f16(acc + L::kColO, v_desc.at(2048 * k), p_desc.at(256 * k), idesc_o, k != 0 ? 1u : more);
        }
        tc_commit_elected(pv_done);
      }
    }
    if (!ok) fail(&g_iq_status_kv, abort_flag, kStatusMmaWait);
    tc_commit_elected(drained);
  } else {
    // --------------------------------------------------------------- softmax
    Walker<N> walk(start);
    Segment g = {};
    const int key = threadIdx.x;                          // key of a tile; dimension of the output
    constexpr uint32_t barrier = 1;
    const uint32_t lane_base = static_cast<uint32_t>(warp) << 21;   // this warp's 32 tensor-memory lanes
    const uint32_t o_at = tmem + lane_base + L::kColO;
    uint32_t tile = 0;
    bool ok = true;        // this thread's waits
    bool stop = false;     // some thread's wait gave up; the same in all of them
    bool first = true;     // no item has been finished here
    bool open = false;     // the last item begins here and goes on in the next CTA
    const long long run = start.per;
    // This thread's part of the values.
    constexpr int kChunks = D / 16, kSteps = kTile * kChunks / kSoftmax, kRowStep = kSoftmax / kChunks;
    const int v_piece = key % 4 + (D == 128 ? key / 8 % 2 * 4 : 0), v_q = key / (2 * kChunks);
    const int v_row = v_q / 4 * 8 + ((v_q % 4) ^ (key / 4 % 2 * 5));
    const uint32_t v_from =
        kSelected ? key * 16 : v_row * D + (D == 128 ? v_piece ^ (v_row & 7) : v_piece ^ (v_row >> 1 & 3)) * 16;
    constexpr int kFromStep = kSelected ? kSoftmax * 16 : kRowStep * D;
    // Selected keys: this thread's codes of the values, for itself alone.
    [[maybe_unused]] auto copy_v = [&](uint32_t t) {
      ok = ok && mbar_wait(&meta_full[t % L::kMetaTiles], t / L::kMetaTiles & 1u, timeout);
      if (!ok) return;
      const int2* rows = s_meta + t % L::kMetaTiles * kTile + v_row;
      uint8_t* to = smem + L::kOffCodesV + t % L::kSlotsV * L::kSlotBytes + v_from;
      int row[kSteps];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) row[j] = rows[j * kRowStep].x;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const bool there = row[j] != none;
        cp_async_16(to + j * kFromStep, a.kv.codes[1] + (there ? static_cast<long long>(row[j]) * D : 0) + v_piece * 16,
                    there ? 16u : 0u);
      }
      cp_async_commit();
    };
    const uint32_t v_to = L::kOffV + (v_piece / 4) * (kTile * 128) + v_row * 128 + (((2 * (v_piece % 4)) ^ (v_row & 7)) << 4);
    while (!stop && walk.next(a, g)) {
      if constexpr (kSelected) copy_v(tile);
      // ---- Q: rows scaled by a power of two, split into two E4M3 terms
      {
        constexpr int kPerRow = kSoftmax / N;     // threads per row
        constexpr int kVals = D / kPerRow;                 // values per thread
        const int r = key / kPerRow, part = key % kPerRow;
        uint4 x[kVals / 8];
        uint32_t m2 = 0;
        const bool there = r < g.rows;
        const int fr = g.r0 + r, tok = fr / a.group;
        const int head = g.h * a.group + fr - tok * a.group;
        if (there) {
          const uint16_t* src = a.q + (g.row0 + tok) * a.ldq + head * static_cast<long long>(D) + part * kVals;
#pragma unroll
          for (int i = 0; i < kVals / 8; ++i) x[i] = reinterpret_cast<const uint4*>(src)[i];
        } else {
#pragma unroll
          for (int i = 0; i < kVals / 8; ++i) x[i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kVals / 8; ++i) {
          m2 = __vmaxu2(m2, x[i].x & 0x7FFF7FFFu);
          m2 = __vmaxu2(m2, x[i].y & 0x7FFF7FFFu);
          m2 = __vmaxu2(m2, x[i].z & 0x7FFF7FFFu);
          m2 = __vmaxu2(m2, x[i].w & 0x7FFF7FFFu);
        }
        uint32_t m1 = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
        for (int w = 1; w < kPerRow; w <<= 1) m1 = max(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, w));
        // Smallest e with 448 * 2^e >= the largest value, at least -118.
        const uint32_t bits = m1 << 16;
        const int e = max(-118, static_cast<int>(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < kVals / 8; ++i) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t c1[4], c2[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float(w[j] << 16) * inv, hi = __uint_as_float(w[j] & 0xFFFF0000u) * inv;
            c1[j] = cvt_e4m3x2(lo, hi);
            c2[j] = cvt_e4m3x2(lo - e4m3_to_float(c1[j]), hi - e4m3_to_float(c1[j] >> 8));
          }
          const int d0 = part * kVals + 8 * i;             // K-major without swizzle: [16 dims][row][16]
          uint8_t* dst = s_q + (d0 >> 4) * (16 * N) + r * 16 + (d0 & 8);
          *reinterpret_cast<uint2*>(dst) = make_uint2(c1[0] | c1[1] << 16, c1[2] | c1[3] << 16);
          *reinterpret_cast<uint2*>(dst + L::kQBytes) = make_uint2(c2[0] | c2[1] << 16, c2[2] | c2[3] << 16);
        }
        if (part == 0) {
          s_bq[r] = query_scale(bits, e);
          s_vis[r] = there ? g.base + tok + 1 : 0;
          s_m[r] = kNoMax;
          s_out[r] = (g.row0 + tok) * a.ldo + head * static_cast<long long>(D);
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
        named_barrier_sync(barrier, kSoftmax);
      }
      const int vis_first = s_vis[0];
      float l[N];
#pragma unroll
      for (int c = 0; c < N; ++c) l[c] = 0.f;

      for (int i = 0; i < g.n; ++i, ++tile) {
        const int pos0 = (g.kt0 + i) * kTile;
        const uint32_t mslot = tile % L::kMetaTiles;
        ok = ok && mbar_wait(&meta_full[mslot], (tile / L::kMetaTiles) & 1u, timeout);
        const int2 data = s_meta[mslot * kTile + key];
        const bool seen = data.x != none;
        const float kf = seen ? a.scale_log2 * ue8m0_to_float(data.y & 0xFF) : 0.f, hide = seen ? 0.f : -INFINITY;
        const bool some_hidden = __any_sync(0xFFFFFFFFu, !seen);
        const bool causal = !kSelected && pos0 + kTile > vis_first;   // some row does not see all keys
        ok = ok && mbar_wait(&s_full[tile & 1u], (tile >> 1) & 1u, timeout);
        tc_fence_after_sync();
        const uint32_t s_at = tmem + lane_base + L::kColS + (tile & 1u) * N;
        const uint64_t kf2 = f2_pack(kf, kf), hide2 = f2_pack(hide, hide);

        // Exponents of the weights: x - m, x rounded first (the product's addend
        // is 0 or -inf); -inf where the row does not see the key.  If one passes
        // kMost anywhere (and for the first tile) the maximum moves first.
        float d[N];
        bool settle = i == 0;
        while (true) {
          if (!settle) {
            if constexpr (N == 32) {
              tmem_ld_32x32b_x32(s_at, d);
              tmem_ld_wait(d);
            } else {
              tmem_ld_32x32b_x16(s_at, d);
              tmem_ld_wait16(d);
            }
#pragma unroll
            for (int c = 0; c < N; c += 4) {
              const ulonglong2 bq = *reinterpret_cast<const ulonglong2*>(s_bq + c);
              const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(s_nm + c);
              f2_unpack(f2_add(f2_fma(f2_mul(f2_pack(d[c], d[c + 1]), bq.x), kf2, hide2), nm.x), d[c], d[c + 1]);
              f2_unpack(f2_add(f2_fma(f2_mul(f2_pack(d[c + 2], d[c + 3]), bq.y), kf2, hide2), nm.y), d[c + 2], d[c + 3]);
            }
            if (some_hidden) {
#pragma unroll
              for (int c = 0; c < N; ++c) d[c] = seen ? d[c] : -INFINITY;
            }
            if (causal) {
#pragma unroll
              for (int c = 0; c < N; ++c) d[c] = pos0 + key < s_vis[c] ? d[c] : -INFINITY;
            }
            float tops[4] = {d[0], d[1], d[2], d[3]};
#pragma unroll
            for (int c = 4; c < N; ++c) tops[c & 3] = fmaxf(tops[c & 3], d[c]);
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            if (named_barrier_and(barrier, kSoftmax, ok && !(top > kMost))) break;
          }
          // Some thread saw a weight that is too large, or gave up waiting.
          stop = !named_barrier_and(barrier, kSoftmax, ok && *abort_flag == 0u);
          if (stop) break;
          // The maximum per column, over the warp, then over the warps.
#pragma unroll 1
          for (int c0 = 0; c0 < N; c0 += 16) {
            float z[16];
            tmem_ld_32x32b_x16(s_at + c0, z);
            tmem_ld_wait16(z);
            float mine = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const bool in = seen && (kSelected || pos0 + key < s_vis[c0 + c]);
              const float m = redux_max(in ? __fmaf_rn(__fmul_rn(z[c], s_bq[c0 + c]), kf, hide) : -INFINITY);
              mine = lane == c ? m : mine;
            }
            if (lane < 16) s_red[warp * N + c0 + lane] = mine;
          }
          named_barrier_sync(barrier, kSoftmax);
          if (key < N) {
            const float old = s_m[key];
            float m = fmaxf(fmaxf(s_red[key], s_red[N + key]), fmaxf(s_red[2 * N + key], s_red[3 * N + key]));
            m = key < g.rows ? fmaxf(old, m) : 1e30f;        // unused columns: weight 0, never in the way
            s_m[key] = m;
            s_nm[key] = -m;
            s_corr[key] = ex2(old - m);
          }
          named_barrier_sync(barrier, kSoftmax);
          if (i > 0) {
            ok = mbar_wait(pv_done, (tile - 1) & 1u, timeout);
            tc_fence_after_sync();
#pragma unroll 1
            for (int c0 = 0; c0 < 2 * N; c0 += 16) {
              float o[16];
              tmem_ld_32x32b_x16(o_at + c0, o);
              tmem_ld_wait16(o);
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                const float4 f = *reinterpret_cast<const float4*>(s_corr + c0 % N + c);
                tmem_st_32x32b_x4(o_at + c0 + c, o[c] * f.x, o[c + 1] * f.y, o[c + 2] * f.z, o[c + 3] * f.w);
              }
            }
            tmem_st_wait();
#pragma unroll
            for (int c = 0; c < N; ++c) l[c] *= s_corr[c];
          }
          settle = false;
        }
        if (stop) break;
        if (i > 0) ok = mbar_wait(pv_done, (tile - 1) & 1u, timeout);   // the buffers of P and V are free

        // ---- weights
        const float fv = seen ? ue8m0_to_float(data.y >> 16) * (1.f / kUp) : 0.f;
        const uint64_t fv2 = f2_pack(fv, fv);
#pragma unroll
        for (int c0 = 0; c0 < N; c0 += 8) {
          uint32_t w[4], w_lo[4];
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            const uint64_t e = f2_pack(ex2(d[c0 + c]), ex2(d[c0 + c + 1])), ev = f2_mul(e, fv2);
            float* lc = l + c0 + c;
            f2_unpack(f2_add(e, f2_pack(lc[0], lc[1])), lc[0], lc[1]);
            float x0, x1;
            f2_unpack(ev, x0, x1);
            w[c / 2] = cvt_bf16x2(x0, x1);
            f2_unpack(f2_sub(ev, f2_pack(__uint_as_float(w[c / 2] << 16), __uint_as_float(w[c / 2] & 0xFFFF0000u))), x0, x1);
            w_lo[c / 2] = cvt_bf16x2(x0, x1);
          }
          // [8 columns][key][8]
          uint8_t* to = s_p + c0 * (kTile * 2) + key * 16;
          *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(to + L::kPBytes) = make_uint4(w_lo[0], w_lo[1], w_lo[2], w_lo[3]);
        }
        // ---- values: 16 codes per step, 16 dimensions of one key, into the
        // 128-byte swizzled rows of 64 BF16 values.  Eight lanes have four pieces of
        // row r and the same four of row r ^ 5: what they load (under the TMA
        // swizzle, which exchanges 16-byte pieces by the row, or with 64-byte
        // rows by pairs of rows) and both halves of what they store touch every
        // bank once.  A thread's rows all have the same r mod 8, so its
        // addresses differ by constants.  Slots behind the sequence's end may
        // hold any bytes, NaN among them, and 0 * NaN is NaN: they become zeros
        // (pages without any key, and unselected keys, arrive as zeros).
        {
          const uint32_t slot = tile % L::kSlotsV;
          if constexpr (kSelected) {
            cp_async_wait<0>();
          } else {
            ok = ok && mbar_wait(&v_full[slot], tile / L::kSlotsV & 1u, timeout);
          }
          const uint8_t* codes = smem + L::kOffCodesV + slot * L::kSlotBytes + v_from;
          uint4 x[kSteps];
#pragma unroll
          for (int j = 0; j < kSteps; ++j) x[j] = *reinterpret_cast<const uint4*>(codes + j * kFromStep);
          if constexpr (kSelected) {
            if (i + 1 < g.n) copy_v(tile + 1);               // its place: with one slot, the one just read
          } else {
            mbar_arrive(&v_empty[slot]);
          }
          if (!kSelected && pos0 + kTile > g.keys) {
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              if (pos0 + v_row + j * kRowStep >= g.keys) x[j] = make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const uint2 h0 = cvt_bf16x4_e4m3(x[j].x), h1 = cvt_bf16x4_e4m3(x[j].y);
            const uint2 h2 = cvt_bf16x4_e4m3(x[j].z), h3 = cvt_bf16x4_e4m3(x[j].w);
            *reinterpret_cast<uint4*>(smem + v_to + j * (kRowStep * 128)) = make_uint4(h0.x, h0.y, h1.x, h1.y);
            *reinterpret_cast<uint4*>(smem + (v_to ^ 16u) + j * (kRowStep * 128)) = make_uint4(h2.x, h2.y, h3.x, h3.y);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        mbar_arrive(p_full);
      }
      if (stop) break;

      // ---- the rows' sums over all keys, and the output
      // Transposing reduction: lane c ends up with column c's sum over the warp.
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) {
#pragma unroll
        for (int c = 0; c < (N == 32 || w < 16 ? w : 16); ++c) {
          if (N == 16 && w == 16) {
            l[c] += __shfl_xor_sync(0xFFFFFFFFu, l[c], 16);
          } else {
            const bool up = (lane & w) != 0;
            const float send = up ? l[c] : l[c + w], keep = up ? l[c + w] : l[c];
            l[c] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, w);
          }
        }
      }
      if (lane < N) s_red[warp * N + lane] = l[0];
      ok = ok && mbar_wait(pv_done, (tile - 1) & 1u, timeout);
      tc_fence_after_sync();
      stop = !named_barrier_and(barrier, kSoftmax, ok);
      if (stop) break;
      const bool whole = g.n == g.kt_total;
      const int part = 2 * blockIdx.x + (first ? 0 : 1);   // an item that goes on from the CTA before comes first
      first = false;
      if (key < N) {
        const float sum = s_red[key] + s_red[N + key] + s_red[2 * N + key] + s_red[3 * N + key];
        s_corr[key] = sum > 0.f ? kUp / sum : 0.f;
        if (!whole && key < g.rows) {
          p.part_ml[static_cast<long long>(part) * N + key] = make_float2(s_m[key], sum);
        }
      }
      named_barrier_sync(barrier, kSoftmax);
#pragma unroll 1
      for (int c0 = 0; c0 < g.rows; c0 += 16) {
        float o[16], o_lo[16];
        tmem_ld_32x32b_x16(o_at + c0, o);
        tmem_ld_32x32b_x16(o_at + N + c0, o_lo);
        tmem_ld_wait16(o);
        tmem_ld_wait16(o_lo);
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] += o_lo[c];
        if (key < D) {
          float* dst = p.part_o + (static_cast<long long>(part) * N + c0) * D + key;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (c0 + c < g.rows) {
              if (whole) {
                a.out[s_out[c0 + c] + key] = __bfloat16_as_ushort(__float2bfloat16_rn(o[c] * s_corr[c0 + c]));
              } else {
                dst[c * D] = o[c];
              }
            }
          }
        }
      }
      // Header of an item that begins here and goes on in the next CTA.
      open = !whole && g.kt0 == 0;
      if (threadIdx.x == 0 && open) {
        p.heads[2 * blockIdx.x] = make_int4(1, static_cast<int>(quotient(g.first + g.kt_total - 1, run)), part, g.rows);
        p.heads[2 * blockIdx.x + 1] = make_int4(g.row0, g.r0, g.h, 0);
      }
      tc_fence_before_sync();
      named_barrier_sync(barrier, kSoftmax);         // the arrays are free again
    }
    if constexpr (kSelected) cp_async_wait<0>();          // also when a wait gave up
    if (stop || !ok) fail(&g_iq_status_kv, abort_flag, kStatusEpilogueWait);
    if (threadIdx.x == 0 && (stop || !open)) p.heads[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    if (!mbar_wait(drained, 0, 2 * timeout)) fail(&g_iq_status_kv, abort_flag, kStatusTeardownWait);
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// K10: joins the partial sums of the items cut between CTAs.  CTA c of K9 or
// K11 left a header if an item begins in its run and ends in that of CTA c1.
// With few rows several warps share one, each adding every kShare-th part with
// four parts in flight; their sums meet in shared memory in a fixed order.  One
// row over 4632 keys, both kernels: four warps per row 13.1 us, two 13.9, eight
// 15.1 (most blocks find no header).  Three parts in flight instead of four cost
// 0.2 us, eight 0.8.
template <int N>
struct JoinLayout {
  static constexpr int kShare = N == 16 ? 4 : (N == 32 ? 2 : 1);   // warps per row
  static constexpr int kWarps = 8;
  static constexpr int kRows = N == 128 ? 16 : kWarps / kShare;    // rows of a block
};

template <int N, int D>
__global__ void __launch_bounds__(JoinLayout<N>::kWarps * 32) kv_attention_join_kernel(const AttnParams p) {
  using J = JoinLayout<N>;
  constexpr int kPer = D / 32;
  __shared__ float s_o[J::kWarps][D];
  __shared__ float2 s_ml[J::kWarps];
  grid_launch_dependents();
  grid_dependency_wait();
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 head = p.heads[2 * c];
  if (head.x == 0 || static_cast<int>(blockIdx.y) * J::kRows >= head.w) return;
  const int4 where = p.heads[2 * c + 1];
  const int parts = head.y - c + 1;
  for (int r0 = 0; r0 < J::kRows; r0 += J::kWarps / J::kShare) {
    const int row = blockIdx.y * J::kRows + r0 + warp / J::kShare, share = warp % J::kShare;
    const bool there = row < head.w;
    // Every part is read once, with the running maximum of a softmax.
    float m = kNoMax, sum = 0.f, o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = 0.f;
    auto add = [&](float part_m, float part_l, const float* part_o) {
      const float top = fmaxf(m, part_m), down = ex2(m - top), w = ex2(part_m - top);
      m = top;
      sum = sum * down + part_l * w;
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[i] = o[i] * down + part_o[i] * w;
    };
    if (there) {
      for (int j0 = share; j0 < parts; j0 += 4 * J::kShare) {
        float2 ml[4];
        float x[4][kPer];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = j0 + u * J::kShare < parts ? j0 + u * J::kShare : j0;
          const long long at = static_cast<long long>(j == 0 ? head.z : 2 * (c + j)) * N + row;
          ml[u] = p.part_ml[at];
          const float* src = p.part_o + at * D + lane * kPer;
          if constexpr (kPer == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            x[u][0] = v.x, x[u][1] = v.y, x[u][2] = v.z, x[u][3] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            x[u][0] = v.x, x[u][1] = v.y;
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (j0 + u * J::kShare < parts) add(ml[u].x, ml[u].y, x[u]);
        }
      }
    }
    if constexpr (J::kShare > 1) {
      if (share > 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) s_o[warp][lane * kPer + i] = o[i];
        if (lane == 0) s_ml[warp] = make_float2(m, sum);
      }
      __syncthreads();
      if (share > 0) continue;                        // one round of rows
#pragma unroll
      for (int w = 1; w < J::kShare; ++w) add(s_ml[warp + w].x, s_ml[warp + w].y, &s_o[warp + w][lane * kPer]);
    }
    if (!there) continue;
    const int fr = where.y + row, tok = fr / p.a.group;
    const float inv = sum > 0.f ? kUp / sum : 0.f;
    uint16_t* dst = p.a.out + (where.x + tok) * p.a.ldo +
                    (where.z * p.a.group + fr - tok * p.a.group) * static_cast<long long>(D) + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      *reinterpret_cast<__nv_bfloat162*>(dst + i) = __floats2bfloat162_rn(o[i] * inv, o[i + 1] * inv);
    }
  }
}

constexpr int kMaxSms = 160;

// Rows per MMA: the smallest instance that holds the rows of one item.  Up to
// 32 rows the keys take the accumulator's lanes (this file); with more, the
// rows do (iq_kv_attention_rows.cu).  Decode over 64 ragged sequences, 8 KV
// heads: 16 rows per item 177 us with N = 16, 202 with 32; 32 rows 210 us with
// N = 32, 239 with 128.  2048 selected keys of 4632 tokens, 32 rows per item:
// 558 us with N = 32, 691 with 128.
int rows_per_mma(long long rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : kManyRows); }

int ctas_per_sm(int n) { return n == kManyRows ? 1 : 2; }

size_t part_bytes(int n, int dim) {
  return 2 * static_cast<size_t>(kMaxSms) * ctas_per_sm(n) *
         (static_cast<size_t>(n) * dim * sizeof(float) + n * sizeof(float2) + sizeof(int4));
}

template <int N, int D>
cudaError_t setup_instance() {
  const cudaError_t err = cudaFuncSetAttribute(kv_attention_kernel<N, D, false>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<N, D>::kSmemBytes);
  if (err != cudaSuccess) return err;
  return cudaFuncSetAttribute(kv_attention_kernel<N, D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Layout<N, D>::kSmemBytes);
}

template <int N, int D>
cudaError_t launch_instance(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnParams& p, int ctas,
                            cudaStream_t stream) {
  cudaError_t err;
  if constexpr (N == kManyRows) {
    err = launch_kv_attention_rows(tm_k, tm_v, p, ctas, stream);
  } else {
    err = launch_dependent(p.a.indices != nullptr ? kv_attention_kernel<N, D, true> : kv_attention_kernel<N, D, false>,
                           dim3(ctas, 1, 1), Layout<N, D>::kThreads, Layout<N, D>::kSmemBytes, stream, tm_k, tm_v, p);
  }
  if (err != cudaSuccess) return err;
  return launch_dependent(kv_attention_join_kernel<N, D>, dim3(ctas, N / JoinLayout<N>::kRows, 1),
                          JoinLayout<N>::kWarps * 32, 0, stream, p);
}

template <int D>
cudaError_t launch_dim(int n, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnParams& p, int ctas,
                       cudaStream_t stream) {
  switch (n) {
    case 16: return launch_instance<16, D>(tm_k, tm_v, p, ctas, stream);
    case 32: return launch_instance<32, D>(tm_k, tm_v, p, ctas, stream);
    default: return launch_instance<kManyRows, D>(tm_k, tm_v, p, ctas, stream);
  }
}

}  // namespace

cudaError_t kv_attention_setup_device() {
  cudaError_t err = setup_instance<16, 64>();
  if (err == cudaSuccess) err = setup_instance<32, 64>();
  if (err == cudaSuccess) err = setup_instance<16, 128>();
  if (err == cudaSuccess) err = setup_instance<32, 128>();
  if (err == cudaSuccess) err = kv_attention_rows_setup_device();
  return err;
}

size_t kv_attention_workspace(int num_rows, int q_heads, int kv_heads, int dim) {
  return part_bytes(rows_per_mma(static_cast<long long>(num_rows) * (q_heads / kv_heads)), dim);
}

cudaError_t launch_kv_attention(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a, void* ws,
                                int sm_count, unsigned long long timeout_ns, cudaStream_t stream) {
  // Rows of one item: a token's heads with selected keys, else the heads of
  // the mean number of tokens per sequence.
  const long long tokens = a.indices != nullptr ? 1 : (a.kv.num_rows + a.kv.num_seqs - 1) / a.kv.num_seqs;
  const int n = rows_per_mma(tokens * a.group);
  const int ctas = ctas_per_sm(n) * (sm_count < kMaxSms ? sm_count : kMaxSms);
  AttnParams p;
  p.a = a;
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2 * static_cast<size_t>(ctas) * n * a.kv.dim);
  p.heads = reinterpret_cast<int4*>(p.part_ml + 2 * static_cast<size_t>(ctas) * n);
  p.timeout_ns = timeout_ns;
  return a.kv.dim == 64 ? launch_dim<64>(n, tm_k, tm_v, p, ctas, stream)
                        : launch_dim<128>(n, tm_k, tm_v, p, ctas, stream);
}

cudaError_t read_kv_status(uint32_t* flags, bool reset) {
  uint32_t v = 0, w = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_iq_status_kv, sizeof(v));
  if (err == cudaSuccess) err = read_kv_rows_status(&w, reset);
  if (err != cudaSuccess) return err;
  if (flags) *flags = v | w;
  if (reset) {
    const uint32_t zero = 0;
    err = cudaMemcpyToSymbol(g_iq_status_kv, &zero, sizeof(zero));
  }
  return err;
}

}  // namespace iq
