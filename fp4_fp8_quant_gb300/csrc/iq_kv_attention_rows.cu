// Attention over the paged 8-bit KV cache with many rows per item: prompts,
// chunks of them, and selected keys under many query heads (include/iq.h,
// section 4; the mathematics of the scales and of the split operands is in
// iq_kv_attention.cu).
//
// K11 kv_attention_rows_kernel.  128 rows of one KV head per item,
//   S [128 rows, 128 keys] = Q x K^T,   O [128 rows, D] += P x V.
// Per tile the tensor cores need 512 cycles for S (two E4M3 terms of Q) and
// 512 for O (BF16); everything else is arranged so that they wait
// for nothing but each other:
//   - one CTA per SM has all of tensor memory: O and three score buffers, whose
//     columns the weights take over.  The scores run up to two tiles ahead of
//     the products, across the items' ends, and no issuer waits for an MMA to
//     complete.  Scores and products have an issuing warp each: what a warp does
//     between two tiles (waits, commits, some hundred instructions) costs as long
//     as a product, and the other warp's MMAs run meanwhile.
//   - two softmax groups of eight warps take alternate tiles; in a group two
//     threads share a row, half of the keys each, and a row's maximum, sum and
//     scale are registers.
//   - the maximum is that of the segment's first tile, so the groups need
//     nothing of one another.  Weights and values are BF16, with the exponents
//     of float32: keys far below that maximum keep their eight significant bits
//     (in half precision those behind a dominant first key would be lost one bit
//     per octave below 2^-8 of it), and the row's sum adds the rounded weights,
//     so that what a weight loses it loses above and below the fraction.  (A
//     second term of the weights, as in iq_kv_attention.cu, takes the prompt below
//     from 360 to 424 us.)  Kept at its value's scale times 2^-40, a weight may
//     grow to 2^40 times the first tile's largest; a segment in which a thread's
//     weights of one tile add up to more is noted and done again at the end of the
//     CTA's run, with the maximum moved and O scaled at every tile.
//   - the values are converted to BF16 by warps of their own, from codes that
//     TMA has staged, without their scales: a multiplication there costs 26 us of
//     a 4632-token prompt, in the weights 11.  Selected keys: the same warps copy
//     the codes of V and of three quarters of K by cp.async, a copy of 16 bytes per
//     lane costing them some 85 cycles; the rest of K the producers gather by TMA,
//     which takes 13 cycles per row (a quarter of K gathered: 709 us for 4632
//     tokens, half 718 us, all 754 us, none 726 us).
//   - four more warps split the next item's Q while the present item's keys
//     pass, and write the output while the next item's pass.
//   - the loops are kept rolled: seven warps with four roles share an SM
//     quarter's instruction cache, and a third of all stalls were for
//     instructions before (4632-token prompt 590 -> 407 us, selected keys 913
//     -> 716 us).
// Measured: a 4632-token prompt, 64 query and 8 KV heads, 360 us = 977 TFLOP/s,
// tensor pipe 46 % active, 0.71 instructions per scheduler and cycle.  A tile takes
// some 2100 cycles: three tiles per turn of the score buffers, and a turn is
// scores, softmax, product and the waits between them.  A prompt whose every
// segment is done again takes 990 us.  2048 selected keys of 4632 tokens, 64
// query heads on one KV head, 706 us, bound by bringing the rows.
//
// Warps: 0..15 softmax, 16..19 values, 20..23 Q and output, 24 and 25 producers
// (even and odd tiles), 26 issuer of the scores, 27 of the products.

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

__device__ uint32_t g_iq_status_kv_rows;

namespace {

constexpr int N = kManyRows;
constexpr int kHalf = kTile / 2;                 // keys of a softmax thread
constexpr int kGroup = 256;                      // threads of a softmax group
constexpr int kSoftmax = 2 * kGroup, kValue = 128, kQ = 128;
constexpr int kThreads = kSoftmax + kValue + kQ + 128;
constexpr int kValueWarp = kSoftmax / 32, kQWarp = kValueWarp + kValue / 32, kProducerWarp = kQWarp + kQ / 32,
              kScoreWarp = kProducerWarp + 2, kProductWarp = kScoreWarp + 1;
constexpr int kSlotsK = 3, kSlotsS = 3;
constexpr int kMetaTiles = 4;                    // tiles whose key data are held
constexpr float kMostSum = kUp;                  // most that a thread's weights of a tile may add up to
constexpr int kEntries = 12;                     // segments announced ahead
constexpr int kGathered = 32;                    // selected keys of a tile whose K is gathered by TMA
constexpr int kNoted = 1024;                     // places to note a segment; the last is also every later one's

// A segment as the producer announces it to the other roles; n = 0 ends a
// round.
struct Entry {
  Segment g;
  int ordinal;       // of the segment in the CTA's run
};
static_assert(sizeof(Entry) <= 80, "entry");

template <int D>
struct RowLayout {
  static constexpr int kSlotBytes = kTile * D;
  static constexpr int kQBytes = N * D;          // one term of Q
  static constexpr int kVBytes = kTile * D * 2;
  static constexpr int kOffCodesV = kSlotsK * kSlotBytes;            // two slots
  static constexpr int kOffV = kOffCodesV + 2 * kSlotBytes;          // two buffers
  static constexpr int kOffQ = kOffV + 2 * kVBytes;                  // two buffers of two terms
  static constexpr int kOffMeta = kOffQ + 4 * kQBytes;               // float kf, hide [kTile], bf16 fv [kTile], int row [kTile] per tile
  static constexpr int kOffBq = kOffMeta + kMetaTiles * kTile * 16;  // float [4][N]: scale of the query row
  static constexpr int kOffM = kOffBq + 4 * N * 4;                   // float [2][N]: maximum
  static constexpr int kOffTop = kOffM + 2 * N * 4;                  // float [2 groups][2 halves][N]
  static constexpr int kOffSum = kOffTop + 4 * N * 4;                // float [2][2 groups][2 halves][N]
  static constexpr int kOffNoted = kOffSum + 8 * N * 4;
  static constexpr int kOffEntry = kOffNoted + kNoted / 8;           // Entry [kEntries]
  static constexpr int kOffBar = kOffEntry + kEntries * 80;
  static constexpr int kNumBars = 2 * kSlotsK + 2 * kMetaTiles + 2 * 6 + 3 * kSlotsS + 14 + kEntries;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffHoles = kOffMisc + 96;                    // int [kMetaTiles]: rows are missing
  static constexpr int kSmemBytes = kOffHoles + kMetaTiles * 4;
  static_assert(kOffV % 1024 == 0 && kOffQ % 1024 == 0, "alignment");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// Tensor memory: output, and three buffers of scores, whose columns the
// weights take over (half h of the keys: columns 64 h to 64 h + 31).
constexpr uint32_t kColO = 0, kColS = 128, kTmemCols = 512;

__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Pairs of halves to E4M3 codes (16 bits), and back.
__device__ __forceinline__ uint32_t cvt_e4m3x2_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}

__device__ __forceinline__ uint32_t cvt_f16x2_e4m3x2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(c)));
  return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Arrives on the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int D, bool kSelected>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                             const __grid_constant__ AttnParams p) {
  using L = RowLayout<D>;
  // All of the shared memory there is: no room for moving to a boundary.
  extern __shared__ __align__(1024) uint8_t smem[];
  float* s_meta = reinterpret_cast<float*>(smem + L::kOffMeta);   // [kMetaTiles][4][kTile]
  float* s_bq = reinterpret_cast<float*>(smem + L::kOffBq);
  float* s_m = reinterpret_cast<float*>(smem + L::kOffM);
  float* s_top = reinterpret_cast<float*>(smem + L::kOffTop);
  float* s_sum = reinterpret_cast<float*>(smem + L::kOffSum);
  int* s_holes = reinterpret_cast<int*>(smem + L::kOffHoles);
  uint32_t* s_noted = reinterpret_cast<uint32_t*>(smem + L::kOffNoted);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* k_empty = k_full + kSlotsK;
  uint64_t* meta_full = k_empty + kSlotsK;
  uint64_t* meta_empty = meta_full + kMetaTiles;
  uint64_t* codes_full = meta_empty + kMetaTiles;   // [2] codes of V (whole pages)
  uint64_t* codes_empty = codes_full + 2;           // [2]
  uint64_t* v_full = codes_full + 4;                // [2] values in BF16
  uint64_t* q_full = codes_full + 6;                // [2]
  uint64_t* q_empty = codes_full + 8;               // [2] the scores of a segment are done
  uint64_t* pv_done = codes_full + 10;              // [2] second product of a tile
  uint64_t* s_full = codes_full + 12;               // [kSlotsS] scores
  uint64_t* s_empty = s_full + kSlotsS;             // [kSlotsS] weights are used
  uint64_t* p_full = s_empty + kSlotsS;             // [kSlotsS] weights are stored
  uint64_t* o_full = p_full + kSlotsS;              // output of a segment
  uint64_t* o_empty = o_full + 1;                   // and read
  uint64_t* m_full = o_full + 2;                    // [2] maximum of a segment
  uint64_t* drained = o_full + 4;
  uint64_t* sum_full = o_full + 5;                  // [2] the rows' sums of a segment
  uint64_t* sum_empty = o_full + 7;                 // [2] and read
  uint64_t* group_done = o_full + 9;                // [2] all threads of a softmax group are here
  uint64_t* drained_s = o_full + 11;
  uint64_t* top_read = o_full + 12;                 // [2] s_top of a softmax group is read
  uint64_t* entry_full = o_full + 14;               // [kEntries]
  auto entry_at = [&](uint32_t i) { return reinterpret_cast<Entry*>(smem + L::kOffEntry + i % kEntries * 80); };
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + 4);
  uint32_t* s_again = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + 8);          // some segment is noted
  volatile uint32_t* s_total = reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc + 12);   // tiles, once known
  Start* s_start = reinterpret_cast<Start*>(smem + L::kOffMisc + 16);
  static_assert(sizeof(Start) <= 80, "start");

  const AttnArgs& a = p.a;
  const uint64_t timeout = p.timeout_ns;
  if ((smem_u32(smem) & 1023u) != 0) {                  // the swizzles would not match; never seen
    if (threadIdx.x == 0) {
      atomicOr(&g_iq_status_kv_rows, kStatusProducerWait);
      p.heads[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  grid_launch_dependents();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int i = 0; i < kSlotsK; ++i) {
      mbar_init(&k_full[i], kSelected ? 1 + kValue : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < kMetaTiles; ++i) {
      mbar_init(&meta_full[i], 1);
      mbar_init(&meta_empty[i], kSelected ? kGroup + kValue : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&codes_full[i], 1);
      mbar_init(&codes_empty[i], kValue);
      mbar_init(&v_full[i], kValue);
      mbar_init(&q_full[i], kQ);
      mbar_init(&q_empty[i], 1);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < kSlotsS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 1);
      mbar_init(&p_full[i], kGroup);
    }
    mbar_init(o_full, 1);
    mbar_init(o_empty, kQ);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sum_full[i], kSoftmax);
      mbar_init(&sum_empty[i], kQ);
      mbar_init(&group_done[i], kGroup);
      mbar_init(&m_full[i], kGroup);
      mbar_init(&top_read[i], kGroup);
    }
    mbar_init(drained, 1);
    mbar_init(drained_s, 1);
    for (int i = 0; i < kEntries; ++i) mbar_init(&entry_full[i], 1);
    *abort_flag = 0u;
    *s_again = 0u;
    *s_total = ~0u;
    for (int i = 0; i < kNoted / 32; ++i) s_noted[i] = 0u;
    fence_mbar_init();
  }
  if (warp == kProductWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
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
  const int none = a.kv.num_pages * a.kv.heads * a.kv.page;   // a row past the end: zeros

  // Every role takes the segments in order as the producer announces them; in
  // a second round the noted ones.  (An entry's place is taken again twelve
  // entries on, one segment ahead of the tiles.  Key data are held for four
  // tiles, so the softmax is by then past tile t + 5 of the entry's first tile
  // t, the products, which give back the score buffers, past t + 2: all roles
  // have read the entry.)
  Segment g = {};
  int ordinal = -1;
  bool again = false;
  uint32_t entry = 0;
  // What a role carries from tile to tile, over both rounds.  Buffers that
  // come in pairs belong to the even and the odd tiles (or segments).
  uint32_t tile = 0, seg = 0, meets = 0, tops = 0;
  // its waits; the same in all lanes of a warp, but for the value warps (all
  // waits are bounded, and no role waits at a CTA barrier inside a round)
  bool ok = true;
  bool open = false;                                    // output: the last item goes on in the next CTA
  auto all = [&](bool yes) { return __all_sync(0xFFFFFFFFu, yes) != 0; };
  auto next_segment = [&] {
    const uint32_t e = entry++;
    ok = ok && mbar_wait(&entry_full[e % kEntries], e / kEntries & 1u, timeout) && *abort_flag == 0u;
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok) return false;
    const Entry* at = entry_at(e);
    g = at->g;
    ordinal = at->ordinal;
    return g.n > 0;
  };

  while (true) {
    if (warp == kProducerWarp || warp == kProducerWarp + 1) {
      // ------------------------------------------------------------ producer
      // Publish the tiles' key data and load their codes, whole pages at once or
      // kGathered selected rows of K.  One warp has the even tiles and one the
      // odd, and the first also finds the segments.  ok is the same in every
      // lane.
      const uint32_t odd = warp - kProducerWarp;
      int last_k = -1, last_v = -1;                          // this warp's last tiles on their way
      auto push = [&](uint32_t t, const int* rows, const uint32_t* sf) {
        const uint32_t mslot = t % kMetaTiles, slot = t % kSlotsK;
        [[maybe_unused]] const bool leader = ((4 * lane) & (a.kv.page - 1)) == 0;
        const bool k_free = mbar_wait(&k_empty[slot], (t / kSlotsK & 1u) ^ 1u, timeout) && *abort_flag == 0u;
        if (!all(k_free)) return false;
        if (lane == 0) mbar_arrive_expect_tx(&k_full[slot], kSelected ? kGathered * D : L::kSlotBytes);
        __syncwarp();
        uint8_t* k_to = smem + slot * L::kSlotBytes + 4 * lane * D;
        if constexpr (kSelected) {
          if (4 * lane < kGathered) tma_gather4(k_to, &tm_k, &k_full[slot], make_int4(rows[0], rows[1], rows[2], rows[3]));
        } else {
          if (leader) tma_load_2d(k_to, &tm_k, &k_full[slot], 0, rows[0]);
        }
        last_k = static_cast<int>(t);
        const bool free = mbar_wait(&meta_empty[mslot], (t / kMetaTiles & 1u) ^ 1u, timeout) && *abort_flag == 0u;
        if (!all(free)) return false;
        float* meta = s_meta + mslot * 4 * kTile + 4 * lane;
        float kf[4], hide[4], fv[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool there = rows[c] != none;
          kf[c] = there ? fabsf(a.scale_log2) * ue8m0_to_float(sf[c] & 0xFFu) : 0.f;
          hide[c] = there ? 0.f : -INFINITY;
          fv[c] = there ? ue8m0_to_float(sf[c] >> 16) * (1.f / kUp) : 0.f;
        }
        *reinterpret_cast<float4*>(meta) = make_float4(kf[0], kf[1], kf[2], kf[3]);
        *reinterpret_cast<float4*>(meta + kTile) = make_float4(hide[0], hide[1], hide[2], hide[3]);
        reinterpret_cast<uint2*>(s_meta + (mslot * 4 + 2) * kTile)[lane] =
            make_uint2(cvt_bf16x2(fv[0], fv[1]), cvt_bf16x2(fv[2], fv[3]));
        *reinterpret_cast<int4*>(meta + 3 * kTile) = make_int4(rows[0], rows[1], rows[2], rows[3]);
        const bool holes = __any_sync(0xFFFFFFFFu, rows[0] == none || rows[1] == none || rows[2] == none || rows[3] == none);
        __syncwarp();
        if (lane == 0) {
          s_holes[mslot] = holes;
          mbar_arrive(&meta_full[mslot]);
        }
        if constexpr (!kSelected) {
          const uint32_t b = t & 1u;
          const bool v_free = mbar_wait(&codes_empty[b], (t >> 1 & 1u) ^ 1u, timeout);
          if (!__all_sync(0xFFFFFFFFu, v_free)) return false;
          if (lane == 0) mbar_arrive_expect_tx(&codes_full[b], L::kSlotBytes);
          __syncwarp();
          if (leader) tma_load_2d(smem + L::kOffCodesV + b * L::kSlotBytes + 4 * lane * D, &tm_v, &codes_full[b], 0, rows[0]);
          last_v = static_cast<int>(t);
        }
        return true;
      };
      const int first_tile = static_cast<int>(tile);
      Walker<N> walk(start);
      ordinal = -1;
      // The segment to come is found and announced before the present one's
      // tiles are published, so that its Q is there in time.
      auto announce = [&] {
        Segment found = {};
        bool more = false;
        while (!more && walk.next(a, found)) {
          ++ordinal;
          const int place = min(ordinal, kNoted - 1);
          more = !again || (s_noted[place >> 5] >> (place & 31) & 1u) != 0u;
        }
        if (!more) found.n = 0;                              // the round's end
        __syncwarp();
        if (lane == 0) {
          Entry* at = entry_at(entry);
          at->g = found;
          at->ordinal = ordinal;
          mbar_arrive(&entry_full[entry % kEntries]);
        }
        ++entry;
        __syncwarp();
      };
      if (odd == 0) announce();
      auto walk_on = [&] {
        if (odd != 0) return next_segment();
        g = entry_at(entry - 1)->g;
        if (g.n == 0) return false;
        announce();
        return true;
      };
      if constexpr (!kSelected) {
        // Pages in order, each lane the page of its own four keys: pages are
        // looked up four tiles ahead, their scales two.
        while (ok && walk_on()) {
          auto find_page = [&](int i) {
            const int pos = (g.kt0 + i) * kTile + 4 * lane;
            return i < g.n && pos < g.keys ? kv_page_of(a.kv, g.b, pos) : -1;
          };
          auto find_scales = [&](int id) {
            const long long at = static_cast<long long>(max(id, 0)) * a.kv.heads + g.h;
            return a.kv.sf[0][at] | static_cast<uint32_t>(a.kv.sf[1][at]) << 16;
          };
          int i = (tile ^ odd) & 1u;
          int pid = find_page(i), pid1 = find_page(i + 2);
          uint32_t sf = find_scales(pid);
          for (; ok && i < g.n; i += 2) {
            const uint32_t sf1 = find_scales(pid1);
            const int pid2 = find_page(i + 4);
            const int pos = (g.kt0 + i) * kTile + 4 * lane;
            const int row0 = static_cast<int>((static_cast<long long>(pid) * a.kv.heads + g.h) * a.kv.page);
            int rows[4];
            const uint32_t sf4[4] = {sf, sf, sf, sf};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              rows[c] = pid >= 0 && pos + c < g.keys ? row0 + ((pos + c) & (a.kv.page - 1)) : none;
            }
            ok = push(tile + i, rows, sf4);
            pid = pid1;
            pid1 = pid2;
            sf = sf1;
          }
          tile += g.n;
        }
      } else {
        // Single rows, four keys per lane.  The three dependent loads
        // (position, page, scales) of a tile are issued four, two and two tiles
        // ahead, the scales when the tile before is published.
        while (ok && walk_on()) {
          int pos[4], pos1[4], pid[4], row[4];
          uint32_t sf[4];                                  // scale bytes of key and value
          const int32_t* list = a.indices + static_cast<long long>(g.list) * a.ld_idx;
          const int32_t* table = a.kv.table + static_cast<long long>(g.b) * a.kv.table_ld;
          const int left = min(a.topk, (g.kt0 + g.n) * kTile);        // this segment's part of the list ends here
          auto find_pos = [&](int i, int* pos) {
            const int j = (g.kt0 + i) * kTile + 4 * lane;
#pragma unroll
            for (int k = 0; k < 4; ++k) pos[k] = j + k < left ? list[j + k] : -1;
          };
          auto find_pid = [&](const int* pos, int* pid) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              pid[k] = static_cast<unsigned>(pos[k]) < static_cast<unsigned>(g.keys) ? table[pos[k] >> a.kv.page_log2] : -1;
            }
          };
          auto find_row = [&](const int* pos, const int* pid, int* row) {     // (rows fit 31 bits)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              row[k] = static_cast<unsigned>(pid[k]) < static_cast<unsigned>(a.kv.num_pages)
                           ? ((pid[k] * a.kv.heads + g.h) << a.kv.page_log2) + (pos[k] & (a.kv.page - 1))
                           : none;
            }
          };
          auto find_scales = [&](const int* row, uint32_t* sf) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int at = row[k] != none ? row[k] >> a.kv.page_log2 : 0;
              sf[k] = a.kv.sf[0][at] | static_cast<uint32_t>(a.kv.sf[1][at]) << 16;
            }
          };
          int i = (tile ^ odd) & 1u;
          find_pos(i, pos);
          find_pos(i + 2, pos1);
          find_pid(pos, pid);
          find_row(pos, pid, row);
          find_scales(row, sf);
          for (; ok && i < g.n; i += 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) pos[k] = pos1[k];
            find_pid(pos, pid);
            find_pos(i + 4, pos1);
            ok = push(tile + i, row, sf);
            find_row(pos, pid, row);
            find_scales(row, sf);
          }
          tile += g.n;
        }
      }
      if (!ok) fail(&g_iq_status_kv_rows, abort_flag, kStatusProducerWait);
      __syncwarp();
      if (lane == 0 && odd == 0) *s_total = tile;            // the value warps stop here
      // Every copy begun here has landed before the CTA ends, also when a
      // wait gave up.  (A slot that a later tile took was waited for there.)
      auto landed = [&](uint64_t* bar, uint32_t phase) {
        if (!mbar_wait(bar, phase & 1u, timeout)) fail(&g_iq_status_kv_rows, abort_flag, kStatusTeardownWait);
      };
      if (last_v >= 0) landed(&codes_full[last_v & 1], last_v >> 1);
      if (last_k >= 0) landed(&k_full[last_k % kSlotsK], last_k / kSlotsK);
      if (last_k - 2 >= first_tile && last_k + 1 >= static_cast<int>(tile)) {
        landed(&k_full[(last_k - 2) % kSlotsK], (last_k - 2) / kSlotsK);
      }
    } else if (warp == kScoreWarp) {
      // ------------------------------------------------------ scores' issuer
      constexpr uint32_t kSwizzle = D == 128 ? 2u : 4u;
      constexpr uint32_t idesc = idesc_f32(128, kTile, 0, 0);
      const uint32_t base = uniform(smem_u32(smem)), acc = uniform(tmem);
      const Desc k_desc = smem_desc(base, 16, 8 * D, kSwizzle), q_desc = smem_desc(base + L::kOffQ, 16 * N, 128, 0);
      while (ok && next_segment()) {
        const uint32_t sb = uniform(seg & 1u);
        ok = all(mbar_wait(&q_full[sb], seg >> 1 & 1u, timeout));
        const Desc q_tile = q_desc.at(sb * 2 * L::kQBytes);
        for (int i = 0; ok && i < g.n; ++i, ++tile) {
          const uint32_t b = uniform(tile % kSlotsS), slot = uniform(tile % kSlotsK);
          ok = mbar_wait(&s_empty[b], (tile / kSlotsS & 1u) ^ 1u, timeout);
          ok = all(ok && mbar_wait(&k_full[slot], tile / kSlotsK & 1u, timeout) && *abort_flag == 0u);
          if (!ok) break;
          if constexpr (kSelected) fence_proxy_async_smem();               // the value warps' copies
          tc_fence_after_sync();
          const Desc k_tile = k_desc.at(slot * L::kSlotBytes);
          const uint32_t d = acc + kColS + b * kTile;
#pragma unroll
          for (int term = 0; term < 2; ++term) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              tc_mma_f8(d, q_tile.at(term * L::kQBytes + 2 * k * (16 * N)), k_tile.at(32 * k), idesc, (term | k) != 0);
            }
          }
          tc_commit_elected(&s_full[b]);
          tc_commit_elected(&k_empty[slot]);
        }
        tc_commit_elected(&q_empty[sb]);
        ++seg;
      }
      if (!ok) fail(&g_iq_status_kv_rows, abort_flag, kStatusMmaWait);
    } else if (warp == kProductWarp) {
      // ---------------------------------------------------- products' issuer
      constexpr uint32_t idesc = idesc_f32(128, D, 0, 1) | kBf16Operands;
      const uint32_t base = uniform(smem_u32(smem)), acc = uniform(tmem);
      const Desc v_desc = smem_desc(base + L::kOffV, D == 128 ? kTile * 128 : 0, 1024, 2);
      while (ok && next_segment()) {
        for (int i = 0; i < g.n; ++i, ++tile) {
          const uint32_t b = uniform(tile & 1u), parity = tile >> 1 & 1u;
          const uint32_t sb = uniform(tile % kSlotsS);
          ok = mbar_wait(&v_full[b], parity, timeout) && mbar_wait(&p_full[sb], tile / kSlotsS & 1u, timeout);
          // The segment before has been read out of O.
          if (i == 0 && seg > 0) ok = ok && mbar_wait(o_empty, (seg - 1) & 1u, timeout);
          ok = all(ok && *abort_flag == 0u);
          if (!ok) break;
          tc_fence_after_sync();
          const Desc v_tile = v_desc.at(b * L::kVBytes);
          const uint32_t w = acc + kColS + sb * kTile, more = uniform(i != 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k) {
            tc_mma_f16_ta(acc + kColO, w + 8 * k + (k >= kHalf / 16 ? kHalf / 2 : 0), v_tile.at(2048 * k), idesc, k != 0 ? 1u : more);
          }
          tc_commit_elected(&pv_done[b]);
          tc_commit_elected(&s_empty[sb]);
          if constexpr (!kSelected) tc_commit_elected(&meta_empty[uniform(tile % kMetaTiles)]);
        }
        tc_commit_elected(o_full);
        ++seg;
      }
      if (!ok) fail(&g_iq_status_kv_rows, abort_flag, kStatusMmaWait);
    } else if (warp >= kQWarp) {
      // ------------------------------------------------------- Q and output
      // Rows scaled by a power of two and split into two E4M3 terms, a
      // segment ahead, a row per thread.  A buffer is free when the scores of
      // the segment before the last are done; the softmax may not yet have
      // read the scales of that one and of the next, so these have four
      // buffers.
      const int tid = threadIdx.x - kQWarp * 32;
      const uint32_t flip = a.scale_log2 < 0.f ? 0x80808080u : 0u;
      auto load_q = [&](const Segment& sg, uint32_t q_seg) {
        const uint32_t b = q_seg & 1u;
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(&q_empty[b], (q_seg >> 1 & 1u) ^ 1u, timeout));
        if (!ok) return;
        // Eight values of BF16 take the place that 16 codes of a term will
        // have: a thread converts in place.
        uint8_t* to = smem + L::kOffQ + b * 2 * L::kQBytes + tid * 16;   // K-major without swizzle: [16 dims][row][16]
        {
          const int fr = sg.r0 + min(tid, sg.rows - 1), tok = fr / a.group;   // rows past the item's repeat its last one
          const int head = sg.h * a.group + fr - tok * a.group;
          const uint16_t* src = a.q + (sg.row0 + tok) * a.ldq + head * static_cast<long long>(D);
#pragma unroll 4
          for (int i = 0; i < D / 16; ++i) {
            cp_async_16(to + i * (16 * N), src + 16 * i, 16);
            cp_async_16(to + i * (16 * N) + L::kQBytes, src + 16 * i + 8, 16);
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
        uint32_t m2 = 0;
#pragma unroll 4
        for (int i = 0; i < D / 16; ++i) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 x = *reinterpret_cast<const uint4*>(to + i * (16 * N) + half * L::kQBytes);
            m2 = __vmaxu2(__vmaxu2(m2, x.x & 0x7FFF7FFFu), x.y & 0x7FFF7FFFu);
            m2 = __vmaxu2(__vmaxu2(m2, x.z & 0x7FFF7FFFu), x.w & 0x7FFF7FFFu);
          }
        }
        // Smallest e with 448 * 2^e >= the largest value, at least -118.
        const uint32_t bits = max(m2 & 0xFFFFu, m2 >> 16) << 16;
        const int e = max(-118, static_cast<int>(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        s_bq[q_seg % 4 * N + tid] = query_scale(bits, e);
#pragma unroll 1
        for (int i = 0; i < D / 16; ++i) {
          uint4* at[2] = {reinterpret_cast<uint4*>(to + i * (16 * N)),
                          reinterpret_cast<uint4*>(to + i * (16 * N) + L::kQBytes)};
          const uint4 x[2] = {*at[0], *at[1]};
          uint32_t c1[8], c2[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4& y = x[j / 4];
            const uint32_t w = j % 4 == 0 ? y.x : (j % 4 == 1 ? y.y : (j % 4 == 2 ? y.z : y.w));
            // Scaled values are halves: eight significant bits from 448 down
            // to 2^-17, and 2^-24 is far below what the second term keeps.
            const uint32_t h = cvt_f16x2(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xFFFF0000u) * inv);
            c1[j] = cvt_e4m3x2_f16x2(h);
            c2[j] = cvt_e4m3x2_f16x2(sub_f16x2(h, cvt_f16x2_e4m3x2(c1[j])));
          }
          // A negative scale changes the sign of the codes, so that the
          // largest product is the largest score.
          *at[0] = make_uint4((c1[0] | c1[1] << 16) ^ flip, (c1[2] | c1[3] << 16) ^ flip, (c1[4] | c1[5] << 16) ^ flip,
                              (c1[6] | c1[7] << 16) ^ flip);
          *at[1] = make_uint4((c2[0] | c2[1] << 16) ^ flip, (c2[2] | c2[3] << 16) ^ flip, (c2[4] | c2[5] << 16) ^ flip,
                              (c2[6] | c2[7] << 16) ^ flip);
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_full[b]);
      };
      // The rows' sums and maxima, then a row's output per thread.
      const long long run = start.per;
      auto write_out = [&](const Segment& sg, int order) {
        const uint32_t sb = seg & 1u;
        ok = ok && mbar_wait(&sum_full[sb], seg >> 1 & 1u, timeout) && mbar_wait(o_full, seg & 1u, timeout);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return;
        tc_fence_after_sync();
        const int r = tid;
        const bool there = r < sg.rows;
        const float* sums = s_sum + sb * 4 * N + r;
        const float l = (sums[0] + sums[N]) + (sums[2 * N] + sums[3 * N]), m = s_m[sb * N + r];
        mbar_arrive(&sum_empty[sb]);
        const bool whole = sg.n == sg.kt_total;
        const int part = 2 * blockIdx.x + (order == 0 ? 0 : 1);   // an item that goes on from the CTA before comes first
        const float inv = l > 0.f ? kUp / l : 0.f;
        const int fr = sg.r0 + r, tok = fr / a.group, head = sg.h * a.group + fr - tok * a.group;
        uint16_t* out = a.out + (sg.row0 + tok) * a.ldo + head * static_cast<long long>(D);
        float* part_o = p.part_o + (static_cast<long long>(part) * N + r) * D;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + kColO;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          float o[16];
          tmem_ld_32x32b_x16(lanes + c0, o);
          tmem_ld_wait16(o);
          if (c0 + 16 == D) {                                // all of O is read
            tc_fence_before_sync();
            mbar_arrive(o_empty);
          }
          if (there && whole) {
#pragma unroll
            for (int c = 0; c < 16; c += 8) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[c + 2 * k] * inv, o[c + 2 * k + 1] * inv);
                w[k] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              *reinterpret_cast<uint4*>(out + c0 + c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (there) {
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
              *reinterpret_cast<float4*>(part_o + c0 + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
            }
          }
        }
        if (there && !whole) p.part_ml[static_cast<long long>(part) * N + r] = make_float2(m, l);
        if (!again) {
          // Header of an item that begins here and goes on in the next CTA.
          open = !whole && sg.kt0 == 0;
          if (tid == 0 && open) {
            p.heads[2 * blockIdx.x] = make_int4(1, static_cast<int>(quotient(sg.first + sg.kt_total - 1, run)), part, sg.rows);
            p.heads[2 * blockIdx.x + 1] = make_int4(sg.row0, sg.r0, sg.h, 0);
          }
        }
      };
      bool there = next_segment();
      if (there) load_q(g, seg);
      while (ok && there) {
        const Segment present = g;
        const int order = ordinal;
        there = next_segment();
        if (there) load_q(g, seg + 1);
        write_out(present, order);
        ++seg;
      }
      if (!ok) fail(&g_iq_status_kv_rows, abort_flag, kStatusEpilogueWait);
      if (tid == 0 && (!ok || !open)) p.heads[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    } else if (warp >= kValueWarp) {
      // -------------------------------------------------------------- values
      // 16 codes per step, 16 dimensions of one key, into 128-byte swizzled
      // rows of 64 BF16 values.  Eight lanes have four pieces of row r and the same
      // four of row r ^ 5: what they load and both halves of what they store
      // touch every bank once.  A thread's rows all have the same r mod 8, so
      // its addresses differ by constants.
      const int tid = threadIdx.x - kValueWarp * 32;
      constexpr int kChunks = D / 16, kSteps = kTile * kChunks / kValue, kRowStep = kValue / kChunks;
      const int c = tid % 4 + (D == 128 ? tid / 8 % 2 * 4 : 0), q = tid / (2 * kChunks);
      const int r_first = q / 4 * 8 + ((q % 4) ^ (tid / 4 % 2 * 5));
      const uint32_t codes_at =
          L::kOffCodesV + (kSelected ? tid * 16 : r_first * D + (D == 128 ? c ^ (r_first & 7) : c ^ (r_first >> 1 & 3)) * 16);
      const uint32_t v_at = L::kOffV + (c / 4) * (kTile * 128) + r_first * 128 + (((2 * (c % 4)) ^ (r_first & 7)) << 4);
      // Waits until a tile's rows are published; false after the last one.
      auto published = [&](uint32_t t) {
        uint64_t* bar = &meta_full[t % kMetaTiles];
        const uint32_t parity = t / kMetaTiles & 1u;
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        while (true) {
          if (mbar_try_wait(bar, parity)) return true;
          if (*s_total == t) return false;
          if (*abort_flag != 0u || globaltimer_ns() - t0 > timeout) {
            ok = false;
            return false;
          }
        }
      };
      auto rows_of = [&](uint32_t t) {
        return reinterpret_cast<const int*>(s_meta + (t % kMetaTiles * 4 + 3) * kTile) + r_first;
      };
      // Selected keys: the rest of K's codes into their slot, the pieces of a
      // row exchanged as the TMA swizzle would, and V's codes, for this thread
      // alone.  (K's place is free: the producer has waited for it.)
      auto copy = [&](uint32_t t) {
        const int* row_of = rows_of(t);
        uint8_t* to = smem + codes_at + (t & 1u) * L::kSlotBytes;
        int rows[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) rows[j] = row_of[j * kRowStep];
        uint8_t* k_to = smem + t % kSlotsK * L::kSlotBytes + r_first * D +
                        (D == 128 ? c ^ (r_first & 7) : c ^ (r_first >> 1 & 3)) * 16;
#pragma unroll
        for (int j = kGathered / kRowStep; j < kSteps; ++j) {
          const bool there = rows[j] != none;
          cp_async_16(k_to + j * (kRowStep * D), a.kv.codes[0] + (there ? static_cast<long long>(rows[j]) * D : 0) + c * 16,
                      there ? 16u : 0u);
        }
        cp_async_arrive(&k_full[t % kSlotsK]);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          const bool there = rows[j] != none;
          cp_async_16(to + j * kValue * 16, a.kv.codes[1] + (there ? static_cast<long long>(rows[j]) * D : 0) + c * 16,
                      there ? 16u : 0u);
        }
        cp_async_commit();
        mbar_arrive(&meta_empty[t % kMetaTiles]);            // the rows are read
      };
      bool there = published(tile);
      [[maybe_unused]] bool there1 = false;                  // the next tile
      if constexpr (kSelected) {
        if (there) copy(tile);
        there1 = there && published(tile + 1);
        if (there1) copy(tile + 1);
      }
      while (there && ok) {
        const uint32_t b = tile & 1u;
        if constexpr (kSelected) {
          if (there1) {
            cp_async_wait<1>();
          } else {
            cp_async_wait<0>();
          }
        } else {
          ok = ok && mbar_wait(&codes_full[b], tile >> 1 & 1u, timeout);
        }
        // The product of tile - 2 is done with this buffer.
        if (tile >= 2) ok = ok && mbar_wait(&pv_done[b], (tile - 2) >> 1 & 1u, timeout);
        if (!ok) break;
        // kAtOnce steps' codes before any is stored: a load behind a store
        // would wait for it.
        const uint8_t* codes = smem + codes_at + b * L::kSlotBytes;
        uint8_t* v_to = smem + v_at + b * L::kVBytes;
        uint8_t* v_next = smem + (v_at ^ 16u) + b * L::kVBytes;                 // the other half's place
        const bool holes = !kSelected && s_holes[tile % kMetaTiles] != 0;
        constexpr int kAtOnce = 4;
#pragma unroll 1
        for (int j0 = 0; j0 < kSteps; j0 += kAtOnce) {
          uint4 x[kAtOnce];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            x[j] = *reinterpret_cast<const uint4*>(codes + j * (kSelected ? kValue * 16 : kRowStep * D));
          }
          if (holes) {
            // Slots behind the sequence's end may hold any bytes, NaN among
            // them, and 0 * NaN is NaN: they become zeros.
            const int* row_of = rows_of(tile) + j0 * kRowStep;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              if (row_of[j * kRowStep] == none) x[j] = make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const uint2 h0 = cvt_bf16x4_e4m3(x[j].x), h1 = cvt_bf16x4_e4m3(x[j].y);
            const uint2 h2 = cvt_bf16x4_e4m3(x[j].z), h3 = cvt_bf16x4_e4m3(x[j].w);
            *reinterpret_cast<uint4*>(v_to + j * (kRowStep * 128)) = make_uint4(h0.x, h0.y, h1.x, h1.y);
            *reinterpret_cast<uint4*>(v_next + j * (kRowStep * 128)) = make_uint4(h2.x, h2.y, h3.x, h3.y);
          }
          codes += kAtOnce * (kSelected ? kValue * 16 : kRowStep * D);
          v_to += kAtOnce * (kRowStep * 128);
          v_next += kAtOnce * (kRowStep * 128);
        }
        fence_proxy_async_smem();
        if constexpr (!kSelected) mbar_arrive(&codes_empty[b]);
        mbar_arrive(&v_full[b]);
        ++tile;
        if constexpr (kSelected) {
          // V two tiles ahead, into the place that this tile's codes leave.
          there = there1;
          there1 = there && published(tile + 1);
          if (there1) copy(tile + 1);
        } else {
          there = ok && published(tile);
        }
      }
      if constexpr (kSelected) cp_async_wait<0>();           // also when a wait gave up
      if (!ok) fail(&g_iq_status_kv_rows, abort_flag, kStatusEpilogueWait);
    } else {
      // ------------------------------------------------------------- softmax
      const int group = warp >> 3, half = warp >> 2 & 1;
      const int r = threadIdx.x & 127;                       // row of the item, tensor-memory lane
      const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;
      auto meet = [&] {                                      // waits for the group's threads
        tc_fence_before_sync();
        mbar_arrive(&group_done[group]);
        ok = ok && mbar_wait(&group_done[group], meets & 1u, timeout);
        ++meets;
        tc_fence_after_sync();
      };
      auto agree = [&] { return ok = __all_sync(0xFFFFFFFFu, ok); };
      while (ok && next_segment()) {
        const uint32_t sb = seg & 1u;
        const bool there = r < g.rows;
        const int vis = there ? g.base + (g.r0 + r) / a.group + 1 : 1 << 30;   // positions below are seen
        const bool idle = (warp & 3) * 32 >= g.rows;         // no row in this warp
        const bool careful = again;                          // the maximum moves with every tile
        const int mine = (tile ^ group) & 1;                 // this group's first tile of the segment: 0 or 1
        bool over = false;                                   // a weight is too large
        float m = kNoMax, l = 0.f, bq = 0.f;

        for (int i = mine; i < g.n; i += 2) {
          const uint32_t t = tile + i, mslot = t % kMetaTiles, slot = t % kSlotsS;
          const uint32_t s_at = tmem + lane_base + kColS + slot * kTile + half * kHalf;
          const float* kf = s_meta + mslot * 4 * kTile + half * kHalf;
          const float* hide = kf + kTile;                    // 0, or -inf where there is no key
          const uint16_t* fv = reinterpret_cast<const uint16_t*>(s_meta + (mslot * 4 + 2) * kTile) + half * kHalf;
          // Keys of this half that the row sees.  (Selected keys that it does
          // not see are not there.)
          const int limit = kSelected ? kTile : vis - (g.kt0 + i) * kTile - half * kHalf;
          const bool cut = !kSelected && __any_sync(0xFFFFFFFFu, limit < kHalf);
          ok = ok && mbar_wait(&meta_full[mslot], t / kMetaTiles & 1u, timeout);
          ok = ok && mbar_wait(&s_full[slot], t / kSlotsS & 1u, timeout) && *abort_flag == 0u;
          if (!agree()) break;
          if (i == mine) bq = s_bq[seg % 4 * N + r];
          tc_fence_after_sync();
          if (i == 0 || careful) {
            // ---- the maximum, over both halves
            float top = -INFINITY;
            if (!idle) {
#pragma unroll 1
              for (int c0 = 0; c0 < kHalf; c0 += 16) {
                float v[16];
                tmem_ld_32x32b_x16(s_at + c0, v);
                tmem_ld_wait16(v);
                float x = -INFINITY;
                if constexpr (kSelected) {
#pragma unroll
                  for (int c = 0; c < 16; c += 4) {
                    const float4 k4 = *reinterpret_cast<const float4*>(kf + c0 + c);
                    const float4 h4 = *reinterpret_cast<const float4*>(hide + c0 + c);
                    x = fmaxf(fmaxf(x, __fmaf_rn(v[c] * bq, k4.x, h4.x)), __fmaf_rn(v[c + 1] * bq, k4.y, h4.y));
                    x = fmaxf(fmaxf(x, __fmaf_rn(v[c + 2] * bq, k4.z, h4.z)), __fmaf_rn(v[c + 3] * bq, k4.w, h4.w));
                  }
                } else {
                  // 16 keys of one page have one factor.
#pragma unroll
                  for (int c = 0; c < 16; ++c) x = fmaxf(x, c0 + c < limit ? v[c] : -INFINITY);
                  if (x != -INFINITY) x = __fmaf_rn(x, bq * kf[c0], hide[c0]);   // (0 * inf would be NaN)
                }
                top = fmaxf(top, x);
              }
            }
            // (A warp of the group may be two tiles back, at the reading below.)
            ok = ok && mbar_wait(&top_read[group], (tops++ & 1u) ^ 1u, timeout);
            s_top[(group * 2 + half) * N + r] = top;
            // Careful: the product of the tile before is done, and its
            // maximum (the other group's) stands in s_m.
            if (i > 0) ok = ok && mbar_wait(&pv_done[group ^ 1], (t - 1) >> 1 & 1u, timeout);
            meet();
            if (!agree()) break;
            const float before = i > 0 ? s_m[sb * N + r] : kNoMax;
            top = fmaxf(before, fmaxf(s_top[group * 2 * N + r], s_top[(group * 2 + 1) * N + r]));
            mbar_arrive(&top_read[group]);
            l *= ex2(m - top);
            m = top;
            const float corr = ex2(before - top);
            if (i > 0 && __any_sync(0xFFFFFFFFu, corr != 1.f)) {
#pragma unroll 1
              for (int c0 = 0; c0 < D / 2; c0 += 16) {
                float o[16];
                const uint32_t o_at = tmem + lane_base + kColO + half * (D / 2) + c0;
                tmem_ld_32x32b_x16(o_at, o);
                tmem_ld_wait16(o);
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                  tmem_st_32x32b_x4(o_at + c, o[c] * corr, o[c + 1] * corr, o[c + 2] * corr, o[c + 3] * corr);
                }
              }
              tmem_st_wait();
            }
            if (careful) meet();                             // every thread has read s_m
            // The segment before the last is written out: s_m is free.
            if (i == 0) ok = ok && mbar_wait(&sum_empty[sb], (seg >> 1 & 1u) ^ 1u, timeout);
            if (half == 0) s_m[sb * N + r] = m;
            if (i == 0) mbar_arrive(&m_full[sb]);
          } else if (i == mine) {
            // The other group has the segment's first tile.  (A barrier for each
            // parity: segment s + 2 arrives behind sum_empty of s, which this
            // thread's sum of s is part of, so no phase is missed; and the phase
            // of s cannot be taken for that of s - 1, whichever group is late.)
            ok = ok && mbar_wait(&m_full[sb], seg >> 1 & 1u, timeout);
            m = s_m[sb * N + r];
          }
          // ---- weights, over this half's scores.  A score is rounded, as it
          // was for the maximum, before that is taken away: their difference
          // would hold what the rounding left out, 2^11 in the exponent for a
          // score of 2^35.  (The addend of the product, 0 or -inf, keeps the
          // compiler from making one step of the product and the difference.)
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          auto weigh = [&](auto is_cut) {
            const uint64_t down2 = f2_pack(-m, -m), bq2 = f2_pack(bq, bq);
#pragma unroll 1
            for (int c0 = 0; c0 < kHalf; c0 += 16) {
              float s[16];
              tmem_ld_32x32b_x16(s_at + c0, s);
              tmem_ld_wait16(s);
              uint32_t w[8];
              if constexpr (kSelected) {
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                  const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(kf + c0 + c);
                  const ulonglong2 h4 = *reinterpret_cast<const ulonglong2*>(hide + c0 + c);
                  const uint2 f4 = *reinterpret_cast<const uint2*>(fv + c0 + c);
                  float x[4];
                  f2_unpack(f2_add(f2_fma(f2_mul(f2_pack(s[c], s[c + 1]), bq2), k4.x, h4.x), down2), x[0], x[1]);
                  f2_unpack(f2_add(f2_fma(f2_mul(f2_pack(s[c + 2], s[c + 3]), bq2), k4.y, h4.y), down2), x[2], x[3]);
#pragma unroll
                  for (int k = 0; k < 4; ++k) x[k] = ex2(x[k]);
                  const uint32_t p0 = cvt_bf16x2(x[0], x[1]), p1 = cvt_bf16x2(x[2], x[3]);
                  add_bf16x2(sum[0], sum[1], p0);
                  add_bf16x2(sum[2], sum[3], p1);
                  w[c / 2] = mul_bf16x2(p0, f4.x);
                  w[c / 2 + 1] = mul_bf16x2(p1, f4.y);
                }
              } else {
                // 16 keys of one page have one factor and one value scale.
                const float f = bq * kf[c0], h = hide[c0];
                const uint64_t f2 = f2_pack(f, f), h2 = f2_pack(h, h);
                const uint32_t fv2 = fv[c0] * 0x10001u;
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                  float x0, x1;
                  f2_unpack(f2_add(f2_fma(f2_pack(s[c], s[c + 1]), f2, h2), down2), x0, x1);
                  if constexpr (decltype(is_cut)::value) {
                    x0 = c0 + c < limit ? x0 : -INFINITY;
                    x1 = c0 + c + 1 < limit ? x1 : -INFINITY;
                  }
                  x0 = ex2(x0);
                  x1 = ex2(x1);
                  const uint32_t p = cvt_bf16x2(x0, x1);
                  add_bf16x2(sum[c & 2], sum[(c & 2) + 1], p);
                  w[c / 2] = mul_bf16x2(p, fv2);
                }
              }
              tmem_st_32x32b_x8(s_at + c0 / 2, w);         // behind what is read
            }
          };
          if (!idle) {
            if (cut) {
              weigh(std::true_type{});
            } else {
              weigh(std::false_type{});
            }
            tmem_st_wait();
          }
          tc_fence_before_sync();
          mbar_arrive(&p_full[slot]);
          if constexpr (kSelected) mbar_arrive(&meta_empty[mslot]);
          const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
          l += all;
          over = over || !(all <= kMostSum);                 // at least the largest weight
        }
        tile += g.n;
        if (over && there && !careful) {
          const int place = min(ordinal, kNoted - 1);
          atomicOr(&s_noted[place >> 5], 1u << (place & 31));
          *s_again = 1u;
        }

        if (!ok) break;
        if (careful && mine < g.n) {
          // The sums refer to the segment's last maximum.
          const uint32_t last = tile - 1;
          ok = ok && mbar_wait(&pv_done[last & 1u], last >> 1 & 1u, timeout);
          l *= ex2(m - s_m[sb * N + r]);
        }
        ok = ok && mbar_wait(&sum_empty[sb], (seg >> 1 & 1u) ^ 1u, timeout);
        s_sum[(sb * 4 + group * 2 + half) * N + r] = l;
        mbar_arrive(&sum_full[sb]);
        ++seg;
      }
      if (!ok) fail(&g_iq_status_kv_rows, abort_flag, kStatusEpilogueWait);
    }

    // The second round, if a segment is noted and nothing gave up.
    __syncthreads();
    if (again || *s_again == 0u || *abort_flag != 0u) break;
    again = true;
    __syncthreads();
    if (threadIdx.x == 0) *s_total = ~0u;
    __syncthreads();
  }

  if (warp == kScoreWarp) tc_commit_elected(drained_s);
  if (warp == kProductWarp) {
    tc_commit_elected(drained);
    if (!mbar_wait(drained, 0, 2 * timeout) || !mbar_wait(drained_s, 0, 2 * timeout)) {
      fail(&g_iq_status_kv_rows, abort_flag, kStatusTeardownWait);
    }
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool kSelected>
cudaError_t setup() {
  return cudaFuncSetAttribute(kv_attention_rows_kernel<D, kSelected>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RowLayout<D>::kSmemBytes);
}

template <int D, bool kSelected>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnParams& p, int ctas,
                   cudaStream_t stream) {
  return launch_dependent(kv_attention_rows_kernel<D, kSelected>, dim3(ctas, 1, 1), kThreads, RowLayout<D>::kSmemBytes, stream,
                          tm_k, tm_v, p);
}

}  // namespace

cudaError_t kv_attention_rows_setup_device() {
  cudaError_t err = setup<64, false>();
  if (err == cudaSuccess) err = setup<64, true>();
  if (err == cudaSuccess) err = setup<128, false>();
  if (err == cudaSuccess) err = setup<128, true>();
  return err;
}

cudaError_t launch_kv_attention_rows(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnParams& p, int ctas,
                                     cudaStream_t stream) {
  if (p.a.indices != nullptr) {
    return p.a.kv.dim == 64 ? launch<64, true>(tm_k, tm_v, p, ctas, stream)
                            : launch<128, true>(tm_k, tm_v, p, ctas, stream);
  }
  return p.a.kv.dim == 64 ? launch<64, false>(tm_k, tm_v, p, ctas, stream)
                          : launch<128, false>(tm_k, tm_v, p, ctas, stream);
}

cudaError_t read_kv_rows_status(uint32_t* flags, bool reset) {
  uint32_t v = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_iq_status_kv_rows, sizeof(v));
  if (err != cudaSuccess) return err;
  if (flags) *flags = v;
  if (reset) {
    const uint32_t zero = 0;
    err = cudaMemcpyToSymbol(g_iq_status_kv_rows, &zero, sizeof(zero));
  }
  return err;
}

}  // namespace iq
