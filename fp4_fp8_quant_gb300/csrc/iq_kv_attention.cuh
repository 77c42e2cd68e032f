// What the two attention kernels over the paged 8-bit KV cache share: the
// products' instructions, the division of the work over the CTAs, and the
// partial sums that are joined afterwards.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "iq_internal.h"
#include "iq_kv.h"
#include "iq_ptx.cuh"

namespace iq {

constexpr int kTile = 128;                 // keys per tile
// What beginning and ending an item of N rows costs, in key tiles.  Measured:
// a 4632-token prompt with 4 369 us, 6 362, 8 372, 10 381; one with dimension 64
// 299, 302, 308, 317; decode over 64 ragged sequences 184 with 2, 173 with 4, 174
// with 6, 177 with 8.
template <int N>
constexpr int kItemTiles = N > 32 ? 6 : 4;
// Weighted values are kept at 1 / kUp of what they are until the output is
// written: weights may grow to kUp times a row's first maximum, and sums of many
// large values stay finite.
constexpr float kUp = 0x1p40f;
constexpr float kNoMax = -3.402823466e38f;  // running maximum of a row that has seen no key: no finite score is below

struct AttnParams {
  AttnArgs a;
  float* part_o;            // [2 * ctas][N][D]  (weighted values / kUp)
  float2* part_ml;          // [2 * ctas][N]  (running maximum, sum)
  int4* heads;              // [2 * ctas] header of the item cut at the end of each CTA's run
  unsigned long long timeout_ns;
};

// ---- instruction pieces

// The MMAs are issued by a whole warp: all lanes run its loop, so that the operands are
// known to be the same in all of them, and one lane is elected for each
// instruction.  (Issued from a branch that one lane alone takes, an MMA costs
// 45 cycles or more to issue, whatever its size; elected, at most what it takes
// to run: 64 cycles at 128x128, 32 at 128x64 with A in tensor memory.)
// Descriptors are two words, of which only the low one, the address, changes
// from instruction to instruction.
struct Desc {
  uint32_t lo, hi;
  __device__ __forceinline__ Desc at(uint32_t bytes) const { return {lo + (bytes >> 4), hi}; }
};

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, Desc a, Desc b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %6, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, Desc a, Desc b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %6, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A from tensor memory.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, Desc b, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on the barrier when everything the elected lane issued has completed.
__device__ __forceinline__ void tc_commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// The same value in every lane, known as such to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Instruction descriptor of both products: E4M3 (kind::f8f6f4) or half
// (kind::f16) operands are type 0, float32 accumulators; a_mn / b_mn: operand
// stored MN-major.
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// With BF16 operands (both, kind::f16).
constexpr uint32_t kBf16Operands = (1u << 7) | (1u << 10);

// Matrix descriptor: start address, leading and stride byte offsets, swizzle
// (0 none, 2 128-byte, 4 64-byte).
__device__ __forceinline__ Desc smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return {(saddr >> 4) | (lbo >> 4) << 16, sbo >> 4 | 1u << 14 | swizzle << 29};
}

// Four rows of a tensor map whose box is one row high.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int4 rows) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(rows.x), "r"(rows.y), "r"(rows.z),
      "r"(rows.w)
      : "memory");
}

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four E4M3 codes -> four halves, exact.
__device__ __forceinline__ uint2 cvt_f16x4_e4m3(uint32_t c) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(c));
  return r;
}

__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Adds two BF16 values to two sums in float32.
__device__ __forceinline__ void add_bf16x2(float& lo, float& hi, uint32_t w) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "add.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
      : "+f"(lo), "+f"(hi)
      : "r"(w));
}

// Four E4M3 codes -> four BF16 values, exact.
__device__ __forceinline__ uint2 cvt_bf16x4_e4m3(uint32_t c) {
  const uint2 h = cvt_f16x4_e4m3(c);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
  return make_uint2(cvt_bf16x2(a.x, a.y), cvt_bf16x2(b.x, b.y));
}

// 2^e, the scale of a query row whose largest magnitude has these bits.  A row
// that holds an infinity (E4M3 has none: its codes would saturate) gets NaN.
__device__ __forceinline__ float query_scale(uint32_t bits, int e) {
  return bits < 0x7F800000u ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __uint_as_float(0x7FC00000u);
}

__device__ __forceinline__ void fail(uint32_t* status, volatile uint32_t* abort_flag, uint32_t bit) {
  atomicOr(status, bit);
  *abort_flag = 1u;
}

// ---- division of the work

// A run of key tiles of one item: rows [r0, r0 + rows) of one KV head.
struct Segment {
  int b, h;
  int r0, rows;      // flattened rows token * group + head, token 0 = packed row `row0`
  int row0;
  int base;          // token i sees positions < base + i + 1
  int keys;          // positions >= keys are not there for any row of the item
  int list;          // packed row whose index list is read (selected keys)
  int kt0, n;        // first key tile, tiles of this segment
  int kt_total;      // tiles of the item
  long long first;   // unit of the item's first tile
};

// Dense items of sequence b.  Rows outside [0, num_rows) are nobody's: neither
// Q nor the output is touched there, whatever row_start holds.
struct SeqInfo {
  int row0, n_rows, base, limit;
};

__device__ __forceinline__ SeqInfo seq_info(const KvArgs& kv, int b) {
  SeqInfo s;
  const int end = kv.row_start[b + 1], len = kv.kv_len[b];
  s.row0 = max(kv.row_start[b], 0);
  const int last = min(end, kv.num_rows);
  s.n_rows = last > s.row0 ? last - s.row0 : 0;
  s.base = len - end + s.row0;
  s.limit = static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(kv.max_pages) << kv.page_log2));
  return s;
}

template <int N>
__device__ __forceinline__ int row_tiles(const SeqInfo& s, int group) {
  return s.n_rows <= 0 ? 0 : (s.n_rows * group + N - 1) / N;
}

// Positions the last row of row tile rt sees.
template <int N>
__device__ __forceinline__ int keys_of(const SeqInfo& s, int group, int rt) {
  const int last = min(s.n_rows * group, (rt + 1) * N) - 1;
  return max(0, min(s.base + last / group + 1, s.limit));
}

__device__ __forceinline__ int key_tiles(int keys) { return max(1, (keys + kTile - 1) / kTile); }

// a / b for a >= 0, b > 0: a division of 64 bits is some hundred instructions.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 31 == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, w);
  return v;
}

__device__ __forceinline__ long long warp_prefix(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, v, w);
    if (lane >= w) v += o;
  }
  return v;
}

// Items and key tiles of a number of row tiles.
struct Load {
  long long items, tiles;
};

// Of all row tiles of the sequence held by lane `owner` (whole warp).
template <int N>
__device__ __forceinline__ Load seq_load_warp(SeqInfo s, int group, int owner) {
  s.n_rows = __shfl_sync(0xFFFFFFFFu, s.n_rows, owner);
  s.base = __shfl_sync(0xFFFFFFFFu, s.base, owner);
  s.limit = __shfl_sync(0xFFFFFFFFu, s.limit, owner);
  const int nrt = row_tiles<N>(s, group);
  long long sum = 0;
  for (int rt = threadIdx.x & 31; rt < nrt; rt += 32) sum += key_tiles(keys_of<N>(s, group, rt));
  return {nrt, warp_sum(sum)};
}

// Of (one KV head of) the sequence s, in every lane its own.
template <int N>
__device__ __forceinline__ Load seq_load(const AttnArgs& a, const SeqInfo& s) {
  const int nrt = row_tiles<N>(s, a.group);
  Load own = {nrt, 0};
  if (nrt <= 4) {
    for (int rt = 0; rt < nrt; ++rt) own.tiles += key_tiles(keys_of<N>(s, a.group, rt));
  }
  for (uint32_t many = __ballot_sync(0xFFFFFFFFu, nrt > 4); many != 0; many &= many - 1) {
    const int owner = __ffs(many) - 1;
    const Load v = seq_load_warp<N>(s, a.group, owner);
    if ((threadIdx.x & 31) == owner) own = v;
  }
  return own;
}

__device__ __forceinline__ SeqInfo seq_info_or_none(const KvArgs& kv, int b) {
  return b < kv.num_seqs ? seq_info(kv, b) : SeqInfo{0, 0, 0, 0};
}

// Where a CTA's run of tiles begins; found by one warp, read by all.  Tiles are
// counted in units: an item has its key tiles behind `cost` units that stand
// for the work of beginning and ending it, so that many short items weigh what
// they cost.
struct Start {
  long long u_begin, u_end, per;   // units of all items, laid end to end
  int cost;
  int b, rt, h, unit;              // dense: the item of u_begin and the unit within it
  SeqInfo s;                       // of sequence b
};

template <int N>
__device__ Start find_start(const AttnArgs& a) {
  Start st;
  const int lane = threadIdx.x & 31;
  Load all = {0, 0}, own = {0, 0};
  SeqInfo s = {0, 0, 0, 0};
  if (a.indices != nullptr) {
    all.items = static_cast<long long>(a.kv.num_rows) * ((a.group + N - 1) / N) * a.kv.heads;
    all.tiles = all.items * key_tiles(a.topk);
  } else {
    for (int b0 = 0; b0 < a.kv.num_seqs; b0 += 32) {
      s = seq_info_or_none(a.kv, b0 + lane);
      own = seq_load<N>(a, s);
      all.items += own.items;
      all.tiles += own.tiles;
    }
    all.items = warp_sum(all.items) * a.kv.heads;
    all.tiles = warp_sum(all.tiles) * a.kv.heads;
  }
  // Where there is at most a tile for every CTA, each gets one.
  st.cost = all.tiles > gridDim.x ? kItemTiles<N> : 0;
  const long long total = all.tiles + st.cost * all.items;
  st.per = quotient(total + gridDim.x - 1, gridDim.x);
  st.u_begin = min(total, st.per * blockIdx.x);
  st.u_end = min(total, st.u_begin + st.per);
  st.b = st.rt = st.h = st.unit = 0;
  st.s = s;
  if (a.indices != nullptr || st.u_begin >= st.u_end) return st;
  long long left = st.u_begin;                       // units before u_begin, from the current point on
  for (int b0 = 0; b0 < a.kv.num_seqs; b0 += 32) {
    if (a.kv.num_seqs > 32) {
      s = seq_info_or_none(a.kv, b0 + lane);
      own = seq_load<N>(a, s);
    }
    const long long units = (own.tiles + st.cost * own.items) * a.kv.heads;
    const long long upto = warp_prefix(units);
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > left);
    if (past == 0) {
      left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
      continue;
    }
    const int j = __ffs(past) - 1;
    left -= __shfl_sync(0xFFFFFFFFu, upto - units, j);
    st.b = b0 + j;
    s.row0 = __shfl_sync(0xFFFFFFFFu, s.row0, j);
    s.n_rows = __shfl_sync(0xFFFFFFFFu, s.n_rows, j);
    s.base = __shfl_sync(0xFFFFFFFFu, s.base, j);
    s.limit = __shfl_sync(0xFFFFFFFFu, s.limit, j);
    st.s = s;
    const int nrt = row_tiles<N>(s, a.group);
    for (int rt0 = 0; rt0 < nrt; rt0 += 32) {
      const int item = rt0 + lane < nrt ? st.cost + key_tiles(keys_of<N>(s, a.group, rt0 + lane)) : 0;
      const long long o = static_cast<long long>(item) * a.kv.heads;
      const long long to = warp_prefix(o);
      const uint32_t p = __ballot_sync(0xFFFFFFFFu, to > left);
      if (p == 0) {
        left -= __shfl_sync(0xFFFFFFFFu, to, 31);
        continue;
      }
      const int i = __ffs(p) - 1;
      left -= __shfl_sync(0xFFFFFFFFu, to - o, i);
      const int each = __shfl_sync(0xFFFFFFFFu, item, i);
      st.rt = rt0 + i;
      st.h = static_cast<int>(quotient(left, each));
      st.unit = static_cast<int>(left - static_cast<long long>(st.h) * each);
      break;
    }
    break;
  }
  return st;
}

// Steps through the segments of a CTA's run, by whole warps.  Every role has
// its own.
template <int N>
struct Walker {
  const Start& st;                                   // in shared memory
  long long u;
  int b, rt, h, unit;

  __device__ __forceinline__ explicit Walker(const Start& start)
      : st(start), u(start.u_begin), b(start.b), rt(start.rt), h(start.h), unit(start.unit) {}

  __device__ __forceinline__ bool next(const AttnArgs& a, Segment& g) {
    const long long u_end = st.u_end;
    const int cost = st.cost;
    do {
      if (u >= u_end) return false;
      int at;                                        // unit within the item
      if (a.indices != nullptr) {
        const int units = cost + key_tiles(a.topk);
        const int splits = (a.group + N - 1) / N;
        const long long item = quotient(u, units), parts = quotient(item, a.kv.heads);
        at = static_cast<int>(u - item * units);
        g.h = static_cast<int>(item - parts * a.kv.heads);
        g.list = static_cast<int>(quotient(parts, splits));
        const int part = static_cast<int>(parts - static_cast<long long>(g.list) * splits);
        g.row0 = g.list;
        g.r0 = part * N;
        g.rows = min(N, a.group - g.r0);
        g.kt_total = key_tiles(a.topk);
        g.b = kv_find_seq(a.kv, g.list);
        g.base = -1;
        if (g.b < a.kv.num_seqs) g.base = a.kv.kv_len[g.b] - a.kv.row_start[g.b + 1] + g.list;
        g.keys = max(0, static_cast<int>(min(static_cast<long long>(g.base) + 1,
                                             static_cast<long long>(a.kv.max_pages) << a.kv.page_log2)));
      } else {
        SeqInfo s = b == st.b ? st.s : seq_info(a.kv, b);
        int nrt = row_tiles<N>(s, a.group);
        while (rt >= nrt) {                          // u < u_end: a sequence with rows follows
          rt = 0;
          if (++b >= a.kv.num_seqs) return false;
          s = seq_info(a.kv, b);
          nrt = row_tiles<N>(s, a.group);
        }
        at = unit;
        unit = 0;
        g.b = b;
        g.h = h;
        g.r0 = rt * N;
        g.rows = min(N, s.n_rows * a.group - g.r0);
        g.row0 = s.row0;
        g.list = 0;
        g.base = s.base;
        g.keys = keys_of<N>(s, a.group, rt);
        g.kt_total = key_tiles(g.keys);
        if (++h == a.kv.heads) {
          h = 0;
          ++rt;
        }
      }
      g.first = u - at + cost;
      const long long to = min(g.first + g.kt_total, u_end);
      const long long from = max(u, g.first);
      g.kt0 = static_cast<int>(from - g.first);
      g.n = static_cast<int>(to - from);
      u = to;
    } while (g.n <= 0);                              // only the units before the item's tiles lie in this run
    return true;
  }
};

// The many-rows kernel (iq_kv_attention_rows.cu): 128 rows per item, one CTA
// per SM.
constexpr int kManyRows = 128;
cudaError_t kv_attention_rows_setup_device();
cudaError_t launch_kv_attention_rows(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnParams& p, int ctas,
                                     cudaStream_t stream);
cudaError_t read_kv_rows_status(uint32_t* flags, bool reset);

}  // namespace iq
