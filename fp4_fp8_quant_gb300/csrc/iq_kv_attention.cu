// Attention over the paged 8-bit KV cache (include/iq.h, section 4):
//   out = sum_s p_s v_s / sum_s p_s,  p_s = 2^(x_s),  x_s = scale log2(e) q . k_s.
//
// K9 kv_attention_kernel.  Both products run on the fifth-generation tensor
// cores on the codes as they lie in the cache: nothing is converted, a key or
// value byte is moved once, from memory to shared memory, by TMA.  The keys
// are the MMA's M side in the first product and its K side in the second, the
// queries its N side in both:
//   S^T [128 keys, N rows]  = K [128, D]  x  Q^T [D, N]
//   O^T [D, N rows]        += V^T [D, 128]  x  P [128, N]
// so a tile does full work whether the rows are one token's heads (N = 16) or
// a chunk of a prompt (N = 64), and decode, chunks and selected keys are one
// kernel.  A row is one (token, query head); the rows of one KV head are taken
// token by token, N at a time.
//
// BF16 times E4M3 without loss.  The MMA multiplies E4M3 by E4M3, and a BF16
// value is the sum of two: with a row scaled by a power of two to at most 448,
// q1 = E4M3(q) leaves a remainder of at most four significant bits, which q2 =
// E4M3(q - q1) holds exactly (down to 2^-19 of the row's largest value).  The
// two products add up in one accumulator.  The weights P are split the same
// way, P = P1 + P2 / 16 (2^-8 of each weight, as BF16 would), with the second
// product's accumulator apart, so that P2 uses E4M3's whole range.
//
// Scales.  A key's scale 2^eK multiplies its scores, one factor per lane of
// the accumulator.  A value's scale 2^eV is folded into the exponent, the
// weight being 2^(x + eV - m) with m the running maximum of x + eV: values
// stay codes, weights stay below 1, and the row's sum takes 2^-eV back out.
//
// The running maximum is lazy: m moves, and the accumulators are scaled, only
// when some weight would pass 2^2.75 times the one m stands for (the weights
// are kept at 2^6 of it, and E4M3 ends at 448 = 2^8.8).
//
// Work is divided by key tiles: the tiles of all (rows, KV head) items, laid
// end to end, are cut into one equal run per CTA (two CTAs per SM), so ragged
// lengths, one long sequence and many short ones load the SMs alike.  An item
// cut between CTAs leaves its partial sums (float32, with m and the sum) in
// the workspace, and K10 joins them in a fixed order.
//
// Warps: 0..3 softmax (one key per thread; the same threads load Q, scale and
// store O, one dimension per thread), 4 producer (page lookups, TMA), 5 MMA
// issuer.  K and V tiles share one ring of slots in the order of use
// (K0 K1 V0 K2 V1 ...); the scores are double buffered, so S of the next tile
// is computed while the softmax works on this one.  Every wait is bounded.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "iq_internal.h"
#include "iq_kv.h"
#include "iq_ptx.cuh"

namespace iq {

__device__ uint32_t g_iq_status_kv;

namespace {

constexpr int kTile = 128;                 // keys per tile (MMA M of the first product, K of the second)
constexpr int kGroupThreads = 128;         // a softmax group: four warps, one key per thread
constexpr float kNoMax = -1e30f;           // running maximum of a row that has seen no key
constexpr float kLift = 4.f;               // exponent of a weight at the running maximum
constexpr float kMaxLifted = 15.f;         // and the largest one taken: 2^15 in half precision
constexpr int kItemTiles = 4;              // what beginning and ending an item costs, in key tiles

template <int N, int D>
struct Layout {
  static constexpr int kCols = N < 32 ? N : 32;   // rows (accumulator columns) of a softmax group
  static constexpr int kGroups = N / kCols;
  static constexpr int kThreads = kGroups * kGroupThreads + 64;
  static constexpr int kCtasPerSm = N == 128 ? 1 : 2;
  static constexpr int kSlotBytes = kTile * D;
  // Slots for the codes: two CTAs per SM leave 64 rows one slot each, enough
  // because a tile's work lasts longer than a load from L2.
  static constexpr int kSlotsK = N == 128 ? 4 : (N == 64 && D == 128 ? 1 : 2);
  static constexpr int kSlotsV = N == 128 ? 3 : (N <= 16 || D == 64 ? 2 : 1);
  static constexpr int kMetaTiles = kSlotsK <= 2 ? 4 : 8;   // tiles whose key scales are held
  static constexpr int kQBytes = N * D;          // one term of Q
  static constexpr int kPBytes = kTile * N * 2;
  static constexpr int kVBytes = kTile * D * 2;  // values in half precision
  static constexpr int kOffCodesV = kSlotsK * kSlotBytes;
  static constexpr int kOffV = kOffCodesV + kSlotsV * kSlotBytes;
  static constexpr int kOffQ = kOffV + kVBytes;
  static constexpr int kOffP = kOffQ + 2 * kQBytes;
  static constexpr int kOffMeta = kOffP + kPBytes;
  static constexpr int kOffOut = kOffMeta + kMetaTiles * kTile * 8;  // long long [N]: where the row's output goes
  static constexpr int kOffRows = kOffOut + N * 8;                   // float m, nm, bq, corr [N], int vis [N]
  static constexpr int kOffRed = kOffRows + 5 * N * 4;               // float [4][N]
  static constexpr int kOffBar = kOffRed + 4 * N * 4;
  static constexpr int kNumBars = 2 * (kSlotsK + kSlotsV) + 2 + 4 + kMetaTiles;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;            // + alignment slack
  // Tensor memory: two score buffers and the output accumulator (a power of two is allocated).
  static constexpr uint32_t kColS = 0, kColO = 2 * N, kTmemCols = 4 * N;
  static_assert(kOffQ % 1024 == 0 && kOffP % 128 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(kSmemBytes <= 226 * 1024 / kCtasPerSm, "shared memory");
  static_assert(kMetaTiles >= kSlotsK + 2, "a tile's key scales stay until its softmax is done");
};

struct Params {
  AttnArgs a;
  float* part_o;            // [2 * ctas][N][D]
  float2* part_ml;          // [2 * ctas][N]  (running maximum, sum)
  int4* heads;              // [2 * ctas] header of the item cut at the end of each CTA's run
  unsigned long long timeout_ns;
};

// ---- instruction pieces

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of both products: E4M3 (kind::f8f6f4) or half
// (kind::f16) operands are type 0, float32 accumulators; a_mn / b_mn: operand
// stored MN-major.
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Matrix descriptor: start address, leading and stride byte offsets, swizzle
// (0 none, 2 128-byte, 4 64-byte).
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(lbo >> 4) << 16 |
         static_cast<uint64_t>(sbo >> 4) << 32 | 1ull << 46 | static_cast<uint64_t>(swizzle) << 61;
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

__device__ __forceinline__ void fail(volatile uint32_t* abort_flag, uint32_t bit) {
  atomicOr(&g_iq_status_kv, bit);
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

// Dense items of sequence b.
struct SeqInfo {
  int row0, n_rows, base, limit;
};

__device__ __forceinline__ SeqInfo seq_info(const KvArgs& kv, int b) {
  SeqInfo s;
  s.row0 = kv.row_start[b];
  s.n_rows = kv.row_start[b + 1] - s.row0;
  const int len = kv.kv_len[b];
  s.base = len - s.n_rows;
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

// Units of an item: its key tiles behind kItemTiles that stand for the work of
// beginning and ending it, so that many short items weigh what they cost.
__device__ __forceinline__ int item_units(int keys) { return kItemTiles + key_tiles(keys); }

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

// Units of all row tiles of the sequence held by lane `owner` (whole warp).
template <int N>
__device__ __forceinline__ long long seq_units_warp(SeqInfo s, int group, int owner) {
  s.n_rows = __shfl_sync(0xFFFFFFFFu, s.n_rows, owner);
  s.base = __shfl_sync(0xFFFFFFFFu, s.base, owner);
  s.limit = __shfl_sync(0xFFFFFFFFu, s.limit, owner);
  const int nrt = row_tiles<N>(s, group);
  long long sum = 0;
  for (int rt = threadIdx.x & 31; rt < nrt; rt += 32) sum += item_units(keys_of<N>(s, group, rt));
  return warp_sum(sum);
}

// Units (of one KV head) of sequence b0 + lane, in every lane its own.
template <int N>
__device__ __forceinline__ long long seq_units(const AttnArgs& a, int b0) {
  const int b = b0 + (threadIdx.x & 31);
  SeqInfo s = {0, 0, 0, 0};
  if (b < a.kv.num_seqs) s = seq_info(a.kv, b);
  const int nrt = row_tiles<N>(s, a.group);
  long long sum = 0;
  if (nrt <= 4) {
    for (int rt = 0; rt < nrt; ++rt) sum += item_units(keys_of<N>(s, a.group, rt));
  }
  for (uint32_t many = __ballot_sync(0xFFFFFFFFu, nrt > 4); many != 0; many &= many - 1) {
    const int owner = __ffs(many) - 1;
    const long long v = seq_units_warp<N>(s, a.group, owner);
    if ((threadIdx.x & 31) == owner) sum = v;
  }
  return sum;
}

// Where a CTA's run of tiles begins; found by one warp, read by all.
struct Start {
  long long u_begin, u_end, per;   // units of all items, laid end to end
  int b, rt, h, unit;              // dense: the item of u_begin and the unit within it
};

template <int N>
__device__ Start find_start(const AttnArgs& a) {
  Start st;
  long long total;
  if (a.indices != nullptr) {
    total = static_cast<long long>(a.kv.num_rows) * ((a.group + N - 1) / N) * a.kv.heads * item_units(a.topk);
  } else {
    total = 0;
    for (int b0 = 0; b0 < a.kv.num_seqs; b0 += 32) total += warp_sum(seq_units<N>(a, b0));
    total *= a.kv.heads;
  }
  st.per = (total + gridDim.x - 1) / gridDim.x;
  st.u_begin = min(total, st.per * blockIdx.x);
  st.u_end = min(total, st.u_begin + st.per);
  st.b = st.rt = st.h = st.unit = 0;
  if (a.indices != nullptr || st.u_begin >= st.u_end) return st;
  const int lane = threadIdx.x & 31;
  long long left = st.u_begin;                       // units before u_begin, from the current point on
  for (int b0 = 0; b0 < a.kv.num_seqs; b0 += 32) {
    const long long own = seq_units<N>(a, b0) * a.kv.heads;
    const long long upto = warp_prefix(own);
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > left);
    if (past == 0) {
      left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
      continue;
    }
    const int j = __ffs(past) - 1;
    left -= __shfl_sync(0xFFFFFFFFu, upto - own, j);
    st.b = b0 + j;
    const SeqInfo s = seq_info(a.kv, st.b);
    const int nrt = row_tiles<N>(s, a.group);
    for (int rt0 = 0; rt0 < nrt; rt0 += 32) {
      const int units = rt0 + lane < nrt ? item_units(keys_of<N>(s, a.group, rt0 + lane)) : 0;
      const long long o = static_cast<long long>(units) * a.kv.heads;
      const long long to = warp_prefix(o);
      const uint32_t p = __ballot_sync(0xFFFFFFFFu, to > left);
      if (p == 0) {
        left -= __shfl_sync(0xFFFFFFFFu, to, 31);
        continue;
      }
      const int i = __ffs(p) - 1;
      left -= __shfl_sync(0xFFFFFFFFu, to - o, i);
      const int each = __shfl_sync(0xFFFFFFFFu, units, i);
      st.rt = rt0 + i;
      st.h = static_cast<int>(left / each);
      st.unit = static_cast<int>(left % each);
      break;
    }
    break;
  }
  return st;
}

// Steps through the segments of a CTA's run.  Every role has its own.
template <int N>
struct Walker {
  long long u, u_end;
  int b, rt, h, unit;

  __device__ __forceinline__ explicit Walker(const Start& s)
      : u(s.u_begin), u_end(s.u_end), b(s.b), rt(s.rt), h(s.h), unit(s.unit) {}

  __device__ __forceinline__ bool next(const AttnArgs& a, Segment& g) {
    do {
      if (u >= u_end) return false;
      int at;                                        // unit within the item
      if (a.indices != nullptr) {
        const int units = item_units(a.topk);
        const int splits = (a.group + N - 1) / N;
        long long item = u / units;
        at = static_cast<int>(u - item * units);
        g.h = static_cast<int>(item % a.kv.heads);
        item /= a.kv.heads;
        const int part = static_cast<int>(item % splits);
        g.list = static_cast<int>(item / splits);
        g.row0 = g.list;
        g.r0 = part * N;
        g.rows = min(N, a.group - g.r0);
        g.kt_total = key_tiles(a.topk);
        g.b = kv_find_seq_thread(a.kv, g.list);
        g.base = -1;
        if (g.b < a.kv.num_seqs) g.base = a.kv.kv_len[g.b] - a.kv.row_start[g.b + 1] + g.list;
        g.keys = max(0, static_cast<int>(min(static_cast<long long>(g.base) + 1,
                                             static_cast<long long>(a.kv.max_pages) << a.kv.page_log2)));
      } else {
        SeqInfo s = seq_info(a.kv, b);
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
      g.first = u - at + kItemTiles;
      const long long to = min(g.first + g.kt_total, u_end);
      const long long from = max(u, g.first);
      g.kt0 = static_cast<int>(from - g.first);
      g.n = static_cast<int>(to - from);
      u = to;
    } while (g.n <= 0);                              // only the units before the item's tiles lie in this run
    return true;
  }
};

// Four keys' places in the cache, as the producer's lane holds them.
struct KeyRows {
  int row[4];        // rows of the codes taken as a matrix [.][D]; num_rows: none
};

template <int N, int D>
__global__ void __launch_bounds__(Layout<N, D>::kThreads, Layout<N, D>::kCtasPerSm)
    kv_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ Params p) {
  using L = Layout<N, D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_q = smem + L::kOffQ;
  uint8_t* s_p = smem + L::kOffP;
  long long* s_out = reinterpret_cast<long long*>(smem + L::kOffOut);
  float2* s_meta = reinterpret_cast<float2*>(smem + L::kOffMeta);    // [L::kMetaTiles][128] (score factor, eV)
  float* s_m = reinterpret_cast<float*>(smem + L::kOffRows);         // running maximum
  float* s_nm = s_m + N;                                             // kLift - maximum
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
  static_assert(sizeof(Start) <= 48, "start");

  const AttnArgs& a = p.a;
  const uint64_t timeout = p.timeout_ns;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kProducerWarp = 4 * L::kGroups, kMmaWarp = kProducerWarp + 1;

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
      mbar_init(&v_empty[i], L::kGroups * kGroupThreads);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(q_full, L::kGroups * kGroupThreads);
    mbar_init(p_full, L::kGroups * kGroupThreads);
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
  const Start start = *s_start;

  if (warp == kProducerWarp) {
    // -------------------------------------------------------------- producer
    Walker<N> walk(start);
    Segment g = {};
    const int none = a.kv.num_pages * a.kv.heads * a.kv.page;   // a row past the end: TMA fills zeros
    const bool leader = a.indices != nullptr || ((4 * lane) & (a.kv.page - 1)) == 0;
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
      if (a.indices != nullptr) {
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

    auto push_k = [&](const int* rows, const float2* meta) {
      const int mslot = pushed % L::kMetaTiles;
      if (!push(&tm_k, k_full, k_empty, smem, L::kSlotsK, pushed, rows)) return false;
      float4* dst = reinterpret_cast<float4*>(s_meta + mslot * kTile + 4 * lane);
      dst[0] = make_float4(meta[0].x, meta[0].y, meta[1].x, meta[1].y);
      dst[1] = make_float4(meta[2].x, meta[2].y, meta[3].x, meta[3].y);
      __syncwarp();
      if (lane == 0) mbar_arrive(&meta_full[mslot]);
      return true;
    };
    // What the softmax needs of a key: score factor and the exponent of the
    // value's scale (-inf: no such key).
    auto key_meta = [&](bool there, uint32_t ek, uint32_t ev) {
      return there ? make_float2(a.scale_log2 * ue8m0_to_float(ek), static_cast<float>(static_cast<int>(ev) - 127))
                   : make_float2(0.f, -INFINITY);
    };

    if (a.indices == nullptr) {
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
          const uint32_t k = __shfl_sync(0xFFFFFFFFu, ek, j + my_page), v = __shfl_sync(0xFFFFFFFFu, ev, j + my_page);
          const int pos = (g.kt0 + i) * kTile + 4 * lane;
          const int row = id >= 0 ? static_cast<int>((static_cast<long long>(id) * a.kv.heads + g.h) * a.kv.page) : none;
          float2 meta[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) meta[c] = key_meta(id >= 0 && pos + c < g.keys, k, v);
          ok = push_k(&row, meta);
          if (i > 0) ok = ok && push_v(&last_row);
          last_row = row;
          if (j == 0) find_scales(next_pid, next_ek, next_ev);
        }
        ok = ok && push_v(&last_row);
      }
    } else {
      // Single rows, four keys per lane, two tiles per step.  The three
      // dependent loads (position, page, scales) of a pair of tiles are issued
      // three, two and one steps ahead, so that none is waited for.
      while (ok && walk.next(a, g)) {
        int pos3[8], pos2[8], pid2[8], row1[8], row0[8], row_last[4];
        uint32_t sf1[8], sf0[8];
        auto find_pos = [&](int pair, int* pos) {
          const int j = (g.kt0 + 2 * pair) * kTile + 4 * lane;
          const int32_t* list = a.indices + static_cast<long long>(g.list) * a.ld_idx;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int at = j + (k >> 2) * kTile + (k & 3);
            pos[k] = 2 * pair + (k >> 2) < g.n && at < a.topk ? list[at] : -1;
          }
        };
        auto find_pid = [&](const int* pos, int* pid) {
#pragma unroll
          for (int k = 0; k < 8; ++k) pid[k] = pos[k] < g.keys ? kv_page_of(a.kv, g.b, pos[k]) : -1;
        };
        auto find_row = [&](const int* pos, const int* pid, int* row) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const long long at = static_cast<long long>(pid[k]) * a.kv.heads + g.h;
            row[k] = pid[k] >= 0 ? static_cast<int>(at * a.kv.page + (pos[k] & (a.kv.page - 1))) : none;
          }
        };
        auto find_scales = [&](const int* row, uint32_t* sf) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sf[k] = 0;
            if (row[k] != none) {
              const int at = row[k] >> a.kv.page_log2;
              sf[k] = a.kv.sf[0][at] | static_cast<uint32_t>(a.kv.sf[1][at]) << 8;
            }
          }
        };
        find_pos(0, pos2);
        find_pos(1, pos3);
        find_pid(pos2, pid2);
        find_row(pos2, pid2, row0);
        find_scales(row0, sf0);
        find_pid(pos3, pid2);
        find_row(pos3, pid2, row1);
        find_pos(2, pos2);
        find_pid(pos2, pid2);
        find_pos(3, pos3);
        for (int p2 = 0; ok && 2 * p2 < g.n; ++p2) {
          int next[8];
          find_scales(row1, sf1);                          // pair p2 + 1
          find_row(pos2, pid2, next);                      // pair p2 + 2
#pragma unroll
          for (int k = 0; k < 8; ++k) pos2[k] = pos3[k];
          find_pid(pos2, pid2);                            // pair p2 + 3
          find_pos(p2 + 4, pos3);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int i = 2 * p2 + half;
            if (i < g.n) {
              float2 meta[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t f = sf0[4 * half + c];
                meta[c] = key_meta(row0[4 * half + c] != none, f & 0xFFu, f >> 8);
              }
              ok = ok && push_k(row0 + 4 * half, meta);
              // Values one tile behind the keys.
              if (half == 1) {
                ok = ok && push_v(row0);
              } else if (i > 0) {
                ok = ok && push_v(row_last);
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) row_last[c] = g.n - 2 * p2 == 1 ? row0[c] : row0[4 + c];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            row0[k] = row1[k];
            sf0[k] = sf1[k];
            row1[k] = next[k];
          }
        }
        ok = ok && push_v(row_last);
      }
    }
    if (!ok) fail(abort_flag, kStatusProducerWait);
    // Every copy has landed before the CTA ends (also when a wait gave up).
    for (int i = max(0, pushed - L::kSlotsK); i < pushed; ++i) {
      if (!mbar_wait(&k_full[i % L::kSlotsK], i / L::kSlotsK & 1, timeout)) fail(abort_flag, kStatusTeardownWait);
    }
    for (int i = max(0, pushed_v - L::kSlotsV); i < pushed_v; ++i) {
      if (!mbar_wait(&v_full[i % L::kSlotsV], i / L::kSlotsV & 1, timeout)) fail(abort_flag, kStatusTeardownWait);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      Walker<N> walk(start);
      Segment g = {};
      constexpr uint32_t kSwizzle = D == 128 ? 2u : 4u;
      const uint32_t idesc_s = idesc_f32(128, N, 0, 0), idesc_o = idesc_f32(128, N, 1, 1);
      const uint32_t k_at = smem_u32(smem), q_at = smem_u32(s_q), p_at = smem_u32(s_p),
                     v_at = smem_u32(smem + L::kOffV);
      uint32_t tile = 0, seg = 0;
      bool ok = true;
      auto scores = [&](uint32_t t) {                    // S of tile t
        const uint32_t slot = t % L::kSlotsK;
        if (!mbar_wait(&k_full[slot], t / L::kSlotsK & 1u, timeout)) return false;
        tc_fence_after_sync();
        const uint32_t d = tmem + L::kColS + (t & 1u) * N;
#pragma unroll
        for (int term = 0; term < 2; ++term) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            tc_mma_f8(d, smem_desc(k_at + slot * L::kSlotBytes + 32 * k, 16, 8 * D, kSwizzle),
                      smem_desc(q_at + term * L::kQBytes + 2 * k * (16 * N), 16 * N, 128, 0), idesc_s,
                      (term | k) != 0);
          }
        }
        tc_commit(&k_empty[slot]);
        tc_commit(&s_full[t & 1u]);
        return true;
      };
      while (ok && walk.next(a, g)) {
        ok = mbar_wait(q_full, seg & 1u, timeout);
        ++seg;
        tc_fence_after_sync();
        ok = ok && scores(tile);
        for (int i = 0; ok && i < g.n; ++i, ++tile) {
          if (i + 1 < g.n) ok = scores(tile + 1);
          ok = ok && mbar_wait(p_full, tile & 1u, timeout) && *abort_flag == 0u;
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k) {
            // V: 16 keys are two groups of eight rows of 64 dimensions; the
            // next 64 dimensions are 128 rows on (with D = 64 the second 64
            // lanes repeat the first).  P: [8 columns][key][8].
            tc_mma_f16(tmem + L::kColO, smem_desc(v_at + 2048 * k, D == 128 ? kTile * 128 : 0, 1024, 2),
                       smem_desc(p_at + 256 * k, 128, kTile * 16, 0), idesc_o, (i | k) != 0);
          }
          tc_commit(pv_done);
        }
      }
      if (!ok) fail(abort_flag, kStatusMmaWait);
      tc_commit(drained);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    // Group w has the rows (columns of S^T and O^T) [col0, col0 + kCols).
    constexpr int kCols = L::kCols;
    Walker<N> walk(start);
    Segment g = {};
    const int key = threadIdx.x % kGroupThreads;          // key of a tile; dimension of the output
    const int group_warp = warp & 3;
    const uint32_t barrier = 1 + warp / 4;
    const int col0 = warp / 4 * kCols;
    const uint32_t lane_base = static_cast<uint32_t>(group_warp) << 21;   // this warp's 32 tensor-memory lanes
    const uint32_t o_at = tmem + lane_base + L::kColO + col0;
    s_out += col0;
    s_m += col0;
    s_nm += col0;
    s_bq += col0;
    s_corr += col0;
    s_vis += col0;
    s_red += 4 * col0;                                    // [4 warps][kCols]
    uint32_t tile = 0;
    bool ok = true;        // this thread's waits
    bool stop = false;     // some thread's wait gave up; the same in the whole group
    bool first = true;     // no item has been finished here
    bool open = false;     // the last item begins here and goes on in the next CTA
    const long long run = start.per;
    while (!stop && walk.next(a, g)) {
      const int rows = min(kCols, g.rows - col0);         // of this group; may be 0 or less
      // ---- Q: rows scaled by a power of two, split into two E4M3 terms
      {
        constexpr int kPerRow = kGroupThreads / kCols;     // threads per row
        constexpr int kVals = D / kPerRow;                 // values per thread
        const int r = key / kPerRow, part = key % kPerRow;
        uint4 x[kVals / 8];
        uint32_t m2 = 0;
        const bool there = r < rows;
        const int fr = g.r0 + col0 + r, tok = fr / a.group;
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
          uint8_t* dst = s_q + (d0 >> 4) * (16 * N) + (col0 + r) * 16 + (d0 & 8);
          *reinterpret_cast<uint2*>(dst) = make_uint2(c1[0] | c1[1] << 16, c1[2] | c1[3] << 16);
          *reinterpret_cast<uint2*>(dst + L::kQBytes) = make_uint2(c2[0] | c2[1] << 16, c2[2] | c2[3] << 16);
        }
        if (part == 0) {
          s_bq[r] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          s_vis[r] = there ? g.base + tok + 1 : 0;
          s_m[r] = kNoMax;
          s_out[r] = (g.row0 + tok) * a.ldo + head * static_cast<long long>(D);
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
        named_barrier_sync(barrier, kGroupThreads);
      }
      const int vis_first = s_vis[0];
      float l[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) l[c] = 0.f;

      for (int i = 0; i < g.n; ++i, ++tile) {
        const int pos0 = (g.kt0 + i) * kTile;
        const uint32_t mslot = tile % L::kMetaTiles;
        ok = ok && mbar_wait(&meta_full[mslot], (tile / L::kMetaTiles) & 1u, timeout);
        const float2 meta = s_meta[mslot * kTile + key];
        const bool seen = meta.y != -INFINITY;
        const bool some_hidden = __any_sync(0xFFFFFFFFu, !seen);
        const bool causal = a.indices == nullptr && pos0 + kTile > vis_first;   // some row does not see all keys
        ok = ok && mbar_wait(&s_full[tile & 1u], (tile >> 1) & 1u, timeout);
        tc_fence_after_sync();
        const uint32_t s_at = tmem + lane_base + L::kColS + (tile & 1u) * N + col0;
        const uint64_t kf2 = f2_pack(meta.x, meta.x), ev2 = f2_pack(meta.y, meta.y);

        // Exponents of the weights: x + eV + kLift - m; -inf where the row
        // does not see the key.  If one passes kMaxLifted anywhere in the
        // group (and for the first tile) the maximum moves first.
        float d[kCols];
        bool settle = i == 0;
        while (true) {
          if (!settle) {
            if constexpr (kCols == 32) {
              tmem_ld_32x32b_x32(s_at, d);
              tmem_ld_wait(d);
            } else {
              tmem_ld_32x32b_x16(s_at, d);
              tmem_ld_wait16(d);
            }
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
              const ulonglong2 bq = *reinterpret_cast<const ulonglong2*>(s_bq + c);
              const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(s_nm + c);
              f2_unpack(f2_fma(f2_mul(f2_pack(d[c], d[c + 1]), bq.x), kf2, f2_add(nm.x, ev2)), d[c], d[c + 1]);
              f2_unpack(f2_fma(f2_mul(f2_pack(d[c + 2], d[c + 3]), bq.y), kf2, f2_add(nm.y, ev2)), d[c + 2], d[c + 3]);
            }
            if (some_hidden) {
#pragma unroll
              for (int c = 0; c < kCols; ++c) d[c] = seen ? d[c] : -INFINITY;
            }
            if (causal) {
#pragma unroll
              for (int c = 0; c < kCols; ++c) d[c] = pos0 + key < s_vis[c] ? d[c] : -INFINITY;
            }
            float tops[4] = {d[0], d[1], d[2], d[3]};
#pragma unroll
            for (int c = 4; c < kCols; ++c) tops[c & 3] = fmaxf(tops[c & 3], d[c]);
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            if (named_barrier_and(barrier, kGroupThreads, ok && !(top > kMaxLifted))) break;
          }
          // Some thread saw its maximum move, or gave up waiting.
          stop = !named_barrier_and(barrier, kGroupThreads, ok && *abort_flag == 0u);
          if (stop) break;
          // The maximum per column, over the warp, then over the warps.
#pragma unroll 1
          for (int c0 = 0; c0 < kCols; c0 += 16) {
            float z[16];
            tmem_ld_32x32b_x16(s_at + c0, z);
            tmem_ld_wait16(z);
            float mine = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const bool in = seen && (a.indices != nullptr || pos0 + key < s_vis[c0 + c]);
              const float m = redux_max(in ? z[c] * s_bq[c0 + c] * meta.x + meta.y : -INFINITY);
              mine = lane == c ? m : mine;
            }
            if (lane < 16) s_red[group_warp * kCols + c0 + lane] = mine;
          }
          named_barrier_sync(barrier, kGroupThreads);
          if (key < kCols) {
            const float old = s_m[key];
            float m = fmaxf(fmaxf(s_red[key], s_red[kCols + key]), fmaxf(s_red[2 * kCols + key], s_red[3 * kCols + key]));
            m = key < rows ? fmaxf(old, m) : 1e30f;        // unused columns: weight 0, never in the way
            s_m[key] = m;
            s_nm[key] = kLift - m;
            s_corr[key] = ex2(old - m);
          }
          named_barrier_sync(barrier, kGroupThreads);
          if (i > 0) {
            ok = mbar_wait(pv_done, (tile - 1) & 1u, timeout);
            tc_fence_after_sync();
#pragma unroll 1
            for (int c0 = 0; c0 < kCols; c0 += 16) {
              float o[16];
              tmem_ld_32x32b_x16(o_at + c0, o);
              tmem_ld_wait16(o);
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                const float4 f = *reinterpret_cast<const float4*>(s_corr + c0 + c);
                tmem_st_32x32b_x4(o_at + c0 + c, o[c] * f.x, o[c + 1] * f.y, o[c + 2] * f.z, o[c + 3] * f.w);
              }
            }
            tmem_st_wait();
#pragma unroll
            for (int c = 0; c < kCols; ++c) l[c] *= s_corr[c];
          }
          settle = false;
        }
        if (stop) break;
        if (i > 0) ok = mbar_wait(pv_done, (tile - 1) & 1u, timeout);   // the buffers of P and V are free

        // ---- weights
        const float fl = seen ? ex2(-meta.y) : 0.f;
        const uint64_t fl2 = f2_pack(fl, fl);
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 8) {
          uint32_t w[4];
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            const float e0 = ex2(d[c0 + c]), e1 = ex2(d[c0 + c + 1]);
            float* lc = l + c0 + c;
            f2_unpack(f2_fma(f2_pack(e0, e1), fl2, f2_pack(lc[0], lc[1])), lc[0], lc[1]);
            w[c / 2] = cvt_f16x2(e0, e1);
          }
          // [8 columns][key][8]
          *reinterpret_cast<uint4*>(s_p + (col0 + c0) * (kTile * 2) + key * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // ---- values: 16 codes per step, 16 dimensions of one key, into the
        // 128-byte swizzled rows of 64 halves.  Slots behind the sequence's
        // end may hold any bytes, NaN among them, and 0 * NaN is NaN: they
        // become zeros (pages without any key, and unselected keys, arrive as
        // zeros).
        {
          const uint32_t slot = tile % L::kSlotsV;
          ok = ok && mbar_wait(&v_full[slot], tile / L::kSlotsV & 1u, timeout);
          constexpr int kChunks = D / 16;                  // per key
          constexpr int kSteps = kTile * kChunks / (L::kGroups * kGroupThreads);
          const uint8_t* codes = smem + L::kOffCodesV + slot * L::kSlotBytes;
          const int c = threadIdx.x % kChunks;
          uint4 x[kSteps];
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const int r = (j * (L::kGroups * kGroupThreads) + threadIdx.x) / kChunks;
            // The codes lie under the TMA swizzle: 16-byte pieces exchanged by
            // the row (128-byte rows) or by pairs of rows (64-byte rows).
            const int at = D == 128 ? (c ^ (r & 7)) : (c ^ (r >> 1 & 3));
            x[j] = *reinterpret_cast<const uint4*>(codes + r * D + at * 16);
          }
          mbar_arrive(&v_empty[slot]);
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const int r = (j * (L::kGroups * kGroupThreads) + threadIdx.x) / kChunks;
            if (a.indices == nullptr && pos0 + r >= g.keys) x[j] = make_uint4(0, 0, 0, 0);
            const uint2 h0 = cvt_f16x4_e4m3(x[j].x), h1 = cvt_f16x4_e4m3(x[j].y);
            const uint2 h2 = cvt_f16x4_e4m3(x[j].z), h3 = cvt_f16x4_e4m3(x[j].w);
            const uint4 lo = make_uint4(h0.x, h0.y, h1.x, h1.y), hi = make_uint4(h2.x, h2.y, h3.x, h3.y);
            uint8_t* row = smem + L::kOffV + (c / 4) * (kTile * 128) + r * 128;
            // Lanes of the upper 64 dimensions store their halves in the other
            // order: a quarter warp then touches every bank once.
            const int odd = c / 4 & 1, first = 2 * (c % 4) + odd;
            *reinterpret_cast<uint4*>(row + ((first ^ (r & 7)) << 4)) = odd ? hi : lo;
            *reinterpret_cast<uint4*>(row + (((first ^ 1) ^ (r & 7)) << 4)) = odd ? lo : hi;
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
        for (int c = 0; c < (kCols == 32 || w < 16 ? w : 16); ++c) {
          if (kCols == 16 && w == 16) {
            l[c] += __shfl_xor_sync(0xFFFFFFFFu, l[c], 16);
          } else {
            const bool up = (lane & w) != 0;
            const float send = up ? l[c] : l[c + w], keep = up ? l[c + w] : l[c];
            l[c] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, w);
          }
        }
      }
      if (lane < kCols) s_red[group_warp * kCols + lane] = l[0];
      ok = ok && mbar_wait(pv_done, (tile - 1) & 1u, timeout);
      tc_fence_after_sync();
      stop = !named_barrier_and(barrier, kGroupThreads, ok);
      if (stop) break;
      const bool whole = g.n == g.kt_total;
      const int part = 2 * blockIdx.x + (first ? 0 : 1);   // an item that goes on from the CTA before comes first
      first = false;
      if (key < kCols) {
        const float sum = s_red[key] + s_red[kCols + key] + s_red[2 * kCols + key] + s_red[3 * kCols + key];
        s_corr[key] = sum > 0.f ? 1.f / sum : 0.f;
        if (!whole && key < rows) {
          p.part_ml[static_cast<long long>(part) * N + col0 + key] = make_float2(s_m[key], sum);
        }
      }
      named_barrier_sync(barrier, kGroupThreads);
#pragma unroll 1
      for (int c0 = 0; c0 < rows; c0 += 16) {
        float o[16];
        tmem_ld_32x32b_x16(o_at + c0, o);
        tmem_ld_wait16(o);
        if (key < D) {
          float* dst = p.part_o + (static_cast<long long>(part) * N + col0 + c0) * D + key;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (c0 + c < rows) {
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
        p.heads[2 * blockIdx.x] = make_int4(1, static_cast<int>((g.first + g.kt_total - 1) / run), part, g.rows);
        p.heads[2 * blockIdx.x + 1] = make_int4(g.row0, g.r0, g.h, 0);
      }
      tc_fence_before_sync();
      named_barrier_sync(barrier, kGroupThreads);         // the group's arrays are free again
    }
    if (stop || !ok) fail(abort_flag, kStatusEpilogueWait);
    if (threadIdx.x == 0 && (stop || !open)) p.heads[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    if (!mbar_wait(drained, 0, 2 * timeout)) fail(abort_flag, kStatusTeardownWait);
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// K11: many rows per item.  The products the other way round,
//   S [128 rows, 128 keys] = Q x K^T,   O [128 rows, D] += P x V,
// one row per softmax thread: its maximum, sum and scale are registers, and
// nothing is exchanged between threads.

template <int D>
struct RowLayout {
  static constexpr int kRows = 128;
  static constexpr int kThreads = 320;           // 4 softmax, 4 value, producer, MMA warps
  static constexpr int kSlotsK = 2;
  static constexpr int kMetaTiles = 4;
  static constexpr int kSlotBytes = kTile * D;
  static constexpr int kQBytes = kRows * D;      // one term of Q
  static constexpr int kVBytes = kTile * D * 2;
  static constexpr int kOffV = kSlotsK * kSlotBytes;
  static constexpr int kOffQ = kOffV + kVBytes;
  static constexpr int kOffMeta = kOffQ + 2 * kQBytes;              // float kf, ev, fl [kTile], int row [kTile] per tile
  static constexpr int kOffBar = kOffMeta + kMetaTiles * kTile * 16;
  static constexpr int kNumBars = 2 * kSlotsK + 2 * kMetaTiles + 6;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;
  // Tensor memory: scores, whose columns the weights take over, and output.
  static constexpr uint32_t kColS = 0, kColO = 128, kTmemCols = 256;
  static_assert(kOffV % 1024 == 0 && kOffQ % 1024 == 0, "alignment");
  static_assert(kSmemBytes <= 113 * 1024, "two CTAs per SM");
};

// A from tensor memory.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <int D, bool kSelected>
__global__ void __launch_bounds__(320, 2)
    kv_attention_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ Params p) {
  using L = RowLayout<D>;
  constexpr int N = L::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_v = smem + L::kOffV;
  uint8_t* s_q = smem + L::kOffQ;
  float* s_meta = reinterpret_cast<float*>(smem + L::kOffMeta);   // [kMetaTiles][4][kTile]
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* k_empty = k_full + L::kSlotsK;
  uint64_t* meta_full = k_empty + L::kSlotsK;
  uint64_t* meta_empty = meta_full + L::kMetaTiles;
  uint64_t* q_full = meta_empty + L::kMetaTiles;
  uint64_t* s_full = q_full + 1;
  uint64_t* p_full = q_full + 2;
  uint64_t* v_full = q_full + 3;
  uint64_t* pv_done = q_full + 4;
  uint64_t* drained = q_full + 5;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + 4);
  Start* s_start = reinterpret_cast<Start*>(smem + L::kOffMisc + 8);

  const AttnArgs& a = p.a;
  const uint64_t timeout = p.timeout_ns;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kProducerWarp = 8, kMmaWarp = 9;

  grid_launch_dependents();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_k);
    for (int i = 0; i < L::kSlotsK; ++i) {
      mbar_init(&k_full[i], kSelected ? 128 : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < L::kMetaTiles; ++i) {
      mbar_init(&meta_full[i], 1);
      mbar_init(&meta_empty[i], 1);
    }
    mbar_init(q_full, 128);
    mbar_init(s_full, 1);
    mbar_init(p_full, 128);
    mbar_init(v_full, 128);
    mbar_init(pv_done, 1);
    mbar_init(drained, 1);
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
  const Start start = *s_start;
  const int none = a.kv.num_pages * a.kv.heads * a.kv.page;   // a row past the end: zeros

  if (warp == kProducerWarp) {
    // -------------------------------------------------------------- producer
    Walker<N> walk(start);
    Segment g = {};
    int pushed = 0;
    bool ok = true;                                   // the same in every lane

    // Publishes a tile's key data; where whole pages are loaded, also loads
    // the keys.
    auto push = [&](const int* rows, const uint32_t* ek, const uint32_t* ev) {
      const int mslot = pushed % L::kMetaTiles;
      const bool free = mbar_wait(&meta_empty[mslot], (pushed / L::kMetaTiles & 1) ^ 1, timeout) && *abort_flag == 0u;
      if (!__all_sync(0xFFFFFFFFu, free)) return false;
      float* meta = s_meta + mslot * 4 * kTile + 4 * lane;
      float kf[4], e[4], fl[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool there = rows[c] != none;
        kf[c] = there ? fabsf(a.scale_log2) * ue8m0_to_float(ek[c]) : 0.f;
        e[c] = there ? static_cast<float>(static_cast<int>(ev[c]) - 127) : -INFINITY;
        fl[c] = there ? ex2(-e[c]) : 0.f;
      }
      *reinterpret_cast<float4*>(meta) = make_float4(kf[0], kf[1], kf[2], kf[3]);
      *reinterpret_cast<float4*>(meta + kTile) = make_float4(e[0], e[1], e[2], e[3]);
      *reinterpret_cast<float4*>(meta + 2 * kTile) = make_float4(fl[0], fl[1], fl[2], fl[3]);
      *reinterpret_cast<int4*>(meta + 3 * kTile) = make_int4(rows[0], rows[1], rows[2], rows[3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&meta_full[mslot]);
      if constexpr (!kSelected) {
        const int slot = pushed % L::kSlotsK;
        const bool k_free = mbar_wait(&k_empty[slot], (pushed / L::kSlotsK & 1) ^ 1, timeout) && *abort_flag == 0u;
        if (!__all_sync(0xFFFFFFFFu, k_free)) return false;
        if (lane == 0) mbar_arrive_expect_tx(&k_full[slot], L::kSlotBytes);
        __syncwarp();
        if (((4 * lane) & (a.kv.page - 1)) == 0) {
          tma_load_2d(smem + slot * L::kSlotBytes + 4 * lane * D, &tm_k, &k_full[slot], 0, rows[0]);
        }
      }
      ++pushed;
      return true;
    };

    if constexpr (!kSelected) {
      // Pages in order: lane l looks up page l of a batch of 32, one batch
      // ahead, pages while the batch begins and their scales a tile later.
      const int per_tile = kTile >> a.kv.page_log2;
      const int my_page = (4 * lane) >> a.kv.page_log2;          // of a tile
      while (ok && walk.next(a, g)) {
        const int page0 = (g.kt0 * kTile) >> a.kv.page_log2;
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
        for (int i = 0; ok && i < g.n; ++i) {
          const int j = (i * per_tile) & 31;
          if (j == 0 && i > 0) {
            pid = next_pid;
            ek = next_ek;
            ev = next_ev;
            next_pid = find_page(i * per_tile + 32);
          }
          const int id = __shfl_sync(0xFFFFFFFFu, pid, j + my_page);
          const uint32_t k = __shfl_sync(0xFFFFFFFFu, ek, j + my_page), v = __shfl_sync(0xFFFFFFFFu, ev, j + my_page);
          const int pos = (g.kt0 + i) * kTile + 4 * lane;
          const int row0 = static_cast<int>((static_cast<long long>(id) * a.kv.heads + g.h) * a.kv.page);
          int rows[4];
          const uint32_t k4[4] = {k, k, k, k}, v4[4] = {v, v, v, v};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            rows[c] = id >= 0 && pos + c < g.keys ? row0 + ((pos + c) & (a.kv.page - 1)) : none;
          }
          ok = push(rows, k4, v4);
          if (j == 0) find_scales(next_pid, next_ek, next_ev);
        }
      }
    } else {
      // Single rows, four keys per lane.  The three dependent loads (position,
      // page, scales) of a tile are issued three, two and one tiles ahead.
      while (ok && walk.next(a, g)) {
        int pos3[4], pos2[4], pid2[4], row1[4], row0[4];
        uint32_t ek1[4], ev1[4], ek0[4], ev0[4];
        auto find_pos = [&](int i, int* pos) {
          const int j = (g.kt0 + i) * kTile + 4 * lane;
          const int32_t* list = a.indices + static_cast<long long>(g.list) * a.ld_idx;
#pragma unroll
          for (int k = 0; k < 4; ++k) pos[k] = i < g.n && j + k < a.topk ? list[j + k] : -1;
        };
        auto find_pid = [&](const int* pos, int* pid) {
#pragma unroll
          for (int k = 0; k < 4; ++k) pid[k] = pos[k] < g.keys ? kv_page_of(a.kv, g.b, pos[k]) : -1;
        };
        auto find_row = [&](const int* pos, const int* pid, int* row) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const long long at = static_cast<long long>(pid[k]) * a.kv.heads + g.h;
            row[k] = pid[k] >= 0 ? static_cast<int>(at * a.kv.page + (pos[k] & (a.kv.page - 1))) : none;
          }
        };
        auto find_scales = [&](const int* row, uint32_t* ek, uint32_t* ev) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ek[k] = ev[k] = 0;
            if (row[k] != none) {
              const int at = row[k] >> a.kv.page_log2;
              ek[k] = a.kv.sf[0][at];
              ev[k] = a.kv.sf[1][at];
            }
          }
        };
        find_pos(0, pos2);
        find_pos(1, pos3);
        find_pid(pos2, pid2);
        find_row(pos2, pid2, row0);
        find_scales(row0, ek0, ev0);
        find_pid(pos3, pid2);
        find_row(pos3, pid2, row1);
        find_pos(2, pos2);
        find_pid(pos2, pid2);
        find_pos(3, pos3);
        for (int i = 0; ok && i < g.n; ++i) {
          int next[4];
          find_scales(row1, ek1, ev1);                     // tile i + 1
          find_row(pos2, pid2, next);                      // tile i + 2
#pragma unroll
          for (int k = 0; k < 4; ++k) pos2[k] = pos3[k];
          find_pid(pos2, pid2);                            // tile i + 3
          find_pos(i + 4, pos3);
          ok = push(row0, ek0, ev0);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            row0[k] = row1[k];
            row1[k] = next[k];
            ek0[k] = ek1[k];
            ev0[k] = ev1[k];
          }
        }
      }
    }
    if (!ok) fail(abort_flag, kStatusProducerWait);
    if constexpr (!kSelected) {
      // Every copy has landed before the CTA ends (also when a wait gave up).
      for (int i = max(0, pushed - L::kSlotsK); i < pushed; ++i) {
        if (!mbar_wait(&k_full[i % L::kSlotsK], i / L::kSlotsK & 1, timeout)) fail(abort_flag, kStatusTeardownWait);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      Walker<N> walk(start);
      Segment g = {};
      constexpr uint32_t kSwizzle = D == 128 ? 2u : 4u;
      const uint32_t idesc_s = idesc_f32(128, kTile, 0, 0), idesc_o = idesc_f32(128, D, 0, 1);
      const uint32_t k_at = smem_u32(smem), q_at = smem_u32(s_q), v_at = smem_u32(s_v);
      uint32_t tile = 0, seg = 0;
      bool ok = true;
      while (ok && walk.next(a, g)) {
        ok = mbar_wait(q_full, seg & 1u, timeout);
        ++seg;
        for (int i = 0; ok && i < g.n; ++i, ++tile) {
          const uint32_t slot = tile % L::kSlotsK;
          ok = mbar_wait(&k_full[slot], tile / L::kSlotsK & 1u, timeout);
          // The weights of the tile before lie in the scores' columns.
          if (tile > 0) ok = ok && mbar_wait(pv_done, (tile - 1) & 1u, timeout);
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int term = 0; term < 2; ++term) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              tc_mma_f8(tmem + L::kColS, smem_desc(q_at + term * L::kQBytes + 2 * k * (16 * N), 16 * N, 128, 0),
                        smem_desc(k_at + slot * L::kSlotBytes + 32 * k, 16, 8 * D, kSwizzle), idesc_s,
                        (term | k) != 0);
            }
          }
          tc_commit(&k_empty[slot]);
          tc_commit(s_full);
          ok = mbar_wait(v_full, tile & 1u, timeout) && mbar_wait(p_full, tile & 1u, timeout) && *abort_flag == 0u;
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k) {
            tc_mma_f16_ta(tmem + L::kColO, tmem + L::kColS + 8 * k,
                          smem_desc(v_at + 2048 * k, D == 128 ? kTile * 128 : 0, 1024, 2), idesc_o, (i | k) != 0);
          }
          tc_commit(&meta_empty[tile % L::kMetaTiles]);
          tc_commit(pv_done);
        }
      }
      if (!ok) fail(abort_flag, kStatusMmaWait);
      tc_commit(drained);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- values
    // From memory through registers into half precision: 16 codes per load,
    // 16 dimensions of one key, stored as 128-byte swizzled rows of 64
    // halves.  A tile's loads are in flight while the tile before is used.
    Walker<N> walk(start);
    Segment g = {};
    const int tid = threadIdx.x - 128;
    constexpr int kChunks = D / 16, kSteps = kTile * kChunks / 128;
    const int c = tid % kChunks;
    uint32_t tile = 0;
    bool ok = true;
    int next_row[kSteps];                              // this thread's rows of the tile to come
    // Reads a tile's rows; selected keys are copied from here too, 16 bytes
    // per thread and step, the pieces of a row exchanged as the TMA swizzle
    // would.
    auto begin = [&](uint32_t t) {
      const uint32_t mslot = t % L::kMetaTiles, slot = t % L::kSlotsK;
      bool good = mbar_wait(&meta_full[mslot], t / L::kMetaTiles & 1u, timeout) && *abort_flag == 0u;
      if constexpr (kSelected) good = good && mbar_wait(&k_empty[slot], (t / L::kSlotsK & 1u) ^ 1u, timeout);
      if (!good) return false;
      const int* row_of = reinterpret_cast<const int*>(s_meta + (mslot * 4 + 3) * kTile);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int r = (j * 128 + tid) / kChunks;
        next_row[j] = row_of[r];
        if constexpr (kSelected) {
          const int at = D == 128 ? (c ^ (r & 7)) : (c ^ (r >> 1 & 3));
          const bool there = next_row[j] != none;
          cp_async_16(smem + slot * L::kSlotBytes + r * D + at * 16,
                      a.kv.codes[0] + (there ? static_cast<long long>(next_row[j]) * D + c * 16 : 0), there ? 16u : 0u);
        }
      }
      if constexpr (kSelected) cp_async_commit();
      return true;
    };
    while (ok && walk.next(a, g)) {
      ok = begin(tile);
      for (int i = 0; ok && i < g.n; ++i, ++tile) {
        uint4 x[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          x[j] = make_uint4(0, 0, 0, 0);
          if (next_row[j] != none) {
            x[j] = ld_dependent_v4(a.kv.codes[1] + static_cast<long long>(next_row[j]) * D + c * 16);
          }
        }
        if (i + 1 < g.n) ok = begin(tile + 1);
        if constexpr (kSelected) {
          if (i + 1 < g.n && ok) {
            cp_async_wait<1>();
          } else {
            cp_async_wait<0>();
          }
          fence_proxy_async_smem();
          mbar_arrive(&k_full[tile % L::kSlotsK]);
        }
        if (tile > 0) ok = ok && mbar_wait(pv_done, (tile - 1) & 1u, timeout);
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          const int r = (j * 128 + tid) / kChunks;
          const uint2 h0 = cvt_f16x4_e4m3(x[j].x), h1 = cvt_f16x4_e4m3(x[j].y);
          const uint2 h2 = cvt_f16x4_e4m3(x[j].z), h3 = cvt_f16x4_e4m3(x[j].w);
          const uint4 lo = make_uint4(h0.x, h0.y, h1.x, h1.y), hi = make_uint4(h2.x, h2.y, h3.x, h3.y);
          uint8_t* row = s_v + (c / 4) * (kTile * 128) + r * 128;
          // Lanes of the upper 64 dimensions store their halves in the other
          // order: a quarter warp then touches every bank once.
          const int odd = c / 4 & 1, first = 2 * (c % 4) + odd;
          *reinterpret_cast<uint4*>(row + ((first ^ (r & 7)) << 4)) = odd ? hi : lo;
          *reinterpret_cast<uint4*>(row + (((first ^ 1) ^ (r & 7)) << 4)) = odd ? lo : hi;
        }
        fence_proxy_async_smem();
        mbar_arrive(v_full);
      }
    }
    if (!ok) fail(abort_flag, kStatusEpilogueWait);
    if constexpr (kSelected) cp_async_wait<0>();       // also when a wait gave up
  } else {
    // --------------------------------------------------------------- softmax
    Walker<N> walk(start);
    Segment g = {};
    const int r = threadIdx.x;                            // row of the item, tensor-memory lane
    const uint32_t lane_base = static_cast<uint32_t>(warp) << 21;
    const uint32_t s_at = tmem + lane_base + L::kColS, o_at = tmem + lane_base + L::kColO;
    uint32_t tile = 0;
    bool ok = true, first = true, open = false;
    const long long run = start.per;
    while (ok && walk.next(a, g)) {
      // ---- Q: the row scaled by a power of two, split into two E4M3 terms
      const bool there = r < g.rows;
      const int fr = g.r0 + r, tok = fr / a.group;
      const int head = g.h * a.group + fr - tok * a.group;
      const int vis = there ? g.base + tok + 1 : 1 << 30;  // positions below are seen
      const bool idle = warp * 32 >= g.rows;              // no row in this warp
      float bq;
      {
        const uint4* src =
            reinterpret_cast<const uint4*>(a.q + (g.row0 + tok) * a.ldq + head * static_cast<long long>(D));
        uint32_t m2 = 0;
        if (there) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 x = src[i];
            m2 = __vmaxu2(__vmaxu2(m2, x.x & 0x7FFF7FFFu), x.y & 0x7FFF7FFFu);
            m2 = __vmaxu2(__vmaxu2(m2, x.z & 0x7FFF7FFFu), x.w & 0x7FFF7FFFu);
          }
        }
        // Smallest e with 448 * 2^e >= the largest value, at least -118.
        const uint32_t bits = max(m2 & 0xFFFFu, m2 >> 16) << 16;
        const int e = max(-118, static_cast<int>(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        bq = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        const uint32_t flip = a.scale_log2 < 0.f ? 0x8080u : 0u;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t c1[8], c2[8];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (there) x = src[2 * i + half];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float lo = __uint_as_float(w[j] << 16) * inv, hi = __uint_as_float(w[j] & 0xFFFF0000u) * inv;
              const uint32_t t = cvt_e4m3x2(lo, hi);
              c1[4 * half + j] = t;
              c2[4 * half + j] = cvt_e4m3x2(lo - e4m3_to_float(t), hi - e4m3_to_float(t >> 8));
            }
          }
          // A negative scale changes the sign of the codes, so that the largest
          // product is the largest score.
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            c1[j] ^= flip;
            c2[j] ^= flip;
          }
          uint8_t* dst = s_q + i * (16 * N) + r * 16;      // K-major without swizzle: [16 dims][row][16]
          *reinterpret_cast<uint4*>(dst) = make_uint4(c1[0] | c1[1] << 16, c1[2] | c1[3] << 16, c1[4] | c1[5] << 16,
                                                      c1[6] | c1[7] << 16);
          *reinterpret_cast<uint4*>(dst + L::kQBytes) = make_uint4(c2[0] | c2[1] << 16, c2[2] | c2[3] << 16,
                                                                   c2[4] | c2[5] << 16, c2[6] | c2[7] << 16);
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      float m = kNoMax, l = 0.f;

      for (int i = 0; i < g.n; ++i, ++tile) {
        const uint32_t mslot = tile % L::kMetaTiles;
        const float* kf = s_meta + mslot * 4 * kTile;
        const float* ev = kf + kTile;
        const float* fl = kf + 2 * kTile;
        ok = ok && mbar_wait(&meta_full[mslot], tile / L::kMetaTiles & 1u, timeout);
        ok = ok && mbar_wait(s_full, tile & 1u, timeout) && *abort_flag == 0u;
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        if (idle) {
          tc_fence_before_sync();
          mbar_arrive(p_full);
          continue;
        }
        // Keys of the tile that the row sees.  (Selected keys that it does not
        // see have eV = -inf.)
        const int limit = kSelected ? kTile : vis - (g.kt0 + i) * kTile;
        const bool cut = !kSelected && __any_sync(0xFFFFFFFFu, limit < kTile);

        // ---- largest x + eV
        float top = -INFINITY;
        auto find_top = [&](auto is_cut) {
#pragma unroll
          for (int c0 = 0; c0 < kTile; c0 += 32) {
            float v[32];
            tmem_ld_32x32b_x32(s_at + c0, v);
            tmem_ld_wait(v);
            if constexpr (kSelected) {
              const uint64_t bq2 = f2_pack(bq, bq);
              float t[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(kf + c0 + c);
                const ulonglong2 e4 = *reinterpret_cast<const ulonglong2*>(ev + c0 + c);
                float x[4];
                f2_unpack(f2_fma(f2_mul(f2_pack(v[c], v[c + 1]), bq2), k4.x, e4.x), x[0], x[1]);
                f2_unpack(f2_fma(f2_mul(f2_pack(v[c + 2], v[c + 3]), bq2), k4.y, e4.y), x[2], x[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) t[k] = fmaxf(t[k], x[k]);
              }
              top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
            } else {
              // 16 keys of one page: one factor and one exponent.
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                if constexpr (decltype(is_cut)::value) {
#pragma unroll
                  for (int c = h; c < h + 16; ++c) v[c] = c0 + c < limit ? v[c] : -INFINITY;
                }
                float t[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  t[c] = fmaxf(fmaxf(v[h + c], v[h + 4 + c]), fmaxf(v[h + 8 + c], v[h + 12 + c]));
                }
                const float most = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                const float x = most * (bq * kf[c0 + h]) + ev[c0 + h];
                // No key seen: -inf whatever the factor (0 * inf is NaN).
                top = fmaxf(top, decltype(is_cut)::value && most == -INFINITY ? -INFINITY : x);
              }
            }
          }
        };
        if (cut) {
          find_top(std::true_type{});
        } else {
          find_top(std::false_type{});
        }
        // The running maximum moves only where a weight would pass 2^15 of
        // what the accumulators are scaled by.
        const bool move = top + (kLift - m) > kMaxLifted;
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float corr = move ? ex2(m - top) : 1.f;
          if (move) m = top;
          l *= corr;
          if (i > 0) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              float o[32];
              tmem_ld_32x32b_x32(o_at + c0, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] *= corr;
              tmem_st_32x32b_x32(o_at + c0, o);
            }
            tmem_st_wait();
          }
        }
        const float nm = kLift - m;

        // ---- weights, over the scores' columns
        uint64_t sum[2] = {0, 0};
        auto weigh = [&](auto is_cut) {
          const uint64_t nm2 = f2_pack(nm, nm), bq2 = f2_pack(bq, bq);
#pragma unroll
          for (int c0 = 0; c0 < kTile; c0 += 32) {
            float v[32];
            tmem_ld_32x32b_x32(s_at + c0, v);
            tmem_ld_wait(v);
            uint32_t w[16];
            if constexpr (kSelected) {
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(kf + c0 + c);
                const ulonglong2 e4 = *reinterpret_cast<const ulonglong2*>(ev + c0 + c);
                const ulonglong2 f4 = *reinterpret_cast<const ulonglong2*>(fl + c0 + c);
                float x[4];
                f2_unpack(f2_fma(f2_mul(f2_pack(v[c], v[c + 1]), bq2), k4.x, f2_add(e4.x, nm2)), x[0], x[1]);
                f2_unpack(f2_fma(f2_mul(f2_pack(v[c + 2], v[c + 3]), bq2), k4.y, f2_add(e4.y, nm2)), x[2], x[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = ex2(x[k]);
                sum[0] = f2_fma(f2_pack(x[0], x[1]), f4.x, sum[0]);
                sum[1] = f2_fma(f2_pack(x[2], x[3]), f4.y, sum[1]);
                w[c / 2] = cvt_f16x2(x[0], x[1]);
                w[c / 2 + 1] = cvt_f16x2(x[2], x[3]);
              }
            } else {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                const float f = bq * kf[c0 + h], n = ev[c0 + h] + nm, fc = fl[c0 + h];
                const uint64_t f2 = f2_pack(f, f), n2 = f2_pack(n, n), fl2 = f2_pack(fc, fc);
                uint64_t part[2] = {0, 0};
#pragma unroll
                for (int c = h; c < h + 16; c += 2) {
                  float x0, x1;
                  f2_unpack(f2_fma(f2_pack(v[c], v[c + 1]), f2, n2), x0, x1);
                  if constexpr (decltype(is_cut)::value) {
                    x0 = c0 + c < limit ? x0 : -INFINITY;
                    x1 = c0 + c + 1 < limit ? x1 : -INFINITY;
                  }
                  x0 = ex2(x0);
                  x1 = ex2(x1);
                  part[c / 2 & 1] = f2_add(part[c / 2 & 1], f2_pack(x0, x1));
                  w[c / 2] = cvt_f16x2(x0, x1);
                }
                sum[0] = f2_fma(part[0], fl2, sum[0]);
                sum[1] = f2_fma(part[1], fl2, sum[1]);
              }
            }
            tmem_st_32x32b_x8(s_at + c0 / 2, w);
            tmem_st_32x32b_x8(s_at + c0 / 2 + 8, w + 8);
          }
        };
        if (cut) {
          weigh(std::true_type{});
        } else {
          weigh(std::false_type{});
        }
        {
          float a0, a1;
          f2_unpack(f2_add(sum[0], sum[1]), a0, a1);
          l += a0 + a1;
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(p_full);
      }
      if (!ok) break;

      // ---- output
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(pv_done, (tile - 1) & 1u, timeout));
      tc_fence_after_sync();
      const bool whole = g.n == g.kt_total;
      const int part = 2 * blockIdx.x + (first ? 0 : 1);   // an item that goes on from the CTA before comes first
      first = false;
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
      for (int c0 = 0; c0 < (idle ? 0 : D); c0 += 32) {
        float o[32];
        tmem_ld_32x32b_x32(o_at + c0, o);
        tmem_ld_wait(o);
        if (there && whole) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + (g.row0 + tok) * a.ldo + head * static_cast<long long>(D) + c0);
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(o[c + 2 * k] * inv, o[c + 2 * k + 1] * inv);
              w[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            dst[c / 8] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (there) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (static_cast<long long>(part) * N + r) * D + c0);
#pragma unroll
          for (int c = 0; c < 32; c += 4) dst[c / 4] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
        }
      }
      if (there && !whole) p.part_ml[static_cast<long long>(part) * N + r] = make_float2(m, l);
      // Header of an item that begins here and goes on in the next CTA.
      open = !whole && g.kt0 == 0;
      if (threadIdx.x == 0 && open) {
        p.heads[2 * blockIdx.x] = make_int4(1, static_cast<int>((g.first + g.kt_total - 1) / run), part, g.rows);
        p.heads[2 * blockIdx.x + 1] = make_int4(g.row0, g.r0, g.h, 0);
      }
      tc_fence_before_sync();
    }
    if (!ok) fail(abort_flag, kStatusEpilogueWait);
    if (threadIdx.x == 0 && (!ok || !open)) p.heads[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    if (!mbar_wait(drained, 0, 2 * timeout)) fail(abort_flag, kStatusTeardownWait);
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// K10: joins the partial sums of the items cut between CTAs.  CTA c of K9 or
// K11 left a header if an item begins in its run and ends in that of CTA c1.
// With few rows several warps share one, each adding every kShare-th part with
// four parts in flight; their sums meet in shared memory in a fixed order.
template <int N>
struct JoinLayout {
  static constexpr int kShare = N == 16 ? 4 : (N == 32 ? 2 : 1);   // warps per row
  static constexpr int kWarps = 8;
  static constexpr int kRows = N == 128 ? 16 : kWarps / kShare;    // rows of a block
};

template <int N, int D>
__global__ void __launch_bounds__(JoinLayout<N>::kWarps * 32) kv_attention_join_kernel(const Params p) {
  using J = JoinLayout<N>;
  constexpr int kPer = D / 32;
  __shared__ float s_o[J::kWarps][D];
  __shared__ float s_l[J::kWarps];
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
    auto part_of = [&](int j) { return static_cast<long long>(j == 0 ? head.z : 2 * (c + j)) * N + row; };
    float m = kNoMax;
    if (there) {
      for (int j = lane; j < parts; j += 32) m = fmaxf(m, p.part_ml[part_of(j)].x);
    }
    m = redux_max(m);
    float o[kPer], sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = 0.f;
    if (there) {
      for (int j0 = share; j0 < parts; j0 += 4 * J::kShare) {
        float2 ml[4];
        float x[4][kPer];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = j0 + u * J::kShare;
          const long long at = part_of(j < parts ? j : j0);
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
          const float w = j0 + u * J::kShare < parts ? ex2(ml[u].x - m) : 0.f;
          sum += w * ml[u].y;
#pragma unroll
          for (int i = 0; i < kPer; ++i) o[i] += w * x[u][i];
        }
      }
    }
    if constexpr (J::kShare > 1) {
      if (share > 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) s_o[warp][lane * kPer + i] = o[i];
        if (lane == 0) s_l[warp] = sum;
      }
      __syncthreads();
      if (share > 0) continue;                        // one round of rows
#pragma unroll
      for (int w = 1; w < J::kShare; ++w) {
        sum += s_l[warp + w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] += s_o[warp + w][lane * kPer + i];
      }
    }
    if (!there) continue;
    const int fr = where.y + row, tok = fr / p.a.group;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    uint16_t* dst = p.a.out + (where.x + tok) * p.a.ldo +
                    (where.z * p.a.group + fr - tok * p.a.group) * static_cast<long long>(D) + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      *reinterpret_cast<__nv_bfloat162*>(dst + i) = __floats2bfloat162_rn(o[i] * inv, o[i + 1] * inv);
    }
  }
}

constexpr int kMaxSms = 160;

// Rows per MMA: the smallest instance that holds the rows of one item, at most 128.
int rows_per_mma(long long rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : 128); }

int ctas_per_sm(int) { return 2; }

size_t part_bytes(int n, int dim) {
  return 2 * static_cast<size_t>(kMaxSms) * ctas_per_sm(n) *
         (static_cast<size_t>(n) * dim * sizeof(float) + n * sizeof(float2) + sizeof(int4));
}

template <int N, int D>
cudaError_t setup_instance() {
  return cudaFuncSetAttribute(kv_attention_kernel<N, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Layout<N, D>::kSmemBytes);
}

template <int N, int D>
cudaError_t launch_instance(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Params& p, int ctas,
                            cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(Layout<N, D>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<N, D>::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kv_attention_kernel<N, D>, tm_k, tm_v, p);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3(ctas, N / JoinLayout<N>::kRows, 1);
  cfg.blockDim = dim3(JoinLayout<N>::kWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_attention_join_kernel<N, D>, p);
}

template <int D, bool kSelected>
cudaError_t setup_rows() {
  return cudaFuncSetAttribute(kv_attention_rows_kernel<D, kSelected>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RowLayout<D>::kSmemBytes);
}

template <int D, bool kSelected>
cudaError_t launch_rows(const CUtensorMap& tm_k, const Params& p, int ctas, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(RowLayout<D>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = RowLayout<D>::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kv_attention_rows_kernel<D, kSelected>, tm_k, p);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3(ctas, 128 / JoinLayout<128>::kRows, 1);
  cfg.blockDim = dim3(JoinLayout<128>::kWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_attention_join_kernel<128, D>, p);
}

}  // namespace

cudaError_t kv_attention_setup_device() {
  cudaError_t err = setup_rows<64, false>();
  if (err == cudaSuccess) err = setup_rows<64, true>();
  if (err == cudaSuccess) err = setup_rows<128, false>();
  if (err == cudaSuccess) err = setup_rows<128, true>();
  if (err == cudaSuccess) err = setup_instance<16, 64>();
  if (err == cudaSuccess) err = setup_instance<32, 64>();
  if (err == cudaSuccess) err = setup_instance<16, 128>();
  if (err == cudaSuccess) err = setup_instance<32, 128>();
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
  Params p;
  p.a = a;
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2 * static_cast<size_t>(ctas) * n * a.kv.dim);
  p.heads = reinterpret_cast<int4*>(p.part_ml + 2 * static_cast<size_t>(ctas) * n);
  p.timeout_ns = timeout_ns;
  if (a.kv.dim == 64) {
    switch (n) {
      case 16: return launch_instance<16, 64>(tm_k, tm_v, p, ctas, stream);
      case 32: return launch_instance<32, 64>(tm_k, tm_v, p, ctas, stream);
      default:
        return a.indices != nullptr ? launch_rows<64, true>(tm_k, p, ctas, stream)
                                    : launch_rows<64, false>(tm_k, p, ctas, stream);
    }
  }
  switch (n) {
    case 16: return launch_instance<16, 128>(tm_k, tm_v, p, ctas, stream);
    case 32: return launch_instance<32, 128>(tm_k, tm_v, p, ctas, stream);
    default:
        return a.indices != nullptr ? launch_rows<128, true>(tm_k, p, ctas, stream)
                                    : launch_rows<128, false>(tm_k, p, ctas, stream);
  }
}

cudaError_t read_kv_status(uint32_t* flags, bool reset) {
  uint32_t v = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_iq_status_kv, sizeof(v));
  if (err != cudaSuccess) return err;
  if (flags) *flags = v;
  if (reset) {
    const uint32_t zero = 0;
    err = cudaMemcpyToSymbol(g_iq_status_kv, &zero, sizeof(zero));
  }
  return err;
}

}  // namespace iq
