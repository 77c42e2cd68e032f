// The router's two ends (include/iq.h, section 5): which experts a token's row
// goes to, and the weighted sum of what comes back.
//
// K14 route_choose_kernel.  A warp per token holds its logits in registers, 32
// experts per register, as integers of the same order.  A lane sorts its own (up to
// 256 experts; see Lane); the k largest are then found one after the other: a
// maximum over the lanes' own largest, then the lowest expert among the lanes that
// hold it.  Softmax sums are float32 over the same registers.
//
// The slots are in (expert, token) order.  A block counts how many of its tokens
// chose each expert; K15 route_place_kernel, a block for the same tokens, takes
// the counts of the blocks before it (with many blocks added up by
// route_prefix_kernel) and of the experts before each expert, and within the block a
// token's rank is the number of lower bits in its expert's mask of tokens.  No
// order of atomics shows.  One block, or a cluster whose blocks read one another's
// counts in shared memory, does all of it in one launch.
//
// Bound by latency and, where an SM has 32 tokens, by the choosing warps'
// instructions.  Per call in a CUDA graph: one token, 64 experts 2.1 us; 256 experts,
// k = 8: 64 tokens 5.4, 512 tokens 6.6, 4632 tokens 10.3 (their logits alone would take
// 0.8), 16384 tokens 23.  Looking through all of a lane's registers again in every
// step, two tokens to a warp: 3.7, 8.7, 10.7, 16.0, 26.4.
//
// K16 combine_kernel.  out = add + sum_j w_j y[slot_j], 8 columns per thread,
// eight rows of a token in flight at a time.  Bound by memory: 4632 tokens of eight
// rows of 7168 columns on top of another (664 MB) 99 us = 6.7 TB/s; 64 tokens 2.8 us.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "iq_kv.h"
#include "iq_moe.h"
#include "iq_ptx.cuh"

namespace iq {

namespace {

constexpr int kFew = 16, kMany = 32;            // tokens of a block, a warp each: bits of the experts' masks
constexpr int kPlaceThreads = 512;
constexpr float kNoScore = -709.78f;             // of less, 1 / (1 + exp(-l)) is 0 in 64 bits too
constexpr int kOneCluster = 8;                   // blocks that can do all of it in one launch

// Entries of a block's counts: four at a time.
__host__ __device__ __forceinline__ int count_stride(int experts) { return (experts + 3) / 4 * 4; }

// Order of the floats as unsigned integers, -0 like +0 and NaN like -inf; no
// float gives 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) != 0u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) != 0u ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, w);
  return v;
}

// exp(x - m) for x <= m, of equal infinities 1.
__device__ __forceinline__ float exp_below(float x, float m) { return x == m ? 1.f : expf(x - m); }

// Far below zero 1 + exp(x) is 1, and exp(-x) soon no float.
__device__ __forceinline__ float sigmoid(float x) { return x < -80.f ? expf(x) : 1.f / (1.f + expf(-x)); }

// The largest of what a lane holds that is left, one after the other.  kRegs up to
// 8: sorted once, so that a step is a shift; with more registers that would be
// dearer than looking through them again.
template <int kRegs, bool kSorted = (kRegs <= 8)>
struct Lane;

template <int kRegs>
struct Lane<kRegs, true> {
  uint32_t v[kRegs];
  uint64_t at;                                       // the registers they came from, four bits each
  __device__ __forceinline__ void begin(const uint32_t (&all)[kRegs]) {
    uint32_t from[kRegs];
#pragma unroll
    for (int i = 0; i < kRegs; ++i) v[i] = all[i], from[i] = i;
    // Odd-even merge sort, falling, equal ones by register.
#pragma unroll
    for (int p = 1; p < kRegs; p *= 2) {
#pragma unroll
      for (int q = p; q > 0; q /= 2) {
#pragma unroll
        for (int j = q % p; j + q < kRegs; j += 2 * q) {
#pragma unroll
          for (int i = 0; i < q; ++i) {
            const int lo = i + j, hi = i + j + q;
            if (hi < kRegs && lo / (2 * p) == hi / (2 * p)) {
              const bool swap = v[lo] < v[hi] || (v[lo] == v[hi] && from[lo] > from[hi]);
              const uint32_t a = swap ? v[hi] : v[lo], b = swap ? v[lo] : v[hi];
              const uint32_t c = swap ? from[hi] : from[lo], d = swap ? from[lo] : from[hi];
              v[lo] = a, v[hi] = b, from[lo] = c, from[hi] = d;
            }
          }
        }
      }
    }
    at = 0;
#pragma unroll
    for (int i = 0; i < kRegs; ++i) at |= static_cast<uint64_t>(from[i]) << (4 * i);
  }
  __device__ __forceinline__ uint32_t best() const { return v[0]; }
  __device__ __forceinline__ int expert(int lane) const { return 32 * static_cast<int>(at & 15) + lane; }
  __device__ __forceinline__ void pop(bool mine) {
#pragma unroll
    for (int i = 0; i < kRegs; ++i) v[i] = mine ? (i + 1 < kRegs ? v[i + 1] : 0u) : v[i];
    at = mine ? at >> 4 : at;
  }
};

template <int kRegs>
struct Lane<kRegs, false> {
  uint32_t v[kRegs];
  uint32_t taken, top;                               // registers that are gone, the largest that is left
  int from;
  __device__ __forceinline__ void look() {           // the lowest register of equal ones
    top = 0u;
    from = 0;
#pragma unroll
    for (int i = 0; i < kRegs; ++i) {
      if ((taken >> i & 1u) == 0u && v[i] > top) {
        top = v[i];
        from = i;
      }
    }
  }
  __device__ __forceinline__ void begin(const uint32_t (&all)[kRegs]) {
#pragma unroll
    for (int i = 0; i < kRegs; ++i) v[i] = all[i];
    taken = 0u;
    look();
  }
  __device__ __forceinline__ uint32_t best() const { return top; }
  __device__ __forceinline__ int expert(int lane) const { return 32 * from + lane; }
  __device__ __forceinline__ void pop(bool mine) {
    if (mine) {
      taken |= 1u << from;
      look();
    }
  }
};

// The experts and weights of token t, by a warp; lane j < k gets expert j.  kRegs:
// 32 experts each.
template <int kRegs>
__device__ __forceinline__ int choose(const RouteArgs& a, int t) {
  const int lane = threadIdx.x & 31;
  uint32_t v[kRegs];
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    const int e = 32 * i + lane;
    v[i] = 0u;
    if (e < a.experts) {
      const long long at = static_cast<long long>(t) * a.ld + e;
      v[i] = ordered(a.bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.logits)[at]) << 16)
                            : static_cast<const float*>(a.logits)[at]);
    }
  }
  Lane<kRegs> left;
  left.begin(v);
  float sum = 0.f;                                   // of this lane's, if all experts count
  if (!a.sigmoid && !a.normalize) {
    const float m = from_ordered(__reduce_max_sync(0xFFFFFFFFu, left.best()));
#pragma unroll
    for (int i = 0; i < kRegs; ++i) sum += left.v[i] != 0u ? exp_below(from_ordered(left.v[i]), m) : 0.f;
  }
  int mine = 0;
  uint32_t mine_v = 0u;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, left.best());
    const int own = left.expert(lane);
    const int e = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, left.best() == top ? static_cast<uint32_t>(own) : 0xFFFFFFFFu));
    if (lane == j) {
      mine = e;
      mine_v = top;
    }
    left.pop((e & 31) == lane);
  }
  const bool there = lane < a.k;
  const float x = from_ordered(mine_v);
  float w = 0.f, total = 1.f;
  if (a.sigmoid) {
    // Shares of scores far below zero are those of exp(x): to float32's precision from
    // -40 on, while the scores themselves end at -103.  Beyond kNoScore they are 0.
    const float m = __shfl_sync(0xFFFFFFFFu, x, 0);
    const bool far = a.normalize && m < -40.f;
    w = there && !(far && m < kNoScore) ? (far ? exp_below(x, m) : sigmoid(x)) : 0.f;
    if (a.normalize) total = warp_add(w);
  } else {
    const float m = __shfl_sync(0xFFFFFFFFu, x, 0);
    if (m != -INFINITY) {                              // (else no expert is left: weights 0)
      w = there ? exp_below(x, m) : 0.f;
      total = warp_add(a.normalize ? w : sum);
    }
  }
  if (there) {
    const long long at = static_cast<long long>(t) * a.k + lane;
    a.weights[at] = total > 0.f ? w / total * a.scale : 0.f;
    a.out_experts[at] = mine;
  }
  return mine;
}

// The places of the block's n pairs among the slots: s_mask [experts] holds who
// chose what, s_base [experts] the slots before the block's own.
template <int kThreads>
__device__ __forceinline__ void place(const RouteArgs& a, const uint32_t* s_mask, const int* s_base, int t0, int n) {
  const int32_t* mine = a.out_experts + static_cast<long long>(t0) * a.k;
  int32_t* slots = a.slots + static_cast<long long>(t0) * a.k;
  for (int s = threadIdx.x; s < n; s += kThreads) {
    const int i = s / a.k, e = mine[s];
    const int rank = s_base[e] + __popc(s_mask[e] & ((1u << i) - 1u));
    slots[s] = rank;
    a.rows[rank] = t0 + i;
  }
}

// Exclusive sums of s_count [experts] over the experts, by the whole block, into
// s_base (added to what stands there) and, by block 0, into row_start.
template <int kThreads>
__device__ __forceinline__ void add_starts(const RouteArgs& a, const int* s_count, int* s_base, int* s_warp) {
  constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int own[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    own[i] = e < a.experts ? s_count[e] : 0;
    sum += own[i];
  }
  int upto = sum;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, upto, w);
    if (lane >= w) upto += o;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int before = upto - sum;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e < a.experts) {
      s_base[e] += before;
      if (blockIdx.x == 0) a.row_start[e] = before;
    }
    before += own[i];
    if (e == a.experts - 1 && blockIdx.x == 0) a.row_start[a.experts] = before;
  }
  __syncthreads();
}

// Threads of K15 that share the adding up of four experts' counts.
__host__ __device__ __forceinline__ int place_share(int experts) {
  const int share = kPlaceThreads / (count_stride(experts) / 4);
  return share < 16 ? share : 16;
}

// How far a block's tokens are from being all of them.
enum Scope { kBlock, kCluster, kGrid };

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int kRegs, Scope kScope, int kTokens>
__global__ void __launch_bounds__(kTokens * 32) route_choose_kernel(const RouteArgs a) {
  __shared__ int s_count[kMaxGroups];
  __shared__ uint32_t s_mask[kScope != kGrid ? kMaxGroups : 1];
  __shared__ int s_base[kScope != kGrid ? kMaxGroups : 1];
  __shared__ int s_total[kScope == kCluster ? kMaxGroups : 1];
  __shared__ int s_warp[kTokens];
  constexpr int kThreads = kTokens * 32;
  grid_launch_dependents();
  for (int e = threadIdx.x; e < a.experts; e += kThreads) {
    s_count[e] = 0;
    if constexpr (kScope != kGrid) {
      s_base[e] = 0;
      s_mask[e] = 0u;
    }
  }
  __syncthreads();
  grid_dependency_wait();
  const int t0 = blockIdx.x * kTokens, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (t0 + warp < a.tokens) {
    const int e = choose<kRegs>(a, t0 + warp);
    if (lane < a.k) {
      atomicAdd(&s_count[e], 1);
      if constexpr (kScope != kGrid) atomicOr(&s_mask[e], 1u << warp);
    }
  }
  if constexpr (kScope == kGrid) {
    __syncthreads();
    const int stride = count_stride(a.experts);
    int* to = a.counts + static_cast<long long>(blockIdx.x) * stride;
    for (int e = threadIdx.x; e < stride; e += kThreads) to[e] = e < a.experts ? s_count[e] : 0;
  } else if constexpr (kScope == kCluster) {
    // The counts of the cluster's blocks before this one, and of all.
    __syncwarp();
    cluster_sync_all();
    const int rank = static_cast<int>(cluster_ctarank()), blocks = gridDim.x;
    for (int e = threadIdx.x; e < a.experts; e += kThreads) {
      int before = 0, total = 0;
#pragma unroll
      for (int r = 0; r < kOneCluster; ++r) {
        if (r < blocks) {
          const int v = ld_cluster(mapa_shared(smem_u32(&s_count[e]), r));
          total += v;
          before += r < rank ? v : 0;
        }
      }
      s_base[e] = before;
      s_total[e] = total;
    }
    __syncwarp();
    cluster_arrive_release();                          // no block leaves before all have read its counts
  }
  if constexpr (kScope != kGrid) {
    __syncthreads();
    add_starts<kThreads>(a, kScope == kCluster ? s_total : s_count, s_base, s_warp);
    place<kThreads>(a, s_mask, s_base, t0, min(kTokens, a.tokens - t0) * a.k);   // experts written by this block
  }
  if constexpr (kScope == kCluster) {
    __syncwarp();
    cluster_wait();
  }
}

// With many blocks: each expert's counts replaced by those of the blocks before,
// and behind the last block its total.  A block takes four experts.
constexpr int kPrefixThreads = 256;

__global__ void __launch_bounds__(kPrefixThreads) route_prefix_kernel(const RouteArgs a, int blocks) {
  __shared__ int4 s_warp[kPrefixThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int quads = count_stride(a.experts) / 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int4* at = reinterpret_cast<int4*>(a.counts) + blockIdx.x;
  int4 sum = make_int4(0, 0, 0, 0);                    // of the pieces before
  for (int b0 = 0; b0 < blocks; b0 += kPrefixThreads) {
    const int b = b0 + threadIdx.x;
    const int4 own = b < blocks ? at[static_cast<long long>(b) * quads] : make_int4(0, 0, 0, 0);
    int4 v = own;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, v.x, w), y = __shfl_up_sync(0xFFFFFFFFu, v.y, w);
      const int z = __shfl_up_sync(0xFFFFFFFFu, v.z, w), u = __shfl_up_sync(0xFFFFFFFFu, v.w, w);
      if (lane >= w) v.x += x, v.y += y, v.z += z, v.w += u;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    int4 before = sum;
    for (int w = 0; w < kPrefixThreads / 32; ++w) {
      const int4 o = s_warp[w];
      if (w < warp) before.x += o.x, before.y += o.y, before.z += o.z, before.w += o.w;
      sum.x += o.x, sum.y += o.y, sum.z += o.z, sum.w += o.w;
    }
    if (b < blocks) {
      at[static_cast<long long>(b) * quads] =
          make_int4(before.x + v.x - own.x, before.y + v.y - own.y, before.z + v.z - own.z, before.w + v.w - own.w);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) at[static_cast<long long>(blocks) * quads] = sum;
}

// kPrefixed: route_prefix_kernel has been there.
template <bool kPrefixed>
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const RouteArgs a) {
  __shared__ int s_count[kMaxGroups];
  __shared__ uint32_t s_mask[kMaxGroups];
  __shared__ int s_base[kMaxGroups];
  __shared__ int s_warp[kPlaceThreads / 32];
  grid_launch_dependents();
  for (int e = threadIdx.x; e < a.experts; e += kPlaceThreads) {
    s_count[e] = 0;
    s_base[e] = 0;
    s_mask[e] = 0u;
  }
  __syncthreads();
  grid_dependency_wait();
  const int t0 = blockIdx.x * a.block_tokens, blocks = gridDim.x;
  const int n = min(a.block_tokens, a.tokens - t0) * a.k;
  const int32_t* mine = a.out_experts + static_cast<long long>(t0) * a.k;
  for (int s = threadIdx.x; s < n; s += kPlaceThreads) {
    const int i = s / a.k;
    atomicOr(&s_mask[mine[s]], 1u << i);
  }
  if constexpr (kPrefixed) {
    const long long stride = count_stride(a.experts);
    for (int e = threadIdx.x; e < a.experts; e += kPlaceThreads) {
      s_base[e] = a.counts[blockIdx.x * stride + e];
      s_count[e] = a.counts[blocks * stride + e];
    }
  } else {
    // Counts of all blocks and of those before this one: a thread adds up four
    // experts, several threads share them where there are few.
    const int quads = count_stride(a.experts) / 4, share = place_share(a.experts);
    const int q = threadIdx.x % quads, part = threadIdx.x / quads;
    if (part < share) {
      int4 all = make_int4(0, 0, 0, 0), before = all;
      const int4* from = reinterpret_cast<const int4*>(a.counts) + q;
#pragma unroll 8
      for (int b = part; b < blocks; b += share) {
        const int4 c = from[static_cast<long long>(b) * quads];
        const int m = b < static_cast<int>(blockIdx.x) ? -1 : 0;
        all.x += c.x, all.y += c.y, all.z += c.z, all.w += c.w;
        before.x += c.x & m, before.y += c.y & m, before.z += c.z & m, before.w += c.w & m;
      }
      const int sum[4] = {all.x, all.y, all.z, all.w}, lower[4] = {before.x, before.y, before.z, before.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * q + i < a.experts) {
          atomicAdd(&s_count[4 * q + i], sum[i]);
          atomicAdd(&s_base[4 * q + i], lower[i]);
        }
      }
    }
  }
  __syncthreads();
  add_starts<kPlaceThreads>(a, s_count, s_base, s_warp);
  place<kPlaceThreads>(a, s_mask, s_base, t0, n);
}

// ---- combination

constexpr int kCombineThreads = 128;

__device__ __forceinline__ void add_scaled(float* o, uint4 v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), o[2 * i]);
    o[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xFFFF0000u), o[2 * i + 1]);
  }
}

// Read once.  (Not by the read-only path: the kernel before this one, which may
// write it, is still running when this one starts.)
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineArgs a) {
  constexpr int kAtOnce = 8;
  grid_launch_dependents();
  grid_dependency_wait();
  const unsigned t = blockIdx.y + blockIdx.z * 65535u;      // past the last token up to 2^31 + 65534
  const int col = (blockIdx.x * kCombineThreads + threadIdx.x) * 8;
  if (t >= static_cast<unsigned>(a.tokens) || col >= a.cols) return;
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  if (a.add != nullptr) add_scaled(o, *reinterpret_cast<const uint4*>(a.add + t * a.ld_add + col), 1.f);
  const int32_t* slots = a.slots + static_cast<long long>(t) * a.k;
  const float* weights = a.weights + static_cast<long long>(t) * a.k;
  for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
    uint4 v[kAtOnce];
    float w[kAtOnce];
    bool there[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int s = j0 + j < a.k ? slots[j0 + j] : -1;
      there[j] = static_cast<unsigned>(s) < static_cast<unsigned>(a.rows);
      w[j] = there[j] ? weights[j0 + j] : 0.f;
      if (there[j]) v[j] = ld_once_v4(a.y + s * a.ldy + col);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (there[j]) add_scaled(o, v[j], w[j]);
    }
  }
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(a.out + t * a.ld_out + col) = make_uint4(r[0], r[1], r[2], r[3]);
}

// Blocks up to which each adds up the counts of all the others itself; with more,
// a kernel between does (256 experts: 512 tokens, 32 blocks, 6.6 us; 1024 tokens, 64
// blocks, 7.8 without it and 7.4 with; 64 experts, 64 blocks, 5.2 and 5.9, 128 blocks
// 6.9 and 6.4).
int summed_blocks(int experts) {
  const int blocks = 4 * place_share(experts);
  return blocks > 32 ? blocks : 32;
}

// Few tokens to a block while an SM has one block at most (256 experts: 1024 tokens
// 7.4 us, with kMany to a block 8.2; 2048 tokens 8.2 and 9.8).
constexpr int kFewTokens = 2048;
int block_tokens(int tokens) { return tokens <= kFewTokens ? kFew : kMany; }
int route_blocks(int tokens) { return (tokens + block_tokens(tokens) - 1) / block_tokens(tokens); }

// Shared memory that keeps a second block off an SM: the choosing warps' instructions
// bound it, so two blocks on one SM, another idle, take twice as long (4632 tokens,
// 256 experts: 13.9 us, with it 10.4).
constexpr int kSpread = 120 * 1024;

template <int kRegs, int kTokens>
cudaError_t launch_places(const RouteArgs& a, int sm_count, cudaStream_t stream) {
  const int blocks = route_blocks(a.tokens);
  cudaError_t err = launch_dependent(route_choose_kernel<kRegs, kGrid, kTokens>, dim3(blocks), kTokens * 32,
                                     blocks <= sm_count ? kSpread : 0, stream, a);
  if (err != cudaSuccess) return err;
  if (blocks <= summed_blocks(a.experts)) return launch_dependent(route_place_kernel<false>, dim3(blocks), kPlaceThreads, 0, stream, a);
  err = launch_dependent(route_prefix_kernel, dim3(count_stride(a.experts) / 4), kPrefixThreads, 0, stream, a, blocks);
  if (err != cudaSuccess) return err;
  return launch_dependent(route_place_kernel<true>, dim3(blocks), kPlaceThreads, 0, stream, a);
}

template <int kRegs>
cudaError_t launch_choose(const RouteArgs& a, int sm_count, cudaStream_t stream) {
  const int blocks = route_blocks(a.tokens);
  if (a.block_tokens == kMany) return launch_places<kRegs, kMany>(a, sm_count, stream);
  if (blocks == 1) return launch_dependent(route_choose_kernel<kRegs, kBlock, kFew>, dim3(1), kFew * 32, 0, stream, a);
  if (blocks > kOneCluster) return launch_places<kRegs, kFew>(a, sm_count, stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kFew * 32, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, route_choose_kernel<kRegs, kCluster, kFew>, a);
}

template <int kRegs>
cudaError_t set_spread() {
  const cudaError_t err =
      cudaFuncSetAttribute(route_choose_kernel<kRegs, kGrid, kFew>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpread);
  if (err != cudaSuccess) return err;
  return cudaFuncSetAttribute(route_choose_kernel<kRegs, kGrid, kMany>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpread);
}

}  // namespace

cudaError_t route_setup_device() {
  for (cudaError_t err : {set_spread<2>(), set_spread<8>(), set_spread<16>(), set_spread<32>()}) {
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// Past kFewTokens blocks are larger and at first fewer; the size does not fall there.
size_t route_workspace(int tokens, int experts) {
  const int blocks = tokens <= kFewTokens ? route_blocks(tokens) : std::max(route_blocks(tokens), route_blocks(kFewTokens));
  return blocks <= kOneCluster ? 0 : (static_cast<size_t>(blocks) + 1) * count_stride(experts) * sizeof(int);
}

cudaError_t launch_route(RouteArgs a, int sm_count, cudaStream_t stream) {
  a.block_tokens = block_tokens(a.tokens);
  const int regs = (a.experts + 31) / 32;
  if (regs <= 2) return launch_choose<2>(a, sm_count, stream);
  if (regs <= 8) return launch_choose<8>(a, sm_count, stream);
  if (regs <= 16) return launch_choose<16>(a, sm_count, stream);
  return launch_choose<32>(a, sm_count, stream);
}

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream) {
  const int rows = a.tokens < 65535 ? a.tokens : 65535;
  return launch_dependent(combine_kernel, dim3((a.cols / 8 + kCombineThreads - 1) / kCombineThreads, rows, (a.tokens + 65534) / 65535),
                          kCombineThreads, 0, stream, a);
}

}  // namespace iq
