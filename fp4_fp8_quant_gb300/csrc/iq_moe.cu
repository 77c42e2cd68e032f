// The router's two ends (include/iq.h, section 5): which experts a token's row
// goes to, and the weighted sum of what comes back.
//
// K14 route_choose_kernel.  A warp per token holds its logits in registers, 32
// experts per register, as integers of the same order.  The k largest are found
// one after the other: a maximum over the lanes' own maxima, then the lowest
// expert among the lanes that hold it; only the lane that gave it up looks
// through its registers again.  Softmax sums are float32 over the same registers.
//
// The slots are in (expert, token) order.  A block counts how many of its 32 tokens
// chose each expert; K15 route_place_kernel, a block for the same tokens, takes
// the counts of the blocks before it (with many blocks added up by
// route_prefix_kernel) and of the experts before each expert, and within the block a
// token's rank is the number of lower bits in its expert's mask of tokens.  No
// order of atomics shows.  Up to 32 tokens one block does all of it in one launch
// (64 tokens in one block took 18 us, two blocks and two launches take 14).
//
// Bound by latency: 8 us for one token, 64 experts, 17 us for 4632 tokens, 256
// experts (their logits alone would take 0.8); 34 us for 16384, where the choosing
// warps' instructions bound it.
//
// K16 combine_kernel.  out = add + sum_j w_j y[slot_j], 8 columns per thread,
// eight rows of a token in flight at a time.  Bound by memory: 4632 tokens of eight
// rows of 7168 columns on top of another (664 MB) 99 us = 6.7 TB/s; 64 tokens 2.8 us.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "iq_fp8.cuh"
#include "iq_kv.h"
#include "iq_moe.h"
#include "iq_ptx.cuh"

namespace iq {

namespace {

constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteTokens = 32;                 // of a block: a bit each in the experts' masks

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

// The experts and weights of kSide tokens t, t + kRouteWarps, ..., one after the
// other's step so that their latencies overlap (those past the last are not
// written); lane j < k gets expert j of each.  kRegs: 32 experts each.
template <int kRegs, int kSide>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, int (&mine)[kSide]) {
  const int lane = threadIdx.x & 31;
  uint32_t v[kSide][kRegs], best[kSide], mine_v[kSide];
  uint32_t taken[kSide];                             // this lane's registers that are gone
  int best_e[kSide];
#pragma unroll
  for (int s = 0; s < kSide; ++s) {
    const int row = min(t + s * kRouteWarps, a.tokens - 1);
#pragma unroll
    for (int i = 0; i < kRegs; ++i) {
      const int e = 32 * i + lane;
      v[s][i] = 0u;
      if (e < a.experts) {
        const long long at = static_cast<long long>(row) * a.ld + e;
        v[s][i] = ordered(a.bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.logits)[at]) << 16)
                                 : static_cast<const float*>(a.logits)[at]);
      }
    }
  }
  auto look = [&](int s) {                           // the lane's largest that is left, the lowest of equal ones
    best[s] = 0u;
    best_e[s] = lane;
#pragma unroll
    for (int i = 0; i < kRegs; ++i) {
      if ((taken[s] >> i & 1u) == 0u && v[s][i] > best[s]) {
        best[s] = v[s][i];
        best_e[s] = 32 * i + lane;
      }
    }
  };
#pragma unroll
  for (int s = 0; s < kSide; ++s) {
    taken[s] = 0u;
    mine[s] = 0;
    mine_v[s] = 0u;
    look(s);
  }
  for (int j = 0; j < a.k; ++j) {
#pragma unroll
    for (int s = 0; s < kSide; ++s) {
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best[s]);
      const int e = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, best[s] == top ? static_cast<uint32_t>(best_e[s]) : 0xFFFFFFFFu));
      if (lane == j) {
        mine[s] = e;
        mine_v[s] = top;
      }
      if ((e & 31) == lane) {
        taken[s] |= 1u << (e >> 5);
        look(s);
      }
    }
  }
  const bool there = lane < a.k;
#pragma unroll
  for (int s = 0; s < kSide; ++s) {
    const float x = from_ordered(mine_v[s]);
    float w = 0.f, total = 1.f;
    if (a.sigmoid) {
      w = there ? 1.f / (1.f + expf(-x)) : 0.f;
      if (a.normalize) total = warp_add(w);
    } else {
      const float m = __shfl_sync(0xFFFFFFFFu, x, 0);
      if (m != -INFINITY) {                            // (else no expert is left: weights 0)
        w = there ? exp_below(x, m) : 0.f;
        if (a.normalize) {
          total = warp_add(w);
        } else {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < kRegs; ++i) sum += v[s][i] != 0u ? exp_below(from_ordered(v[s][i]), m) : 0.f;
          total = warp_add(sum);
        }
      }
    }
    if (there && t + s * kRouteWarps < a.tokens) {
      const long long at = static_cast<long long>(t + s * kRouteWarps) * a.k + lane;
      a.weights[at] = total > 0.f ? w / total * a.scale : 0.f;
      a.out_experts[at] = mine[s];
    }
  }
}

// The place of the block's tokens among the slots: s_mask [experts] holds who
// chose what, s_base [experts] the slots before the block's own.
__device__ __forceinline__ void place(const RouteArgs& a, const uint32_t* s_mask, const int* s_base, int t, int j, int e) {
  const int rank = s_base[e] + __popc(s_mask[e] & ((1u << (t % kRouteTokens)) - 1u));
  a.slots[static_cast<long long>(t) * a.k + j] = rank;
  a.rows[rank] = t;
}

// Exclusive sums of s_count [experts] over the experts, by the whole block, into
// s_base (added to what stands there) and, by block 0, into row_start.
__device__ __forceinline__ void add_starts(const RouteArgs& a, const int* s_count, int* s_base, int* s_warp) {
  constexpr int kPer = kMaxGroups / kRouteThreads;
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

template <int kRegs, bool kOne>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const RouteArgs a) {
  __shared__ int s_count[kMaxGroups];
  __shared__ uint32_t s_mask[kOne ? kMaxGroups : 1];
  __shared__ int s_base[kOne ? kMaxGroups : 1];
  __shared__ int s_warp[kRouteWarps];
  grid_launch_dependents();
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
    s_count[e] = 0;
    if constexpr (kOne) {
      s_base[e] = 0;
      s_mask[e] = 0u;
    }
  }
  __syncthreads();
  grid_dependency_wait();
  const int t0 = blockIdx.x * kRouteTokens, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kSide = kRegs <= 8 ? 2 : 1;
  for (int i = warp; i < kRouteTokens && t0 + i < a.tokens; i += kSide * kRouteWarps) {
    int e[kSide];
    choose<kRegs, kSide>(a, t0 + i, e);
#pragma unroll
    for (int s = 0; s < kSide; ++s) {
      const int at = i + s * kRouteWarps;
      if (lane < a.k && t0 + at < a.tokens) {
        atomicAdd(&s_count[e[s]], 1);
        if constexpr (kOne) atomicOr(&s_mask[e[s]], 1u << at);
      }
    }
  }
  __syncthreads();
  if constexpr (kOne) {
    add_starts(a, s_count, s_base, s_warp);
    for (int s = threadIdx.x; s < a.tokens * a.k; s += kRouteThreads) {
      const int t = s / a.k;
      place(a, s_mask, s_base, t, s - t * a.k, a.out_experts[s]);       // written by this block
    }
  } else {
    const int stride = count_stride(a.experts);
    int* to = a.counts + static_cast<long long>(blockIdx.x) * stride;
    for (int e = threadIdx.x; e < stride; e += kRouteThreads) to[e] = e < a.experts ? s_count[e] : 0;
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
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const RouteArgs a) {
  __shared__ int s_count[kMaxGroups];
  __shared__ uint32_t s_mask[kMaxGroups];
  __shared__ int s_base[kMaxGroups];
  __shared__ int s_warp[kRouteWarps];
  grid_launch_dependents();
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
    s_count[e] = 0;
    s_base[e] = 0;
    s_mask[e] = 0u;
  }
  __syncthreads();
  grid_dependency_wait();
  const int t0 = blockIdx.x * kRouteTokens, blocks = gridDim.x;
  const int n = min(kRouteTokens, a.tokens - t0) * a.k;
  const int32_t* mine = a.out_experts + static_cast<long long>(t0) * a.k;
  for (int s = threadIdx.x; s < n; s += kRouteThreads) {
    const int i = s / a.k;
    atomicOr(&s_mask[mine[s]], 1u << i);
  }
  if constexpr (kPrefixed) {
    const long long stride = count_stride(a.experts);
    for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
      s_base[e] = a.counts[blockIdx.x * stride + e];
      s_count[e] = a.counts[blocks * stride + e];
    }
  } else {
    // Counts of all blocks and of those before this one: a thread adds up four
    // experts, several threads share them where there are few.
    const int quads = count_stride(a.experts) / 4, share = kRouteThreads / quads;
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
  add_starts(a, s_count, s_base, s_warp);
  for (int s = threadIdx.x; s < n; s += kRouteThreads) {
    const int i = s / a.k;
    place(a, s_mask, s_base, t0 + i, s - i * a.k, mine[s]);
  }
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
      if (there[j]) v[j] = ld_stream_v4(a.y + s * a.ldy + col);
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
// a kernel between does (256 experts, 4632 tokens: 20.5 us without it, 17.4 with;
// 1024 tokens 16.4 with either).
constexpr int kSummedBlocks = 64;

int route_blocks(int tokens) { return (tokens + kRouteTokens - 1) / kRouteTokens; }

template <int kRegs>
cudaError_t launch_choose(const RouteArgs& a, cudaStream_t stream) {
  const int blocks = route_blocks(a.tokens);
  if (blocks == 1) return launch_dependent(route_choose_kernel<kRegs, true>, dim3(1), kRouteThreads, 0, stream, a);
  cudaError_t err = launch_dependent(route_choose_kernel<kRegs, false>, dim3(blocks), kRouteThreads, 0, stream, a);
  if (err != cudaSuccess) return err;
  if (blocks <= kSummedBlocks) return launch_dependent(route_place_kernel<false>, dim3(blocks), kRouteThreads, 0, stream, a);
  err = launch_dependent(route_prefix_kernel, dim3(count_stride(a.experts) / 4), kPrefixThreads, 0, stream, a, blocks);
  if (err != cudaSuccess) return err;
  return launch_dependent(route_place_kernel<true>, dim3(blocks), kRouteThreads, 0, stream, a);
}

}  // namespace

size_t route_workspace(int tokens, int experts) {
  const int blocks = route_blocks(tokens);
  return blocks <= 1 ? 0 : (static_cast<size_t>(blocks) + 1) * count_stride(experts) * sizeof(int);
}

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  const int regs = (a.experts + 31) / 32;
  if (regs <= 2) return launch_choose<2>(a, stream);
  if (regs <= 8) return launch_choose<8>(a, stream);
  if (regs <= 16) return launch_choose<16>(a, stream);
  return launch_choose<32>(a, stream);
}

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream) {
  const int rows = a.tokens < 65535 ? a.tokens : 65535;
  return launch_dependent(combine_kernel, dim3((a.cols / 8 + kCombineThreads - 1) / kCombineThreads, rows, (a.tokens + 65534) / 65535),
                          kCombineThreads, 0, stream, a);
}

}  // namespace iq
