// Attention over the paged 8-bit KV cache (include/iq.h, section 4).
//
// K9 kv_attention_kernel.  One warp per (row, query head) walks the row's keys
// 32 at a time: lane j looks up key j's page and scales, the warp forms the 32
// dot products one key after the other (each lane holds dim / 32 dimensions),
// lane j keeps key j's score, and the softmax is carried along as a running
// maximum and sum (base 2, float32).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "iq_internal.h"
#include "iq_kv.h"
#include "iq_ptx.cuh"

namespace iq {

namespace {

constexpr int kSimpleWarps = 4;

template <int kDim>
__global__ void __launch_bounds__(kSimpleWarps * 32) kv_attention_kernel(AttnArgs a) {
  constexpr int kPer = kDim / 32;   // dimensions per lane: 2 or 4
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int hq = blockIdx.x * kSimpleWarps + (threadIdx.x >> 5);
  const int t = blockIdx.y + blockIdx.z * 32768;
  if (hq >= a.q_heads || t >= a.kv.num_rows) return;
  const int h = hq / a.group;
  const int b = kv_find_seq(a.kv, t);
  int visible = 0;
  if (b < a.kv.num_seqs) visible = max(0, a.kv.kv_len[b] - a.kv.row_start[b + 1] + t + 1);
  const int n = a.indices != nullptr ? a.topk : visible;
  float q[kPer], o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.ldq + hq * kDim + lane * kPer + i]) << 16);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int s0 = 0; s0 < n; s0 += 32) {
    int pos = s0 + lane < n ? s0 + lane : -1;
    if (a.indices != nullptr && pos >= 0) pos = a.indices[t * a.ld_idx + pos];
    if (pos >= visible) pos = -1;
    const int pid = b < a.kv.num_seqs ? kv_page_of(a.kv, b, pos) : -1;
    const long long tile = static_cast<long long>(pid) * a.kv.heads + h;
    const long long at = (tile * a.kv.page + (pos & (a.kv.page - 1))) * kDim;
    const float kf = pid >= 0 ? ue8m0_to_float(a.kv.sf[0][tile]) : 0.f;
    const float vf = pid >= 0 ? ue8m0_to_float(a.kv.sf[1][tile]) : 0.f;
    const uint32_t ok = __ballot_sync(0xFFFFFFFFu, pid >= 0);
    if (ok == 0) continue;
    float score = -INFINITY;
    for (uint32_t todo = ok; todo != 0; todo &= todo - 1) {
      const int j = __ffs(todo) - 1;
      const uint8_t* k = a.kv.codes[0] + __shfl_sync(0xFFFFFFFFu, at, j) + lane * kPer;
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) d += q[i] * e4m3_to_float(k[i]);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, w);
      if (lane == j) score = d * kf * a.scale_log2;
    }
    float mx = score;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
    const float m_new = fmaxf(m, mx);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float p = exp2f(score - base), c = exp2f(m - base);
    m = m_new;
    l = l * c + p;   // this lane's share of the sum
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] *= c;
    const float pv = p * vf;
    for (uint32_t todo = ok; todo != 0; todo &= todo - 1) {
      const int j = __ffs(todo) - 1;
      const uint8_t* v = a.kv.codes[1] + __shfl_sync(0xFFFFFFFFu, at, j) + lane * kPer;
      const float w = __shfl_sync(0xFFFFFFFFu, pv, j);
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[i] += w * e4m3_to_float(v[i]);
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, w);
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    a.out[t * a.ldo + hq * kDim + lane * kPer + i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
  }
}

}  // namespace

cudaError_t launch_kv_attention(const AttnArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.q_heads + kSimpleWarps - 1) / kSimpleWarps, a.kv.num_rows < 32768 ? a.kv.num_rows : 32768,
                     (a.kv.num_rows + 32767) / 32768);
  cfg.blockDim = dim3(kSimpleWarps * 32, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.kv.dim == 64 ? cudaLaunchKernelEx(&cfg, kv_attention_kernel<64>, a)
                        : cudaLaunchKernelEx(&cfg, kv_attention_kernel<128>, a);
}

}  // namespace iq
