// Helpers of the kernels that reduce a row of logits: packed (value, index)
// keys, the base-2 log-sum-exp state, and sorting networks over a warp.
#pragma once

#include "ddt_common.cuh"

namespace ddt {

// loads from shared memory of a CTA of the cluster (address from map_to_rank)
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ unsigned long long topk_key(float v, int idx) {
  return (static_cast<unsigned long long>(float_order_key(v)) << 32) |
         static_cast<unsigned long long>(~static_cast<uint32_t>(idx));
}

__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

constexpr float kLog2e = 1.4426950408889634f;

// 2^x by the hardware approximation (relative error about 2^-22; subnormal
// results flushed to zero)
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log-sum-exp state in base 2: m = running max of x log2(e), s = sum of
// 2^(x log2(e) - m)
__device__ __forceinline__ void lse_merge(float& m, float& s, float m2, float s2) {
  const float M = fmaxf(m, m2);
  if (M == -INFINITY) return;
  s = (m == -INFINITY ? 0.0f : s * ex2_ftz(m - M)) + (m2 == -INFINITY ? 0.0f : s2 * ex2_ftz(m2 - M));
  m = M;
}

// Bitonic network over the warp's 32 lanes, one key per lane: the full sort
// leaves lane 0 with the largest key; the merge sorts a bitonic sequence.
__device__ __forceinline__ unsigned long long warp_sort_desc(unsigned long long x, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const unsigned long long y = __shfl_xor_sync(DDT_FULL_MASK, x, j);
      // blocks of k lanes alternate direction; the lower lane of a pair keeps
      // the larger key in a descending block
      const bool keep_max = ((lane & j) == 0) == ((lane & k) == 0);
      x = keep_max ? (y > x ? y : x) : (y < x ? y : x);
    }
  }
  return x;
}

__device__ __forceinline__ unsigned long long warp_merge_desc(unsigned long long x, int lane) {
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const unsigned long long y = __shfl_xor_sync(DDT_FULL_MASK, x, j);
    x = ((lane & j) == 0) ? (y > x ? y : x) : (y < x ? y : x);
  }
  return x;
}

}  // namespace ddt
