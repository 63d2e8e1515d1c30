// Accumulated attention weight of cached rows, CUDA-core form (float32
// arithmetic, any d_qk <= 1024): float32 inputs, and the bf16 shapes that the
// tensor-core kernel does not cover.
//
// What it computes is fixed in ddt.h (ddt_cache_weights): for every cached
// row j, sum over the selected verify rows r of e^(scale q_r . k_j - lse_r).
//
// A CTA owns 64 keys of a request and walks the request's query rows 32 at a
// time: a 64 x 32 tile of dot products in registers (4 keys x 2 rows per
// thread), operands staged through shared memory 32 dims at a time. Each key
// belongs to one CTA, so its sum is formed in a fixed order (per thread over
// the row tiles, then over the 16 threads that share the key) without
// atomics. Bound by the FMA rate for long row lists, by latency for short ones.
#include <algorithm>

#include "ddt_kernels.cuh"
#include "topk_keys.cuh"

namespace ddt {
namespace cw {

constexpr int kThreads = 256;
constexpr int kKeys = 64, kRows = 32, kDims = 32;

template <typename T>
__device__ __forceinline__ float elem(const T* p);
template <>
__device__ __forceinline__ float elem<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float elem<uint16_t>(const uint16_t* p) { return bf16_bits_to_float(__ldg(p)); }

template <typename T>
__global__ void __launch_bounds__(kThreads) cache_weights_simt_kernel(WeightsParams p) {
  __shared__ float s_k[kDims][kKeys + 4];
  __shared__ float s_q[kDims][kRows + 2];
  __shared__ float s_lse[kRows];
  __shared__ int s_sees[kRows];
  __shared__ long long s_row[kRows];
  __shared__ float s_sum[kThreads / 16][kKeys];
  __shared__ int s_m, s_bad;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int b = (int)(blockIdx.x / (unsigned)p.tiles), tile0 = (int)(blockIdx.x % (unsigned)p.tiles);
  const int len = p.cache_len[b], n = p.n_nodes[b];
  const int64_t off = p.cache_off[b];
  const int32_t* list = p.nodes ? p.nodes + (int64_t)b * p.M : nullptr;
  // entries of the list: up to its first negative one, each below n_nodes
  int m = n;
  if (tid == 0) {
    s_m = p.M;
    s_bad = n < 0 || n > p.N ? 1 : 0;
  }
  __syncthreads();
  if (list) {
    for (int j = tid; j < p.M; j += kThreads)
      if (__ldg(list + j) < 0) atomicMin(&s_m, j);
    __syncthreads();
    m = s_m;
    for (int j = tid; j < m; j += kThreads)
      if (__ldg(list + j) >= n) s_bad = 1;
  }
  __syncthreads();
  const bool oob = off < 0 || len < 0 || off > p.kv_rows - len;
  const int st = oob ? DDT_ERR_BOUNDS : s_bad ? DDT_ERR_INPUT : DDT_OK;
  if (tile0 == 0 && tid == 0 && p.dev_status) p.dev_status[b] = st;
  if (st != DDT_OK) return;

  const int d = p.d_qk;
  const int rows = m * p.H;  // (entry, head)
  const T* kv = static_cast<const T*>(p.kv) + off * d;
  const float sl2 = p.scale * kLog2e;
  for (int tile = tile0; (int64_t)tile * kKeys < len; tile += p.tiles) {
    const int k0 = tile * kKeys;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int r0 = 0; r0 < rows; r0 += kRows) {
      if (tid < kRows) {
        const int r = r0 + tid;
        float l = -INFINITY;
        int sees = 0;
        long long row = 0;
        if (r < rows) {
          const int e = r / p.H, h = r - e * p.H;
          row = ((long long)b * p.N + (list ? __ldg(list + e) : e)) * p.H + h;
          l = __ldg(p.lse + row);
          sees = p.causal ? len - m + 1 + e : len;
        }
        // a row without visible keys (lse -inf) gives no weight to anything
        s_lse[tid] = l * kLog2e;
        s_sees[tid] = l == -INFINITY ? 0 : sees;
        s_row[tid] = row;
      }
      float acc[4][2] = {};
      for (int c0 = 0; c0 < d; c0 += kDims) {
        __syncthreads();
        for (int e = tid; e < kKeys * kDims; e += kThreads) {
          const int k = e / kDims, c = e % kDims;
          s_k[c][k] = (k0 + k < len && c0 + c < d) ? elem(kv + (int64_t)(k0 + k) * d + c0 + c) : 0.0f;
        }
        for (int e = tid; e < kRows * kDims; e += kThreads) {
          const int r = e / kDims, c = e % kDims;
          s_q[c][r] = (r0 + r < rows && c0 + c < d) ? elem(static_cast<const T*>(p.q) + s_row[r] * d + c0 + c) : 0.0f;
        }
        __syncthreads();
#pragma unroll 8
        for (int c = 0; c < kDims; ++c) {
          const float4 kk = *reinterpret_cast<const float4*>(&s_k[c][4 * tx]);
          const float2 qq = *reinterpret_cast<const float2*>(&s_q[c][2 * ty]);
          acc[0][0] = fmaf(kk.x, qq.x, acc[0][0]);
          acc[1][0] = fmaf(kk.y, qq.x, acc[1][0]);
          acc[2][0] = fmaf(kk.z, qq.x, acc[2][0]);
          acc[3][0] = fmaf(kk.w, qq.x, acc[3][0]);
          acc[0][1] = fmaf(kk.x, qq.y, acc[0][1]);
          acc[1][1] = fmaf(kk.y, qq.y, acc[1][1]);
          acc[2][1] = fmaf(kk.z, qq.y, acc[2][1]);
          acc[3][1] = fmaf(kk.w, qq.y, acc[3][1]);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = 2 * ty + u;
        const float l2 = s_lse[r];
        const int sees = s_sees[r];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (k0 + 4 * tx + i < sees) sum[i] += exp2f(fmaf(acc[i][u], sl2, -l2));
      }
      __syncthreads();  // the tile's rows are done with before they are replaced
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[ty][4 * tx + i] = sum[i];
    __syncthreads();
    if (tid < kKeys && k0 + tid < len) {
      float w = 0.0f;
#pragma unroll
      for (int y = 0; y < kThreads / 16; ++y) w += s_sum[y][tid];
      const int64_t j = off + k0 + tid;
      p.score[j] = p.prev ? fmaf(p.decay, p.prev[j], w) : w;
    }
    __syncthreads();
  }
}

}  // namespace cw

int launch_cache_weights_simt(WeightsParams p, int max_cache_len, cudaStream_t stream) {
  using namespace cw;
  p.tiles = std::max(1, (max_cache_len + kKeys - 1) / kKeys);
  const long long grid = (long long)p.tiles * p.B;
  if (grid > 0x7fffffffLL) return DDT_ERR_UNSUPPORTED;
  if (p.in_dtype == DDT_F32)
    return launch_pdl(cache_weights_simt_kernel<float>, (unsigned)grid, kThreads, 0, stream, p);
  return launch_pdl(cache_weights_simt_kernel<uint16_t>, (unsigned)grid, kThreads, 0, stream, p);
}

}  // namespace ddt
