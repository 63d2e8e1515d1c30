// Accumulated attention weight of cached rows, CUDA-core form (float32
// arithmetic, any d_qk <= 1024): float32 inputs, and the bf16 shapes that the
// tensor-core kernel does not cover.
//
// What it computes is fixed in ddt.h (ddt_cache_weights): for every cached
// row j, sum over the selected verify rows r of e^(scale q_r . k_j - lse_r).
//
// A CTA owns 128 keys of a request and walks the request's query rows 128 at a
// time: a 128 x 128 tile of dot products in registers (8 keys x 8 rows per
// thread, 64 products for 16 values read from shared memory, two CTAs per SM),
// operands through two stages of 16 dims, the next one's loads in flight under
// this one's products. For few rows the tile is 64 x 32 with stages of 32 dims
// (fewer trips: their loads' latency is all that counts). Each key belongs to
// one CTA, so its sum is formed in a fixed order (per thread over the row
// tiles, then over the 16 threads that share the key) without atomics. Bound by
// the fma and shared memory rates for long row lists, by latency for short
// ones. Measured (float32, 72 TFLOP/s at most):
//   4 x 8192 rows of 576 x 8192 keys     8.15 ms, 38 TFLOP/s
//   4 x 1024 rows of 128 x 8192 keys     254 us, 34 TFLOP/s
//   16 rows of 576 x 4096 keys           25 us (64 CTAs, 18 stages each)
// (A 64 x 32 tile without the second stage gave 15 TFLOP/s; 128 x 64 with packed
// pairs of keys 25, bound by its reads of shared memory.)
#include <algorithm>

#include "ddt_kernels.cuh"
#include "topk_keys.cuh"

namespace ddt {
namespace cw {

constexpr int kThreads = 256;

// n (4 or 8) consecutive elements of a row, from x on: its first `in` (or none) exist.
// vec: rows start on 16 bytes and have a multiple of eight elements.
template <int n>
__device__ __forceinline__ void load_row(const float* x, int in, bool vec, float (&v)[n]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < n; i += 4) {
      const float4 y = in > 0 ? __ldg(reinterpret_cast<const float4*>(x + i)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      v[i] = y.x, v[i + 1] = y.y, v[i + 2] = y.z, v[i + 3] = y.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = i < in ? __ldg(x + i) : 0.0f;
}
template <int n>
__device__ __forceinline__ void load_row(const uint16_t* x, int in, bool vec, float (&v)[n]) {
  if (vec) {
    uint32_t w[n / 2];
    if constexpr (n == 8) {
      const uint4 y = in > 0 ? __ldg(reinterpret_cast<const uint4*>(x)) : make_uint4(0u, 0u, 0u, 0u);
      w[0] = y.x, w[1] = y.y, w[2] = y.z, w[3] = y.w;
    } else {
      const uint2 y = in > 0 ? __ldg(reinterpret_cast<const uint2*>(x)) : make_uint2(0u, 0u);
      w[0] = y.x, w[1] = y.y;
    }
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      v[i] = __uint_as_float(w[i / 2] << 16);
      v[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = i < in ? bf16_bits_to_float(__ldg(x + i)) : 0.0f;
}

// KP keys and RP rows per thread: (8, 8) or (4, 2).
template <typename T, int KP, int RP>
__global__ void __launch_bounds__(kThreads, 2) cache_weights_simt_kernel(WeightsParams p) {
  constexpr int kKeys = 16 * KP, kRows = 16 * RP;
  constexpr int kDims = KP == 8 ? 16 : 32;                       // of a stage
  constexpr int kPK = KP * kDims / 16, kPR = RP * kDims / 16;    // one thread's loads for it
  __shared__ __align__(16) float s_k[2][kDims][kKeys];
  __shared__ __align__(16) float s_q[2][kDims][kRows];
  __shared__ float s_lse[kRows];
  __shared__ int s_sees[kRows];
  __shared__ long long s_row[kRows];
  __shared__ float s_sum[16][kKeys];
  __shared__ int s_m, s_bad;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int tx = (tid & 7) | (tid >> 5 & 1) << 3, ty = (tid >> 3 & 3) | (tid >> 6) << 2;  // 8 x 4 threads in a warp
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
  const T* q = static_cast<const T*>(p.q);
  const bool vec = d % 8 == 0 && (reinterpret_cast<uintptr_t>(p.kv) | reinterpret_cast<uintptr_t>(p.q)) % 16 == 0;
  const float sl2 = p.scale * kLog2e;
  // this thread's part of a stage: kPK dims of one key, kPR dims of one row
  const int lk = tid % kKeys, ck = tid / kKeys * kPK, lr = tid % kRows, cr = tid / kRows * kPR;
  for (int tile = tile0; (int64_t)tile * kKeys < len; tile += p.tiles) {
    const int k0 = tile * kKeys;
    const T* key = lk < len - k0 ? kv + (int64_t)(k0 + lk) * d + ck : nullptr;
    float sum[KP] = {};
    for (int r0 = 0; r0 < rows; r0 += kRows) {
      if (tid < kRows) {
        const int r = r0 + tid;
        float l = -INFINITY;
        int sees = 0;
        long long row = -1;
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
      __syncthreads();
      const T* row = s_row[lr] >= 0 ? q + s_row[lr] * d + cr : nullptr;
      float vk[kPK], vq[kPR];
      auto load = [&](int c0) {
        load_row(key + c0, key ? d - c0 - ck : 0, vec, vk);
        load_row(row + c0, row ? d - c0 - cr : 0, vec, vq);
      };
      auto store = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kPK; ++i) s_k[buf][ck + i][lk] = vk[i];
#pragma unroll
        for (int i = 0; i < kPR; ++i) s_q[buf][cr + i][lr] = vq[i];
      };
      float acc[KP][RP] = {};
      load(0);
      store(0);
      __syncthreads();
      int buf = 0;
      for (int c0 = 0; c0 < d; c0 += kDims, buf ^= 1) {
        const bool more = c0 + kDims < d;
        if (more) load(c0 + kDims);
#pragma unroll 4
        for (int c = 0; c < kDims; ++c) {
          __align__(16) float kk[KP], qq[RP];
#pragma unroll
          for (int i = 0; i < KP; i += 4)
            *reinterpret_cast<float4*>(&kk[i]) = *reinterpret_cast<const float4*>(&s_k[buf][c][16 * i + 4 * tx]);
          if constexpr (RP == 2) {
            *reinterpret_cast<float2*>(&qq[0]) = *reinterpret_cast<const float2*>(&s_q[buf][c][2 * ty]);
          } else {
#pragma unroll
            for (int u = 0; u < RP; u += 4)
              *reinterpret_cast<float4*>(&qq[u]) = *reinterpret_cast<const float4*>(&s_q[buf][c][16 * u + 4 * ty]);
          }
#pragma unroll
          for (int i = 0; i < KP; ++i)
#pragma unroll
            for (int u = 0; u < RP; ++u) acc[i][u] = fmaf(kk[i], qq[u], acc[i][u]);
        }
        if (more) store(buf ^ 1);  // its last readers are behind the barrier before this stage
        __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < RP; ++u) {
        const int r = RP == 2 ? 2 * ty + u : 16 * (u & ~3) + 4 * ty + (u & 3);
        const float l2 = s_lse[r];
        const int sees = s_sees[r];
#pragma unroll
        for (int i = 0; i < KP; ++i)
          if (k0 + 16 * (i & ~3) + 4 * tx + (i & 3) < sees) sum[i] += exp2f(fmaf(acc[i][u], sl2, -l2));
      }
      __syncthreads();  // the tile's rows are done with before they are replaced
    }
#pragma unroll
    for (int i = 0; i < KP; ++i) s_sum[ty][16 * (i & ~3) + 4 * tx + (i & 3)] = sum[i];
    __syncthreads();
    if (tid < kKeys && tid < len - k0) {
      float w = 0.0f;
#pragma unroll
      for (int y = 0; y < 16; ++y) w += s_sum[y][tid];
      const int64_t j = off + k0 + tid;
      p.score[j] = p.prev ? fmaf(p.decay, p.prev[j], w) : w;
    }
    __syncthreads();
  }
}

template <typename T, int KP, int RP>
static int launch_tile(WeightsParams p, int max_cache_len, cudaStream_t stream) {
  constexpr int kKeys = 16 * KP;
  // a request's tiles, as far as the grid allows: a CTA takes every p.tiles-th
  p.tiles = std::max(1, max_cache_len / kKeys + (max_cache_len % kKeys != 0 ? 1 : 0));
  p.tiles = std::min(p.tiles, 0x7fffffff / p.B);
  return launch_pdl(cache_weights_simt_kernel<T, KP, RP>, (unsigned)(p.tiles * p.B), kThreads, 0, stream, p);
}
template <typename T>
static int launch_type(const WeightsParams& p, int max_cache_len, cudaStream_t stream) {
  // The shorter estimated time: waves of two CTAs per SM times tiles of rows,
  // of which a large one takes 3.2 times a small one's time (128 dims: 17 and
  // 5.4 us, the latter mostly latency). 256 rows x 8192 keys: 39 us with 64
  // large tiles, 47 with 128 small ones; 4 x 48 rows x 8192 keys: 33 and 40; 35
  // rows x 536 keys of 40 dims: 11.1 and 7.3.
  const long long rows = (long long)(p.nodes ? p.M : p.N) * p.H, slots = 2LL * sm_count();
  auto time = [&](long long keys, long long rows_per, int unit) {
    const long long ctas = (max_cache_len / keys + 1) * p.B;
    return (ctas + slots - 1) / slots * ((rows + rows_per - 1) / rows_per) * unit;
  };
  return time(128, 128, 32) <= time(64, 32, 10) ? launch_tile<T, 8, 8>(p, max_cache_len, stream)
                                                : launch_tile<T, 4, 2>(p, max_cache_len, stream);
}

}  // namespace cw

int launch_cache_weights_simt(WeightsParams p, int max_cache_len, cudaStream_t stream) {
  return p.in_dtype == DDT_F32 ? cw::launch_type<float>(p, max_cache_len, stream)
                               : cw::launch_type<uint16_t>(p, max_cache_len, stream);
}

}  // namespace ddt
