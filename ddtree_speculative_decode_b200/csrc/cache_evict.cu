// Eviction of latent-cache rows by their accumulated attention weight.
//
// What it computes is fixed in ddt.h (ddt_cache_evict): per layer and request
// the first `sink` rows, the last `recent` rows and the best-scored rows
// between them stay, `keep` in all, in their order.
//
// evict_select_kernel: one cluster of C CTAs per (layer, request), C from 1 to 8
// so that the launch fills the device; each CTA has a slice of the request's
// rows as 32-bit keys in score order (protected rows above every score, NaN
// below every score) in shared memory. The keep-th largest key T is found by
// histograms of 2048 bins laid over the keys' own range (so that scores of a
// few binades still spread over all bins, and few atomics meet), each over the
// bin of the one before that holds T; a bin of at most 512 keys is finished by
// counting ranks. Typically one histogram and one count; a bitwise search over
// the same keys took 32 CTA-wide counts (14 us against 5 for 4096 rows).
// Ranges, histograms and counts are joined through distributed shared memory.
// Rows above T stay, and of those equal to T the lowest ones that fill the
// number: one ordered pass with prefix counts writes the kept rows' indices.
//
// The rows: bound by HBM, each kept row read and written once. Into another
// region (evict_copy_kernel) rows go independently: a CTA takes a block of rows
// and their scores. (Letting the selection's clusters copy their own rows, so
// that one request's selection runs under another's copy, was slower: 82
// against 60 us for 64 clusters, whose threads keep fewer loads in flight.) In
// place, row j is written from row src[j] >= j, so row i must be read before it
// is overwritten: in evict_shift_kernel a CTA takes a 128-byte column of a
// request's rows (one more CTA their scores) and walks it upwards in chunks,
// every chunk read into registers before it is written (later chunks read only
// rows above the ones written so far, so the next chunk's loads are already
// under way), and no CTA waits for another. With few layers and requests the
// columns are as narrow as 32 bytes, for more CTAs. Rows before the first
// evicted one already lie in place and are left alone.
//
// Measured (bf16 rows of 576, half of the rows kept unless said; kernels only):
//   1 x 4096 rows                 11 to 14 us, copy; 15 us in place (latency)
//   1 x 32768 rows                21 us, copy; 50 us in place (few CTAs)
//   61 layers of 4096 rows        58 us, copy (5.0 TB/s); 65 us in place
//   16 layers of 4 x 32768 rows   405 to 416 us, copy (6.0 TB/s); 460 to 470 us in place
// A few rows of a full cache, in place (nearly every row moves a few places):
//   9 of 16393 rows, 61 layers    397 us (5.2 TB/s of rows that move); one layer 40 us
//   9 of 16 x 4105, 61 layers     1454 us (5.8 TB/s)
#include <algorithm>
#include <mutex>

#include "ddt_kernels.cuh"
#include "sm100_ptx.cuh"

namespace ddt {
namespace evict {

using sm100::cluster_ctarank;
using sm100::cluster_sync;
using sm100::map_to_rank;
using sm100::smem_u32;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinsPer = kBins / kSelThreads;  // of one thread
constexpr int kRank = 512;           // keys of a bin that are ranked by counting
constexpr int kSelKeys = 40 * 1024;  // keys a CTA holds in shared memory; longer slices re-read their scores
constexpr int kMaxC = 8;
constexpr int kMaxLen = 1 << 30;  // rows of a request: row numbers are added up in 32 bits

__device__ __forceinline__ uint32_t ld_remote(const void* mine, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(mine), (uint32_t)rank)) : "memory");
  return v;
}
__device__ __forceinline__ void st_remote(const void* mine, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_u32(mine), (uint32_t)rank)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_remote(const void* mine, int rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(map_to_rank(smem_u32(mine), (uint32_t)rank)), "r"(v)
               : "memory");
  return old;
}

// score order: larger score, larger key; NaN lowest
__device__ __forceinline__ uint32_t score_key(float x) { return x == x ? float_order_key(x) : 0u; }

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_hist[kBins], s_sum[kBins];
  __shared__ uint32_t s_rank[kRank];
  __shared__ uint32_t s_min, s_max, s_T, s_n;
  __shared__ uint32_t s_lo[kMaxC], s_hi[kMaxC], s_gt[kMaxC], s_tie[kMaxC], s_first[kMaxC];  // by the cluster's CTA
  __shared__ int s_bin, s_above, s_inbin, s_ties;
  __shared__ int s_scan[2][kSelWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.cluster, rank = C > 1 ? (int)cluster_ctarank() : 0;
  auto meet = [&]() {
    if (C > 1) cluster_sync();
    else __syncthreads();
  };
  const unsigned lb = blockIdx.x / (unsigned)C;
  const int layer = (int)(lb / (unsigned)p.B), b = (int)(lb % (unsigned)p.B);
  const int len = p.cache_len[b], keep = p.keep[b];
  const int64_t off = p.cache_off[b], doff = p.kv_dst ? p.dst_off[b] : off;
  // the request's verdict, the same on every layer (the host has checked that
  // the layers' stride does not overflow)
  const int count = min(len, keep);
  int st = DDT_OK;
  const int64_t last = (int64_t)(p.n_layers - 1);
  const int64_t room = p.kv_rows - len - last * p.layer_stride_rows;
  const int64_t droom = p.kv_dst ? p.dst_rows - max(count, 0) - last * p.dst_layer_stride_rows : room;
  if (off < 0 || len < 0 || len > kMaxLen || room < 0 || off > room || doff < 0 || droom < 0 || doff > droom)
    st = DDT_ERR_BOUNDS;
  else if (keep < 0 || (len > keep && (int64_t)keep < (int64_t)p.sink + p.recent))
    st = DDT_ERR_INPUT;
  else if (count > p.max_keep)
    st = DDT_ERR_CAPACITY;
  const bool head = rank == 0 && tid == 0;
  if (layer == 0 && head && p.dev_status) p.dev_status[b] = st;
  int32_t* src = p.src + (int64_t)lb * p.max_keep;
  const int kept = st == DDT_OK ? count : 0;
  for (int j = kept + rank * kSelThreads + tid; j < p.max_keep; j += C * kSelThreads) src[j] = -1;
  int2* plan = p.plan + lb;
  if (st != DDT_OK) {  // the same on the whole cluster, as every branch on len and keep
    if (head) *plan = make_int2(-1, 0);
    return;
  }
  const float* score = p.score + (int64_t)layer * p.layer_stride_rows + off;
  if (len <= keep) {  // everything stays
    for (int i = rank * kSelThreads + tid; i < len; i += C * kSelThreads) src[i] = i;
    if (head) *plan = make_int2(len, len);
    return;
  }
  const int per = (len + C - 1) / C, i0 = min(len, rank * per), i1 = min(len, i0 + per);
  const bool held = per <= p.held_keys;
  const int tail = len - p.recent;
  auto row_key = [&](int i, float x) { return (i < p.sink || i >= tail) ? 0xffffffffu : score_key(x); };
  if (tid == 0) {
    s_min = 0xffffffffu;
    s_max = 0u;
  }
  __syncthreads();
  // the scored rows between the protected ones; `want` of them stay
  const int m0 = min(p.sink, len), m1 = max(m0, tail), want = keep - (len - (m1 - m0));
  const int a0 = max(i0, m0), a1 = min(i1, m1);  // of this slice
  {
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll 8
    for (int i = i0 + tid; i < i1; i += kSelThreads) {
      const uint32_t k = row_key(i, score[i]);
      if (held) s_key[i - i0] = k;
      if (i >= m0 && i < m1) {
        lo = min(lo, k);
        hi = max(hi, k);
      }
    }
    lo = __reduce_min_sync(DDT_FULL_MASK, lo);
    hi = __reduce_max_sync(DDT_FULL_MASK, hi);
    if (lane == 0) {
      atomicMin(&s_min, lo);
      atomicMax(&s_max, hi);
    }
  }
  if (C > 1) {
    cluster_sync();  // the slice's range is known, and every CTA of the cluster runs
    if (tid < C) {
      st_remote(&s_lo[rank], tid, s_min);
      st_remote(&s_hi[rank], tid, s_max);
    }
    cluster_sync();
    if (tid == 0)
      for (int c = 0; c < C; ++c) {
        s_min = min(s_min, s_lo[c]);
        s_max = max(s_max, s_hi[c]);
      }
  }
  __syncthreads();
  auto key_at = [&](int i) { return held ? s_key[i - i0] : row_key(i, score[i]); };

  // ---- T: kept are the keys above T and, of those equal to it, the first
  // `ties`
  uint32_t T = 0xfffffffeu;  // want = 0: only the protected rows are above
  int ties = 0;
  if (want > 0) {
    uint32_t lo = s_min, range = s_max - s_min;
    int above = 0;  // scored rows above the current range
    for (;;) {      // at most three rounds: 11 bits of the range each
      const int bits = 32 - __clz((int)range), shift = max(0, bits - 11);
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0u;
      if (tid == 0) s_n = 0u;
      __syncthreads();
#pragma unroll 4
      for (int i = a0 + tid; i < a1; i += kSelThreads) {
        const uint32_t d = key_at(i) - lo;
        if (d <= range) atomicAdd(&s_hist[d >> shift], 1u);
      }
      meet();
      if (C > 1) {
        // each CTA adds up its share of the bins for everyone
        const int share = kBins / C, first = rank * share;
        for (int i = first + tid; i < first + share; i += kSelThreads) {
          uint32_t n = 0u;
          for (int c = 0; c < C; ++c) n += ld_remote(&s_hist[i], c);
          for (int c = 0; c < C; ++c) st_remote(&s_sum[i], c, n);
        }
        cluster_sync();
      }
      // the bin that holds the want-th largest: thread t has kBinsPer bins
      const uint32_t* bins = C > 1 ? s_sum : s_hist;
      int h[kBinsPer], suf = 0;  // of this thread's and the higher lanes' bins
#pragma unroll
      for (int q = 0; q < kBinsPer; ++q) {
        h[q] = (int)bins[kBinsPer * tid + q];
        suf += h[q];
      }
      const int own = suf;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(DDT_FULL_MASK, suf, o);
        if (lane + o < 32) suf += y;
      }
      if (lane == 0) s_scan[0][warp] = suf;
      __syncthreads();
      const int higher = __reduce_add_sync(DDT_FULL_MASK, lane > warp && lane < kSelWarps ? s_scan[0][lane] : 0);
      int up = above + higher + suf - own;  // rows above this thread's bins
#pragma unroll
      for (int q = kBinsPer - 1; q >= 0; --q) {
        if (up < want && want <= up + h[q]) {
          s_bin = kBinsPer * tid + q;
          s_above = up;
          s_inbin = h[q];
        }
        up += h[q];
      }
      __syncthreads();
      above = s_above;
      lo += (uint32_t)s_bin << shift;
      const int n = s_inbin;
      if (shift == 0) {
        T = lo;
        ties = want - above;
        break;
      }
      if (above + n == want) {  // the whole bin stays (lo > 0: some row goes)
        T = lo - 1u;
        break;
      }
      range = (1u << shift) - 1u;
      if (n > kRank) {
        meet();  // nobody reads this round's histogram any more
        continue;
      }
      for (int i = a0 + tid; i < a1; i += kSelThreads) {
        const uint32_t k = key_at(i);
        if (k - lo <= range) {
          const uint32_t at = C > 1 ? add_remote(&s_n, 0, 1u) : atomicAdd(&s_n, 1u);
          st_remote(&s_rank[at], 0, k);
        }
      }
      meet();
      if (C > 1 && rank > 0)
        for (int i = tid; i < n; i += kSelThreads) s_rank[i] = ld_remote(&s_rank[i], 0);
      __syncthreads();
      if (tid < n) {
        const uint32_t k = s_rank[tid];
        int more = 0, same = 0;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
          const uint32_t y = s_rank[i];
          more += y > k ? 1 : 0;
          same += y == k ? 1 : 0;
        }
        if (above + more < want && want <= above + more + same) {  // equal keys agree
          s_T = k;
          s_ties = want - above - more;
        }
      }
      __syncthreads();
      T = s_T;
      ties = s_ties;
      break;
    }
  }

  // ---- rows above T and rows equal to it before this slice
  int base_gt = 0, base_tie = 0;
  if (C > 1) {
    int gt = 0, tie = 0;
    for (int i = i0 + tid; i < i1; i += kSelThreads) {
      const uint32_t k = key_at(i);
      gt += k > T ? 1 : 0;
      tie += k == T ? 1 : 0;
    }
    gt = __reduce_add_sync(DDT_FULL_MASK, gt);
    tie = __reduce_add_sync(DDT_FULL_MASK, tie);
    if (lane == 0) {
      s_scan[0][warp] = gt;
      s_scan[1][warp] = tie;
    }
    __syncthreads();
    gt = __reduce_add_sync(DDT_FULL_MASK, lane < kSelWarps ? s_scan[0][lane] : 0);
    tie = __reduce_add_sync(DDT_FULL_MASK, lane < kSelWarps ? s_scan[1][lane] : 0);
    if (tid < C) {
      st_remote(&s_gt[rank], tid, (uint32_t)gt);
      st_remote(&s_tie[rank], tid, (uint32_t)tie);
    }
    cluster_sync();
    for (int c = 0; c < rank; ++c) {
      base_gt += (int)s_gt[c];
      base_tie += (int)s_tie[c];
    }
  }

  // ---- the kept rows in order: chunks of four consecutive rows per thread
  __syncthreads();  // s_scan is free
  int par = 0, hole = len;
  for (int c0 = i0; c0 < i1; c0 += 4 * kSelThreads) {
    const int r0 = c0 + 4 * tid;
    uint32_t k[4];
    int mine = 0;  // rows above T in the low half, rows equal to T in the high half
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = r0 + q;
      k[q] = i < i1 ? key_at(i) : 0u;
      if (i < i1) mine += k[q] > T ? 1 : k[q] == T ? (1 << 16) : 0;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(DDT_FULL_MASK, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[par][warp] = inc;
    __syncthreads();
    const int w = lane < kSelWarps ? s_scan[par][lane] : 0;
    int before = __reduce_add_sync(DDT_FULL_MASK, lane < warp ? w : 0);
    const int all = __reduce_add_sync(DDT_FULL_MASK, w);
    par ^= 1;
    before += inc - mine;
    int gt = base_gt + (before & 0xffff), tie = base_tie + (before >> 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = r0 + q;
      if (i >= i1) break;
      const bool is_gt = k[q] > T, is_tie = k[q] == T;
      if (is_gt || (is_tie && tie < ties)) src[gt + min(tie, ties)] = i;
      else hole = min(hole, i);
      gt += is_gt ? 1 : 0;
      tie += is_tie ? 1 : 0;
    }
    base_gt += all & 0xffff;
    base_tie += all >> 16;
  }
  // the first row that goes: no row before it moves
  hole = __reduce_min_sync(DDT_FULL_MASK, hole);
  __syncthreads();
  if (tid == 0) s_min = (uint32_t)len;
  __syncthreads();
  if (lane == 0) atomicMin(&s_min, (uint32_t)hole);
  __syncthreads();
  if (tid == 0) st_remote(&s_first[rank], 0, s_min);
  meet();  // the slices' lists are complete
  if (head) {
    uint32_t first = s_first[0];
    for (int c = 1; c < C; ++c) first = min(first, s_first[c]);
    *plan = make_int2(keep, (int)first);
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveU = 8;

// Rows into another region: CTA (layer, request, block of rows).
template <typename Tv>
__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(EvictParams p) {
  pdl_wait();
  const unsigned lb = blockIdx.x / (unsigned)p.blocks, blk = blockIdx.x % (unsigned)p.blocks;
  const int layer = (int)(lb / (unsigned)p.B), b = (int)(lb % (unsigned)p.B);
  const int2 plan = p.plan[lb];
  if (layer == 0 && blk == 0 && threadIdx.x == 0) p.new_len[b] = max(plan.x, 0);
  const int r0 = (int)blk * p.block_rows, r1 = min(plan.x, r0 + p.block_rows);
  if (r0 >= r1) return;
  const int vpr = p.row_vecs;
  const Tv* from = reinterpret_cast<const Tv*>(p.kv) + ((int64_t)layer * p.layer_stride_rows + p.cache_off[b]) * vpr;
  Tv* to = reinterpret_cast<Tv*>(p.kv_dst) + ((int64_t)layer * p.dst_layer_stride_rows + p.dst_off[b] + r0) * vpr;
  const int32_t* src = p.src + (int64_t)lb * p.max_keep + r0;
  const float* sfrom = p.score + (int64_t)layer * p.layer_stride_rows + p.cache_off[b];
  float* sto = p.score_dst + (int64_t)layer * p.dst_layer_stride_rows + p.dst_off[b] + r0;
  for (int r = threadIdx.x; r < r1 - r0; r += kMoveThreads) sto[r] = sfrom[__ldg(src + r)];
  const int n = (r1 - r0) * vpr;
  for (int e0 = threadIdx.x; e0 < n; e0 += kMoveThreads * kMoveU) {
    Tv v[kMoveU];
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) {
      const int e = e0 + u * kMoveThreads;
      if (e < n) {
        const int r = e / vpr;
        v[u] = __ldcs(from + (int64_t)__ldg(src + r) * vpr + (e - r * vpr));
      }
    }
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) {
      const int e = e0 + u * kMoveThreads;
      if (e < n) __stcs(to + e, v[u]);
    }
  }
}

// The shift of one column: rows plan.y .. plan.x - 1, `row` of `step` rows per
// chunk and step being this thread's.
template <typename Tv>
__device__ __forceinline__ void shift_column(Tv* kv, int stride, bool on, const int32_t* src, int2 plan, int row, int step) {
  // chunk by chunk: the indices two chunks and the rows one chunk ahead
  Tv v[kMoveU];
  int at[kMoveU];
  auto indices = [&](int j0) {
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) {
      const int j = j0 + row + u * step;
      at[u] = on && j < plan.x ? src[j] : -1;
    }
  };
  auto rows = [&]() {
#pragma unroll
    for (int u = 0; u < kMoveU; ++u)
      if (at[u] >= 0) v[u] = kv[(int64_t)at[u] * stride];
  };
  indices(plan.y);
  rows();
  indices(plan.y + step * kMoveU);
  for (int j0 = plan.y; j0 < plan.x; j0 += step * kMoveU) {  // the same trips for the whole CTA
    Tv w[kMoveU];
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) w[u] = v[u];
    rows();
    indices(j0 + 2 * step * kMoveU);
    __syncthreads();  // the chunk is read, by everyone, before any of it is overwritten
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) {
      const int j = j0 + row + u * step;
      if (on && j < plan.x) kv[(int64_t)j * stride] = w[u];
    }
  }
}

// In place: CTA (layer, request, column of p.col vectors), the last of a
// request its scores.
template <typename Tv>
__global__ void __launch_bounds__(kMoveThreads) evict_shift_kernel(EvictParams p) {
  pdl_wait();
  const unsigned lb = blockIdx.x / (unsigned)p.blocks, blk = blockIdx.x % (unsigned)p.blocks;
  const int layer = (int)(lb / (unsigned)p.B), b = (int)(lb % (unsigned)p.B), tid = threadIdx.x;
  const int2 plan = p.plan[lb];
  const int64_t row0 = (int64_t)layer * p.layer_stride_rows + p.cache_off[b];
  if (layer == 0 && blk == 0 && tid == 0) p.new_len[b] = plan.x >= 0 ? plan.x : p.cache_len[b];
  const int32_t* src = p.src + (int64_t)lb * p.max_keep;
  if ((int)blk == p.blocks - 1) {
    shift_column(p.score + row0, 1, true, src, plan, tid, kMoveThreads);
    return;
  }
  const int c = (int)blk * p.col + tid % p.col;
  shift_column(reinterpret_cast<Tv*>(p.kv) + row0 * p.row_vecs + c, p.row_vecs, c < p.row_vecs, src, plan, tid / p.col,
               kMoveThreads / p.col);
}

// Dynamic shared memory of the selection's keys, opted in once per device.
static bool opt_in() {
  static std::mutex mu;
  static bool done[kMaxDevices] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev])
    done[dev] = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4) ==
                cudaSuccess;
  return done[dev];
}

static int launch_select(const EvictParams& p, cudaStream_t stream) {
  if (!opt_in()) return DDT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.n_layers * p.B * p.cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)p.held_keys * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, p) == cudaSuccess ? DDT_OK : DDT_ERR_CUDA;
}

// The move's split; false: more CTAs than a launch may have.
template <typename Tv>
static bool split_move(EvictParams& p) {
  p.row_vecs = p.row_bytes / (int)sizeof(Tv);
  const long long lbs = (long long)p.n_layers * p.B;
  if (p.kv_dst) {
    // blocks of two trips per thread, smaller ones when they would not give
    // every SM four CTAs
    const long long vecs = (long long)p.max_keep * lbs * p.row_vecs, most = kMoveThreads * kMoveU * 2;
    const long long per = std::min(most, std::max<long long>(kMoveThreads, vecs / (4 * sm_count())));
    p.block_rows = std::max(1, (int)(per / p.row_vecs));
    p.blocks = std::max(1, (p.max_keep + p.block_rows - 1) / p.block_rows);
  } else {
    p.col = 128 / (int)sizeof(Tv);
    while (p.col * (int)sizeof(Tv) > 32 && lbs * ((p.row_vecs + p.col - 1) / p.col) < 4 * sm_count()) p.col >>= 1;
    p.blocks = (p.row_vecs + p.col - 1) / p.col + 1;  // and the scores
  }
  return lbs * p.blocks <= 0x7fffffffLL;
}

template <typename Tv>
static int launch_move(const EvictParams& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)p.n_layers * (unsigned)p.B * (unsigned)p.blocks;
  return p.kv_dst ? launch_pdl(evict_copy_kernel<Tv>, grid, kMoveThreads, 0, stream, p)
                  : launch_pdl(evict_shift_kernel<Tv>, grid, kMoveThreads, 0, stream, p);
}

}  // namespace evict

size_t evict_workspace_bytes(int B, int n_layers, int max_cache_len) {
  (void)max_cache_len;
  return ((size_t)B * n_layers * sizeof(int2) + 255) / 256 * 256;
}

int launch_cache_evict(EvictParams p, int max_cache_len, void* workspace, cudaStream_t stream) {
  using namespace evict;
  p.plan = static_cast<int2*>(workspace);
  const long long lbs = (long long)p.n_layers * p.B;
  // CTAs per (layer, request): one for short caches, otherwise as many as there
  // are SMs for. A cluster's meetings cost what about 8000 rows do: with the
  // copy, one request of 6000 rows takes 12.6 us with one CTA and 14.2 with
  // eight, of 12000 16.7 and 15.4, of 32768 28.6 and 17.1 (4096 rows kept); 64
  // of 8192 take 63 us with one, 65 with two and 75 with four, two per SM.
  // Clusters of eight do not fill the device (their SMs are neighbours): 16 of
  // 24000 take 49 us with eight CTAs, 40 with four, 42 with two.
  p.cluster = max_cache_len < 10240 ? 1 : kMaxC;
  while (p.cluster > 1 && lbs * p.cluster > (p.cluster > 4 ? sm_count() / 2 : sm_count())) p.cluster >>= 1;
  if (lbs * p.cluster > 0x7fffffffLL) return DDT_ERR_UNSUPPORTED;
  // shared memory for the longest slice the caller announces; a longer one (or
  // one beyond what is set aside) re-reads its scores instead
  const int slice = (std::min(max_cache_len, kMaxLen) + p.cluster - 1) / p.cluster;
  p.held_keys = std::min(kSelKeys, (slice + 1023) / 1024 * 1024);
  auto al = [](const void* q, uintptr_t a) { return reinterpret_cast<uintptr_t>(q) % a == 0; };
  const bool wide = p.row_bytes % 16 == 0 && al(p.kv, 16) && al(p.kv_dst, 16);
  if (!(wide ? split_move<uint4>(p) : split_move<uint32_t>(p))) return DDT_ERR_UNSUPPORTED;  // before anything is written
  const int st = launch_select(p, stream);
  if (st != DDT_OK) return st;
  return wide ? launch_move<uint4>(p, stream) : launch_move<uint32_t>(p, stream);
}

}  // namespace ddt
