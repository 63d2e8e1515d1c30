// Eviction of latent-cache rows by their accumulated attention weight.
//
// What it computes is fixed in ddt.h (ddt_cache_evict): per layer and request
// the first `sink` rows, the last `recent` rows and the best-scored rows
// between them stay, `keep` in all, in their order.
//
// evict_select_kernel: one CTA per (layer, request). Rows become 32-bit keys
// in score order (protected rows above every score, NaN below every score),
// held in shared memory. The keep-th largest key T is found by histograms of
// 2048 bins laid over the keys' own range (so that scores of a few binades
// still spread over all bins, and few atomics meet), each over the bin of the
// one before that holds T; a bin of at most 512 keys is finished by counting
// ranks. Typically one histogram and one count; a bitwise search over the same
// keys took 32 CTA-wide counts (14 us against 5 for 4096 rows). Rows above T
// stay, and of those equal to T the lowest ones that fill the number: one
// ordered pass with a CTA-wide prefix count writes the kept rows' indices and,
// in place, moves the scores (a score moves to its own index or a lower one,
// and a chunk is read before it is written).
//
// evict_copy_kernel and evict_shift_kernel move the rows. Bound: HBM, each kept
// row read and written once. Into another region rows go independently: a CTA
// takes a block of rows (and its scores). In place, row j is written from row src[j] >= j, so row i
// must be read before it is overwritten: a CTA takes a 128-byte column of a
// request's rows and walks it upwards in chunks, every chunk read into
// registers before it is written (later chunks read only rows above the ones
// written so far, so the next chunk's loads are already under way), and no
// CTA waits for another. With few layers and requests the columns are as
// narrow as 32 bytes, for more CTAs. Rows before the first
// evicted one already lie in place and are left alone.
#include <algorithm>
#include <mutex>

#include "ddt_kernels.cuh"

namespace ddt {
namespace evict {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kRank = 512;           // keys of a bin that are ranked by counting
constexpr int kSelKeys = 48 * 1024;  // keys held in shared memory; longer caches re-read their scores
constexpr int kMaxLen = 1 << 30;  // rows of a request: row numbers are added up in 32 bits

// score order: larger score, larger key; NaN lowest
__device__ __forceinline__ uint32_t score_key(float x) { return x == x ? float_order_key(x) : 0u; }

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ int s_hist[kBins];
  __shared__ uint32_t s_rank[kRank];
  __shared__ uint32_t s_min, s_max, s_T;
  __shared__ int s_bin, s_above, s_inbin, s_n, s_ties;
  __shared__ int s_scan[2][kSelWarps];
  __shared__ int s_hole;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int layer = (int)(blockIdx.x / (unsigned)p.B), b = (int)(blockIdx.x % (unsigned)p.B);
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
  if (layer == 0 && tid == 0 && p.dev_status) p.dev_status[b] = st;
  int32_t* src = p.src + ((int64_t)layer * p.B + b) * p.max_keep;
  const int kept = st == DDT_OK ? count : 0;
  for (int j = kept + tid; j < p.max_keep; j += kSelThreads) src[j] = -1;
  int2* plan = p.plan + (int64_t)layer * p.B + b;
  if (st != DDT_OK) {
    if (tid == 0) *plan = make_int2(-1, 0);
    return;
  }
  float* score = p.score + (int64_t)layer * p.layer_stride_rows + off;
  if (len <= keep) {  // everything stays
    for (int i = tid; i < len; i += kSelThreads) src[i] = i;
    if (tid == 0) *plan = make_int2(len, len);
    return;
  }
  const bool held = len <= p.held_keys;
  const int tail = len - p.recent;
  auto row_key = [&](int i, float x) { return (i < p.sink || i >= tail) ? 0xffffffffu : score_key(x); };
  if (tid == 0) {
    s_hole = len;
    s_min = 0xffffffffu;
    s_max = 0u;
  }
  __syncthreads();
  // the scored rows between the protected ones; `want` of them stay
  const int m0 = min(p.sink, len), m1 = max(m0, tail), want = keep - (len - (m1 - m0));
  {
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll 8
    for (int i = tid; i < len; i += kSelThreads) {
      const uint32_t k = row_key(i, score[i]);
      if (held) s_key[i] = k;
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
  __syncthreads();
  auto key_at = [&](int i) { return held ? s_key[i] : score_key(score[i]); };

  // ---- T: kept are the keys above T and, of those equal to it, the first
  // `ties`
  uint32_t T = 0xfffffffeu;  // want = 0: only the protected rows are above
  int ties = 0;
  if (want > 0) {
    uint32_t lo = s_min, range = s_max - s_min;
    int above = 0;  // scored rows above the current range
    for (;;) {      // at most three rounds: 11 bits of the range each
      const int bits = 32 - __clz((int)range), shift = max(0, bits - 11);
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
      if (tid == 0) s_n = 0;
      __syncthreads();
#pragma unroll 4
      for (int i = m0 + tid; i < m1; i += kSelThreads) {
        const uint32_t d = key_at(i) - lo;
        if (d <= range) atomicAdd(&s_hist[d >> shift], 1);
      }
      __syncthreads();
      // the bin that holds the want-th largest: thread t has bins 2t, 2t + 1
      const int h0 = s_hist[2 * tid], h1 = s_hist[2 * tid + 1];
      int suf = h0 + h1;  // of this thread's and the higher lanes' bins
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(DDT_FULL_MASK, suf, o);
        if (lane + o < 32) suf += y;
      }
      if (lane == 0) s_scan[0][warp] = suf;
      __syncthreads();
      const int higher = __reduce_add_sync(DDT_FULL_MASK, lane > warp ? s_scan[0][lane] : 0);
      const int up1 = above + higher + suf - h0 - h1, up0 = up1 + h1;  // rows above bin 2t + 1, above bin 2t
      if (up1 < want && want <= up1 + h1) {
        s_bin = 2 * tid + 1;
        s_above = up1;
        s_inbin = h1;
      } else if (up0 < want && want <= up0 + h0) {
        s_bin = 2 * tid;
        s_above = up0;
        s_inbin = h0;
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
      if (n > kRank) continue;
      for (int i = m0 + tid; i < m1; i += kSelThreads) {
        const uint32_t k = key_at(i);
        if (k - lo <= range) s_rank[atomicAdd(&s_n, 1)] = k;
      }
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

  // ---- the kept rows in order: chunks of four consecutive rows per thread
  __syncthreads();  // s_scan is free
  int base_gt = 0, base_tie = 0, par = 0, hole = len;
  for (int c0 = 0; c0 < len; c0 += 4 * kSelThreads) {
    const int i0 = c0 + 4 * tid;
    float x[4];
    uint32_t k[4];
    int mine = 0;  // rows above T in the low half, rows equal to T in the high half
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + q;
      const bool read = i < len && (!p.kv_dst || !held);  // into another region the copy moves the scores
      x[q] = read ? score[i] : 0.0f;
      k[q] = i < len ? (held ? s_key[i] : row_key(i, x[q])) : 0u;
      if (i < len) mine += k[q] > T ? 1 : k[q] == T ? (1 << 16) : 0;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(DDT_FULL_MASK, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[par][warp] = inc;
    __syncthreads();  // and every score of the chunk is in registers
    int before = lane < warp ? s_scan[par][lane] : 0, all = s_scan[par][lane];
    before = __reduce_add_sync(DDT_FULL_MASK, before);
    all = __reduce_add_sync(DDT_FULL_MASK, all);
    par ^= 1;
    before += inc - mine;
    int gt = base_gt + (before & 0xffff), tie = base_tie + (before >> 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + q;
      if (i >= len) break;
      const bool is_gt = k[q] > T, is_tie = k[q] == T;
      if (is_gt || (is_tie && tie < ties)) {
        const int j = gt + min(tie, ties);
        src[j] = i;
        if (!p.kv_dst && j != i) score[j] = x[q];
      } else {
        hole = min(hole, i);
      }
      gt += is_gt ? 1 : 0;
      tie += is_tie ? 1 : 0;
    }
    base_gt += all & 0xffff;
    base_tie += all >> 16;
  }
  hole = __reduce_min_sync(DDT_FULL_MASK, hole);
  if (lane == 0) atomicMin(&s_hole, hole);
  __syncthreads();
  if (tid == 0) *plan = make_int2(keep, s_hole);
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

// Rows in place: CTA (layer, request, column of p.col vectors).
template <typename Tv>
__global__ void __launch_bounds__(kMoveThreads) evict_shift_kernel(EvictParams p) {
  pdl_wait();
  const unsigned lb = blockIdx.x / (unsigned)p.blocks, blk = blockIdx.x % (unsigned)p.blocks;
  const int layer = (int)(lb / (unsigned)p.B), b = (int)(lb % (unsigned)p.B);
  const int2 plan = p.plan[lb];
  if (layer == 0 && blk == 0 && threadIdx.x == 0) p.new_len[b] = plan.x >= 0 ? plan.x : p.cache_len[b];
  const int vpr = p.row_vecs;
  const int c = (int)blk * p.col + (int)threadIdx.x % p.col;
  const bool on = c < vpr;
  Tv* kv = reinterpret_cast<Tv*>(p.kv) + ((int64_t)layer * p.layer_stride_rows + p.cache_off[b]) * vpr + c;
  const int32_t* src = p.src + (int64_t)lb * p.max_keep;
  const int step = kMoveThreads / p.col, row = (int)threadIdx.x / p.col;
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
      if (at[u] >= 0) v[u] = kv[(int64_t)at[u] * vpr];
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
      if (on && j < plan.x) kv[(int64_t)j * vpr] = w[u];
    }
  }
}

// The selection's shared-memory opt-in, once per device.
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

template <typename Tv>
static int launch_move(EvictParams p, cudaStream_t stream) {
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
    p.blocks = (p.row_vecs + p.col - 1) / p.col;
  }
  if (lbs * p.blocks > 0x7fffffffLL) return DDT_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)(lbs * p.blocks);
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
  // shared memory for the longest cache the caller announces; a longer one
  // (or one beyond what an SM holds) re-reads its scores instead
  p.held_keys = std::min(kSelKeys, (std::min(max_cache_len, kMaxLen) + 1023) / 1024 * 1024);
  const int smem = p.held_keys * 4;
  if (smem > 32 * 1024 && !opt_in()) return DDT_ERR_CUDA;
  const int st = launch_pdl(evict_select_kernel, (unsigned)(p.n_layers * p.B), kSelThreads, (size_t)smem, stream, p);
  if (st != DDT_OK) return st;
  auto al = [](const void* q, uintptr_t a) { return reinterpret_cast<uintptr_t>(q) % a == 0; };
  if (p.row_bytes % 16 == 0 && al(p.kv, 16) && al(p.kv_dst, 16)) return launch_move<uint4>(p, stream);
  return launch_move<uint32_t>(p, stream);
}

}  // namespace ddt
