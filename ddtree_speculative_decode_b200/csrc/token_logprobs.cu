// Log probabilities of given tokens at selected verify rows, with the rows'
// entropy and their top alternatives.
//
// What it computes is fixed in ddt.h (ddt_token_logprobs). With m the row's
// largest logit, one pass over the row gives
//   s = sum_v e^(x_v - m),  u = sum_v e^(x_v - m) (x_v - m)
// and from them logsumexp = m + ln s, log p_t = (x_t - m) - ln s and the
// entropy ln s - u / s (both terms are >= 0, so nothing cancels). Partial
// (m, s, u) of two parts of a row join exactly: with d = m - M,
// s e^d and (u + d s) e^d are the sums relative to M.
//
// Bound: HBM, every logit of a selected row read once. At 6.5 TB/s an SM gets
// about 12 bf16 logits per cycle, so a logit may cost 10 issue slots and 1.3
// turns of the ex2 units: the sums run on packed float pairs relative to an
// integer power of two (one fma gives a pair's exponents), and that reference
// moves only when a logit exceeds it by 2^16, so almost never after the first
// loads.
//
// Work split: a fixed grid of 256-thread CTAs (three per SM) in clusters of up
// to 8. Full waves take a row per CTA; the rows left over are shared by C CTAs
// of a cluster each, C chosen on the device from their number (the shortest
// estimated makespan: rounds of rows x (slice + a fixed cost per slice)). A
// slice's result goes to the group's first CTA through distributed shared
// memory; the cluster barrier for it is split (arrive after a row, wait after
// the next one), so the join of a row overlaps the next row's loads.
//
// Loads: every thread copies its own vectors into its own slots of a
// three-stage ring in shared memory (cp.async), three rounds of four vectors
// ahead and across row ends, so the memory stays busy while a row is joined;
// a thread reads only what it copied, so the ring needs no barrier.
//
// Top alternatives: packed keys (order-preserving value bits << 32 | ~index:
// the larger key is the larger value at the lower index). The pass over the row
// keeps only, per thread and place in the round (a unit: every 1024th vector),
// the largest value so far. At the end each warp publishes the j-th largest of
// its threads' largest values; the r-th largest of the warps' is a bound that
// at least r j >= K values of the slice reach (r = min(K, 4), j = ceil(K / r)).
// The few units whose largest value reaches it are read once more, by the whole
// warp, for the keys of the values that do. (Collecting keys on the way, by a
// bound that rises with the row, took 5 instructions per logit instead of 1 and
// had to give up on rising rows.) If more than kPick values reach the bound
// (rows of few distinct values), the slice is read once more with care.
//
// Measured (bf16, rows of 163840; us): 512 rows 34.7 without alternatives, 45
// with 8, 58 with 32; 2048 rows 111 without (6.0 TB/s), 136 with 8; 4096 rows
// 244 to 274 with one (4.9 to 5.5 TB/s); instructions per logit 7.7 with none or
// one, 9.7 with 8, of which the row's end is the difference. Constant rows, which
// are all read again with care: one 84 (an ordinary one 9 with 1 or 8
// alternatives), 64 136 (14), 512 700 (41 to 45); 512 rows of 300 distinct
// values 400 to 440.
#include <algorithm>
#include <mutex>

#include "ddt_kernels.cuh"
#include "sm100_ptx.cuh"
#include "topk_keys.cuh"

namespace ddt {
namespace tlp {

using sm100::cluster_ctarank;
using sm100::cluster_sync;
using sm100::map_to_rank;
using sm100::smem_u32;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kU = 4;             // vectors per thread and round
constexpr int kRound = kU * kThreads;
constexpr int kStages = 3;        // rounds of the ring
constexpr int kRingBytes = kStages * kRound * 16;
constexpr int kMaxC = 8;          // CTAs that may share a row
constexpr int kOwn = 256;         // rows of one CTA in a launch that follows a node list
constexpr int kStep = 64;         // threads that add keys between two looks in the careful pass
constexpr int kBest = 4;          // warps whose published values make the bound
constexpr int kCand = 768;        // keys of the careful pass's buffer
constexpr int kFew = 8;           // up to this many alternatives the warps' bound is tight enough
constexpr int kPick = 128;        // keys that reach the bound
constexpr float kFar = -150.0f;   // e^kFar and 2^kFar are zero in float32
constexpr float kUsual = 1e6f;    // below this, a logit in base 2 is off by less than one before it is rounded
constexpr float kUsualTop = 999999.9375f;  // the largest float below kUsual
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kAhead = 16.0f;   // base-2 exponents may exceed the reference by this much

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// pairs of floats in one 64-bit register
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (m, s, u) of part of a row: m its largest logit (NaN if one is), s = sum
// e^d and u = sum e^d d with d = x - m. Empty: m = -inf, s = u = 0.
struct Sums {
  float m, s, u;
};
// The join of kLanes lanes' parts (a power of two), in every one of them: their
// largest m, and the sums relative to it.
template <int kLanes>
__device__ __forceinline__ Sums join(Sums a) {
  float M = a.m;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(DDT_FULL_MASK, M, o));
  const float d = fmaxf(a.m - M, kFar), e = ex2_ftz(d * kLog2e);  // an empty part has s = u = 0: any finite d does
  a.u = (a.u + d * a.s) * e;
  a.s *= e;
  a.m = M;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(DDT_FULL_MASK, a.s, o);
    a.u += __shfl_xor_sync(DDT_FULL_MASK, a.u, o);
  }
  return a;
}

// How many of n keys in shared memory are larger than this one (keys differ):
// its place among them. Independent broadcasts and compares, a third of a
// sorting network's latency for the 10 to 40 keys that are left.
__device__ __forceinline__ int rank_of(unsigned long long key, const unsigned long long* keys, int n) {
  int r = 0;
#pragma unroll 4
  for (int i = 0; i + 1 < n; i += 2) {
    const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(keys + i);
    r += (k.x > key ? 1 : 0) + (k.y > key ? 1 : 0);
  }
  if (n & 1) r += keys[n - 1] > key ? 1 : 0;
  return r;
}

struct Part {  // one CTA's share of a row
  Sums sums;
  float pad;
  uint32_t bounds[kWarps];      // its warps' published values
  unsigned long long keys[32];  // its best keys (0: none), in any order
};

template <bool kBF16>
struct Vec {
  static constexpr int kPer = kBF16 ? 8 : 4;
};

template <bool kBF16>
__device__ __forceinline__ float value_of(const uint4& r, int t) {
  const uint32_t w = t < (kBF16 ? 2 : 1) ? r.x : t < (kBF16 ? 4 : 2) ? r.y : t < (kBF16 ? 6 : 3) ? r.z : r.w;
  if (!kBF16) return __uint_as_float(w);
  return __uint_as_float((t & 1) ? (w & 0xffff0000u) : (w << 16));
}

// two neighbouring values, raised to at least -1e38 (0xfe96 in bf16), where
// the exponential is zero and the exponent still finite
template <bool kBF16>
__device__ __forceinline__ void pair_of(const uint4& r, int t, float& a, float& b) {
  if (kBF16) {
    uint32_t w = t < 2 ? r.x : t < 4 ? r.y : t < 6 ? r.z : r.w;
    asm("max.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(0xfe96fe96u));
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
  } else {
    a = fmaxf(value_of<kBF16>(r, t), -1e38f);
    b = fmaxf(value_of<kBF16>(r, t + 1), -1e38f);
  }
}

// Running maxima of whole vectors, NaN if one is: packed for bf16.
template <bool kBF16>
struct Max;
template <>
struct Max<true> {
  __nv_bfloat162 v;
  __device__ __forceinline__ Max() {}
  __device__ __forceinline__ static __nv_bfloat162 h(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  __device__ __forceinline__ explicit Max(const uint4& r) : v(__hmax2_nan(__hmax2_nan(h(r.x), h(r.y)), __hmax2_nan(h(r.z), h(r.w)))) {}
  __device__ __forceinline__ void add(const Max& o) { v = __hmax2_nan(v, o.v); }
  __device__ __forceinline__ float value() const { return max_nan(__low2float(v), __high2float(v)); }
};
template <>
struct Max<false> {
  float v;
  __device__ __forceinline__ Max() {}
  __device__ __forceinline__ explicit Max(const uint4& r) {
    v = max_nan(max_nan(__uint_as_float(r.x), __uint_as_float(r.y)), max_nan(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  __device__ __forceinline__ void add(const Max& o) { v = max_nan(v, o.v); }
  __device__ __forceinline__ float value() const { return v; }
};

// An end of a row: the elements before full0 (side 0, at the back of the
// vector) or from full1 on (side 1, at its front); the rest is -inf, which no
// sum and no key takes.
template <bool kBF16>
__device__ __noinline__ uint4 load_edge(const unsigned char* row, int V, int full0, int full1, int side) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  const int pos = side ? full1 : full0 - Vec<kBF16>::kPer, lo = side ? full1 : 0, hi = side ? V : full0;
#pragma unroll
  for (int t = 0; t < Vec<kBF16>::kPer; ++t) {
    const int i = pos + t;
    const bool in = i >= lo && i < hi;
    if (kBF16) {
      const uint32_t x = in ? reinterpret_cast<const uint16_t*>(row)[i] : 0xff80u;
      w[t / 2] |= x << (16 * (t & 1));
    } else {
      w[t] = in ? reinterpret_cast<const uint32_t*>(row)[i] : 0xff800000u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The values of a vector that reach tv, one bit each (no -inf).
template <bool kBF16>
__device__ __forceinline__ unsigned hits_of(const uint4& v, float tv) {
  unsigned hits = 0u;
#pragma unroll
  for (int q = 0; q < Vec<kBF16>::kPer; ++q) {
    const float x = value_of<kBF16>(v, q);
    hits |= x >= tv && x > -INFINITY ? 1u << q : 0u;
  }
  return hits;
}
// Writes their keys to buf[at ..], as far as they fit in room and reach T;
// place_of gives each its place.
template <bool kBF16, typename F>
__device__ __forceinline__ void write_keys(const uint4& v, unsigned hits, int at, unsigned long long T,
                                           unsigned long long* buf, int room, F place_of) {
  while (hits) {
    const int q = __ffs(hits) - 1;
    hits &= hits - 1u;
    float x;
    if (kBF16) {
      const uint32_t w = q < 2 ? v.x : q < 4 ? v.y : q < 6 ? v.z : v.w;
      x = __uint_as_float((q & 1) ? (w & 0xffff0000u) : (w << 16));
    } else {
      x = __uint_as_float(q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w);
    }
    const unsigned long long key = topk_key(x, at + q);
    if (key < T) continue;
    const int slot = place_of();
    if (slot < room) buf[slot] = key;
  }
}
// Careful pass: any number of values, places by count.
template <bool kBF16>
__device__ __noinline__ void append_keys(uint4 v, int at, unsigned long long T, float tv, unsigned long long* cand,
                                         int* count) {
  write_keys<kBF16>(v, hits_of<kBF16>(v, tv), at, T, cand, kCand, [&]() { return atomicAdd(count, 1); });
}
// The keys of one lane's values, from its place on.
template <bool kBF16>
__device__ __noinline__ void place_keys(uint4 v, unsigned hits, int at, unsigned long long* buf, int place) {
  write_keys<kBF16>(v, hits, at, 1ull, buf, kPick, [&]() { return place++; });
}

// One key per lane into descending order; rolled and out of line, as is the
// merge: both run once or a few times per row, and a row's latency is mostly
// the code that has to be fetched for it.
__device__ __noinline__ unsigned long long sort_list(unsigned long long x, int lane) {
#pragma unroll 1
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
      const unsigned long long y = __shfl_xor_sync(DDT_FULL_MASK, x, j);
      x = (((lane & j) == 0) == ((lane & k) == 0)) == (y > x) ? y : x;
    }
  }
  return x;
}
// merge of two lists sorted over the lanes (descending): the 32 best, sorted
__device__ __noinline__ unsigned long long merge_lists(unsigned long long a, unsigned long long b, int lane) {
  const unsigned long long r = __shfl_sync(DDT_FULL_MASK, b, 31 - lane);
  unsigned long long x = a > r ? a : r;
#pragma unroll 1
  for (int j = 16; j > 0; j >>= 1) {
    const unsigned long long y = __shfl_xor_sync(DDT_FULL_MASK, x, j);
    x = ((lane & j) == 0) == (y > x) ? y : x;
  }
  return x;
}

// Sorts the buffer's first n keys into its 32 best: every warp its share,
// then warp 0 the warps' lists. Warp 0 returns the list over its lanes. The
// caller's barrier comes before; one barrier inside.
__device__ __forceinline__ unsigned long long best_of(const unsigned long long* cand, int n,
                                                      unsigned long long (*lists)[32], int warp, int lane) {
  unsigned long long l = 0ull;
  for (int c = warp * 32; c < n; c += kThreads) {
    const int i = c + lane;
    l = merge_lists(l, sort_list(i < n ? cand[i] : 0ull, lane), lane);
  }
  lists[warp][lane] = l;
  __syncthreads();
  if (warp == 0) {
    const int used = min(kWarps, (n + 31) / 32);
#pragma unroll 1
    for (int w = 1; w < used; ++w) l = merge_lists(l, lists[w][lane], lane);
  }
  return l;
}

// The K best keys of a slice of which too many values reach the bound: its whole
// vectors [v0, v1) once more (and the row's ends, if it has them), kStep
// threads at a time between looks at the buffer's level, the bound raised to
// the K-th best key whenever the buffer could run full. Leaves the 32 best.
template <bool kBF16>
__device__ __noinline__ void careful_keys(const unsigned char* row, int V, int full0, int full1, int v0, int v1, bool ends,
                                          int K, unsigned long long* cand, int* count,
                                          unsigned long long (*lists)[32]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = Vec<kBF16>::kPer;
  unsigned long long T = 1ull;
  __syncthreads();
  if (tid == 0) *count = 0;
  __syncthreads();
  for (int r0 = v0; r0 < v1 + (ends ? kStep : 0); r0 += kStep) {
    const bool end = r0 >= v1;  // the last trip
    const int i = r0 + tid;
    const bool mine = end ? tid < 2 : tid < kStep && i < v1;
    if (mine) {
      const int pos = end ? (tid == 0 ? full0 - kPer : full1) : full0 + i * kPer;
      const uint4 x = end ? load_edge<kBF16>(row, V, full0, full1, tid)
                          : __ldg(reinterpret_cast<const uint4*>(row + (long long)pos * (kBF16 ? 2 : 4)));
      append_keys<kBF16>(x, pos, T, T == 1ull ? -INFINITY : key_value(T), cand, count);
    }
    __syncthreads();
    const int level = *count;
    __syncthreads();  // everyone has read the level before the next trip adds to it: one branch for the whole CTA
    if (level > kCand - kStep * 8) {
      const unsigned long long l = best_of(cand, level, lists, warp, lane);
      if (warp == 0) cand[lane] = l;
      if (tid == 0) *count = 32;
      __syncthreads();
      const unsigned long long kth = cand[K - 1];
      T = kth > T ? kth : T;
    }
    if (end) break;
  }
  const unsigned long long l = best_of(cand, *count, lists, warp, lane);
  if (warp == 0) cand[lane] = l;
  __syncthreads();
}

// The r-th largest of the warps' published values (0 if fewer are published).
__device__ __forceinline__ uint32_t nth_largest(const uint32_t* values, int r, int lane) {
  uint32_t x = lane < kWarps ? *const_cast<const volatile uint32_t*>(values + lane) : 0u, top = 0u;
#pragma unroll 1
  for (int i = 0; i < r; ++i) {
    top = __reduce_max_sync(DDT_FULL_MASK, x);
    const unsigned who = __ballot_sync(DDT_FULL_MASK, x == top);
    if (lane == __ffs(who) - 1) x = 0u;
  }
  return top;
}

template <bool kBF16, bool kTop>
__global__ void __launch_bounds__(kThreads, 3) token_logprobs_kernel(LogprobsParams p) {
  extern __shared__ __align__(16) unsigned char s_ring[];  // [kStages][kU][kThreads] vectors
  __shared__ int s_list[kOwn];  // this CTA's entries of a node list
  __shared__ int s_row[kOwn];   // and their logits rows, -1: no such node
  __shared__ int s_wcount[kWarps];
  __shared__ Sums s_sums[2][kWarps];
  __shared__ __align__(16) Part s_part[2][kMaxC];
  __shared__ unsigned long long s_cand[kTop ? kCand : 1];
  __shared__ unsigned long long s_lists[kTop ? kWarps : 1][32];
  __shared__ __align__(16) unsigned long long s_pick[kTop ? kPick : 1], s_last[kTop ? kMaxC * 32 : 1];
  __shared__ int s_count, s_picked[3];  // s_picked, s_bound: by the row's number, read after the row's last barrier
  __shared__ uint32_t s_max[kTop ? kThreads : 1];  // the threads' largest values, upper halves of their keys
  __shared__ uint16_t s_unit[kTop ? kWarps : 1][kU * 32];  // a warp's units that reach the bound
  __shared__ uint4 s_ends[2];
  __shared__ __align__(16) uint32_t s_bound[3][kWarps];  // by the row's number: the warps' j-th largest values, 0 for none
  constexpr int kPer = Vec<kBF16>::kPer;
  constexpr int kElt = kBF16 ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int csize = p.cluster;
  const int crank = csize > 1 ? (int)cluster_ctarank() : 0;
  const int V = p.V, K = p.K;

  pdl_wait();
  pdl_launch_dependents();

  // ---- the selected entries: all of them, or those of the list whose node is
  // not negative, counted by warps over their eighths of it, four neighbouring
  // entries per lane (every CTA reads the whole list, so a list of 16384
  // entries must not cost it more than a few hundred instructions per warp)
  int live = p.R, before = 0;
  const int eighth = (p.R + 128 * kWarps - 1) / (128 * kWarps) * 128, e0 = warp * eighth, e1 = min(p.R, e0 + eighth);
  const int32_t* list = p.nodes ? p.nodes + p.e0 : nullptr;
  auto four = [&](int e) {  // entries e .. e + 3, -1 behind the end
    int4 x = make_int4(-1, -1, -1, -1);
    if (e + 3 < e1 && reinterpret_cast<uintptr_t>(list) % 16 == 0) return __ldg(reinterpret_cast<const int4*>(list + e));
    if (e < e1) x.x = __ldg(list + e);
    if (e + 1 < e1) x.y = __ldg(list + e + 1);
    if (e + 2 < e1) x.z = __ldg(list + e + 2);
    if (e + 3 < e1) x.w = __ldg(list + e + 3);
    return x;
  };
  if (p.nodes) {
#pragma unroll 4
    for (int e = e0 + 4 * lane; e < e1; e += 128) {
      const int4 x = four(e);
      before += (x.x >= 0 ? 1 : 0) + (x.y >= 0 ? 1 : 0) + (x.z >= 0 ? 1 : 0) + (x.w >= 0 ? 1 : 0);
    }
    before = __reduce_add_sync(DDT_FULL_MASK, before);
    // skipped entries: each CTA writes those of its share of the list
    const int share = (p.R + (int)gridDim.x - 1) / (int)gridDim.x, s0 = (int)blockIdx.x * share;
    for (int e = s0 + tid; e < min(p.R, s0 + share); e += kThreads) {
      if (__ldg(list + e) >= 0) continue;
      const long long o = p.e0 + e;
      p.logp[o] = 0.0f;
      if (p.entropy) p.entropy[o] = 0.0f;
      for (int k = 0; k < K; ++k) {
        p.top_logp[o * K + k] = -INFINITY;
        p.top_tok[o * K + k] = -1;
      }
      if (p.dev_status) p.dev_status[o] = DDT_OK;
    }
    if (lane == 0) s_wcount[warp] = before;
    __syncthreads();
    const int n = lane < kWarps ? s_wcount[lane] : 0;
    live = __reduce_add_sync(DDT_FULL_MASK, n);
    before = __reduce_add_sync(DDT_FULL_MASK, lane < warp ? n : 0);
  }
  if (live == 0) return;  // the same on every CTA

  // ---- full waves of a row per CTA, then C CTAs per row for the rows left
  // over: the C with the shortest makespan; a slice costs its vectors plus
  // about `fixed` vectors' time for its set-up and join
  const int grid = (int)gridDim.x;
  const int waves = live / grid, rest = live - waves * grid;
  int lc = p.log_share;  // log2 of C
  if (lc < 0) {
    lc = 0;
    // Measured (163840 bf16 values a row; us with rows left over whole, in halves
    // and in quarters): 512 rows (68 left) 45.1, 37.8, 34.3, with 8 alternatives
    // 54.9, 47.6, 44.7; 600 rows (156 left) 46.0, 38.8, 40.6 and 55.4, 48.3, 56.2;
    // 800 rows (356 left) 46.9, 50.1, 54.1 and 58.2, 65.5, 80.3. These
    // constants choose the shortest of each.
    const int fixed = kTop ? 1500 : 500;
    float best = 0.0f;
    for (int l = 0; rest > 0 && (1 << l) <= csize; ++l) {
      const unsigned g = (unsigned)grid >> l;
      const float cost = (float)(((unsigned)rest + g - 1u) / g) * (float)((V / kPer >> l) + fixed);
      if (l == 0 || cost < best) {
        best = cost;
        lc = l;
      }
    }
  }
  const int C = 1 << lc;
  const int groups = grid >> lc;
  const int group = (int)blockIdx.x >> lc, part = (int)blockIdx.x & (C - 1);
  const int lead = crank - part;  // the group's first CTA, as a rank of the cluster
  const int rows = waves + (rest + groups - 1) / groups;  // of every CTA, some of the last ones empty
  if (p.nodes) {  // this CTA's share of the selected entries, in order
    auto mine = [&](int e, int node, int ord) {
      const bool full = ord < waves * grid;
      const unsigned d = full ? (unsigned)grid : (unsigned)groups, x = full ? (unsigned)ord : (unsigned)(ord - waves * grid);
      const unsigned turn = x / d;
      if (x - turn * d != (full ? blockIdx.x : (unsigned)group)) return;
      const int it = (full ? 0 : waves) + (int)turn;
      s_list[it] = e;
      s_row[it] = node < p.N ? (int)((unsigned)(p.e0 + e) / (unsigned)p.M) * p.N + node : -1;
    };
    const unsigned lower = (1u << lane) - 1u;
#pragma unroll 2
    for (int c = e0; c < e1; c += 128) {
      const int e = c + 4 * lane;
      const int4 x = four(e);
      const unsigned v0 = __ballot_sync(DDT_FULL_MASK, x.x >= 0), v1 = __ballot_sync(DDT_FULL_MASK, x.y >= 0);
      const unsigned v2 = __ballot_sync(DDT_FULL_MASK, x.z >= 0), v3 = __ballot_sync(DDT_FULL_MASK, x.w >= 0);
      if ((v0 | v1 | v2 | v3) == 0u) continue;
      int ord = before + __popc(v0 & lower) + __popc(v1 & lower) + __popc(v2 & lower) + __popc(v3 & lower);
      before += __popc(v0) + __popc(v1) + __popc(v2) + __popc(v3);
      if (x.x >= 0) mine(e, x.x, ord++);
      if (x.y >= 0) mine(e + 1, x.y, ord++);
      if (x.z >= 0) mine(e + 2, x.z, ord++);
      if (x.w >= 0) mine(e + 3, x.w, ord);
    }
    __syncthreads();
  }
  if (C > 1) cluster_sync();      // every CTA of the cluster runs before its shared memory is written

  // the it-th row of this CTA: its entry (-1: none), its logits (null: none)
  // and its share
  auto locate = [&](int it, long long& entry, const unsigned char*& row) {
    const int ord = it < waves ? it * grid + (int)blockIdx.x : waves * grid + (it - waves) * groups + group;
    entry = -1;
    row = nullptr;
    if (it >= rows || ord >= live) return;
    long long r;
    if (p.nodes) {
      entry = p.e0 + s_list[it];
      r = s_row[it];
    } else {
      entry = ord;
      const unsigned b = (unsigned)ord / (unsigned)p.M;
      r = (long long)b * p.N + ((unsigned)ord - b * (unsigned)p.M);
    }
    if (r >= 0) row = static_cast<const unsigned char*>(p.logits) + r * p.row_stride * kElt;
  };
  // whole 16-byte vectors of memory in the row: from element full0 on, nfull
  // of them; what is before and behind are the row's ends
  auto shape = [&](const unsigned char* row, int& full0, int& nfull) {
    const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / kElt);
    full0 = min(V, mis ? kPer - mis : 0);
    nfull = (V - full0) / kPer;
  };
  auto share = [&](int it, int nfull, int& v0, int& v1) {
    const int l = it < waves ? 0 : lc, k = it < waves ? 0 : part;
    const int per = (nfull + (1 << l) - 1) >> l;
    v0 = min(nfull, k * per);
    v1 = min(nfull, v0 + per);
  };

  // ---- the copies run ahead of the sums, round by round over all rows
  const uint32_t ring = smem_u32(s_ring) + (uint32_t)tid * 16u;
  int f_it = -1, f_left = 0;  // the row being copied and its vectors left, the same for the CTA
  uint32_t f_slot = 0u;       // byte offset of the stage
  const unsigned char* f_src = nullptr;
  auto fetch_round = [&]() {  // of a row with a whole round left
#pragma unroll
    for (int u = 0; u < kU; ++u) copy_async(ring + f_slot + (uint32_t)(u * kThreads * 16), f_src + u * kThreads * 16);
    copy_commit();
    f_src += kRound * 16;
    f_left -= kRound;
    f_slot = f_slot == (kStages - 1) * kRound * 16 ? 0u : f_slot + kRound * 16;
  };
  auto fetch = [&]() {
    while (f_left <= 0 && f_it + 1 < rows) {
      ++f_it;
      long long entry;
      const unsigned char* row;
      locate(f_it, entry, row);
      if (row) {
        int full0, nfull, v0, v1;
        shape(row, full0, nfull);
        share(f_it, nfull, v0, v1);
        f_left = v1 - v0;
        f_src = row + (long long)full0 * kElt + (long long)(v0 + tid) * 16;
      }
    }
    if (f_left >= kRound) {
      fetch_round();
      return;
    }
    if (f_left > 0) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (f_left > tid + u * kThreads)
          copy_async(ring + f_slot + (uint32_t)(u * kThreads * 16), f_src + u * kThreads * 16);
    }
    copy_commit();
    f_src += kRound * 16;
    f_left -= kRound;
    f_slot = f_slot == (kStages - 1) * kRound * 16 ? 0u : f_slot + kRound * 16;
  };
#pragma unroll 1
  for (int g = 0; g < kStages; ++g) fetch();
  uint32_t slot = (uint32_t)tid * 16u;  // of this thread, in the stage the sums are at

  // the join of a finished row by warp 0 of the group's first CTA
  float xt = 0.0f, xt_prev = 0.0f;
  long long ent_prev = -1;
  int st = DDT_OK, st_prev = DDT_OK;
  auto finish = [&](int buf, int c, long long entry, float x, int status) {
    const Part* q = s_part[buf];
    Sums a = lane < c ? q[lane].sums : Sums{-INFINITY, 0.0f, 0.0f};
    a = join<kMaxC>(a);
    a.m = __shfl_sync(DDT_FULL_MASK, a.m, 0);
    a.s = __shfl_sync(DDT_FULL_MASK, a.s, 0);
    a.u = __shfl_sync(DDT_FULL_MASK, a.u, 0);
    // a NaN or +inf logit, or no finite one
    const bool bad = status != DDT_OK || !(fabsf(a.m) <= 3.402823466e38f);
    const float lns = log2f(a.s) * kLn2;
    if (lane == 0) {
      p.logp[entry] = bad ? -INFINITY : (x - a.m) - lns;
      if (p.entropy) p.entropy[entry] = bad ? 0.0f : fmaxf(lns - a.u / a.s, 0.0f);
      if (p.dev_status) p.dev_status[entry] = bad ? DDT_ERR_INPUT : DDT_OK;
    }
    if (kTop) {
      // The bound of the whole row, from the warps of all its slices (at
      // least min(K, kBest) of them publish, unless the row is short), and the
      // keys that reach it: about K. Independent steps throughout: this is
      // the end of a row's latency.
      uint32_t x0 = lane < 4 * c ? q[lane >> 2].bounds[(lane & 3) * 2] : 0u;
      uint32_t x1 = lane < 4 * c ? q[lane >> 2].bounds[(lane & 3) * 2 + 1] : 0u;
      const int full = __popc(__ballot_sync(DDT_FULL_MASK, x0 != 0u)) + __popc(__ballot_sync(DDT_FULL_MASK, x1 != 0u));
      // every warp's value is its j-th largest with j >= ceil(K / kBest)
      const int need = min(K, kBest);
      uint32_t top = 0u;
      if (full >= need) {
#pragma unroll 1
        for (int i = 0; i < need; ++i) {
          top = __reduce_max_sync(DDT_FULL_MASK, max(x0, x1));
          const unsigned who = __ballot_sync(DDT_FULL_MASK, max(x0, x1) == top);
          if (lane == __ffs(who) - 1) {
            if (x0 >= x1) x0 = 0u;
            else x1 = 0u;
          }
        }
      }
      int n = 0;
#pragma unroll
      for (int r = 0; r < kMaxC; ++r) {
        const unsigned long long key = r < c ? q[r].keys[lane] : 0ull;
        const bool keep = !bad && key != 0ull && (uint32_t)(key >> 32) >= top;
        const unsigned votes = __ballot_sync(DDT_FULL_MASK, keep);
        if (keep) s_last[n + __popc(votes & ((1u << lane) - 1u))] = key;
        n += __popc(votes);
      }
      __syncwarp();
#pragma unroll 1
      for (int i = lane; i < n; i += 32) {
        const unsigned long long key = s_last[i];
        const int r = rank_of(key, s_last, n);
        if (r < K) {
          p.top_logp[entry * K + r] = (key_value(key) - a.m) - lns;
          p.top_tok[entry * K + r] = static_cast<int32_t>(~static_cast<uint32_t>(key));
        }
      }
      for (int r = n + lane; r < K; r += 32) {  // fewer tokens than K are possible
        p.top_logp[entry * K + r] = -INFINITY;
        p.top_tok[entry * K + r] = -1;
      }
    }
  };

  if (kTop) {
    if (tid < 3 * kWarps) s_bound[tid / kWarps][tid % kWarps] = 0u;
    if (tid == 0) s_picked[0] = s_picked[1] = s_picked[2] = 0;
    __syncthreads();
  }
  int turn3 = 2;  // it mod 3
#pragma unroll 1
  for (int it = 0; it < rows + (C > 1 ? 1 : 0); ++it) {  // shared rows are joined a turn later
    const bool whole = it < waves || C == 1;  // this CTA has the whole row
    const int buf = it & 1;
    turn3 = turn3 == 2 ? 0 : turn3 + 1;
    long long ent;
    const unsigned char* row;
    locate(it, ent, row);
    const bool on = ent >= 0;  // the same for the CTAs of a group
    Sums a = {-INFINITY, 0.0f, 0.0f};
    float tv = -INFINITY;  // at least K values of the slice reach it
    bool plain = true;     // the buffer held every key that reaches it
    if (kTop) {  // the next row's; nobody uses them before this row's barriers
      const int next3 = turn3 == 2 ? 0 : turn3 + 1;
      if (lane == 0) s_bound[next3][warp] = 0u;
      if (tid == 0) s_picked[next3] = 0;
    }
    if (on) {
      const int t = __ldg(p.tok + ent);
      st = DDT_ERR_INPUT;
      if (row) {
        int full0, nfull, v0, v1;
        shape(row, full0, nfull);
        share(it, nfull, v0, v1);
        const int full1 = full0 + nfull * kPer;
        const bool has_ends = (full0 > 0 || full1 < V) && (whole || part == 0);
        bool ends = has_ends;  // still to come
        const uint32_t inf = kBF16 ? 0xff80ff80u : 0xff800000u;
        const uint4 none = make_uint4(inf, inf, inf, inf);  // a vector past the slice counts as all -inf
        // Running sums as packed pairs, s2 = sum 2^y and u2 = sum 2^y y with y
        // = x log2 e - ref: exact up to one rounding because ref is an integer
        // (near the thread's largest logit in base 2); limit: the logit that
        // moves it.
        uint64_t s2 = 0ull, u2 = 0ull;
        float ref = 0.0f, limit = -INFINITY;
        const int first = min(kThreads, max(v1 - v0, ends ? 2 : 0));  // threads with values in round 0
        const int tr = max(1, min(min(K, kBest), (first + 31) / 32)), tj = (K + tr - 1) / tr;
        // this warp's tj-th largest of its threads' largest values
        auto publish = [&]() {
          uint32_t x = a.m > -INFINITY ? float_order_key(a.m) : 0u, top = 0u;
          const bool enough = __popc(__ballot_sync(DDT_FULL_MASK, x != 0u)) >= tj;  // otherwise it publishes none
          if (K > kFew) s_max[tid] = x >> 16;
#pragma unroll 1
          for (int q = 0; enough && q < tj; ++q) {
            top = __reduce_max_sync(DDT_FULL_MASK, x);
            const unsigned who = __ballot_sync(DDT_FULL_MASK, x == top);
            if (lane == __ffs(who) - 1) x = 0u;
          }
          if (lane == 0) *const_cast<volatile uint32_t*>(&s_bound[turn3][warp]) = top;
        };
        auto bound = [&]() {
          const uint32_t t = nth_largest(s_bound[turn3], tr, lane);
          if (t == 0u) return;
          tv = fmaxf(tv, key_value((unsigned long long)t << 32));
          if (K <= kFew) return;
          // Raised to the K-th largest of the threads' largest values (their
          // keys' upper halves, cut towards smaller values), by bisection: half
          // as many units and values reach it. 512 rows of 163840: 69 -> 60 us
          // with 32 alternatives, 58 -> 51 with 20; with 8 the bisection costs
          // what it saves (45 -> 44.5 us, 512 rows of 32000: 23 -> 24).
          uint32_t key[kWarps], hi = 0u, lo = t >> 16;
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            key[i] = s_max[i * 32 + lane];
            hi = max(hi, key[i]);
          }
          hi = __reduce_max_sync(DDT_FULL_MASK, hi);
#pragma unroll 1
          while (lo < hi) {
            const uint32_t mid = (lo + hi + 1u) >> 1;
            int n = 0;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) n += key[i] >= mid ? 1 : 0;
            if (__reduce_add_sync(DDT_FULL_MASK, n) >= K) lo = mid;
            else hi = mid - 1u;
          }
          tv = fmaxf(tv, key_value((unsigned long long)lo << 48));
        };
        // one round's sums; rm: the largest of its values (NaN if one is)
        auto sums = [&](const uint4 (&v)[kU], float rm) {
          if (!(rm <= limit)) {  // far larger than before (or the first), or a NaN, which stays
            const float M = max_nan(rm, a.m);
            float k, e;
            if (fabsf(a.m) < kUsual) {  // base 2 relative to ref -> base e relative to the old maximum
              k = fmaf(a.m, -kLog2e, ref);
              e = ex2_ftz(k);
              u2 = mul2(fma2(pack2(k, k), s2, u2), pack2(e * kLn2, e * kLn2));
              s2 = mul2(s2, pack2(e, e));
            }
            k = fmaxf(a.m - M, kFar);  // -> relative to the new one (nothing yet: sums of 0)
            e = ex2_ftz(k * kLog2e);
            u2 = mul2(fma2(pack2(k, k), s2, u2), pack2(e, e));
            s2 = mul2(s2, pack2(e, e));
            limit = M;
            if (fabsf(M) < kUsual) {  // -> base 2 relative to the new ref
              ref = ceilf(M * kLog2e);
              // no further than the usual logits: what passes it changes the sums' form here
              limit = fminf((ref + kAhead) * kLn2, kUsualTop);
              k = fmaf(M, kLog2e, -ref);
              e = ex2_ftz(k);
              u2 = mul2(fma2(u2, pack2(kLog2e, kLog2e), mul2(pack2(k, k), s2)), pack2(e, e));
              s2 = mul2(s2, pack2(e, e));
            }
            a.m = M;
          }
          a.m = max_nan(a.m, rm);
          if (fabsf(a.m) < kUsual) {
            const uint64_t nr2 = pack2(-ref, -ref), l2 = pack2(kLog2e, kLog2e);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
#pragma unroll
              for (int q = 0; q < kPer; q += 2) {
                float x0, x1, y0, y1;
                pair_of<kBF16>(v[u], q, x0, x1);
                const uint64_t y = fma2(pack2(x0, x1), l2, nr2);
                unpack2(y, y0, y1);
                const uint64_t e = pack2(ex2_ftz(y0), ex2_ftz(y1));
                s2 = add2(s2, e);
                u2 = fma2(e, y, u2);
              }
            }
          } else if (a.m != -INFINITY) {
            // rows of extreme values: s2 and u2 are sums of e^d and e^d d, d =
            // x - m, cut where the exponential is zero
#pragma unroll
            for (int u = 0; u < kU; ++u) {
#pragma unroll
              for (int q = 0; q < kPer; ++q) {
                const float d = fmaxf(value_of<kBF16>(v[u], q) - a.m, kFar), e = ex2_ftz(d * kLog2e);
                s2 = add2(s2, pack2(e, 0.0f));
                u2 = fma2(pack2(e, 0.0f), pack2(d, 0.0f), u2);
              }
            }
          }
        };
        Max<kBF16> um[kU];  // the largest values of this thread's units
        if (kTop) {
#pragma unroll
          for (int u = 0; u < kU; ++u) um[u] = Max<kBF16>(none);
        }
        auto largest = [&](const uint4 (&v)[kU]) {
          Max<kBF16> m(v[0]);
          if (kTop) um[0].add(m);
#pragma unroll
          for (int u = 1; u < kU; ++u) {
            const Max<kBF16> x(v[u]);
            if (kTop) um[u].add(x);
            m.add(x);
          }
          return m.value();
        };
        auto next_slot = [&](uint32_t x) { return x >= (kStages - 1) * kRound * 16 ? x - (kStages - 1) * kRound * 16 : x + kRound * 16; };
        int left = v1 - v0;
        // whole rounds: no conditions but the rare ones
#pragma unroll 1
        for (; left >= kRound; left -= kRound) {
          uint4 v[kU];
          copy_wait<kStages - 1>();
          const unsigned char* from = s_ring + slot;
#pragma unroll
          for (int u = 0; u < kU; ++u) v[u] = *reinterpret_cast<const uint4*>(from + u * kThreads * 16);
          slot = next_slot(slot);
          sums(v, largest(v));
          // this round's slots are free
          if (f_left >= kRound) fetch_round();
          else fetch();
        }
#pragma unroll 1
        for (; left > 0 || ends; left -= kRound) {
          uint4 v[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) v[u] = none;
          if (left > 0) {
            copy_wait<kStages - 1>();
            const unsigned char* from = s_ring + slot;
#pragma unroll
            for (int u = 0; u < kU; ++u)
              if (left > tid + u * kThreads) v[u] = *reinterpret_cast<const uint4*>(from + u * kThreads * 16);
            slot = next_slot(slot);
          } else {  // the row's ends
            ends = false;
            if (tid < 2) v[0] = s_ends[tid] = load_edge<kBF16>(row, V, full0, full1, tid);
          }
          sums(v, largest(v));
          if (left > 0) fetch();
        }
        // the given token's logit: its index has arrived by now, and the join
        // wants it much later
        st = t >= 0 && t < V ? DDT_OK : DDT_ERR_INPUT;
        if ((whole || part == 0) && warp == 0) {
          xt = 0.0f;
          if (st == DDT_OK) xt = kBF16 ? bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(row) + t))
                                       : __ldg(reinterpret_cast<const float*>(row) + t);
        }
        if (kTop) {
          publish();
          __syncthreads();
          bound();
          // one vector per lane and place: their keys that reach the bound go to the
          // CTA's list, in the places of one count
          auto pick = [&](const uint4 (&x)[kU], const int (&at)[kU]) {
            unsigned hits[kU];
            int own = 0;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              hits[u] = Max<kBF16>(x[u]).value() >= tv ? hits_of<kBF16>(x[u], tv) : 0u;
              own += __popc(hits[u]);
            }
            int place = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int y = __shfl_up_sync(DDT_FULL_MASK, place, o);
              if (lane >= o) place += y;
            }
            const int all = __shfl_sync(DDT_FULL_MASK, place, 31);
            if (all == 0) return true;
            int base = 0;
            if (lane == 0) base = atomicAdd(&s_picked[turn3], all);
            base = __shfl_sync(DDT_FULL_MASK, base, 0);
            place += base - own;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              if (hits[u]) place_keys<kBF16>(x[u], hits[u], at[u], s_pick, place);
              place += __popc(hits[u]);
            }
            return base + all <= kPick;  // otherwise the careful pass follows
          };
          int n = 0;  // units of this warp that reach the bound
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const float m = um[u].value();
            const bool reach = m >= tv && m > -INFINITY;
            const unsigned votes = __ballot_sync(DDT_FULL_MASK, reach);
            if (reach) s_unit[warp][n + __popc(votes & ((1u << lane) - 1u))] = (uint16_t)(u * kThreads + tid);
            n += __popc(votes);
          }
          __syncwarp();
          const unsigned char* vecs = row + (long long)full0 * kElt + (long long)v0 * 16;
          // all vectors of all these units, over the warp's lanes
          const unsigned per = (unsigned)(v1 - v0 + kRound - 1) / kRound, items = (unsigned)n * per;
#pragma unroll 1
          for (unsigned i0 = (unsigned)lane; i0 - (unsigned)lane < items; i0 += 32 * kU) {
            uint4 x[kU];
            int at[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              const unsigned i = i0 + 32 * u, unit = i / per;
              const int k = i < items ? (int)((i - unit * per) * kRound + s_unit[warp][unit]) : v1 - v0;
              at[u] = full0 + (v0 + k) * kPer;
              x[u] = k < v1 - v0 ? __ldg(reinterpret_cast<const uint4*>(vecs + (long long)k * 16)) : none;
            }
            if (!pick(x, at)) break;
          }
          if (has_ends && warp == 0) {
            uint4 x[kU];
            int at[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) x[u] = none, at[u] = 0;
            if (lane < 2) {
              x[0] = s_ends[lane];
              at[0] = lane == 0 ? full0 - kPer : full1;
            }
            pick(x, at);
          }
        }
        float s0, s1, u0, u1;
        unpack2(s2, s0, s1);
        unpack2(u2, u0, u1);
        a.s = s0 + s1;
        a.u = u0 + u1;
        if (fabsf(a.m) < kUsual) {  // from base 2 relative to ref to base e relative to m
          const float k = fmaf(a.m, -kLog2e, ref), ek = ex2_ftz(k);  // -kAhead <= k <= 1
          a.u = (a.u + k * a.s) * ek * kLn2;
          a.s *= ek;
        }
      }
      a = join<32>(a);
      if (lane == 0) s_sums[buf][warp] = a;
    }
    __syncthreads();
    if (kTop && on && s_picked[turn3] > kPick) {  // many equal values: the same for the whole CTA
      long long e2;
      const unsigned char* row2;
      locate(it, e2, row2);
      int full0, nfull, v0, v1;
      shape(row2, full0, nfull);
      share(it, nfull, v0, v1);
      const int full1 = full0 + nfull * kPer;
      careful_keys<kBF16>(row2, V, full0, full1, v0, v1, (full0 > 0 || full1 < V) && (whole || part == 0), K, s_cand,
                          &s_count, s_lists);
      if (warp == 0) s_pick[lane] = s_cand[lane];
      if (tid == 0) s_picked[turn3] = 32;
      plain = false;
      __syncthreads();
    }
    // the shared row before this one is complete in the group's first CTA
    __syncwarp();
    const bool turn = C > 1 && it > waves;
    if (turn) cluster_wait();
    if (warp == 0 && on) {
      const Sums b = join<kWarps>(lane < kWarps ? s_sums[buf][lane] : Sums{-INFINITY, 0.0f, 0.0f});
      const int to = whole ? 0 : part;
      Part* dst = &s_part[buf][to];
      // the slice's keys: all that are left if that is at most 32, else the 32 best
      const int n = kTop ? s_picked[turn3] : 0;
      const uint32_t base = map_to_rank(smem_u32(dst), (uint32_t)(to != 0 ? lead : crank));
      if (lane == 0) {
        st_cluster_f32(base, b.m);
        st_cluster_f32(base + 4, b.s);
        st_cluster_f32(base + 8, b.u);
      }
      if (kTop && lane < kWarps) st_cluster_u32(base + 16 + 4 * lane, plain ? s_bound[turn3][lane] : 0u);
      if (kTop && n <= 32) {
        st_cluster_u64(base + 16 + 4 * kWarps + 8 * lane, lane < n ? s_pick[lane] : 0ull);
      } else if (kTop) {
        for (int i = lane; i < n; i += 32) {
          const unsigned long long key = s_pick[i];
          const int r = rank_of(key, s_pick, n);
          if (r < 32) st_cluster_u64(base + 16 + 4 * kWarps + 8 * r, key);
        }
      }
      __syncwarp();
    }
    if (warp == 0) {
      const bool now = whole && on, before = turn && part == 0 && ent_prev >= 0;
      if (now || before)
        finish(now ? buf : buf ^ 1, now ? 1 : C, now ? ent : ent_prev, now ? xt : xt_prev, now ? st : st_prev);
      __syncwarp();
    }
    ent_prev = on ? ent : -1;
    st_prev = st;
    xt_prev = xt;
    if (C > 1 && it >= waves && it < rows) cluster_arrive();
  }
  copy_wait<0>();
}

template <bool kBF16, bool kTop>
static cudaLaunchConfig_t config(cudaLaunchAttribute* attr, int grid, int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRingBytes;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// CTAs of the kernel resident at once in such clusters on the current device
// (0: such clusters cannot be scheduled; -1: no such device), looked up once per
// device (with the shared-memory opt-in set).
template <bool kBF16, bool kTop>
static int resident_ctas(int cluster) {
  static std::mutex mu;
  static int known[kMaxDevices][kMaxC + 1];
  static bool have[kMaxDevices][kMaxC + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  std::lock_guard<std::mutex> lock(mu);
  if (!have[dev][cluster]) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config<kBF16, kTop>(attr, 4096, cluster, nullptr);
    if (cudaFuncSetAttribute(token_logprobs_kernel<kBF16, kTop>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRingBytes) != cudaSuccess)
      return -1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, token_logprobs_kernel<kBF16, kTop>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    known[dev][cluster] = n * cluster;
    have[dev][cluster] = true;
  }
  return known[dev][cluster];
}

template <bool kBF16, bool kTop>
static int launch_t(LogprobsParams p, cudaStream_t stream) {
  // slices of at least 4 KB; no more CTAs than the rows can use
  const int elt = kBF16 ? 2 : 4;
  const long long all = (long long)p.B * p.M;
  int slots = 0;
  auto fit = [&](int& cluster) {  // the largest cluster up to this one that can be scheduled, with slices of 4 KB
    while (cluster > 1 && (long long)p.V * elt < 4096LL * cluster) cluster >>= 1;
    for (;; cluster >>= 1) {
      slots = resident_ctas<kBF16, kTop>(cluster);
      if (slots != 0 || cluster == 1) break;
    }
    if (slots == 0) slots = 3 * sm_count();
  };
  // A node list selects few rows as a rule: clusters of 8 (a long list: of 4),
  // the split decided on the device. All rows: clusters of 4 (they leave fewer SMs unused) and
  // full waves if the rows fill the device; fewer rows are split so that one
  // wave of CTAs lies evenly on the SMs. One CTA alone keeps an SM about 45 %
  // busy, two 80 %.
  // Measured, lists (163840 bf16 values a row; us in clusters of 8 and of 4):
  // 2048 entries, 16 selected 10.6 and 11.4, 512 selected 45.5 and 37.4; 4096
  // entries, 16 selected 11.3 and 12.3, 592 selected 55.7 and 43.5.
  // All rows (us with 1, 2, 4 and 8 CTAs a row): 8 rows 11.1, 8.1, 6.1, 5.4; 32
  // rows 11.6, 8.5, 7.2, 8.2; 64 rows 12.0, 8.9, 10.1; 100 rows 12.3, 11.9,
  // 10.7; 148 rows 12.9, 15.3; 200 rows 17.9, 15.5. The estimate takes the
  // last column: right at the ends, up to a fifth too slow between (32, 64, 148
  // rows), two fifths for short rows with alternatives (48 rows of 32000 with 8:
  // 12.6 with 8 CTAs a row, 8.8 with 2).
  int cluster = p.nodes && all <= 2048 ? kMaxC : 4;
  fit(cluster);
  p.log_share = -1;
  if (!p.nodes && all < slots) {
    static const float load[4] = {0.0f, 2.2f, 2.5f, 3.0f};
    const float fixed = kTop ? 0.2f : 0.05f;  // of a row's time, per slice
    float best = -1.0f;
    int pick = 1;
    for (int l = 0; l < 4; ++l) {
      int c = 1 << l;
      fit(c);
      if (slots < 0) return DDT_ERR_CUDA;
      const long long ctas = all << l;
      if (c != 1 << l || ctas > slots) break;
      const float cost = load[std::min(3LL, (ctas + sm_count() - 1) / sm_count())] * (1.0f / c + fixed);
      if (best < 0.0f || cost < best) {
        best = cost;
        pick = c;
        p.log_share = l;
      }
    }
    cluster = pick;
    slots = (int)all * cluster;
  }
  if (slots < 0) return DDT_ERR_CUDA;
  p.cluster = cluster;
  const long long most = std::max(1, slots / cluster);
  const long long total = (long long)p.B * p.M;
  const long long ctas = most * cluster;
  const long long step = p.nodes ? std::min(1LL << 20, ctas * (kOwn / 2)) : total;
  for (long long e0 = 0; e0 < total; e0 += step) {
    p.e0 = e0;
    p.R = (int)std::min(step, total - e0);
    // A short list (a path among a tree's nodes) gets one CTA per SM rather
    // than three, which leaves room for the next kernel to start under this
    // one (8 rows of a list of 64: 7.2 against 9.0 us).
    const long long clusters = p.nodes ? std::max<long long>(p.R / 4, sm_count() / cluster) : p.R;
    const int grid = (int)(std::min({most, clusters, (long long)p.R}) * cluster);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config<kBF16, kTop>(attr, grid, cluster, stream);
    if (cudaLaunchKernelEx(&cfg, token_logprobs_kernel<kBF16, kTop>, p) != cudaSuccess) return DDT_ERR_CUDA;
  }
  return DDT_OK;
}

}  // namespace tlp

int launch_token_logprobs(LogprobsParams p, cudaStream_t stream) {
  if (p.logits_dtype == DDT_BF16)
    return p.K > 0 ? tlp::launch_t<true, true>(p, stream) : tlp::launch_t<true, false>(p, stream);
  return p.K > 0 ? tlp::launch_t<false, true>(p, stream) : tlp::launch_t<false, false>(p, stream);
}

}  // namespace ddt
