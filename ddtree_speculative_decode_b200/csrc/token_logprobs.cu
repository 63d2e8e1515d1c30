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
// about 12 bf16 logits per cycle, so a logit may cost about 10 issue slots
// and 1.3 exponentials' worth of its one ex2 unit per cycle and quarter: the
// sums run on packed float pairs (about 5 slots per logit) and the top
// alternatives must cost next to nothing per logit (see below).
//
// Work split: a fixed grid of 256-thread CTAs (four per SM) in clusters of up
// to 8; C of them (C | cluster size) share a row, C chosen on the device from
// the number of selected rows: the C that gives the shortest estimated
// makespan (rounds of rows x (slice + a fixed cost per slice)). Many rows: C
// = 1, no exchange at all; few rows: C = 8 for latency. The slices' partial
// results go to the group's first CTA through distributed shared memory;
// the cluster barrier they need is split (arrive after a row, wait after the
// next one), so the join of a row overlaps the next row's loads.
//
// Top alternatives: packed keys (order-preserving value bits << 32 | ~index:
// the larger key is the larger value at the lower index). The first round of
// loads gives a bound T that at least K keys of the slice reach: each warp
// sorts its threads' best keys, and T is the r-th largest over the warps of
// the warp's j-th best (r = min(K, 4), j = ceil(K / r)). From then on a
// vector costs one compare of its maximum with T's value and a vote; keys
// that reach T are appended to a buffer in shared memory. A round in which
// many threads hold such a value (rising rows) raises T from that round's
// best keys first, which bounds what one round can append. The buffer is
// sorted into the K best at the end of the slice, or when it runs full.
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
constexpr int kU = 4;             // 16-byte vectors in flight per thread
constexpr int kMaxC = 8;          // CTAs that may share a row
constexpr int kListMax = 4096;    // entries of a launch that follows a node list
constexpr int kManyThreads = 40;  // more threads than this at T or above: raise T first
// keys appended between two looks at the buffer's level: a round's from at
// most kManyThreads threads, or one vector of every thread
constexpr int kRoundMax = kManyThreads * kU * 8 > kThreads * 8 ? kManyThreads * kU * 8 : kThreads * 8;
constexpr int kCand = 512 + kRoundMax;
constexpr float kFar = -150.0f;   // 2^kFar is zero in float32: the floor of the base-2 exponents

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
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
// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (m, s, u) of part of a row: m the largest logit (NaN if one is), s and u in
// base 2: s = sum 2^y, u = sum 2^y y with y = (x - m) log2 e. Empty: m = -inf.
struct Sums {
  float m, s, u;
};
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  const float M = max_nan(a.m, b.m);
  // an empty part (m = -inf) has s = u = 0: any finite exponent does
  const float da = fmaxf((a.m - M) * kLog2e, kFar), db = fmaxf((b.m - M) * kLog2e, kFar);
  const float ea = ex2_ftz(da), eb = ex2_ftz(db);
  return {M, a.s * ea + b.s * eb, (a.u + da * a.s) * ea + (b.u + db * b.s) * eb};
}

struct Part {  // one CTA's share of a row
  Sums sums;
  float pad;
  unsigned long long keys[32];
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

template <bool kBF16>
__device__ __forceinline__ float vec_max(const uint4& r) {  // NaN if one is
  if (kBF16) {
    auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 a = __hmax2_nan(__hmax2_nan(h(r.x), h(r.y)), __hmax2_nan(h(r.z), h(r.w)));
    return max_nan(__low2float(a), __high2float(a));
  }
  return max_nan(max_nan(__uint_as_float(r.x), __uint_as_float(r.y)),
                 max_nan(__uint_as_float(r.z), __uint_as_float(r.w)));
}

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

// Appends the vector's keys that reach T to the CTA's buffer.
template <bool kBF16>
__device__ __noinline__ void append_keys(uint4 v, int at, unsigned long long T, unsigned long long* cand, int* count) {
#pragma unroll
  for (int q = 0; q < Vec<kBF16>::kPer; ++q) {
    const float x = value_of<kBF16>(v, q);
    const unsigned long long key = topk_key(x, at + q);
    if (x > -INFINITY && key >= T) {
      const int slot = atomicAdd(count, 1);
      if (slot < kCand) cand[slot] = key;  // always: see kRoundMax
    }
  }
}

// merge of two lists sorted over the lanes (descending): the 32 best, sorted
__device__ __forceinline__ unsigned long long merge_lists(unsigned long long a, unsigned long long b, int lane) {
  const unsigned long long r = __shfl_sync(DDT_FULL_MASK, b, 31 - lane);
  return warp_merge_desc(a > r ? a : r, lane);
}

template <bool kBF16, bool kTop>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_kernel(LogprobsParams p) {
  __shared__ uint16_t s_list[kListMax];
  __shared__ int s_wcount[kWarps], s_live;
  __shared__ Sums s_sums[2][kWarps];
  __shared__ __align__(16) Part s_part[2][kMaxC];
  __shared__ unsigned long long s_cand[kTop ? kCand : 1];
  __shared__ unsigned long long s_lists[kTop ? kWarps : 1][32];
  __shared__ int s_count;
  constexpr int kPer = Vec<kBF16>::kPer;
  constexpr int kElt = kBF16 ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int csize = p.cluster;
  const int crank = csize > 1 ? (int)cluster_ctarank() : 0;
  const int V = p.V, K = p.K;

  pdl_wait();
  pdl_launch_dependents();

  // ---- the selected entries: all of them, or those of the list whose node is
  // not negative; the others are written as skipped by the CTAs in turn
  int live = p.R;
  if (p.nodes) {
    if (tid == 0) s_live = 0;
    __syncthreads();
    int base = 0;
    for (int c0 = 0; c0 < p.R; c0 += kThreads) {
      const int e = c0 + tid;
      const bool on = e < p.R && __ldg(p.nodes + p.e0 + e) >= 0;
      const unsigned votes = __ballot_sync(DDT_FULL_MASK, on);
      if (lane == 0) s_wcount[warp] = __popc(votes);
      __syncthreads();
      int at = base + __popc(votes & ((1u << lane) - 1u));
      int all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int n = s_wcount[w];
        at += w < warp ? n : 0;
        all += n;
      }
      base += all;
      if (on) s_list[at] = (uint16_t)e;
      if (!on && e < p.R && e % (int)gridDim.x == (int)blockIdx.x) {
        const long long o = p.e0 + e;
        p.logp[o] = 0.0f;
        if (p.entropy) p.entropy[o] = 0.0f;
        for (int k = 0; k < K; ++k) {
          p.top_logp[o * K + k] = -INFINITY;
          p.top_tok[o * K + k] = -1;
        }
        if (p.dev_status) p.dev_status[o] = DDT_OK;
      }
      __syncthreads();
    }
    live = base;
  }
  if (live == 0) return;  // the same on every CTA

  // ---- CTAs per row: the C with the shortest makespan; a slice costs its
  // vectors plus about kSliceCost vectors' time for its set-up and join
  constexpr int kSliceCost = 1500;
  int C = 1;
  {
    long long best = -1;
    for (int c = 1; c <= csize; c <<= 1) {
      const long long groups = gridDim.x / c;
      const long long cost = ((live + groups - 1) / groups) * (V / kPer / c + kSliceCost);
      if (best < 0 || cost < best) {
        best = cost;
        C = c;
      }
    }
  }
  const int groups = (int)gridDim.x / C;
  const int group = (int)blockIdx.x / C, part = (int)blockIdx.x % C;
  const int lead = crank - part;  // the group's first CTA, as a rank of the cluster
  const int rounds = (live + groups - 1) / groups;
  if (C > 1) cluster_sync();      // every CTA of the cluster runs before its shared memory is written

  // the join of a finished row by warp 0 of the group's first CTA
  float xt = 0.0f, xt_prev = 0.0f;
  long long ent = -1, ent_prev = -1;
  int st = DDT_OK, st_prev = DDT_OK;
  auto finish = [&](int buf) {
    const Part* q = s_part[buf];
    Sums a = lane < C ? q[lane].sums : Sums{-INFINITY, 0.0f, 0.0f};
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      const Sums b = {__shfl_xor_sync(DDT_FULL_MASK, a.m, o), __shfl_xor_sync(DDT_FULL_MASK, a.s, o),
                      __shfl_xor_sync(DDT_FULL_MASK, a.u, o)};
      a = join(a, b);
    }
    a.m = __shfl_sync(DDT_FULL_MASK, a.m, 0);
    a.s = __shfl_sync(DDT_FULL_MASK, a.s, 0);
    a.u = __shfl_sync(DDT_FULL_MASK, a.u, 0);
    // a NaN or +inf logit, or no finite one
    const bool bad = st_prev != DDT_OK || !(fabsf(a.m) <= 3.402823466e38f);
    const float lns = log2f(a.s) * 0.6931471805599453f;
    if (lane == 0) {
      p.logp[ent_prev] = bad ? -INFINITY : (xt_prev - a.m) - lns;
      if (p.entropy) p.entropy[ent_prev] = bad ? 0.0f : fmaxf(lns - 0.6931471805599453f * (a.u / a.s), 0.0f);
      if (p.dev_status) p.dev_status[ent_prev] = bad ? DDT_ERR_INPUT : DDT_OK;
    }
    if (kTop) {
      unsigned long long best = q[0].keys[lane];
      for (int r = 1; r < C; ++r) best = merge_lists(best, q[r].keys[lane], lane);
      if (lane < K) {
        const bool has = !bad && best != 0ull;
        p.top_logp[ent_prev * K + lane] = has ? (key_value(best) - a.m) - lns : -INFINITY;
        p.top_tok[ent_prev * K + lane] = has ? static_cast<int32_t>(~static_cast<uint32_t>(best)) : -1;
      }
    }
  };

  if (kTop && tid == 0) s_count = 0;
  for (int it = 0; it < rounds; ++it) {
    const int ord = group + it * groups;
    const bool on = ord < live;  // the same for the CTAs of a group
    const int buf = it & 1;
    Sums a = {-INFINITY, 0.0f, 0.0f};
    unsigned long long T = 0ull;  // at least K keys of the slice reach it (0: not known yet)
    if (on) {
      const int e = p.nodes ? (int)s_list[ord] : ord;
      const long long o = p.e0 + e;
      const int b = (int)(o / p.M), j = (int)(o % p.M);
      const int node = p.nodes ? __ldg(p.nodes + o) : j;
      const int t = __ldg(p.tok + o);
      const bool ok = node < p.N && t >= 0 && t < V;
      ent = o;
      st = ok ? DDT_OK : DDT_ERR_INPUT;
      if (node < p.N) {
        const unsigned char* row =
            static_cast<const unsigned char*>(p.logits) + ((long long)b * p.N + node) * p.row_stride * kElt;
        if (part == 0 && warp == 0) {
          xt = 0.0f;
          if (ok) xt = kBF16 ? bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(row) + t))
                             : __ldg(reinterpret_cast<const float*>(row) + t);
        }
        // Items of the row: 0 and 1 are its ends, where a 16-byte vector of
        // memory lies only partly in it (none if aligned); item i >= 2 is the
        // whole vector at element full0 + (i - 2) kPer.
        const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / kElt);
        const int full0 = min(V, mis ? kPer - mis : 0);
        const int nfull = (V - full0) / kPer;
        const int full1 = full0 + nfull * kPer;
        auto pos_of = [&](int i) { return i >= 2 ? full0 + (i - 2) * kPer : i == 0 ? full0 - kPer : full1; };
        const int nitem = nfull + 2;
        const int per = (nitem + C - 1) / C;
        const int v0 = min(nitem, part * per), v1 = min(nitem, v0 + per);
        // a vector past the slice counts as all -inf
        const uint32_t inf = kBF16 ? 0xff80ff80u : 0xff800000u;
        const uint4 none = make_uint4(inf, inf, inf, inf);
        uint64_t s2 = 0ull, u2 = 0ull;  // packed sums relative to a.m
        for (int r0 = v0; r0 < v1; r0 += kU * kThreads) {  // the same trips for the whole CTA
          uint4 v[kU];
          const unsigned char* src = row + (long long)full0 * kElt + (long long)(r0 + tid - 2) * 16;
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int i = r0 + tid + u * kThreads;
            v[u] = none;
            if (i < v1 && (u > 0 || i >= 2)) v[u] = __ldcs(reinterpret_cast<const uint4*>(src) + u * kThreads);
          }
          if (r0 + tid < min(2, v1)) v[0] = load_edge<kBF16>(row, V, full0, full1, r0 + tid);
          float vm[kU];
          float rm = -INFINITY;
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            vm[u] = vec_max<kBF16>(v[u]);
            rm = max_nan(rm, vm[u]);
          }
          if (!(rm <= a.m)) {  // a larger value, or a NaN, which stays
            const float M = max_nan(rm, a.m);
            const float d = fmaxf((a.m - M) * kLog2e, kFar), ed = ex2_ftz(d);
            const uint64_t d2 = pack2(d, d), e2 = pack2(ed, ed);
            u2 = mul2(fma2(d2, s2, u2), e2);
            s2 = mul2(s2, e2);
            a.m = M;
          }
          const float nm = a.m == -INFINITY ? 0.0f : -a.m;  // all -inf so far: every term below is 0
          const uint64_t nm2 = pack2(nm, nm), l2 = pack2(kLog2e, kLog2e);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
#pragma unroll
            for (int q = 0; q < kPer; q += 2) {
              const uint64_t y = mul2(add2(pack2(value_of<kBF16>(v[u], q), value_of<kBF16>(v[u], q + 1)), nm2), l2);
              float y0, y1;
              unpack2(y, y0, y1);
              y0 = fmaxf(y0, kFar);
              y1 = fmaxf(y1, kFar);
              const uint64_t e = pack2(ex2_ftz(y0), ex2_ftz(y1));
              s2 = add2(s2, e);
              u2 = fma2(e, pack2(y0, y1), u2);
            }
          }
          if (kTop) {
            // raise T from this round's best keys: in the first round, or when
            // so many threads hold a value at T that they could fill the buffer
            auto reaches = [&](float x) { return x > -INFINITY && (T == 0ull || x >= key_value(T)); };
            const bool first = r0 == v0;
            int holders = __syncthreads_count(reaches(rm));
            if (first || holders > kManyThreads) {
              unsigned long long best = 0ull;
              if (rm > -INFINITY) {  // the lowest index of this thread's largest value
                int at = 0;
#pragma unroll
                for (int u = kU - 1; u >= 0; --u) {
                  if (vm[u] == rm) {
                    int k = kPer;
#pragma unroll
                    for (int q = kPer - 1; q >= 0; --q)
                      if (value_of<kBF16>(v[u], q) == rm) k = q;
                    at = pos_of(r0 + tid + u * kThreads) + k;
                  }
                }
                best = topk_key(rm, at);
              }
              best = warp_sort_desc(best, lane);
              s_lists[warp][lane] = best;
              __syncthreads();
              const int r = min(K, 4), jj = (K + r - 1) / r - 1;
              const unsigned long long c = lane < kWarps ? s_lists[lane][jj] : 0ull;
              int above = 0;  // warps whose j-th best is larger (equal: the lower warp first)
#pragma unroll
              for (int w = 0; w < kWarps; ++w) {
                const unsigned long long d = __shfl_sync(DDT_FULL_MASK, c, w);
                above += (d > c || (d == c && w < lane)) ? 1 : 0;
              }
              const unsigned pick = __ballot_sync(DDT_FULL_MASK, lane < kWarps && above == r - 1);
              const unsigned long long cand = __shfl_sync(DDT_FULL_MASK, c, __ffs(pick) - 1);
              T = cand > T ? cand : T;
              holders = __syncthreads_count(reaches(rm));
            }
            // still many (rows of few distinct values): look at the buffer's
            // level after every vector instead of after the round
            const bool many = holders > kManyThreads;
            if (!many) {
#pragma unroll
              for (int u = 0; u < kU; ++u)
                if (reaches(vm[u])) append_keys<kBF16>(v[u], pos_of(r0 + tid + u * kThreads), T, s_cand, &s_count);
            }
#pragma unroll 1
            for (int u = many ? 0 : kU - 1; u < kU; ++u) {
              if (many) {
                const int i = r0 + tid + u * kThreads;  // read again: a register array cannot be indexed by u
                if (i < v1) {
                  const uint4 x = i < 2 ? load_edge<kBF16>(row, V, full0, full1, i)
                                        : __ldg(reinterpret_cast<const uint4*>(src) + u * kThreads);
                  if (reaches(vec_max<kBF16>(x))) append_keys<kBF16>(x, pos_of(i), T, s_cand, &s_count);
                }
              }
              __syncthreads();
              if (s_count > kCand - kRoundMax) {  // the same for the whole CTA
                // sort the buffer into its 32 best, which stay as its first entries
                const int n = min(s_count, kCand);
                unsigned long long l = 0ull;
                for (int c = warp * 32; c < n; c += kThreads) {
                  const int i = c + lane;
                  l = merge_lists(l, warp_sort_desc(i < n ? s_cand[i] : 0ull, lane), lane);
                }
                s_lists[warp][lane] = l;
                __syncthreads();
                if (warp == 0) {
#pragma unroll 1
                  for (int w = 1; w < kWarps; ++w) l = merge_lists(l, s_lists[w][lane], lane);
                  s_cand[lane] = l;
                  if (lane == 0) s_count = 32;
                }
                __syncthreads();
                const unsigned long long kth = s_cand[K - 1];
                T = kth > T ? kth : T;
              }
            }
          }
        }
        float s0, s1, u0, u1;
        unpack2(s2, s0, s1);
        unpack2(u2, u0, u1);
        a.s = s0 + s1;
        a.u = u0 + u1;
      }
#pragma unroll
      for (int q = 16; q > 0; q >>= 1) {
        const Sums c = {__shfl_xor_sync(DDT_FULL_MASK, a.m, q), __shfl_xor_sync(DDT_FULL_MASK, a.s, q),
                        __shfl_xor_sync(DDT_FULL_MASK, a.u, q)};
        a = join(a, c);
      }
      if (lane == 0) s_sums[buf][warp] = a;
    }
    __syncthreads();
    unsigned long long l = 0ull;
    if (kTop) {
      const int n = min(s_count, kCand);
      for (int c = warp * 32; c < n; c += kThreads) {
        const int i = c + lane;
        l = merge_lists(l, warp_sort_desc(i < n ? s_cand[i] : 0ull, lane), lane);
      }
      s_lists[warp][lane] = l;
      __syncthreads();
      if (tid == 0) s_count = 0;
      if (warp == 0) {
        const int lists = min(kWarps, (n + 31) / 32);
#pragma unroll 1
        for (int w = 1; w < lists; ++w) l = merge_lists(l, s_lists[w][lane], lane);
      }
    }
    // the row before this one is complete in the group's first CTA
    __syncwarp();
    if (C > 1 && it > 0) {
      cluster_wait();
      if (part == 0 && warp == 0 && ent_prev >= 0) finish(buf ^ 1);
    }
    if (warp == 0 && on) {
      Sums b = lane < kWarps ? s_sums[buf][lane] : Sums{-INFINITY, 0.0f, 0.0f};
#pragma unroll
      for (int q = 4; q > 0; q >>= 1) {
        const Sums c = {__shfl_xor_sync(DDT_FULL_MASK, b.m, q), __shfl_xor_sync(DDT_FULL_MASK, b.s, q),
                        __shfl_xor_sync(DDT_FULL_MASK, b.u, q)};
        b = join(b, c);
      }
      Part* dst = &s_part[buf][part];
      if (C > 1 && part != 0) {
        const uint32_t base = map_to_rank(smem_u32(dst), (uint32_t)lead);
        if (lane == 0) {
          st_cluster_f32(base, b.m);
          st_cluster_f32(base + 4, b.s);
          st_cluster_f32(base + 8, b.u);
        }
        if (kTop) st_cluster_u64(base + 16 + 8 * lane, l);
      } else {
        if (lane == 0) dst->sums = b;
        if (kTop) dst->keys[lane] = l;
        __syncwarp();
      }
    }
    __syncwarp();
    ent_prev = on ? ent : -1;
    st_prev = st;
    xt_prev = xt;
    if (C > 1) {
      cluster_arrive();
    } else if (warp == 0 && on) {
      finish(buf);
    }
  }
  if (C > 1) {
    cluster_wait();
    if (part == 0 && warp == 0 && ent_prev >= 0) finish((rounds - 1) & 1);
  }
}

template <bool kBF16, bool kTop>
static cudaLaunchConfig_t config(cudaLaunchAttribute* attr, int grid, int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 0;
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

// CTAs of the kernel resident at once in clusters of 8 on the current device
// (0: such clusters cannot be scheduled), looked up once per device.
template <bool kBF16, bool kTop>
static int resident_ctas() {
  static std::mutex mu;
  static int known[kMaxDevices];
  static bool have[kMaxDevices] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!have[dev]) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config<kBF16, kTop>(attr, 4096, kMaxC, nullptr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, token_logprobs_kernel<kBF16, kTop>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    known[dev] = n * kMaxC;
    have[dev] = true;
  }
  return known[dev];
}

template <bool kBF16, bool kTop>
static int launch_t(LogprobsParams p, cudaStream_t stream) {
  // slices of at least 4 KB; no more CTAs than the rows can use
  const int elt = kBF16 ? 2 : 4;
  const int slots = resident_ctas<kBF16, kTop>();
  int cluster = kMaxC;
  while (cluster > 1 && (slots == 0 || (long long)p.V * elt < 4096LL * cluster)) cluster >>= 1;
  const long long most = std::max(1, (slots > 0 ? slots : 4 * sm_count()) / cluster);
  p.cluster = cluster;
  const long long total = (long long)p.B * p.M;
  const long long step = p.nodes ? kListMax : total;
  for (long long e0 = 0; e0 < total; e0 += step) {
    p.e0 = e0;
    p.R = (int)std::min(step, total - e0);
    const int grid = (int)(std::min<long long>(most, p.R) * cluster);
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
