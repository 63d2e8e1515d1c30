// Accumulated attention weight of cached rows on the tensor cores, sm_100a:
// bf16 rows of 64 .. 576 dims (a multiple of 64).
//
// What it computes is fixed in ddt.h (ddt_cache_weights): for every cached
// row j, sum over the selected verify rows' heads of e^(scale q . k_j - lse).
//
// The keys are the MMA's M side and the query rows its N side, so a key is a
// tensor-memory lane: one thread owns a key (with one other, which takes the
// other half of the columns), adds up its weights over the columns in
// registers, and no reduction across lanes is needed. e^(s - lse) is
// 2^(s scale log2 e - lse log2 e): one fma and one ex2 per (key, row).
//
// An item is 256 keys of one request (a CTA pair, 128 keys per CTA, tcgen05
// cta_group::2, M = 256) times the request's query rows, or a share of them.
// The CTA's 128 keys stay in shared memory for the item (d / 64 slabs of 16
// KB), the query rows stream through a ring of stages (half of a tile's up
// to 256 rows x 64 dims each, the pair holds the other half; 4 stages of 16 KB,
// more smaller ones when the tiles are small), fetched by
// node from the caller's list: a unit is a node's heads or an even share of
// them (padded to 8 rows, at most 128), which are consecutive rows of q. Units
// that follow one another come in one box (4 x 8192 rows x 32768 keys: 962 ->
// 946 us).
// The issuing thread's own steps bound small tiles: two waits, four MMAs and
// two commits per 64 dims took it 670 cycles whatever the tile's size. So a
// stage has one commit, which releases its query rows and, in an item's last
// tile, the keys they were multiplied with, and small tiles put three slabs
// into a stage (single tokens of 16 requests: 25.2 -> 20.4 us). The next item's
// keys arrive under this item's last MMAs. Accumulators: two of 256 columns, so the
// exponentials of a tile run under the next tile's MMAs.
//
// Bound: the tensor pipe for 4 and more nodes of 64 heads (256 x 256 x 576
// per 4600 cycles; the exponentials take 2050); the rounds of key tiles, the
// plan and the drain for single tokens (16 requests of 1024 to 8192 rows: 313
// tiles on 74 pairs, 20.5 us, 3.9 TB/s).
//
// Items are dealt to a persistent grid of pairs in order. With few key tiles
// the query rows are split into S shares (the S of the shortest estimated
// makespan, computed alike in every CTA); shares write partial sums to the
// workspace and the last one to arrive adds them up in order, so the result
// does not depend on who is last.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "ddt_kernels.cuh"
#include "sm100_ptx.cuh"
#include "topk_keys.cuh"

namespace ddt {
namespace cwt {

using namespace sm100;

constexpr int kThreads = 320;        // warp 0 TMA, warp 1 MMA + TMEM, warps 2..9 weights
constexpr int kMaxSlabs = 9;
constexpr int kMaxStages = 16;
constexpr int kRingBytes = 64 * 1024;  // stages of query rows
constexpr int kKeys = 128;             // keys of one CTA
constexpr int kTile = 2 * kKeys;       // of the pair: M = 256
constexpr int kSlabBytes = kKeys * 128;  // 128 keys x 64 dims bf16
constexpr int kMaxB = 256;           // requests of one launch
constexpr int kMaxShares = 16;
constexpr int kMaxParts = 320;       // (key tile, share) partials of a split launch
constexpr uint64_t kLandNs = 100000; // pause before leaving when a wait gave up

constexpr int kBarAFull = 0;                          // [kMaxSlabs] leader: a stage's keys (both CTAs)
constexpr int kBarBFull = kBarAFull + kMaxSlabs;      // [kMaxStages] leader: a stage of query rows
constexpr int kBarBEmpty = kBarBFull + kMaxStages;    // [kMaxStages] each CTA
constexpr int kBarAccFull = kBarBEmpty + kMaxStages;     // [2] each CTA
constexpr int kBarAccEmpty = kBarAccFull + 2;         // [2] leader: read by 8 warps x 2 CTAs
constexpr int kNumBars = kBarAccEmpty + 2;

struct Shared {  // behind the slabs and stages
  unsigned long long bars[kNumBars];
  uint32_t tmem;
  int aborted;
  int shares, total, last;
  alignas(16) float lse2[2][256];
  alignas(16) int sees[2][256];
  float sums[2][kKeys];  // a key's parts
  int64_t off[kMaxB];
  int len[kMaxB];        // -1: the request is skipped
  int m[kMaxB];          // entries of its list
  int tile0[kMaxB + 1];  // key tiles before it
  int item0[kMaxB + 1];  // items before it
};

struct Params {
  WeightsParams w;
  int b0, nb;            // requests [b0, b0 + nb) of the call
  int slabs;             // d / 64
  int unit;              // query rows of one unit (a multiple of 8, at most 128)
  int chunks;            // units per node
  int per_half;          // units that fit half a tile's 128 columns
  int adjacent;          // the rows of one unit follow those of the one before (every node, no padding)
  int per_tile;          // stages of a tile
  int row_bytes;         // of one slab of a stage's query rows
  int stages, stage_bytes;  // of the ring of query rows
  float sl2;             // scale log2 e
  int* abort;
  unsigned* counters;    // [kMaxParts][2] arrivals, zero between calls
  float* parts;          // [kMaxParts][256] partial sums
  uint64_t wait_ns;
};

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ bool bar_red_and(int id, int nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}

// The items of this launch in order, one cursor per role.
struct Cursor {
  int item, b;
  __device__ explicit Cursor(int first) : item(first), b(0) {}
  // false: no more items. Else the request, its key tile and the share's units
  // [u0, u1), dealt in tiles of `per` units.
  __device__ bool get(const Shared& s, const Params& p, int& kt, int& share, int& nshare, int& u0, int& u1, int& per) {
    if (item >= s.total) return false;
    while (item >= s.item0[b + 1]) ++b;
    const int units = s.m[b] * p.chunks;
    nshare = max(1, min(s.shares, units));
    kt = item - s.item0[b];
    share = 0;
    u0 = 0;
    u1 = units;
    if (nshare > 1) {
      share = kt % nshare;
      kt /= nshare;
      const int base = units / nshare, more = units - base * nshare;
      u0 = share * base + min(share, more);
      u1 = u0 + base + (share < more ? 1 : 0);
    }
    const int most = 2 * p.per_half, n = u1 - u0;
    per = n;
    if (n > most) {
      const int tiles = (n + most - 1) / most;
      per = (n + tiles - 1) / tiles;
    }
    return true;
  }
};

// One query tile: `nu` units from u on, h0 of them in the first half; nh
// columns per half.
struct Tile {
  int nu, h0, nh;
  __device__ Tile(const Params& p, int u, int u1, int per) {
    nu = min(per, u1 - u);
    h0 = (nu + 1) / 2;
    nh = (h0 * p.unit + 31) / 32 * 32;
  }
};

// kKps: slabs of one stage
template <int kKps>
__global__ void __launch_bounds__(kThreads, 1)
    cache_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_pair, const __grid_constant__ CUtensorMap tm_half,
                            Params p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sA = smem_u32(smem), sB = sA + (uint32_t)(p.slabs * kSlabBytes);
  Shared& s = *reinterpret_cast<Shared*>(smem + p.slabs * kSlabBytes + kRingBytes);
  const uint32_t bar0 = smem_u32(s.bars);
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  const WeightsParams& w = p.w;
  int* abort = p.abort;
  const uint64_t wlim = p.wait_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxSlabs; ++i) {
      mbar_init(bar(kBarAFull + i), 1);
    }
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(bar(kBarBFull + i), 1);
      mbar_init(bar(kBarBEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarAccFull + i), 1);
      mbar_init(bar(kBarAccEmpty + i), 16);
    }
    fence_mbar_init_cluster();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_pair);
    prefetch_tmap(&tm_half);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&s.tmem), 512);
    tmem_relinquish_pair();
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();
  // a workspace whose status word holds a timeout: no work (the leader's
  // reading counts for the pair; it writes it into the other CTA once that
  // one is known to run)
  const int held = leader && threadIdx.x == 32 ? *reinterpret_cast<volatile int*>(abort) : 0;

  // ---- every request's rows and list: alike in every CTA
  for (int i = warp; i < p.nb; i += kThreads / 32) {
    const int b = p.b0 + i;
    const int len = w.cache_len[b], n = w.n_nodes[b];
    const int64_t off = w.cache_off[b];
    int m = n;
    bool bad = n < 0 || n > w.N;
    if (w.nodes) {
      const int32_t* list = w.nodes + (int64_t)b * w.M;
      m = 0;
      for (int c = 0; c < w.M; c += 32) {
        const int e = c + lane < w.M ? __ldg(list + c + lane) : -1;
        const unsigned neg = __ballot_sync(DDT_FULL_MASK, e < 0), over = __ballot_sync(DDT_FULL_MASK, e >= n);
        const int k = neg ? __ffs(neg) - 1 : 32;
        m += k;
        if (over & (k == 32 ? 0xffffffffu : (1u << k) - 1u)) bad = true;
        if (k < 32) break;
      }
    }
    const bool oob = off < 0 || len < 0 || off > w.kv_rows - len;
    if (lane == 0) {
      s.len[i] = oob || bad ? -1 : len;
      s.m[i] = oob || bad ? 0 : m;
      s.off[i] = off;
      if (blockIdx.x == 0 && w.dev_status)
        w.dev_status[b] = *reinterpret_cast<volatile int*>(abort) != 0 ? DDT_ERR_TIMEOUT
                          : oob                                         ? DDT_ERR_BOUNDS
                          : bad                                         ? DDT_ERR_INPUT
                                                                        : DDT_OK;
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (leader && threadIdx.x == 32) {
    st_cluster_u32(map_to_rank(smem_u32(&s.aborted), 0), (uint32_t)held);
    st_cluster_u32(map_to_rank(smem_u32(&s.aborted), 1), (uint32_t)held);
  }
  __syncthreads();
  if (warp == 0) {
    // prefix of key tiles and the longest list, then the shares
    int tiles = 0, longest = 0;
    for (int c = 0; c < p.nb; c += 32) {
      const int i = c + lane;
      const int t = i < p.nb && s.len[i] > 0 ? (s.len[i] + kTile - 1) / kTile : 0;
      longest = max(longest, i < p.nb ? s.m[i] : 0);
      int inc = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(DDT_FULL_MASK, inc, o);
        if (lane >= o) inc += y;
      }
      if (i < p.nb) s.tile0[i] = tiles + inc - t;
      tiles += __shfl_sync(DDT_FULL_MASK, inc, 31);
    }
    longest = __reduce_max_sync(DDT_FULL_MASK, longest);
    const int most = 2 * p.per_half, units = longest * p.chunks;
    // lane S - 1 prices S shares: rounds of items times an item's columns (in
    // units) plus about a third of a tile for its keys and its end
    const int S = lane + 1;
    const bool may = S <= min(kMaxShares, max(units, 1)) && (S == 1 || tiles <= kMaxParts / S);
    uint32_t cost = 0xffffffffu;
    if (may && S > 1) {  // tiles * S is small
      const int rounds = (tiles * S + npairs - 1) / npairs;
      cost = (uint32_t)min((long long)rounds * (3 * ((units + S - 1) / S) + 2 * most), 0x7ffffffLL) << 5 | (uint32_t)lane;
    } else if (may) {
      cost = (uint32_t)min((long long)((tiles + npairs - 1) / npairs) * (3 * units + most), 0x7ffffffLL) << 5;
    }
    const int arg = (int)(__reduce_min_sync(DDT_FULL_MASK, cost) & 31u) + 1;
    int items = 0;
    for (int c = 0; c < p.nb; c += 32) {
      const int i = c + lane;
      int t = 0;
      if (i < p.nb && s.len[i] > 0) t = (s.len[i] + kTile - 1) / kTile * max(1, min(arg, s.m[i] * p.chunks));
      int inc = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(DDT_FULL_MASK, inc, o);
        if (lane >= o) inc += y;
      }
      if (i < p.nb) s.item0[i] = items + inc - t;
      items += __shfl_sync(DDT_FULL_MASK, inc, 31);
    }
    if (lane == 0) {
      s.item0[p.nb] = items;
      s.shares = arg;
      s.total = items;
    }
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s.tmem);
  const bool aborted = *reinterpret_cast<volatile int*>(&s.aborted) != 0;

  bool ok = true;  // no wait of this thread gave up
  if (aborted) {
    // straight to the teardown
  } else if (warp == 0) {
    // ============================================================ TMA producer
    // the whole warp: lane j issues the box of unit j of this CTA's half, whose
    // row it works out once per tile (one thread issuing every box with its
    // index arithmetic took 1400 cycles per stage, three times the MMAs' 512)
    const uint32_t afull0 = map_to_rank(bar(kBarAFull), 0), bfull0 = map_to_rank(bar(kBarBFull), 0);
    int slot = 0, issued = 0;
    uint32_t phase = 0;
    Cursor cur(pair);
    int kt, share, nshare, u0, u1, per;
    bool ahead = true;  // the first item's keys need no wait: all their loads go first
    for (; ok && cur.get(s, p, kt, share, nshare, u0, u1, per); cur.item += npairs) {
      if (u0 >= u1) continue;
      const int b = p.b0 + cur.b;
      const int yk = (int)(s.off[cur.b] + kt * kTile + kKeys * (int)rank);
      const int32_t* list = w.nodes ? w.nodes + (int64_t)b * w.M : nullptr;
      auto keys = [&](int j) {  // the keys' slabs of stage j of a tile
        const int k0 = j * kKps, k1 = min(p.slabs, k0 + kKps);
        if (leader) mbar_arrive_expect_tx(bar(kBarAFull + j), 2u * kSlabBytes * (uint32_t)(k1 - k0));
        for (int k = k0; k < k1; ++k)
          tma_load_2d_pair(sA + (uint32_t)(k * kSlabBytes), &tm_k, 64 * k, yk, afull0 + 8u * (uint32_t)j);
      };
      if (ahead && lane < p.per_tile) keys(lane);  // a lane per stage: one after the other took 2100 cycles
      for (int u = u0; u < u1 && ok; u += per) {
        const Tile tile(p, u, u1, per);
        // as few boxes as the rows allow: this CTA's whole half, a node's two
        // units, or single ones
        const int first = u + (leader ? 0 : tile.h0), count = leader ? tile.h0 : tile.nu - tile.h0;
        const bool half = p.adjacent && count * p.unit == 128, pairs = p.chunks == 2 && (first & 1) == 0 && (count & 1) == 0;
        const int step = half ? count : pairs ? 2 : 1;
        const CUtensorMap* map = half ? &tm_half : pairs ? &tm_pair : &tm_q;
        // lane = box + boxes * slab of the stage
        const int boxes = (count + step - 1) / step, box = kKps == 1 ? lane : lane % max(boxes, 1);
        const int slab = kKps == 1 ? 0 : lane / max(boxes, 1);
        const bool mine = box < boxes && slab < kKps;
        int yq = 0;
        if (mine) {
          const int un = first + box * step, e = un / p.chunks, c = un - e * p.chunks;
          yq = (b * w.N + (list ? __ldg(list + e) : e)) * w.H + c * p.unit;
        }
        const uint32_t dst = sB + (uint32_t)(box * step * p.unit * 128 + slab * p.row_bytes);
        for (int j = 0; j < p.per_tile; ++j) {
          if (u == u0 && !ahead) {
            // the keys of this stage are free when the last tile's stage j is
            // done with: known already if its slot has been filled again
            const int g = issued - p.per_tile;  // that stage's number
            if (g + p.stages >= issued) {
              if (!mbar_wait(bar(kBarBEmpty + g % p.stages), (uint32_t)((g / p.stages) & 1), abort, wlim)) ok = false;
              ok = __all_sync(DDT_FULL_MASK, ok);
              if (!ok) break;
            }
            if (lane == 0) keys(j);
          }
          if (!mbar_wait(bar(kBarBEmpty + slot), phase ^ 1u, abort, wlim)) ok = false;
          ok = __all_sync(DDT_FULL_MASK, ok);
          if (!ok) break;
          const int k0 = j * kKps, n = kKps == 1 ? 1 : min(p.slabs - k0, kKps);
          if (leader && lane == 0)
            mbar_arrive_expect_tx(bar(kBarBFull + slot), (uint32_t)(n * tile.nu * p.unit * 128));
          __syncwarp();
          ++issued;
          if (mine && slab < n)
            tma_load_2d_pair(dst + (uint32_t)(slot * p.stage_bytes), map, 64 * (k0 + slab), yq, bfull0 + 8u * (uint32_t)slot);
          if (++slot == p.stages) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      ahead = false;
    }
  } else if (warp == 1 && lane == 0 && leader) {
    // ============================================================ MMA issuer
    int slot = 0, at = 0;
    uint32_t phase = 0, aphase = 0;
    Cursor cur(pair);
    int kt, share, nshare, u0, u1, per;
    for (; ok && cur.get(s, p, kt, share, nshare, u0, u1, per); cur.item += npairs) {
      if (u0 >= u1) continue;
      for (int u = u0; u < u1 && ok; u += per, ++at) {
        const Tile tile(p, u, u1, per);
        const uint32_t idesc = idesc_bf16_f32(kTile, 2 * tile.nh, false, false);
        const int buf = at & 1;
        if (!mbar_wait(bar(kBarAccEmpty + buf), (uint32_t)((at >> 1) & 1) ^ 1u, abort, wlim)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * 256);
        for (int j = 0; j < p.per_tile; ++j) {
          if ((u == u0 && !mbar_wait(bar(kBarAFull + j), aphase, abort, wlim)) ||
              !mbar_wait(bar(kBarBFull + slot), phase, abort, wlim)) {
            ok = false;
            break;
          }
          const int k0 = j * kKps, n = kKps == 1 ? 1 : min(p.slabs - k0, kKps);
#pragma unroll
          for (int i = 0; i < kKps; ++i) {
            if (i < n) {
              const uint64_t da = smem_desc_sw128(sA + (uint32_t)((k0 + i) * kSlabBytes), 16, 1024);
              const uint64_t db = smem_desc_sw128(sB + (uint32_t)(slot * p.stage_bytes + i * p.row_bytes), 16, 1024);
              mma_pair_ss(d, da, db, idesc, (j | i) != 0 ? 1u : 0u);
#pragma unroll
              for (int q = 1; q < 4; ++q) mma_pair_ss(d, da + 2 * q, db + 2 * q, idesc, 1u);
            }
          }
          mma_commit_pair_mc(bar(kBarBEmpty + slot), (uint16_t)0x3u);
          if (++slot == p.stages) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (ok) mma_commit_pair_mc(bar(kBarAccFull + buf), (uint16_t)0x3u);
      }
      aphase ^= 1u;
    }
  } else if (warp >= 2) {
    // ============================================================ weights
    // thread = lane 32 q + lane of the CTA's tensor memory = that key of the
    // CTA; of the two warps per lane quarter each takes every other chunk of 32
    // columns
    const int q = warp & 3, h = warp >= 6 ? 1 : 0, et = (int)threadIdx.x - 64;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t empty0 = map_to_rank(bar(kBarAccEmpty), 0);
    const int row = 32 * q + lane;
    int at = 0;
    Cursor cur(pair);
    int kt, share, nshare, u0, u1, per;
    for (; cur.get(s, p, kt, share, nshare, u0, u1, per); cur.item += npairs) {
      const int b = p.b0 + cur.b, len = s.len[cur.b], m = s.m[cur.b];
      const int32_t* list = w.nodes ? w.nodes + (int64_t)b * w.M : nullptr;
      const int key0 = kt * kTile + kKeys * (int)rank, key = key0 + row, key1 = min(len, key0 + kKeys);
      // the log-sum-exp of column et of a tile and how many keys it sees (0:
      // no query row there, or one without visible keys)
      auto column = [&](int u, float& l2, int& sees) {
        const Tile tile(p, u, u1, per);
        const int half = et >> 7, c = et & 127, j = c / p.unit;
        l2 = 0.0f;
        sees = 0;
        if (c < tile.nh && j < (half ? tile.nu - tile.h0 : tile.h0)) {
          const int un = u + half * tile.h0 + j, e = un / p.chunks, head = (un - e * p.chunks) * p.unit + c - j * p.unit;
          if (head < w.H) {
            const int node = list ? __ldg(list + e) : e;
            const float l = __ldg(w.lse + ((long long)b * w.N + node) * w.H + head);
            l2 = l * kLog2e;
            sees = l == -INFINITY ? 0 : w.causal ? len - m + 1 + e : len;
          }
        }
      };
      float sum = 0.0f;
      float l2 = 0.0f;
      int sees = 0;
      // what the end of the item needs, fetched under its tiles
      const int64_t j = s.off[cur.b] + key0 + et;
      const float old = w.prev && et < kKeys && key0 + et < len ? w.prev[j] : 0.0f;
      if (u0 < u1) column(u0, l2, sees);
      for (int u = u0; u < u1; u += per, ++at) {
        const int buf = at & 1;
        const Tile tile(p, u, u1, per);
        s.lse2[buf][et] = l2;
        s.sees[buf][et] = sees;
        const bool plain = bar_red_and(1, 256, (et & 127) >= tile.nh || sees >= key1);
        if (u + per < u1) column(u + per, l2, sees);  // the next tile's, under this one
        if (ok && !mbar_wait(bar(kBarAccFull + buf), (uint32_t)((at >> 1) & 1), abort, wlim)) ok = false;
        tc_fence_after();
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const int nchunks = 2 * tile.nh / 32;
#pragma unroll 1
        for (int c = h; c < nchunks; c += 2) {
          uint32_t r[32];
          tmem_ld32(lane_addr + (uint32_t)(buf * 256 + 32 * c), r);
          tmem_wait_ld();
          const int col = 32 * c >= tile.nh ? 128 + 32 * c - tile.nh : 32 * c;  // of lse2 and sees
          const float4* pl = reinterpret_cast<const float4*>(&s.lse2[buf][col]);
          if (plain) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = pl[i];
              acc[0] += ex2_ftz(fmaf(__uint_as_float(r[4 * i]), p.sl2, -l.x));
              acc[1] += ex2_ftz(fmaf(__uint_as_float(r[4 * i + 1]), p.sl2, -l.y));
              acc[2] += ex2_ftz(fmaf(__uint_as_float(r[4 * i + 2]), p.sl2, -l.z));
              acc[3] += ex2_ftz(fmaf(__uint_as_float(r[4 * i + 3]), p.sl2, -l.w));
            }
          } else {
            const int4* ps = reinterpret_cast<const int4*>(&s.sees[buf][col]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = pl[i];
              const int4 v = ps[i];
              if (key < v.x) acc[0] += ex2_ftz(fmaf(__uint_as_float(r[4 * i]), p.sl2, -l.x));
              if (key < v.y) acc[1] += ex2_ftz(fmaf(__uint_as_float(r[4 * i + 1]), p.sl2, -l.y));
              if (key < v.z) acc[2] += ex2_ftz(fmaf(__uint_as_float(r[4 * i + 2]), p.sl2, -l.z));
              if (key < v.w) acc[3] += ex2_ftz(fmaf(__uint_as_float(r[4 * i + 3]), p.sl2, -l.w));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive_local(bar(kBarAccEmpty + buf));
          else mbar_arrive_cluster(empty0 + 8u * (uint32_t)buf);
        }
        sum += (acc[0] + acc[1]) + (acc[2] + acc[3]);  // tile by tile: short chains of additions
      }
      // ---- the key's parts, then the shares
      s.sums[h][row] = sum;
      // one wait that gave up spoils the CTA's item: a key's parts come from
      // two warps, a share's from eight
      const bool good = bar_red_and(1, 256, ok);
      if (et < kKeys) {  // whose row is et: key0 + et
        const int key = key0 + et;
        sum = s.sums[0][et] + s.sums[1][et];
        bool write = good;
        if (nshare > 1) {
          const int part = s.tile0[cur.b] + kt;
          float* mine = p.parts + ((int64_t)part * s.shares) * kTile + kKeys * (int)rank + et;
          __stcg(mine + share * kTile, sum);
          named_bar_sync(2, kKeys);
          if (et == 0) {
            // the barrier orders the CTA's partial sums before this thread's
            // release; its acquire, and the next barrier, the others' before
            // their reading
            unsigned* cnt = p.counters + 2 * part + rank;
            unsigned old_count = 0u;
            if (good) asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(old_count) : "l"(cnt) : "memory");
            s.last = good && old_count == (unsigned)nshare - 1u;
            if (s.last) *cnt = 0u;
          }
          named_bar_sync(2, kKeys);
          write = good && *reinterpret_cast<volatile int*>(&s.last) != 0;
          if (write) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kMaxShares; ++i) sum += i < nshare ? __ldcg(mine + i * kTile) : 0.0f;
          }
        }
        if (write && key < len) w.score[j] = w.prev ? fmaf(w.decay, old, sum) : sum;
      }
      named_bar_sync(1, 256);  // s.sums is free again
    }
  }
  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  if (__syncthreads_or(!ok)) {
    // Copies and MMAs that nobody waited for may be in flight: every role of
    // this CTA has issued its last ones, and they take a few microseconds. The
    // pair leaves together, so one CTA's pause is both's.
    const uint64_t t = global_timer_ns();
    while (global_timer_ns() - t < kLandNs) __nanosleep(1000);
    __syncwarp();
  }
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    return nullptr;
  }();
  return fn;
}

// [rows][d] bf16, row-major: boxes of 64 dims x box_rows rows, 128-byte swizzle
static bool make_map(CUtensorMap* m, const void* base, uint64_t d, uint64_t rows, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static size_t smem_bytes(int slabs) {
  return (size_t)slabs * kSlabBytes + kRingBytes + sizeof(Shared) + 1024;
}

// CTA pairs resident at once on the current device, looked up once per device
// (with the shared-memory opt-in set).
template <int kKps>
static int device_pairs() {
  static std::mutex mu;
  static int pairs[kMaxDevices] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  std::lock_guard<std::mutex> lock(mu);
  if (pairs[dev] == 0) {
    if (cudaFuncSetAttribute(cache_weights_tc_kernel<kKps>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes(kMaxSlabs)) != cudaSuccess)
      return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 64);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(kMaxSlabs);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, cache_weights_tc_kernel<kKps>, &cfg) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = sm_count() / 2;
    }
    pairs[dev] = n;
  }
  return pairs[dev];
}

}  // namespace cwt

bool weights_tc_supported(int d_qk, int in_dtype, const void* q, const void* kv) {
  return in_dtype == DDT_BF16 && d_qk >= 64 && d_qk <= 64 * cwt::kMaxSlabs && d_qk % 64 == 0 &&
         reinterpret_cast<uintptr_t>(q) % 16 == 0 && reinterpret_cast<uintptr_t>(kv) % 16 == 0;
}

size_t weights_tc_workspace_bytes() { return 256 + cwt::kMaxParts * 2 * sizeof(unsigned) + cwt::kMaxParts * 256 * sizeof(float); }

namespace cwt {
template <int kKps>
static int launch(Params p, int max_cache_len, cudaStream_t stream) {
  const WeightsParams& w = p.w;
  const int pairs = device_pairs<kKps>();
  if (pairs <= 0) return DDT_ERR_CUDA;
  CUtensorMap tk, tq, tp, th;
  const uint64_t q_rows = (uint64_t)w.B * w.N * w.H;
  if (!make_map(&tk, w.kv, (uint64_t)w.d_qk, (uint64_t)w.kv_rows, kKeys) ||
      !make_map(&tq, w.q, (uint64_t)w.d_qk, q_rows, (uint32_t)p.unit) ||
      !make_map(&tp, w.q, (uint64_t)w.d_qk, q_rows, (uint32_t)std::min(128, 2 * p.unit)) ||
      !make_map(&th, w.q, (uint64_t)w.d_qk, q_rows, 128))
    return DDT_ERR_CUDA;
  for (p.b0 = 0; p.b0 < w.B; p.b0 += kMaxB) {
    p.nb = std::min(kMaxB, w.B - p.b0);
    // every pair that could get an item, counting shares
    const long long tiles = std::max(1LL, (long long)p.nb * (max_cache_len / kTile + (max_cache_len % kTile != 0 ? 1 : 0)));
    const long long items = tiles * std::min<long long>(kMaxShares, std::max(1LL, (long long)w.M * p.chunks));
    const unsigned grid = 2u * (unsigned)std::min<long long>(pairs, items);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(p.slabs);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, cache_weights_tc_kernel<kKps>, tk, tq, tp, th, p) != cudaSuccess) return DDT_ERR_CUDA;
  }
  return DDT_OK;
}
}  // namespace cwt

int launch_cache_weights_tc(WeightsParams w, int max_cache_len, void* workspace, cudaStream_t stream) {
  using namespace cwt;
  Params p{};
  p.w = w;
  p.slabs = w.d_qk / 64;
  // A node's heads in `chunks` units: the split that wastes the fewest of the
  // tile's columns on padding; of equal ones two units per node rather than
  // one, so that an odd number of nodes still fills both halves of the pair.
  int best = -1;
  for (int c = 1; c <= std::max(1, w.H / 16) || (w.H + c - 1) / c > 128; ++c) {
    const int unit = ((w.H + c - 1) / c + 7) / 8 * 8;
    if (unit > 128) continue;
    const int used = (int)(1000000LL * w.H / ((long long)c * unit) * (128 / unit * unit) / 128);
    if (used > best || (used == best && c == 2)) {
      best = used;
      p.unit = unit;
      p.chunks = c;
    }
  }
  p.per_half = 128 / p.unit;
  p.adjacent = !w.nodes && p.unit * p.chunks == w.H;
  // stages as large as half a tile of this launch can be
  const long long units = std::min(2LL * p.per_half, (long long)w.M * p.chunks);
  p.row_bytes = (int)(((units + 1) / 2 * p.unit + 31) / 32 * 32 * 128);
  const int kps = 3 * p.row_bytes <= kRingBytes / 4 && 3 * ((units + 1) / 2) <= 32 ? 3 : 1;
  p.per_tile = (p.slabs + kps - 1) / kps;
  p.stage_bytes = kps * p.row_bytes;
  p.stages = std::min(kMaxStages, kRingBytes / p.stage_bytes);
  p.sl2 = w.scale * kLog2e;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.abort = reinterpret_cast<int*>(ws);
  p.counters = reinterpret_cast<unsigned*>(ws + 256);
  p.parts = reinterpret_cast<float*>(ws + 256 + kMaxParts * 2 * sizeof(unsigned));
  p.wait_ns = wait_limit_ns();
  return kps == 3 ? launch<3>(p, max_cache_len, stream) : launch<1>(p, max_cache_len, stream);
}

}  // namespace ddt
