// Eviction from the paged cache by accumulated attention weight.
//
// Per (sequence, KV head): the keep-th largest of n keys (a radix select, 8
// bits a round), then the kept slots at or behind `keep` (movers) into the
// dropped slots before it (holes), both ascending.  Moving only those costs
// 4 d elements each; keeping the slots in order would rewrite nearly the whole
// cache for every slot dropped near its front.
//
// One thread-block cluster per (sequence, KV head), so that one sequence's 8
// heads still occupy the GPU.  Each block holds the keys of a contiguous
// share of the slots in shared memory (read from HBM once; a share beyond
// key_cap is read again each round); the blocks' digit counts, tie counts and
// move counts are read from one another's shared memory after a cluster
// barrier.  The select is a chain of short phases (some 1 us each); the moves
// are bound by HBM.
#pragma once

#include <cooperative_groups.h>

#include "paged.cuh"

namespace hga {
namespace pev {

namespace cg = cooperative_groups;

constexpr int kMaxC = 8;  // blocks per cluster, at most (portable size)
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKeyCap = 48 * 1024;  // keys in one block's shared memory, at most

// Rank of a slot: tokens that are kept by position above every weight, a NaN
// weight below every other.
__device__ __forceinline__ uint32_t slot_key(float w, int p, int64_t last, int sinks, int recent) {
  if (p < sinks || int64_t(p) > last - recent) return 0xffffffffu;
  return w == w ? ordered_key(w) : 0u;
}

struct Shared {
  int hist[4][256];  // one per round, so that a round needs one cluster barrier
  int tot[256];
  int warp_n[2][kWarps];
  int n_equal, n_holes, n_movers, bad;
  // the select's state: keys whose bits above `shift` exceed prefix's are kept,
  // of those that equal them `need` more (all: the whole bin)
  uint32_t prefix;
  int shift, need, all;
};

// Exclusive prefix over the block's warps of x (warp-uniform), and the total.
__device__ __forceinline__ int warp_prefix(int* table, int x, int warp, int lane, int& total) {
  if (lane == 0) table[warp] = x;
  __syncthreads();
  const int v = lane < kWarps ? table[lane] : 0;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  total = __shfl_sync(0xffffffffu, incl, kWarps - 1);
  const int before = __shfl_sync(0xffffffffu, incl - v, warp);
  __syncthreads();
  return before;
}

// grid (nc, n_kv_heads, batch) in clusters of (nc, 1, 1); dynamic shared
// memory: key_cap keys.  moves: [batch, n_kv_heads, capacity] entries of
// (page, row): holes from 0, movers from capacity / 2 (there are at most
// min(keep, n - keep) of each).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    paged_evict_kernel(PagedView cache, const int32_t* __restrict__ n_slots,
                       const int64_t* __restrict__ pos, int keep, int sinks, int recent,
                       int key_cap, int2* __restrict__ moves) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank()), nc = int(cluster.num_blocks());
  const int h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 4 * 256; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) {
    sh.bad = 0;
    sh.prefix = 0u;
    sh.shift = 32;
    sh.need = keep;
    sh.all = 0;
  }
  pdl_wait();
  // the whole cluster reads the same count and leaves here
  const int n = rank == 0 && tid == 0 ? checked_slots(cache, n_slots, b) : n_slots[b];
  if (n <= keep || int64_t(n) > cache.capacity()) return;
  __syncthreads();
  const int64_t last = pos[b];
  const int32_t* table = cache.table + int64_t(b) * cache.max_pages;
  const int share = (((n + nc - 1) / nc) + 3) & ~3;
  const int lo = min(n, rank * share);
  const int n_loc = min(n, lo + share) - lo;

  // ---- keys of this block's share, four slots at a time ---------------------
  auto keys4 = [&](int i) {
    const int s = lo + i;
    const int page = table[cache.page_of(s)];
    if (!cache.has(page)) {
      sh.bad = 1;
      return make_uint4(0u, 0u, 0u, 0u);
    }
    const int64_t at = cache.record(page, h, cache.row_of(s));
    const float4 w = *reinterpret_cast<const float4*>(cache.weight + at);
    const int4 p = *reinterpret_cast<const int4*>(cache.slot_pos + at);
    return make_uint4(slot_key(w.x, p.x, last, sinks, recent),
                      slot_key(w.y, p.y, last, sinks, recent),
                      slot_key(w.z, p.z, last, sinks, recent),
                      slot_key(w.w, p.w, last, sinks, recent));
  };
#pragma unroll 4
  for (int i = tid * 4; i < n_loc; i += kThreads * 4) {
    const uint4 k = keys4(i);
    if (i < key_cap) *reinterpret_cast<uint4*>(keys + i) = k;
  }
  __syncthreads();
  auto key_at = [&](int i) -> uint32_t {
    if (i < key_cap) return keys[i];
    const int s = lo + i, page = table[cache.page_of(s)];
    if (!cache.has(page)) return 0u;
    const int64_t at = cache.record(page, h, cache.row_of(s));
    return slot_key(cache.weight[at], cache.slot_pos[at], last, sinks, recent);
  };

  // ---- the keep-th largest key -----------------------------------------------
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round;
    const uint32_t prefix = sh.prefix;
    int* hist = sh.hist[round];
    // weights share their leading digits, and many may be equal: the lanes of
    // a warp with the same digit count once
    for (int base = 0; base < n_loc; base += kThreads) {
      const int i = base + tid;
      const uint32_t k = i < n_loc ? key_at(i) : 0u;
      const bool in_bin =
          i < n_loc && (round == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8)));
      const unsigned live = __ballot_sync(0xffffffffu, in_bin);
      if (in_bin) {
        const uint32_t digit = (k >> shift) & 255u;
        const unsigned peers = __match_any_sync(live, digit);
        if (lane == __ffs(peers) - 1) atomicAdd(&hist[digit], __popc(peers));
      }
    }
    cluster.sync();
    if (tid < 256) {
      int sum = 0;
      for (int r = 0; r < nc; ++r) sum += cluster.map_shared_rank(hist, r)[tid];
      sh.tot[tid] = sum;
    }
    bool bad = false;
    if (round == 0)
      for (int r = 0; r < nc; ++r) bad = bad || *cluster.map_shared_rank(&sh.bad, r) != 0;
    __syncthreads();
    if (bad) {  // the same for every thread of the cluster: nothing was written
      if (rank == 0 && tid == 0) latch_status(HGA_ERR_DEVICE_CHECK);
      cluster.sync();
      return;
    }
    if (warp == 0) {
      // lane l owns digits 255-8l .. 248-8l (descending)
      int local = 0;
#pragma unroll
      for (int t = 0; t < 8; ++t) local += sh.tot[255 - 8 * lane - t];
      int incl = local;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int need = sh.need;
      const unsigned ball = __ballot_sync(0xffffffffu, incl - local < need && incl >= need);
      if (lane == __ffs(ball) - 1) {
        int above = incl - local;
        for (int t = 0; t < 8; ++t) {
          const int digit = 255 - 8 * lane - t, c = sh.tot[digit];
          if (above + c >= need) {
            sh.prefix = prefix | (uint32_t(digit) << shift);
            sh.shift = shift;
            sh.need = need - above;
            sh.all = c == need - above;
            break;
          }
          above += c;
        }
      }
    }
    __syncthreads();
    if (sh.all) break;  // the whole bin is kept: the other digits do not matter
  }
  const int shift = sh.shift, need = sh.need;
  const bool all = sh.all;
  const uint32_t edge = sh.prefix >> shift;

  // ---- each warp's run of slots, in steps of 32 -------------------------------
  const int run = ((n_loc + kWarps - 1) / kWarps + 31) & ~31;
  const int i0 = min(n_loc, warp * run), i1 = min(n_loc, i0 + run);
  const unsigned below = (1u << lane) - 1u;
  auto cluster_prefix = [&](int* mine, int& total) {
    int before = 0;
    total = 0;
    for (int r = 0; r < nc; ++r) {
      const int x = *cluster.map_shared_rank(mine, r);
      before += r < rank ? x : 0;
      total += x;
    }
    return before;
  };
  int ties = 0;  // keys equal to the edge before this warp's run
  if (!all) {
    int c = 0, total;
    for (int i = i0; i < i1; i += 32)
      c += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && (key_at(i + lane) >> shift) == edge));
    ties = warp_prefix(sh.warp_n[0], c, warp, lane, total);
    if (tid == 0) sh.n_equal = total;
    cluster.sync();
    ties += cluster_prefix(&sh.n_equal, total);
  }
  // calls f(slot, is a hole, is a mover, holes and movers as lane masks) per step
  auto sweep = [&](auto&& f) {
    int rank_eq = ties;
    for (int i = i0; i < i1; i += 32) {
      const bool in = i + lane < i1;
      const uint32_t k = in ? key_at(i + lane) >> shift : 0u;
      bool kept = in && k > edge;
      const bool eq = in && k == edge;
      if (all) {
        kept = kept || eq;
      } else {
        const unsigned m = __ballot_sync(0xffffffffu, eq);
        kept = kept || (eq && rank_eq + __popc(m & below) < need);
        rank_eq += __popc(m);
      }
      const int s = lo + i + lane;
      const bool hole = in && !kept && s < keep, mover = kept && s >= keep;
      f(s, hole, mover, __ballot_sync(0xffffffffu, hole), __ballot_sync(0xffffffffu, mover));
    }
  };
  int c_holes = 0, c_movers = 0;
  sweep([&](int, bool, bool, unsigned mh, unsigned mm) {
    c_holes += __popc(mh);
    c_movers += __popc(mm);
  });
  int total;
  int at_hole = warp_prefix(sh.warp_n[0], c_holes, warp, lane, total);
  if (tid == 0) sh.n_holes = total;
  int at_mover = warp_prefix(sh.warp_n[1], c_movers, warp, lane, total);
  if (tid == 0) sh.n_movers = total;
  cluster.sync();
  int n_moves;
  at_hole += cluster_prefix(&sh.n_holes, n_moves);
  at_mover += cluster_prefix(&sh.n_movers, n_moves);
  const int64_t cap = cache.capacity();
  int2* holes = moves + (int64_t(b) * cache.n_kv_heads + h) * cap;
  int2* movers = holes + cap / 2;
  sweep([&](int s, bool hole, bool mover, unsigned mh, unsigned mm) {
    if (hole || mover) {
      const int2 where = make_int2(table[cache.page_of(s)], cache.row_of(s));
      if (hole) holes[at_hole + __popc(mh & below)] = where;
      else movers[at_mover + __popc(mm & below)] = where;
    }
    at_hole += __popc(mh);
    at_mover += __popc(mm);
  });
  cluster.sync();

  // ---- the moves: kPairs at a time per warp, 16 bytes per lane and load -------
  constexpr int kRow = D * int(sizeof(T)) / 16;       // pieces of a row
  constexpr int kLoads = 8;                           // in flight per lane
  constexpr int kPairs = kLoads * 32 / (2 * kRow);    // K row and V row of each
  static_assert(kPairs >= 1 && kPairs <= 32);
  uint4* kp = static_cast<uint4*>(cache.k);
  uint4* vp = static_cast<uint4*>(cache.v);
  auto piece = [&](int2 where) {  // first 16-byte piece of that row
    return cache.elem(where.x, h, where.y, D) * int(sizeof(T)) / 16;
  };
  for (int j0 = (warp * nc + rank) * kPairs; j0 < n_moves; j0 += kWarps * nc * kPairs) {
    const int left = min(kPairs, n_moves - j0);
    int64_t src = 0, dst = 0;
    if (lane < left) {
      const int2 to = __ldcg(holes + j0 + lane), from = __ldcg(movers + j0 + lane);
      src = piece(from);
      dst = piece(to);
      const int64_t rs = cache.record(from.x, h, from.y), rd = cache.record(to.x, h, to.y);
      cache.weight[rd] = cache.weight[rs];
      cache.slot_pos[rd] = cache.slot_pos[rs];
    }
    uint4 x[kLoads];
    int64_t to[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = i * 32 + lane, pair = idx / (2 * kRow), e = idx % (2 * kRow);
      const int64_t from = __shfl_sync(0xffffffffu, src, pair);
      to[i] = __shfl_sync(0xffffffffu, dst, pair) + e % kRow;
      if (pair < left) x[i] = (e < kRow ? kp : vp)[from + e % kRow];
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = i * 32 + lane, pair = idx / (2 * kRow), e = idx % (2 * kRow);
      if (pair < left) (e < kRow ? kp : vp)[to[i]] = x[i];
    }
  }
}

}  // namespace pev
}  // namespace hga
