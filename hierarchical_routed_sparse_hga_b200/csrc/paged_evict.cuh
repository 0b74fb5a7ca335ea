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
// share of the slots in shared memory (read from HBM once; what is beyond
// key_cap is read again each time); the blocks read one another's digit
// counts, tie counts and move counts after a cluster barrier.
//
//  1. the keep-th largest key by radix select, 8 bits a round (the blocks read
//     one another's counts: 11 bits would be 8 KiB from each, and slower);
//     after the first digit only the keys of its bin are looked at, and the
//     select ends where the rest of a bin is kept whole (mostly after three);
//  2. a bit per slot (kept or not), ranks of holes and movers within the block
//     from the words' population counts, a list of (page, row) of both; each
//     block has the list entries of its own slots, holes from the front and
//     movers from the back, so the blocks need not know one another's numbers;
//  3. the moves, each 16-byte piece read and written once.
// 1 and 2 (paged_evict_kernel) are a chain of short phases; loops are kept
// rolled where they can be, since each runs once and its instructions are
// fetched for that one time.  3 is bound by HBM and wants the whole GPU and
// other registers, so it is a launch of its own (paged_move_kernel) unless
// there is little to move.
#pragma once

#include <cooperative_groups.h>

#include "paged.cuh"

namespace hga {
namespace pev {

namespace cg = cooperative_groups;

constexpr int kMaxC = 8;  // blocks per cluster, at most (portable size)
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
// A block's share up to which the moves are not a launch of their own: 1 x 1500
// slots cut to 1024 (a share of 188) 12.2 us against 12.9 and one launch less;
// 1 x 4096 cut to 2048 (512) 14.6 against 13.4.
constexpr int kFewSlots = 256;
constexpr int kKeyCap = 44 * 1024;  // keys in one block's shared memory, at most

// Rank of a slot: tokens that are kept by position above every weight, a NaN
// weight below every other.
__device__ __forceinline__ uint32_t slot_key(float w, int p, int64_t last, int sinks, int recent) {
  if (p < sinks || int64_t(p) > last - recent) return 0xffffffffu;
  return w == w ? ordered_key(w) : 0u;
}

constexpr int kBins = 256;
constexpr int kRounds = 4;
constexpr int kCands = 256;             // keys of the first digit's bin that a warp lists
constexpr int kGroup4 = 128;            // slots of a group: four to a lane
constexpr int kGroups = kThreads;       // groups whose ranks are formed at once
constexpr int kChunk = kGroups * kGroup4;

struct alignas(16) Shared {
  int hist[kRounds][kBins];  // one per round, so that a round needs one cluster barrier
  uint32_t cand[kWarps][kCands];
  // group g: bit l of word j is slot 4 l + j
  uint4 equal_bits[kGroups], kept_bits[kGroups];
  int equal_rank[kGroups];
  int2 rank[kGroups];  // of the first hole and mover
  int2 warp_sum[kWarps];
  int unlisted, n_equal, bad;
  int2 n_moves, before[kMaxC + 1];  // the block's holes and movers; of the blocks before each
  // the select's state: keys whose bits from `shift` up exceed prefix's are
  // kept, of those that equal them `need` more (all: every one)
  uint32_t prefix;
  int shift, need, all;
};

// Exclusive prefix over the block's threads of x and y, and their totals.
__device__ __forceinline__ int2 thread_prefix(int2* table, int x, int y, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 incl = make_int2(x, y);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int px = __shfl_up_sync(0xffffffffu, incl.x, o);
    const int py = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += px;
      incl.y += py;
    }
  }
  if (lane == 31) table[warp] = incl;
  __syncthreads();
  int2 before = make_int2(incl.x - x, incl.y - y);
  total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int2 t = table[w];
    if (w < warp) {
      before.x += t.x;
      before.y += t.y;
    }
    total.x += t.x;
    total.y += t.y;
  }
  __syncthreads();
  return before;
}

// first slot of block `rank`'s share
__device__ __forceinline__ int share_begin(int n, int rank, int nc) {
  return min(n, rank * ((((n + nc - 1) / nc) + 3) & ~3));
}

// Exclusive prefix over a cluster's blocks of their holes and movers, by one
// warp, from the lanes' own c (lane r: block r's): before[0 .. kMaxC].
__device__ __forceinline__ void blocks_before(int2 c, int lane, int2* before) {
  int2 incl = c;
#pragma unroll
  for (int o = 1; o < kMaxC; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o);
    const int y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
    }
  }
  if (lane < kMaxC) before[lane + 1] = incl;
  if (lane == 0) before[0] = make_int2(0, 0);
}

// The moves of a (sequence, head) of n slots, kPairs at a time per warp, 16
// bytes per lane and load: warp `worker` of `workers`.  The j-th hole takes the
// j-th mover; sources lie at or behind slot `keep` and destinations before it,
// so the moves may run in any order.  list: the blocks' holes and movers;
// before: their numbers before each of the nc blocks.
template <typename T, int D>
__device__ __forceinline__ void move_rows(const PagedView& cache, int h, int n, int nc,
                                          const int2* list, const int2* before, int worker,
                                          int workers) {
  const int lane = threadIdx.x & 31;
  const int n_moves = before[kMaxC].x;
  constexpr int kRow = D * int(sizeof(T)) / 16;       // pieces of a row
  constexpr int kLoads = 4;                           // in flight per lane
  constexpr int kPairs = kLoads * 32 / (2 * kRow);    // K row and V row of each
  static_assert(kPairs >= 1 && kPairs <= 32);
  uint4* kp = static_cast<uint4*>(cache.k);
  uint4* vp = static_cast<uint4*>(cache.v);
  auto piece = [&](int2 where) {  // first 16-byte piece of that row
    return cache.elem(where.x, h, where.y, D) * int(sizeof(T)) / 16;
  };
  const int j_step = workers * kPairs;
  int2 to_where = make_int2(0, 0), from_where = to_where;
  auto fetch = [&](int j) {  // of the pair that this lane looks after
    if (lane < kPairs && j + lane < n_moves) {
      int rh = 0, rm = 0;
      for (int r = 1; r < nc; ++r) {
        rh += j + lane >= before[r].x ? 1 : 0;
        rm += j + lane >= before[r].y ? 1 : 0;
      }
      to_where = __ldcg(list + share_begin(n, rh, nc) + (j + lane - before[rh].x));
      from_where = __ldcg(list + share_begin(n, rm + 1, nc) - 1 - (j + lane - before[rm].y));
    }
  };
  int j0 = worker * kPairs;
  fetch(j0);
  for (; j0 < n_moves; j0 += j_step) {
    const int left = min(kPairs, n_moves - j0);
    const int64_t src = piece(from_where), dst = piece(to_where);
    float w = 0.f;
    int p = 0;
    int64_t rd = 0;
    if (lane < left) {
      const int64_t rs = cache.record(from_where.x, h, from_where.y);
      rd = cache.record(to_where.x, h, to_where.y);
      w = cache.weight[rs];
      p = cache.slot_pos[rs];
    }
    fetch(j0 + j_step);
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
    if (lane < left) {
      cache.weight[rd] = w;
      cache.slot_pos[rd] = p;
    }
  }
}

// grid (nc, n_kv_heads, batch) in clusters of (nc, 1, 1); dynamic shared
// memory: Shared, then key_cap keys.  counts: [batch, n_kv_heads, kMaxC] numbers
// of holes and movers of each block.  moves: [batch, n_kv_heads, capacity]
// entries of (page, row).  D > 0: the moves of rows of D elements of T follow
// in this launch (counts is not used); D = 0: in paged_move_kernel's.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, D > 0 ? 1 : 2)
    paged_evict_kernel(PagedView cache, const int32_t* __restrict__ n_slots,
                       const int64_t* __restrict__ pos, int keep, int sinks, int recent,
                       int key_cap, int2* __restrict__ counts, int2* __restrict__ moves) {
  extern __shared__ __align__(16) unsigned char ev_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(ev_raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ev_raw + sizeof(Shared));
  static_assert(sizeof(Shared) % 16 == 0);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank()), nc = int(cluster.num_blocks());
  const int h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kRounds * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) {
    sh.bad = 0;
    sh.unlisted = 0;
    sh.prefix = 0u;
    sh.shift = 32;
    sh.need = keep;
    sh.all = 0;
  }
  pdl_wait();
  // the whole cluster reads the same count and leaves here
  const int n = rank == 0 && tid == 0 ? checked_slots(cache, n_slots, b) : n_slots[b];
  const int64_t pair = int64_t(b) * cache.n_kv_heads + h;
  if constexpr (D == 0) pdl_launch_dependents();
  if (n <= keep || int64_t(n) > cache.capacity()) {
    if (D == 0 && tid == 0) counts[pair * kMaxC + rank] = make_int2(0, 0);
    return;
  }
  __syncthreads();
  const int64_t last = pos[b];
  const int32_t* table = cache.table + int64_t(b) * cache.max_pages;
  const int lo = share_begin(n, rank, nc), n_loc = share_begin(n, rank + 1, nc) - lo;

  // ---- keys of this block's share, four slots at a time -----------------------
  constexpr int kBatch = 4;  // of four slots, their loads in flight together
  auto at4 = [&](int i) -> int64_t {  // first record of slots lo + i ..; -1: none
    if (i >= n_loc) return -1;
    const int page = __ldg(table + cache.page_of(lo + i));
    if (cache.has(page)) return cache.record(page, h, cache.row_of(lo + i));
    sh.bad = 1;
    return -1;
  };
#pragma unroll 1
  for (int base = tid * 4; base < n_loc; base += kBatch * kThreads * 4) {
    int64_t at[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) at[u] = at4(base + u * kThreads * 4);
    float4 w[kBatch];
    int4 p[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (at[u] >= 0) {
        w[u] = *reinterpret_cast<const float4*>(cache.weight + at[u]);
        p[u] = *reinterpret_cast<const int4*>(cache.slot_pos + at[u]);
      }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = base + u * kThreads * 4;
      if (at[u] >= 0 && i < key_cap)
        *reinterpret_cast<uint4*>(keys + i) =
            make_uint4(slot_key(w[u].x, p[u].x, last, sinks, recent),
                       slot_key(w[u].y, p[u].y, last, sinks, recent),
                       slot_key(w[u].z, p[u].z, last, sinks, recent),
                       slot_key(w[u].w, p[u].w, last, sinks, recent));
    }
  }
  __syncthreads();
  auto key_at = [&](int i) -> uint32_t {
    if (i < key_cap) return keys[i];
    const int s = lo + i, page = __ldg(table + cache.page_of(s));
    if (!cache.has(page)) return 0u;
    const int64_t at = cache.record(page, h, cache.row_of(s));
    return slot_key(cache.weight[at], cache.slot_pos[at], last, sinks, recent);
  };

  auto key4_at = [&](int i) -> uint4 {  // i a multiple of 4, below n_loc
    if (i < key_cap) return *reinterpret_cast<const uint4*>(keys + i);
    return make_uint4(key_at(i), i + 1 < n_loc ? key_at(i + 1) : 0u,
                      i + 2 < n_loc ? key_at(i + 2) : 0u, i + 3 < n_loc ? key_at(i + 3) : 0u);
  };

  // ---- the keep-th largest key -----------------------------------------------
  int n_cand = 0;  // keys on this warp's list
#pragma unroll 1
  for (int round = 0; round < kRounds; ++round) {
    const int shift = 24 - 8 * round;
    const uint32_t bin = round == 0 ? 0u : sh.prefix >> (shift + 8);
    int* hist = sh.hist[round];
    if (round >= 2 && sh.unlisted == 0) {
      for (int i = lane; i < n_cand; i += 32) {
        const uint32_t k = sh.cand[warp][i];
        if ((k >> (shift + 8)) == bin) atomicAdd(&hist[(k >> shift) & (kBins - 1)], 1);
      }
    } else {
      // four keys per lane: each alone would wait for its own chain
#pragma unroll 1
      for (int i0 = warp * kGroup4; i0 < n_loc; i0 += kThreads * 4) {
        const int i = i0 + lane * 4;
        const uint4 q = i < n_loc ? key4_at(i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t k[4] = {q.x, q.y, q.z, q.w};
        bool in_bin[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          in_bin[j] = i + j < n_loc && (round == 0 || (k[j] >> (shift + 8)) == bin);
          if (in_bin[j]) atomicAdd(&hist[(k[j] >> shift) & (kBins - 1)], 1);
        }
        if (round == 1) {  // list the bin's keys
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const unsigned m = __ballot_sync(0xffffffffu, in_bin[j]);
            const int at = n_cand + __popc(m & ((1u << lane) - 1u));
            if (in_bin[j] && at < kCands) sh.cand[warp][at] = k[j];
            n_cand += __popc(m);
          }
        }
      }
      if (round == 1 && n_cand > kCands && lane == 0) sh.unlisted = 1;
    }
    cluster.sync();  // every block's counts of this round
    // thread t < 256: digit 255 - t of the whole cluster
    int x[kMaxC], bad = 0;
#pragma unroll
    for (int r = 0; r < kMaxC; ++r) {  // in flight together
      x[r] = 0;
      if (r < nc && tid < kBins)
        x[r] = cluster.map_shared_rank(&sh, r)->hist[round][kBins - 1 - tid];
    }
    if (round == 0 && tid < nc) bad = cluster.map_shared_rank(&sh, tid)->bad;
    if (round == 0 && __syncthreads_or(bad)) {
      // the same for the whole cluster; nothing was written
      if (rank == 0 && tid == 0) latch_status(HGA_ERR_DEVICE_CHECK);
      if (D == 0 && tid == 0) counts[pair * kMaxC + rank] = make_int2(0, 0);
      cluster.sync();
      return;
    }
    int count = 0;
#pragma unroll
    for (int r = 0; r < kMaxC; ++r) count += x[r];
    const int need = sh.need;
    int2 total;
    const int above = thread_prefix(sh.warp_sum, count, 0, total).x;
    if (above < need && above + count >= need) {  // in one thread of the block
      sh.prefix |= uint32_t(kBins - 1 - tid) << shift;
      sh.shift = shift;
      sh.need = need - above;
      sh.all = count == need - above;
    }
    __syncthreads();
    if (sh.all) break;  // the whole bin is kept: the other digits do not matter
  }
  const int shift = sh.shift, need = sh.need;
  const bool all = sh.all;
  const uint32_t edge = sh.prefix >> shift;

  // ---- holes and movers --------------------------------------------------------
  // bits below slot `limit` of word j of a group that begins at slot s
  auto lanes_below = [&](int limit, int s, int j) -> unsigned {
    const int c = (limit - s - j + 3) >> 2;
    return c >= 32 ? ~0u : c > 0 ? (1u << c) - 1u : 0u;
  };
  auto popc4 = [](const uint4& m) {
    return __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
  };
  const unsigned below = (1u << lane) - 1u;
  // the keys that equal the edge, by group, and how many come before each
  auto rank_equal = [&](int c0, int n_groups) {
#pragma unroll 1
    for (int g = warp; g < n_groups; g += kWarps) {
      const int i = c0 + g * kGroup4 + lane * 4;
      const uint4 q = i < n_loc ? key4_at(i) : make_uint4(0u, 0u, 0u, 0u);
      const uint4 m = make_uint4(
          __ballot_sync(0xffffffffu, i < n_loc && (q.x >> shift) == edge),
          __ballot_sync(0xffffffffu, i + 1 < n_loc && (q.y >> shift) == edge),
          __ballot_sync(0xffffffffu, i + 2 < n_loc && (q.z >> shift) == edge),
          __ballot_sync(0xffffffffu, i + 3 < n_loc && (q.w >> shift) == edge));
      if (lane == 0) sh.equal_bits[g] = m;
    }
    __syncthreads();
    int2 total;
    const int c = tid < n_groups ? popc4(sh.equal_bits[tid]) : 0;
    sh.equal_rank[tid] = thread_prefix(sh.warp_sum, c, 0, total).x;
    __syncthreads();
    return total.x;
  };
  // With ties, a pass over the chunks for their number, then the lists (a
  // single chunk's tie ranks stand from the first).
  int2* list = moves + pair * cache.capacity() + lo;
  const bool one_chunk = n_loc <= kChunk;
  int ties = 0;  // keys equal to the edge before the chunk
  if (!all) {
#pragma unroll 1
    for (int c0 = 0; c0 < n_loc; c0 += kChunk)
      ties += rank_equal(c0, (min(kChunk, n_loc - c0) + kGroup4 - 1) / kGroup4);
    if (tid == 0) sh.n_equal = ties;
    cluster.sync();
    ties = 0;
    for (int r = 0; r < rank; ++r) ties += *cluster.map_shared_rank(&sh.n_equal, r);
  }
  // D = 0: no more of another block's memory is read, but this block's is not
  // to be left before the others are done with it
  if constexpr (D == 0) cluster.barrier_arrive();
  int2 at = make_int2(0, 0);  // holes and movers before the chunk
#pragma unroll 1
  for (int c0 = 0; c0 < n_loc; c0 += kChunk) {
    const int n_groups = (min(kChunk, n_loc - c0) + kGroup4 - 1) / kGroup4;
    const int equals = all || one_chunk ? 0 : rank_equal(c0, n_groups);
#pragma unroll 1
    for (int g = warp; g < n_groups; g += kWarps) {
      const int i = c0 + g * kGroup4 + lane * 4;
      const uint4 q = i < n_loc ? key4_at(i) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t k[4] = {q.x >> shift, q.y >> shift, q.z >> shift, q.w >> shift};
      bool kept[4];
      if (all) {
#pragma unroll
        for (int j = 0; j < 4; ++j) kept[j] = i + j < n_loc && k[j] >= edge;
      } else {
        const uint4 eq = sh.equal_bits[g];
        int rank_eq = ties + sh.equal_rank[g] +
                      popc4(make_uint4(eq.x & below, eq.y & below, eq.z & below, eq.w & below));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool same = i + j < n_loc && k[j] == edge;
          kept[j] = (i + j < n_loc && k[j] > edge) || (same && rank_eq < need);
          rank_eq += same ? 1 : 0;
        }
      }
      const uint4 m = make_uint4(
          __ballot_sync(0xffffffffu, kept[0]), __ballot_sync(0xffffffffu, kept[1]),
          __ballot_sync(0xffffffffu, kept[2]), __ballot_sync(0xffffffffu, kept[3]));
      if (lane == 0) sh.kept_bits[g] = m;
    }
    __syncthreads();
    int n_hole = 0, n_mover = 0;  // of this thread's group
    if (tid < n_groups) {
      const uint4 m = sh.kept_bits[tid];
      const unsigned bits[4] = {m.x, m.y, m.z, m.w};
      const int s = lo + c0 + tid * kGroup4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n_hole += __popc(~bits[j] & lanes_below(min(keep, lo + n_loc), s, j));
        n_mover += __popc(bits[j] & ~lanes_below(keep, s, j));
      }
    }
    int2 total;
    sh.rank[tid] = thread_prefix(sh.warp_sum, n_hole, n_mover, total);
    __syncthreads();
    // a warp per group, four slots (of one page) per lane
#pragma unroll 1
    for (int g = warp; g < n_groups; g += kWarps) {
      const uint4 m = sh.kept_bits[g];
      const unsigned bits[4] = {m.x, m.y, m.z, m.w};
      const int s = lo + c0 + g * kGroup4, mine = s + lane * 4;
      const int page = mine < n ? __ldg(table + cache.page_of(mine)) : 0;
      int hole = at.x + sh.rank[g].x, mover = at.y + sh.rank[g].y;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned low = lanes_below(min(keep, lo + n_loc), s, j);
        hole += __popc(~bits[j] & low & below);
        mover += __popc(bits[j] & ~low & below);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool kept = (bits[j] >> lane & 1u) != 0u, first = mine + j < keep;
        if (mine + j < lo + n_loc && kept != first)  // a hole or a mover
          list[first ? hole++ : n_loc - 1 - mover++] =
              make_int2(page, cache.row_of(mine + j));
      }
    }
    at.x += total.x;
    at.y += total.y;
    ties += equals;
    __syncthreads();  // the next chunk overwrites the bits
  }
  if constexpr (D == 0) {
    if (tid == 0) counts[pair * kMaxC + rank] = at;
    cluster.barrier_wait();
  } else {
    if (tid == 0) sh.n_moves = at;
    cluster.sync();
    if (warp == 0)
      blocks_before(lane < nc ? cluster.map_shared_rank(&sh, lane)->n_moves : make_int2(0, 0),
                    lane, sh.before);
    __syncthreads();
    cluster.barrier_arrive();  // no more of another block's memory is read
    move_rows<T, D>(cache, h, n, nc, moves + pair * cache.capacity(), sh.before,
                    warp * nc + rank, kWarps * nc);
    __syncthreads();
    __threadfence();
    pdl_launch_dependents();
    cluster.barrier_wait();
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;

// grid (x, n_kv_heads, batch): the moves of each (sequence, head) by x blocks;
// nc: blocks of paged_evict_kernel per (sequence, head)
template <typename T, int D>
__global__ void __launch_bounds__(kMoveThreads)
    paged_move_kernel(PagedView cache, const int32_t* __restrict__ n_slots, int nc,
                      const int2* __restrict__ counts, const int2* __restrict__ moves) {
  __shared__ int2 before[kMaxC + 1];
  const int h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t pair = int64_t(b) * cache.n_kv_heads + h;
  pdl_wait();
  if (warp == 0)
    blocks_before(lane < nc ? counts[pair * kMaxC + lane] : make_int2(0, 0), lane, before);
  __syncthreads();
  move_rows<T, D>(cache, h, n_slots[b], nc, moves + pair * cache.capacity(), before,
                  warp * int(gridDim.x) + int(blockIdx.x), kMoveWarps * int(gridDim.x));
  // as at the end of paged_join_kernel
  __syncthreads();
  __threadfence();
  pdl_launch_dependents();
}

}  // namespace pev
}  // namespace hga
