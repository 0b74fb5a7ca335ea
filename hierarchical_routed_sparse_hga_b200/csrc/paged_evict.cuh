// Eviction from the paged cache by accumulated attention weight.
#pragma once

#include "paged.cuh"

namespace hga {
namespace pev {

constexpr int kThreads = 512;

// Rank of a slot: tokens that are kept by position above every weight, a NaN
// weight below every other.
__device__ __forceinline__ uint32_t slot_key(float w, int p, int64_t last, int sinks, int recent) {
  if (p < sinks || int64_t(p) > last - recent) return 0xffffffffu;
  return w == w ? ordered_key(w) : 0u;
}

// One CTA per (KV head, sequence).  keys, flags: [batch, n_kv_heads, cap];
// moves: [batch, n_kv_heads, cap], holes in the first cap/2 entries, movers
// in the others (there are at most min(keep, n - keep) of each).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    paged_evict_kernel(PagedView cache, const int32_t* __restrict__ n_slots,
                       const int64_t* __restrict__ pos, int keep, int sinks, int recent,
                       uint32_t* __restrict__ keys, uint8_t* __restrict__ flags,
                       int32_t* __restrict__ moves) {
  __shared__ int hist[256];
  __shared__ int scratch[kThreads / 32 + 1];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  pdl_wait();
  const int n = checked_slots(cache, n_slots, b);
  if (n <= keep) return;
  const int32_t* table = cache.table + int64_t(b) * cache.max_pages;
  bool bad = false;
  for (int i = tid; i <= cache.page_of(n - 1); i += kThreads) bad = bad || !cache.has(table[i]);
  if (__syncthreads_or(bad)) {
    if (tid == 0) latch_status(HGA_ERR_DEVICE_CHECK);
    return;
  }
  const int64_t head = int64_t(b) * cache.n_kv_heads + h, cap = cache.capacity();
  uint32_t* key = keys + head * cap;
  uint8_t* sel = flags + head * cap;
  int32_t* hole = moves + head * cap;
  int32_t* mover = hole + cap / 2;
  auto record = [&](int s) { return cache.record(table[cache.page_of(s)], h, cache.row_of(s)); };
  auto elem = [&](int s) { return cache.elem(table[cache.page_of(s)], h, cache.row_of(s), D); };
  const int64_t last = pos[b];
  for (int s = tid; s < n; s += kThreads)
    key[s] = slot_key(cache.weight[record(s)], cache.slot_pos[record(s)], last, sinks, recent);
  __syncthreads();
  block_topk(key, n, keep, sel, hist, scratch);
  const int n_moves = block_enumerate(
      keep, [&](int s) { return sel[s] == 0; }, [&](int s, int r) { hole[r] = s; }, scratch);
  block_enumerate(
      n - keep, [&](int i) { return sel[keep + i] != 0; },
      [&](int i, int r) { mover[r] = keep + i; }, scratch);
  __syncthreads();
  T* kp = static_cast<T*>(cache.k);
  T* vp = static_cast<T*>(cache.v);
  for (int64_t i = tid; i < int64_t(n_moves) * D; i += kThreads) {
    const int j = int(i / D), e = int(i % D);
    kp[elem(hole[j]) + e] = kp[elem(mover[j]) + e];
    vp[elem(hole[j]) + e] = vp[elem(mover[j]) + e];
    if (e == 0) {
      cache.weight[record(hole[j])] = cache.weight[record(mover[j])];
      cache.slot_pos[record(hole[j])] = cache.slot_pos[record(mover[j])];
    }
  }
}

}  // namespace pev
}  // namespace hga
