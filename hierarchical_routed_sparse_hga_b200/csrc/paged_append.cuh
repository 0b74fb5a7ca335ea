// New tokens into the paged cache: RoPE of Q and K at each token's position,
// Q head-major, K and V into the rows of the token's slot, its records reset
// (rotate-half RoPE with angles reduced in double precision, as in
// prepare.cuh).  Memory-bound: each projection element is read once and
// written once.
#pragma once

#include "paged.cuh"

namespace hga {

constexpr int kAppendThreads = 256;

// One CTA per (new token i, sequence b); D/16 lanes per row, each holding 8
// rotation pairs (elements 8c .. 8c+7 and D/2 + 8c .. D/2 + 8c+7).
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads)
    paged_append_kernel(PagedView cache, const T* __restrict__ q_proj,
                        const T* __restrict__ k_proj, const T* __restrict__ v_proj,
                        int64_t q_row_stride, int64_t kv_row_stride, int s_new,
                        const int32_t* __restrict__ n_new, const int32_t* __restrict__ n_slots,
                        const int64_t* __restrict__ pos, int n_q_heads, double log2_base,
                        T* __restrict__ q_out) {
  constexpr int HALF = D / 2, LANES = D / 16, SLOTS = kAppendThreads / LANES;
  __shared__ float2 cs[HALF];
  const int i = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int n_kv = cache.n_kv_heads;
  pdl_wait();
  const int n = checked_slots(cache, n_slots, b);
  const int m = n_new ? n_new[b] : s_new;
  const int64_t first = pos[b] - m + 1;
  const bool bad = n < 0 || m < 0 || m > s_new || m > n ||
                   (m > 0 && (first < 0 || pos[b] > 0x7fffffffLL));
  if (bad) {
    if (n >= 0 && tid == 0) latch_status(HGA_ERR_DEVICE_CHECK);
    return;
  }
  if (i >= m) return;
  const int64_t p = first + i;
  if (log2_base > 0.0) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    for (int e = tid; e < HALF; e += kAppendThreads) {
      const double ang = double(p) * exp2(-(2.0 * e / D) * log2_base);
      const double red = fma(-rint(ang * (1.0 / kTwoPi)), kTwoPi, ang);
      float s, c;
      sincosf(float(red), &s, &c);
      cs[e] = make_float2(c, s);
    }
    __syncthreads();
  }
  const int slot = n - m + i;
  const int row = cache.row_of(slot);
  const int page = cache.table[int64_t(b) * cache.max_pages + cache.page_of(slot)];
  const bool stored = cache.has(page);
  if (!stored && tid == 0) latch_status(HGA_ERR_DEVICE_CHECK);
  const int64_t tok = int64_t(b) * s_new + i;
  const int nq = q_proj ? n_q_heads : 0;
  const int c = tid % LANES;
  for (int r = tid / LANES; r < nq + 2 * n_kv; r += SLOTS) {
    const T* src;
    T* dst;
    bool turn = log2_base > 0.0;
    if (r < nq) {
      src = q_proj + tok * q_row_stride + int64_t(r) * D;
      dst = q_out + ((int64_t(b) * n_q_heads + r) * s_new + i) * D;
    } else {
      if (!stored) continue;
      const int h = (r - nq) % n_kv;
      const bool is_v = r - nq >= n_kv;
      src = (is_v ? v_proj : k_proj) + tok * kv_row_stride + int64_t(h) * D;
      dst = static_cast<T*>(is_v ? cache.v : cache.k) + cache.elem(page, h, row, D);
      turn = turn && !is_v;
    }
    float y1[8], y2[8];
    load8(src + 8 * c, y1);
    load8(src + HALF + 8 * c, y2);
    if (turn) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = cs[8 * c + e];
        const float a = y1[e], z = y2[e];
        y1[e] = a * w.x - z * w.y;
        y2[e] = z * w.x + a * w.y;
      }
    }
    store8(dst + 8 * c, y1);
    store8(dst + HALF + 8 * c, y2);
  }
  if (stored)
    for (int h = tid; h < n_kv; h += kAppendThreads) {
      if (cache.weight) cache.weight[cache.record(page, h, row)] = 0.f;
      if (cache.slot_pos) cache.slot_pos[cache.record(page, h, row)] = int32_t(p);
    }
}

}  // namespace hga
