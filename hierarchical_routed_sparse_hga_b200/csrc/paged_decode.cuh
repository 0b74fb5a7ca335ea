// Attention of one new token per sequence over its paged cache.
#pragma once

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace hga {
namespace pdec {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxG = 8;

// One CTA per (KV head, sequence).  A warp takes one slot at a time, D/32
// elements per lane, with an online softmax per query head; the warps'
// (max, sum, output) partials are merged in warp order.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    paged_decode_kernel(PagedView cache, const T* __restrict__ q,
                        const int32_t* __restrict__ n_slots, int G, int accumulate,
                        float scale_log2, T* __restrict__ o, float* __restrict__ lse) {
  constexpr int E = D / 32;
  __shared__ float qs[kMaxG][D];
  __shared__ float wo[kWarps][kMaxG][D];
  __shared__ float wm[kWarps][kMaxG], wl[kWarps][kMaxG], ls[kMaxG];
  const int h = blockIdx.x, b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  const int n = checked_slots(cache, n_slots, b);
  if (n < 0) return;
  const int64_t row0 = (int64_t(b) * cache.n_kv_heads + h) * G;
  for (int i = tid; i < G * D; i += kThreads) qs[i / D][i % D] = to_float(q[row0 * D + i]);
  __syncthreads();
  const int32_t* table = cache.table + int64_t(b) * cache.max_pages;
  const T* kp = static_cast<const T*>(cache.k);
  const T* vp = static_cast<const T*>(cache.v);
  auto score = [&](int64_t at, int g) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(to_float(kp[at + e * 32 + lane]), qs[g][e * 32 + lane], s);
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    return s * scale_log2;
  };
  float m[kMaxG], l[kMaxG], acc[kMaxG][E];
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[g][e] = 0.f;
  }
  for (int s = warp; s < n; s += kWarps) {
    const int page = table[cache.page_of(s)];
    if (!cache.has(page)) {
      if (lane == 0) latch_status(HGA_ERR_DEVICE_CHECK);
      continue;
    }
    const int64_t at = cache.elem(page, h, cache.row_of(s), D);
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = to_float(vp[at + e * 32 + lane]);
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      if (g >= G) break;
      const float x = score(at, g);
      const float top = fmaxf(m[g], x);
      if (top == -INFINITY) continue;  // no weight yet
      const float a = exp2f(m[g] - top), p = exp2f(x - top);
      m[g] = top;
      l[g] = l[g] * a + p;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[g][e] = fmaf(p, v[e], acc[g][e] * a);
    }
  }
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    if (lane == 0) {
      wm[warp][g] = m[g];
      wl[warp][g] = l[g];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) wo[warp][g][e * 32 + lane] = acc[g][e];
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += kThreads) {
    const int g = i / D, e = i % D;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w][g]);
    for (int w = 0; w < kWarps; ++w) {
      if (wl[w][g] == 0.f) continue;
      const float a = exp2f(wm[w][g] - M);
      L = fmaf(a, wl[w][g], L);
      O = fmaf(a, wo[w][g][e], O);
    }
    o[(row0 + g) * D + e] = from_float<T>(L == 0.f ? 0.f : O / L);
    if (e == 0) {
      ls[g] = L == 0.f ? -INFINITY : M + log2f(L);
      lse[row0 + g] = ls[g] * 0.6931471805599453f;
    }
  }
  if (!accumulate) return;
  __syncthreads();
  for (int s = warp; s < n; s += kWarps) {
    const int page = table[cache.page_of(s)];
    if (!cache.has(page)) continue;
    const int64_t at = cache.elem(page, h, cache.row_of(s), D);
    float w = 0.f;
    for (int g = 0; g < G; ++g) w += exp2f(score(at, g) - ls[g]);
    if (lane == 0) atomicAdd(&cache.weight[cache.record(page, h, cache.row_of(s))], w);
  }
}

}  // namespace pdec
}  // namespace hga
