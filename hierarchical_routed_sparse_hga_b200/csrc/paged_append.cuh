// New tokens into the paged cache: RoPE of Q and K at each token's position,
// Q head-major, K and V into the rows of the token's slot, its records reset
// (rotate-half RoPE with angles reduced in double precision, as in
// prepare.cuh).  Memory-bound: each projection element is read once and
// written once.
//
// Warps work on their own, without block barriers but the last: the chain in front of a
// token's rows (counts, page, angles) takes longer than the rows themselves,
// so what counts is that many tokens are at different points of it: two rows
// per lane in flight (4 x 8192 tokens, ragged: 92 us, 5.5 TB/s; with four rows and
// fewer warps 96 us), in blocks of four warps (of eight: 96 us).  A prompt takes
// one warp per token; with few tokens (up to four an SM) kTokenWarps share one,
// and each makes the token's table of angles for itself: 8 tokens 2.8 us (one
// warp each: 6.9), 512 tokens 4.7 us (7.0), from about 1000 tokens on no gain.
#pragma once

#include "paged.cuh"

namespace hga {

constexpr int kAppendWarps = 4;  // of a block
constexpr int kTokenWarps = 8;

// grid: ceil(batch * s_new * per_tok / kAppendWarps); per_tok warps share a
// token (row tok % s_new of sequence tok / s_new).  D/16 lanes per row, each
// holding 8 rotation pairs (elements 8c .. 8c+7 and D/2 + 8c .. D/2 + 8c+7),
// several rows' loads in flight.  ratio: base^(-2/D), 0 for no rotation.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kAppendWarps)
    paged_append_kernel(PagedView cache, const T* __restrict__ q_proj,
                        const T* __restrict__ k_proj, const T* __restrict__ v_proj,
                        int64_t q_row_stride, int64_t kv_row_stride, int tokens, int s_new,
                        int per_tok, const int32_t* __restrict__ n_new,
                        const int32_t* __restrict__ n_slots, const int64_t* __restrict__ pos,
                        int n_q_heads, double ratio, T* __restrict__ q_out) {
  constexpr int HALF = D / 2, LANES = D / 16, ROWS = 32 / LANES;
  constexpr int kBatch = sizeof(T) == 2 ? 2 : 1;  // rows in flight per lane
  __shared__ __align__(16) float2 table[kAppendWarps][HALF];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_kv = cache.n_kv_heads;
  const int64_t unit = int64_t(blockIdx.x) * kAppendWarps + warp;
  const int tok = int(unit / per_tok), part = int(unit % per_tok);
  pdl_wait();
  if (tok < tokens) {
    const int b = tok / s_new, i = tok % s_new;
    const int nq = q_proj ? n_q_heads : 0, heads = nq + 2 * n_kv;  // rows of a token
    const int c = lane % LANES, sub = lane / LANES;
    const T* q_row = q_proj + int64_t(tok) * q_row_stride;
    const T* k_row = k_proj + int64_t(tok) * kv_row_stride;
    const T* v_row = v_proj + int64_t(tok) * kv_row_stride;
    // row r of the token: query heads, then keys, then values
    auto row = [&](int u, int r0) { return (r0 + u * per_tok) * ROWS + sub; };
    Raw8<T> x1[kBatch], x2[kBatch];
    auto load = [&](int r0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int r = row(u, r0);
        if (r >= heads) continue;
        const T* src = r < nq ? q_row + r * D
                              : r < nq + n_kv ? k_row + (r - nq) * D : v_row + (r - nq - n_kv) * D;
        x1[u].load(src + 8 * c);
        x2[u].load(src + HALF + 8 * c);
      }
    };
    load(part);  // whether or not the row is a token: it is there
    const int n = n_slots[b], m = n_new ? n_new[b] : s_new;
    const int64_t last = pos[b], first = last - m + 1;
    const bool bad = n < 0 || int64_t(n) > cache.capacity() || m < 0 || m > s_new || m > n ||
                     (m > 0 && (first < 0 || last > 0x7fffffffLL));
    if (bad && lane == 0) latch_status(HGA_ERR_DEVICE_CHECK);
    if (!bad && i < m) {
      const int slot = n - m + i, slot_row = cache.row_of(slot);
      const int page = cache.table[int64_t(b) * cache.max_pages + cache.page_of(slot)];
      const int p = int(first + i);
      if (ratio > 0.0) {
        constexpr double kTwoPi = 6.283185307179586476925286766559;
        for (int e = lane; e < HALF; e += 32) {
          // theta = ratio^e by squaring
          double theta = 1.0, power = ratio;
#pragma unroll
          for (int bits = e, k = 0; k < (D == 128 ? 6 : 5); ++k, bits >>= 1, power *= power)
            if (bits & 1) theta *= power;
          const double ang = double(p) * theta;
          const double red = fma(-rint(ang * (1.0 / kTwoPi)), kTwoPi, ang);
          float s, co;
          sincosf(float(red), &s, &co);
          table[warp][e] = make_float2(co, s);
        }
        __syncwarp();
      }
      const bool stored = cache.has(page);
      if (!stored && lane == 0) latch_status(HGA_ERR_DEVICE_CHECK);
      T* q_dst = q_out + (int64_t(b) * n_q_heads * s_new + i) * D;
      const int64_t at = stored ? cache.elem(page, 0, slot_row, D) : 0;
      T* k_dst = static_cast<T*>(cache.k) + at;
      T* v_dst = static_cast<T*>(cache.v) + at;
      for (int r0 = part;;) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int r = row(u, r0);
          if (r >= heads || (r >= nq && !stored)) continue;
          float y1[8], y2[8];
          x1[u].get(y1);
          x2[u].get(y2);
          if (r < nq + n_kv && ratio > 0.0) {
            const float4* cs = reinterpret_cast<const float4*>(&table[warp][8 * c]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 w = cs[e];  // (cos, sin) of two pairs
              const float a0 = y1[2 * e], z0 = y2[2 * e], a1 = y1[2 * e + 1], z1 = y2[2 * e + 1];
              y1[2 * e] = a0 * w.x - z0 * w.y;
              y2[2 * e] = z0 * w.x + a0 * w.y;
              y1[2 * e + 1] = a1 * w.z - z1 * w.w;
              y2[2 * e + 1] = z1 * w.z + a1 * w.w;
            }
          }
          T* dst = r < nq ? q_dst + int64_t(r) * s_new * D
                          : r < nq + n_kv ? k_dst + (int64_t(r - nq) << cache.page_shift) * D
                                          : v_dst + (int64_t(r - nq - n_kv) << cache.page_shift) * D;
          store8(dst + 8 * c, y1);
          store8(dst + HALF + 8 * c, y2);
        }
        r0 += kBatch * per_tok;
        if (r0 * ROWS >= heads) break;
        load(r0);
      }
      if (part == 0 && stored)
        for (int h = lane; h < n_kv; h += 32) {
          if (cache.weight) cache.weight[cache.record(page, h, slot_row)] = 0.f;
          if (cache.slot_pos) cache.slot_pos[cache.record(page, h, slot_row)] = p;
        }
    }
  }
  // The next kernel on the stream may read Q before its own wait (the routing
  // does).  The first warp's trigger counts for the whole block, so it comes
  // after the last one's stores.
  __syncthreads();
  __threadfence();
  pdl_launch_dependents();
}

}  // namespace hga
