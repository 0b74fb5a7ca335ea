// Attention of one new token per sequence over its paged cache.
//
//   s_j = scale q.k_j,  O = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m)   (s in base 2)
//
// Every key and value is read once and meets G <= 8 queries: 4 G flops for
// the 4 (bf16) or 8 (float32) bytes of a K and a V element, far below what the
// tensor cores need to be busy, so the kernel is bound by HBM.  What it has to
// do is keep enough loads in flight on every SM whatever the lengths are.
//
// Split.  The slots of each (sequence, KV head) are cut into units of kUnit
// slots; the units of the whole batch, in order, are dealt out to the blocks
// in equal contiguous runs.  The counts are read on the device, so a ragged
// batch or one long sequence fills the GPU like any other, and a captured
// graph follows the lengths.  A block's run covers at most two incomplete
// (sequence, head) pieces, its first and its last; their partial results go
// to the workspace and paged_join_kernel joins them.
//
// Tile.  A warp takes 4 KiB of K and 4 KiB of V at a time straight into
// registers, 16 bytes per lane and load, in the layout that the matrix
// instruction wants, so nothing passes through shared memory:
//   S [heads x slots] = Q K^T: Q is the 16-row operand (rows >= G are 0), a K
//     row is a column; which element of d stands at which k index is free as
//     long as Q and K agree, so each lane keeps the 16-byte pieces it loaded;
//   O^T [d x heads] = V^T P^T: V^T is the 16-row operand, rows in an order
//     that lets a lane keep its 16-byte pieces (bf16 pairs of two slots are
//     formed with byte permutes), and P^T is exactly the fragment that S left
//     in the lane's registers.
// The warps of a block take the tiles of a piece in turn; their results are
// merged through shared memory in warp order.  All orders are fixed, so
// results are deterministic.
//
// Precision.  Statistics and sums are float32.  P enters its product as two
// bf16 parts (high and remainder, 16 bits): one part alone would add an error
// as large as the rounding of a bf16 output.  Float32 operands are split into
// two tf32 parts and the three largest of the four products are summed: each
// product is good to 2^-21, which plain tf32 (2^-11) is not.
#pragma once

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace hga {
namespace pdec {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 2;
constexpr int kBlocks = 148 * kBlocksPerSm;  // of the B200's 148 SMs
constexpr int kMaxG = 8;
constexpr float kLn2 = 0.6931471805599453f;
// the reference point of the running softmax moves only when a score exceeds
// it by more than this (in base 2): the weights stay below 2^8, no precision
// is lost in float32, and nearly every tile is spared the rescaling
constexpr float kSlack = 8.f;

template <typename T, int D>
struct Tile {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kSlab = kBf16 ? 16 : 8;            // slots of one P V step
  static constexpr int kSlabs = 4096 / (kSlab * D * int(sizeof(T)));
  static constexpr int kSlots = kSlab * kSlabs;           // slots of a tile
  static constexpr int kNt = kSlab / 8;                   // 8-slot columns of S per slab
  static constexpr int kKc = D * int(sizeof(T)) / 64;     // 16-byte pieces of a K row per lane
  static constexpr int kVt = kSlab / 4;                   // V rows per lane and slab
  static constexpr int kVc = D * int(sizeof(T)) / 128;    // 16-byte pieces of a V row per lane
  static constexpr int kMt = D / 16;                      // 16-row tiles of O^T
  static constexpr int kUnit = kWarps * kSlots;
};

// what the decode kernel leaves for the join kernel, at the head of the workspace
struct Work {
  int64_t* first;   // [batch + 1]: units before each sequence; the last: all of them
  float* part;      // [2 * kBlocks][G * (D + 2)]: m[G], l[G], o[G][D] of an incomplete piece
  float* scores;    // [units][kUnit / kSlots][G][kSlots], in base 2; nullptr: not kept
};

// blocks in use, the run of block c, and the block that holds unit u
__host__ __device__ __forceinline__ int blocks_for(int64_t units) {
  return int(units < kBlocks ? units : kBlocks);
}
__device__ __forceinline__ int64_t run_begin(int c, int64_t units, int blocks) {
  return int64_t(c) * units / blocks;
}
__device__ __forceinline__ int block_of(int64_t u, int64_t units, int blocks) {
  return int(((u + 1) * blocks - 1) / units);
}
// where block c puts the piece of a (sequence, head) that begins at unit u0:
// its first piece is slot 0, its last slot 1
__device__ __forceinline__ int part_slot(int c, int64_t u0, int64_t units, int blocks) {
  return 2 * c + (u0 > run_begin(c, units, blocks) ? 1 : 0);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x = hi + lo in two tf32 numbers (the first cut off, so that it never
// overflows; an infinite x has no remainder)
struct Split {
  uint32_t hi, lo;
  __device__ __forceinline__ explicit Split(uint32_t x) {
    hi = x & 0xffffe000u;
    const float rest = __uint_as_float(x) - __uint_as_float(hi);
    lo = __float_as_uint((x & 0x7fffffffu) < 0x7f800000u ? rest : 0.f) & 0xffffe000u;
  }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// one warp's running softmax over its slots: reference m and sum l of head
// lane / 4 (the sum over this lane's slots only), and O^T
template <typename T, int D>
struct Acc {
  using L = Tile<T, D>;
  float m, l, o[L::kMt][4];
};

// Adds the tile in kr, vr.  live: slots of each slab that count (the others'
// K and V registers hold 0).  out: where the scores go (nullptr: nowhere).
template <typename T, int D, typename KR>
__device__ __forceinline__ void score_tile(const KR& kr, const uint4* qf, float scale_log2,
                                           float (&s)[Tile<T, D>::kSlabs][Tile<T, D>::kNt][2]) {
  using L = Tile<T, D>;
#pragma unroll
  for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
    for (int nt = 0; nt < L::kNt; ++nt) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < L::kKc; ++j) {
        const uint4 k = kr[sl][nt][j], a = qf[j];
        if constexpr (L::kBf16) {
          mma_bf16(c, a.x, 0u, a.y, 0u, k.x, k.y);
          mma_bf16(c, a.z, 0u, a.w, 0u, k.z, k.w);
        } else {
          const Split ax(a.x), ay(a.y), az(a.z), aw(a.w), kx(k.x), ky(k.y), kz(k.z), kw(k.w);
          mma_tf32(c, ax.lo, 0u, ay.lo, 0u, kx.hi, ky.hi);
          mma_tf32(c, ax.hi, 0u, ay.hi, 0u, kx.lo, ky.lo);
          mma_tf32(c, ax.hi, 0u, ay.hi, 0u, kx.hi, ky.hi);
          mma_tf32(c, az.lo, 0u, aw.lo, 0u, kz.hi, kw.hi);
          mma_tf32(c, az.hi, 0u, aw.hi, 0u, kz.lo, kw.lo);
          mma_tf32(c, az.hi, 0u, aw.hi, 0u, kz.hi, kw.hi);
        }
      }
      s[sl][nt][0] = c[0] * scale_log2;
      s[sl][nt][1] = c[1] * scale_log2;
    }
}

template <typename T, int D, typename VR>
__device__ __forceinline__ void add_tile(Acc<T, D>& acc, const VR& vr,
                                         float (&s)[Tile<T, D>::kSlabs][Tile<T, D>::kNt][2],
                                         int lane) {
  using L = Tile<T, D>;
  float top = -INFINITY;
#pragma unroll
  for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
    for (int nt = 0; nt < L::kNt; ++nt) top = fmaxf(top, fmaxf(s[sl][nt][0], s[sl][nt][1]));
  if (__any_sync(0xffffffffu, top > acc.m + kSlack)) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = fmaxf(top, acc.m);
    const float a = top == -INFINITY ? 1.f : exp2f(acc.m - top);
    acc.m = top;
    acc.l *= a;
    const float a0 = __shfl_sync(0xffffffffu, a, (lane & 3) * 8);
    const float a1 = __shfl_sync(0xffffffffu, a, (lane & 3) * 8 + 4);
#pragma unroll
    for (int t = 0; t < L::kMt; ++t) {
      acc.o[t][0] *= a0;
      acc.o[t][1] *= a1;
      acc.o[t][2] *= a0;
      acc.o[t][3] *= a1;
    }
  }
#pragma unroll
  for (int sl = 0; sl < L::kSlabs; ++sl) {
    float p[L::kNt][2];
#pragma unroll
    for (int nt = 0; nt < L::kNt; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = s[sl][nt][i];
        p[nt][i] = x == -INFINITY ? 0.f : sm100::ex2_approx(x - acc.m);
        acc.l += p[nt][i];
      }
    if constexpr (L::kBf16) {
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        hi[nt] = bf16_pair(p[nt][0], p[nt][1]);
        lo[nt] = bf16_pair(p[nt][0] - __uint_as_float(hi[nt] << 16),
                           p[nt][1] - __uint_as_float(hi[nt] & 0xffff0000u));
      }
#pragma unroll
      for (int x = 0; x < L::kVc; ++x)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          auto word = [&](int r) {
            const uint4& u = vr[sl][r][x];
            return w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w;
          };
          const uint32_t a0 = __byte_perm(word(0), word(1), 0x5410);
          const uint32_t a1 = __byte_perm(word(0), word(1), 0x7632);
          const uint32_t a2 = __byte_perm(word(2), word(3), 0x5410);
          const uint32_t a3 = __byte_perm(word(2), word(3), 0x7632);
          mma_bf16(acc.o[x * 4 + w], a0, a1, a2, a3, lo[0], lo[1]);
          mma_bf16(acc.o[x * 4 + w], a0, a1, a2, a3, hi[0], hi[1]);
        }
    } else {
      const Split p0(__float_as_uint(p[0][0])), p1(__float_as_uint(p[0][1]));
#pragma unroll
      for (int x = 0; x < L::kVc; ++x)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint4 u0 = vr[sl][0][x], u1 = vr[sl][1][x];
          const Split a0(w ? u0.z : u0.x), a1(w ? u0.w : u0.y);
          const Split a2(w ? u1.z : u1.x), a3(w ? u1.w : u1.y);
          float(&c)[4] = acc.o[x * 2 + w];
          mma_tf32(c, a0.lo, a1.lo, a2.lo, a3.lo, p0.hi, p1.hi);
          mma_tf32(c, a0.hi, a1.hi, a2.hi, a3.hi, p0.lo, p1.lo);
          mma_tf32(c, a0.hi, a1.hi, a2.hi, a3.hi, p0.hi, p1.hi);
        }
    }
  }
}

template <typename T, int D>
struct Shared {
  float wo[kWarps][kMaxG][D];
  float wm[kWarps][kMaxG], wl[kWarps][kMaxG];
  int64_t scan[kWarps];
  int64_t seq_first;  // units before the sequence in which the block's run begins
  int seq;
};

// grid kBlocks
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    paged_decode_kernel(PagedView cache, const T* __restrict__ q,
                        const int32_t* __restrict__ n_slots, int batch, int G, float scale_log2,
                        T* __restrict__ o, float* __restrict__ lse, Work work) {
  using L = Tile<T, D>;
  __shared__ Shared<T, D> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n8 = lane >> 2, q4 = lane & 3;
  const int n_kv = cache.n_kv_heads;
  pdl_wait();
  pdl_launch_dependents();

  // ---- the block's run of units -------------------------------------------
  auto units_of = [&](int b) -> int64_t {
    const int n = n_slots[b];
    return n > 0 && int64_t(n) <= cache.capacity()
               ? int64_t(n_kv) * ((n + L::kUnit - 1) / L::kUnit)
               : 0;
  };
  const int per = (batch + kThreads - 1) / kThreads;
  const int b_lo = min(batch, tid * per), b_hi = min(batch, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    mine += units_of(b);
    const int n = n_slots[b];
    if (blockIdx.x == 0 && (n < 0 || int64_t(n) > cache.capacity()))
      latch_status(HGA_ERR_DEVICE_CHECK);
  }
  int64_t incl = mine;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, w);
    if (lane >= w) incl += x;
  }
  if (lane == 31) sh.scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, units = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.scan[w];
    units += sh.scan[w];
  }
  if (blockIdx.x == 0) {
    int64_t at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      work.first[b] = at;
      at += units_of(b);
    }
    if (tid == 0) work.first[batch] = units;
  }
  // idle sequences have no unit: nothing to attend to
  for (int b = blockIdx.x; b < batch; b += kBlocks) {
    if (n_slots[b] != 0) continue;
    const int64_t row = int64_t(b) * n_kv * G;
    for (int64_t i = tid; i < int64_t(n_kv) * G * D; i += kThreads)
      o[row * D + i] = from_float<T>(0.f);
    for (int i = tid; i < n_kv * G; i += kThreads) lse[row + i] = -INFINITY;
  }
  const int blocks = blocks_for(units);
  if (int(blockIdx.x) >= blocks) return;
  const int64_t run_lo = run_begin(blockIdx.x, units, blocks);
  const int64_t run_hi = run_begin(blockIdx.x + 1, units, blocks);
  if (before <= run_lo && run_lo < before + mine) {
    int64_t at = before;
    int b = b_lo;
    while (run_lo >= at + units_of(b)) at += units_of(b++);
    sh.seq = b;
    sh.seq_first = at;
  }
  __syncthreads();
  int b = sh.seq;
  int64_t seq_first = sh.seq_first;

  // ---- its pieces -----------------------------------------------------------
  for (int64_t u = run_lo; u < run_hi;) {
    int64_t seq_units = units_of(b);
    while (u >= seq_first + seq_units) {
      seq_first += seq_units;
      seq_units = units_of(++b);
    }
    const int n = n_slots[b];
    const int head_units = int(seq_units / n_kv);
    const int h = int((u - seq_first) / head_units);
    const int64_t head_first = seq_first + int64_t(h) * head_units;
    const int64_t u_end = min(run_hi, head_first + head_units);
    const int t_lo = int(u - head_first) * L::kUnit;
    const int t_hi = int(min(int64_t(n), (u_end - head_first) * L::kUnit));
    const int64_t row0 = (int64_t(b) * n_kv + h) * G;
    const int32_t* table = cache.table + int64_t(b) * cache.max_pages;
    const T* kh = static_cast<const T*>(cache.k) + (int64_t(h) << cache.page_shift) * D;
    const T* vh = static_cast<const T*>(cache.v) + (int64_t(h) << cache.page_shift) * D;
    float* score_out = work.scores ? work.scores + head_first * L::kUnit * G : nullptr;

    uint4 qf[L::kKc];
#pragma unroll
    for (int j = 0; j < L::kKc; ++j) {
      qf[j] = make_uint4(0u, 0u, 0u, 0u);
      if (n8 < G)
        qf[j] = *reinterpret_cast<const uint4*>(
            reinterpret_cast<const char*>(q + (row0 + n8) * D) + 16 * (q4 + 4 * j));
    }
    Acc<T, D> acc;
    acc.m = -INFINITY;
    acc.l = 0.f;
#pragma unroll
    for (int t = 0; t < L::kMt; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc.o[t][i] = 0.f;

    // first slot of each slab of the tile at hand, how many of its slots
    // count (0 on a page outside the pool), and its first row's offset
    int live[L::kSlabs];
    int64_t base[L::kSlabs];
    auto locate = [&](int t) {
#pragma unroll
      for (int sl = 0; sl < L::kSlabs; ++sl) {
        const int s0 = t + sl * L::kSlab;
        live[sl] = max(0, min(L::kSlab, t_hi - s0));
        base[sl] = 0;
        if (live[sl] > 0) {
          const int page = table[cache.page_of(s0)];
          if (!cache.has(page)) {
            live[sl] = 0;
            if (lane == 0) latch_status(HGA_ERR_DEVICE_CHECK);
          } else {
            base[sl] = int64_t(page) * cache.page_stride + int64_t(cache.row_of(s0)) * D;
          }
        }
      }
    };
    uint4 kr[L::kSlabs][L::kNt][L::kKc], vr[L::kSlabs][L::kVt][L::kVc];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto load_k = [&]() {
#pragma unroll
      for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
        for (int nt = 0; nt < L::kNt; ++nt) {
          const uint4* src = reinterpret_cast<const uint4*>(kh + base[sl] + (nt * 8 + n8) * D);
#pragma unroll
          for (int j = 0; j < L::kKc; ++j)
            kr[sl][nt][j] = nt * 8 + n8 < live[sl] ? __ldcs(src + q4 + 4 * j) : zero;
        }
    };
    auto load_v = [&]() {
#pragma unroll
      for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
        for (int r = 0; r < L::kVt; ++r) {
          const int t = 2 * q4 + (r & 1) + 8 * (r >> 1);
          const uint4* src = reinterpret_cast<const uint4*>(vh + base[sl] + t * D);
#pragma unroll
          for (int x = 0; x < L::kVc; ++x)
            vr[sl][r][x] = t < live[sl] ? __ldcs(src + n8 + 8 * x) : zero;
        }
    };

    int t = t_lo + warp * L::kSlots;
    if (t < t_hi) {
      locate(t);
      load_k();
      load_v();
    }
    while (t < t_hi) {
      float s[L::kSlabs][L::kNt][2];
      score_tile<T, D>(kr, qf, scale_log2, s);
#pragma unroll
      for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
        for (int nt = 0; nt < L::kNt; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (nt * 8 + 2 * q4 + i >= live[sl]) s[sl][nt][i] = -INFINITY;
      if (score_out && n8 < G) {
        float* dst = score_out + int64_t(t) * G + n8 * L::kSlots + 2 * q4;
#pragma unroll
        for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
          for (int nt = 0; nt < L::kNt; ++nt)
            *reinterpret_cast<float2*>(dst + sl * L::kSlab + nt * 8) =
                make_float2(s[sl][nt][0], s[sl][nt][1]);
      }
      // the next tile's K is requested before this tile's softmax, its V after
      // the product that frees the registers
      t += L::kUnit;
      if (t < t_hi) {
        locate(t);
        load_k();
      }
      add_tile<T, D>(acc, vr, s, lane);
      if (t < t_hi) load_v();
    }

    // ---- the warps' results, in warp order --------------------------------
    float l = acc.l;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (q4 == 0) {
      sh.wm[warp][n8] = acc.m;
      sh.wl[warp][n8] = l;
    }
    {
      constexpr int kPer = 16 / int(sizeof(T));  // elements of a 16-byte piece
#pragma unroll
      for (int x = 0; x < L::kVc; ++x)
#pragma unroll
        for (int w = 0; w < kPer / 2; ++w) {
          const float(&c)[4] = acc.o[x * (kPer / 2) + w];
          const int e = kPer * (n8 + 8 * x) + 2 * w;
          *reinterpret_cast<float2*>(&sh.wo[warp][2 * q4][e]) = make_float2(c[0], c[2]);
          *reinterpret_cast<float2*>(&sh.wo[warp][2 * q4 + 1][e]) = make_float2(c[1], c[3]);
        }
    }
    __syncthreads();
    const bool whole = u == head_first && u_end == head_first + head_units;
    float* part = work.part +
                  int64_t(part_slot(blockIdx.x, head_first, units, blocks)) * G * (D + 2);
    for (int i = tid; i < G * D; i += kThreads) {
      const int g = i / D, e = i % D;
      float M = -INFINITY, sum = 0.f, out = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.wm[w][g]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = sh.wm[w][g] == -INFINITY && sh.wl[w][g] == 0.f ? 0.f
                                                                        : exp2f(sh.wm[w][g] - M);
        sum = fmaf(a, sh.wl[w][g], sum);
        out = fmaf(a, sh.wo[w][g][e], out);
      }
      if (whole) {
        o[(row0 + g) * D + e] = from_float<T>(sum == 0.f ? 0.f : out / sum);
        if (e == 0) lse[row0 + g] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
      } else {
        part[2 * G + i] = out;
        if (e == 0) {
          part[g] = M;
          part[G + g] = sum;
        }
      }
    }
    __syncthreads();  // the next piece overwrites the warps' results
    u = u_end;
  }
}

// ---------------------------------------------------------------------------
// Joins the incomplete pieces, and adds the weights.  Blocks [0, joins):
// one per (sequence, query head), they merge the partial results in block
// order.  The others (accumulate) share the units out among themselves again:
// LSE of the G heads, then weight[slot] += sum_g 2^(s_g - LSE_g) from the
// scores that the decode kernel left (in L2 for the most part).
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

// (m, l) over the pieces of a (sequence, head), for head g: by one warp
__device__ __forceinline__ void join_stats(const Work& work, int G, int stride, int c0, int c1,
                                           int64_t head_first, int64_t units, int blocks, int g,
                                           int lane, float& M, float& sum) {
  M = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32)
    M = fmaxf(M, work.part[int64_t(part_slot(c, head_first, units, blocks)) * stride + g]);
#pragma unroll
  for (int w = 16; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  sum = 0.f;
  for (int c = c0 + lane; c <= c1; c += 32) {
    const float* p = work.part + int64_t(part_slot(c, head_first, units, blocks)) * stride;
    if (p[g] == -INFINITY && p[G + g] == 0.f) continue;
    sum = fmaf(exp2f(p[g] - M), p[G + g], sum);
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
}

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
    paged_join_kernel(PagedView cache, const int32_t* __restrict__ n_slots, int batch, int G,
                      int joins, T* __restrict__ o, float* __restrict__ lse, Work work) {
  using L = Tile<T, D>;
  constexpr int kRows = kJoinThreads / D;
  __shared__ float red[kRows][D];
  __shared__ float head_lse[kMaxG];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_kv = cache.n_kv_heads;
  const int stride = G * (D + 2);
  pdl_wait();
  const int64_t units = work.first[batch];
  const int blocks = blocks_for(units);
  if (int(blockIdx.x) < joins) {
    const int64_t row = blockIdx.x;
    const int b = int(row / (n_kv * G)), h = int(row / G % n_kv), g = int(row % G);
    const int head_units = int((work.first[b + 1] - work.first[b]) / n_kv);
    if (head_units > 0) {
      const int64_t head_first = work.first[b] + int64_t(h) * head_units;
      const int c0 = block_of(head_first, units, blocks);
      const int c1 = block_of(head_first + head_units - 1, units, blocks);
      if (c0 < c1) {
        float M, sum;
        join_stats(work, G, stride, c0, c1, head_first, units, blocks, g, lane, M, sum);
        const int e = tid % D, r = tid / D;
        float out = 0.f;
#pragma unroll 8
        for (int c = c0 + r; c <= c1; c += kRows) {
          const float* p = work.part + int64_t(part_slot(c, head_first, units, blocks)) * stride;
          const float a = p[g] == -INFINITY && p[G + g] == 0.f ? 0.f : exp2f(p[g] - M);
          out = fmaf(a, p[2 * G + g * D + e], out);
        }
        red[r][e] = out;
        __syncthreads();
        if (r == 0) {
#pragma unroll
          for (int i = 1; i < kRows; ++i) out += red[i][e];
          o[row * D + e] = from_float<T>(sum == 0.f ? 0.f : out / sum);
          if (e == 0) lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
        }
      }
    }
  } else if (units > 0) {
    const int n_add = int(gridDim.x) - joins, me = int(blockIdx.x) - joins;
    const int adders = int(units < n_add ? units : n_add);
    const int64_t run_hi = me < adders ? run_begin(me + 1, units, adders) : 0;
    int64_t u = me < adders ? run_begin(me, units, adders) : 0;
    int b = 0;
    if (u < run_hi) {  // the sequence of unit u
      int lo = 0, hi = batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (work.first[mid] <= u) lo = mid;
        else hi = mid - 1;
      }
      b = lo;
    }
    while (u < run_hi) {
      while (u >= work.first[b + 1]) ++b;
      const int head_units = int((work.first[b + 1] - work.first[b]) / n_kv);
      const int h = int((u - work.first[b]) / head_units);
      const int64_t head_first = work.first[b] + int64_t(h) * head_units;
      const int64_t u_end = min(run_hi, head_first + head_units);
      const int n = n_slots[b];
      const int t_lo = int(u - head_first) * L::kUnit;
      const int t_hi = int(min(int64_t(n), (u_end - head_first) * L::kUnit));
      const int c0 = block_of(head_first, units, blocks);
      const int c1 = block_of(head_first + head_units - 1, units, blocks);
      __syncthreads();
      if (warp < G) {
        float x;
        if (c0 < c1) {
          float M, sum;
          join_stats(work, G, stride, c0, c1, head_first, units, blocks, warp, lane, M, sum);
          x = sum == 0.f ? INFINITY : M + log2f(sum);
        } else {
          x = lse[(int64_t(b) * n_kv + h) * G + warp] / kLn2;
          if (x == -INFINITY) x = INFINITY;
        }
        if (lane == 0) head_lse[warp] = x;
      }
      __syncthreads();
      const int32_t* table = cache.table + int64_t(b) * cache.max_pages;
      const float* score = work.scores + head_first * L::kUnit * G;
      for (int t = t_lo + tid; t < t_hi; t += kJoinThreads) {
        const int page = table[cache.page_of(t)];
        if (!cache.has(page)) continue;
        const float* s = score + int64_t(t / L::kSlots) * L::kSlots * G + t % L::kSlots;
        float w = 0.f;
        for (int g = 0; g < G; ++g) w += exp2f(s[g * L::kSlots] - head_lse[g]);
        // two sequences may share a page: an addition, not a store
        atomicAdd(&cache.weight[cache.record(page, h, cache.row_of(t))], w);
      }
      u = u_end;
    }
  }
  // the next kernel on the stream may read what this call wrote before its
  // own wait: let it start only once every store is visible
  __syncthreads();
  __threadfence();
  pdl_launch_dependents();
}

}  // namespace pdec
}  // namespace hga
