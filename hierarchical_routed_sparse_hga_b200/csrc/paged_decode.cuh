// Attention of one new token per sequence over its paged cache.
//
//   x_j = q.k_j,  p_j = 2^((x_j - m) scale / ln 2),  O = sum_j p_j v_j / sum_j p_j,
//   LSE = m scale + ln sum_j p_j
//
// (the scale comes after the difference: two scores that are close keep their
// distance, and LSE is rounded once)
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
// Precision.  Statistics and sums are float32.  P enters its product as three
// bf16 parts, which hold all of its 24 bits (two hold 16, and the remainder
// shows in bf16 outputs).  The matrix unit cuts its sums off instead of rounding
// them, so it forms short ones only (16 slots, 16 or 32 elements of d) and
// additions sum those: sums of bf16 products over 64 tiles come out 0.9 * 2^-24 off
// (root mean square), 4.3 in the unit throughout, which would take 1.5 % less
// time.  Float32 operands are split into two tf32 parts (22 bits) and all four
// products are summed: each is good to 2^-20, where one part alone is good to
// 2^-9.  An infinite key or value counts as in the formula: the parts of its factor
// have one sign and none is 0.
#pragma once

#include <cooperative_groups.h>

#include <algorithm>

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace hga {
namespace pdec {

// 12 warps on an SM: with 168 registers a thread a tile of K and of V and the
// output stay in registers; 16 warps of 128 spill, and read 8 x 32768 slots
// (bf16, 8 heads, d = 128; 1.07 GB) in 202 us instead of 163 (6.6 TB/s).
// Small blocks, so that one merges its warps while another reads.
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 3;
constexpr int kBlocks = 148 * kBlocksPerSm;  // of the B200's 148 SMs
constexpr int kMaxG = 8;

// fills the parts of a factor that would be 0, below half a step of float32
constexpr float kTiny = 0x1p-26f;

// What a product q.k counts.  The reference point of the running softmax moves
// only when a product exceeds it by more than `slack`, 8 in base 2: the
// weights stay below 2^8, no precision is lost in float32, and nearly every
// tile is spared the rescaling.
struct Scale {
  float score;  // of the products in the scores
  float log2;   // the same in base 2
  float slack;  // finite, so that a reference of -inf always moves
  explicit Scale(float scale)
      : score(scale), log2(scale * 1.4426950408889634f), slack(std::min(8.f / log2, 1e37f)) {}
};

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

// What a block of the decode kernel leaves for the join kernel: where its run
// begins, and the head that begins in its last piece and goes on in the next
// block's run (tail_units 0: none does).  Units are counted in 32 bits: the
// call refuses tables that could hold more.
struct alignas(16) Run {
  int32_t units;       // of the whole batch
  int32_t seq;         // in which the run begins; -1: the block has no run
  int32_t seq_first;   // units before it
  int32_t tail_head;   // sequence * n_kv_heads + head
  int32_t tail_first;  // units before the head
  int32_t tail_units;  // units of the head
  int32_t tail_part;   // slot of its first partial result
  int32_t tail_n;      // number of its partial results
};

struct Work {
  Run* runs;        // [kBlocks]
  float* part;      // [2 * kBlocks][G * (D + 2)]: m[G], l[G], o[G][D] of an incomplete piece
  float* scores;    // [units][kUnit / kSlots][G][kSlots], q.k; nullptr: not kept
  float2* stats;    // [batch * n_q_heads] (maximum, sum) of the heads in one piece, with scores
};

// A piece costs about as much as kHeadUnits units on top of those it has (its
// queries, its first pages and rows, its merge, all waited for in turn), so
// each head counts that many more where the runs are cut: position p of a
// head that begins at unit u0 is its unit p - u0 - kHeadUnits.  Without it a
// block that gets many short sequences is the last to end: 64 sequences of 0
// to 8190 slots take 186 us instead of 168.
constexpr int kHeadUnits = 2;

// The runs of the blocks in use: q units each, the first r one more.
struct Runs {
  int blocks, q, r;
  __device__ __forceinline__ explicit Runs(int units) {
    blocks = min(units, kBlocks);
    q = blocks > 0 ? units / blocks : 0;
    r = units - q * blocks;
  }
  __device__ __forceinline__ int begin(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int block_of(int u) const {
    const int wide = r * (q + 1);
    return u < wide ? u / (q + 1) : r + (u - wide) / q;
  }
  // partial results of a head of `units` units from unit `first` on: the
  // blocks' pieces of it; a block puts its first piece in slot 0 of its two,
  // its last in slot 1 (only the head's first block can have it as its last)
  __device__ __forceinline__ void pieces(int first, int units, int& part, int& n) const {
    const int c0 = block_of(first);
    n = block_of(first + units - 1) - c0 + 1;
    part = 2 * c0 + (first > begin(c0) ? 1 : 0);
  }
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4],
                                         const uint32_t (&b)[2]) {
  mma_bf16(c, a[0], a[1], a[2], a[3], b[0], b[1]);
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x = hi + lo in two tf32 numbers of 11 bits: hi cut off (it never overflows),
// lo rounded.  Of an infinity lo is 0: inf - inf is the NaN of all ones, whose
// rounding carries into the sign.  filled (Q, P: the factors of K and V): lo
// has the sign of x and is never 0, at least 2^-26 x, so that both parts of
// it times an infinity are the same infinity.
struct Split {
  uint32_t hi, lo;
  __device__ __forceinline__ explicit Split(uint32_t x, bool filled = false) {
    hi = x & 0xffffe000u;
    const float f = __uint_as_float(x);
    float rest = f - __uint_as_float(hi);
    if (filled && fabsf(rest) < fabsf(f) * kTiny) rest = f * kTiny;
    lo = (__float_as_uint(rest) + 0x1000u) & 0xffffe000u;
  }
};

// the upper 16 bits of x[0] and x[1] as a pair of bf16 numbers; rest: what they leave
__device__ __forceinline__ uint32_t bf16_parts(const float (&x)[2], float (&rest)[2]) {
  const uint32_t a = __float_as_uint(x[0]), b = __float_as_uint(x[1]);
  rest[0] = x[0] - __uint_as_float(a & 0xffff0000u);
  rest[1] = x[1] - __uint_as_float(b & 0xffff0000u);
  return __byte_perm(a, b, 0x7632);
}

// one warp's running softmax over its slots: reference m and sum l of head
// lane / 4 (the sum over this lane's slots only), and O^T
template <typename T, int D>
struct Acc {
  using L = Tile<T, D>;
  float m, l, o[L::kMt][4];
};

// The queries in shared memory: held in registers next to a tile of K and of
// V and the output they would not fit.  Rows padded so that two rows' pieces
// lie in different banks.  float32: split, the remainders kLo pieces behind.
template <typename T, int D>
struct Queries {
  static constexpr int kParts = sizeof(T) == 2 ? 1 : 2;
  static constexpr int kRow = D + 64 / int(sizeof(T));
  static constexpr int kLo = kMaxG * kRow * int(sizeof(T)) / 16;
  alignas(16) T row[kParts][kMaxG][kRow];
};

// Products q.k of the tile in kr, by lane: heads lane / 4, two slots per column
// of 8.  q: this lane's first piece of its query row.
template <typename T, int D, typename KR>
__device__ __forceinline__ void score_tile(const KR& kr, const uint4* q,
                                           float (&s)[Tile<T, D>::kSlabs][Tile<T, D>::kNt][2]) {
  using L = Tile<T, D>;
#pragma unroll
  for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
    for (int nt = 0; nt < L::kNt; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) s[sl][nt][i] = 0.f;
  // The matrix unit sums 32 (float32: 16) elements of d at a time, additions
  // sum those.  (All 128 in the unit: scores 2.5 * 2^-24 short in the mean instead
  // of 0.7; 16 at a time 0.4, but 2.5 us more at 8 x 32768 slots.)
  if constexpr (L::kBf16) {
#pragma unroll
    for (int j = 0; j < L::kKc; ++j) {
      const uint4 a = q[4 * j];
#pragma unroll
      for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
        for (int nt = 0; nt < L::kNt; ++nt) {
          const uint4 k = kr[sl][nt][j];
          float c0[4] = {};
          mma_bf16(c0, a.x, 0u, a.y, 0u, k.x, k.y);
          mma_bf16(c0, a.z, 0u, a.w, 0u, k.z, k.w);
#pragma unroll
          for (int i = 0; i < 2; ++i) s[sl][nt][i] += c0[i];
        }
    }
  } else {
    // (4 x 16384 slots come out 4.7e-7 off, plain float32 sums 1.2e-6, sums in
    // the unit alone 2.8e-6)
#pragma unroll
    for (int j = 0; j < L::kKc; ++j) {
      const uint4 a = q[4 * j], a_lo = q[Queries<T, D>::kLo + 4 * j];
#pragma unroll
      for (int sl = 0; sl < L::kSlabs; ++sl) {
        const uint4 k = kr[sl][0][j];
        const Split kx(k.x), ky(k.y), kz(k.z), kw(k.w);
        float c[4] = {};  // Q's high parts, and its low ones in the 8 rows below
        mma_tf32(c, a.x, a_lo.x, a.y, a_lo.y, kx.lo, ky.lo);
        mma_tf32(c, a.z, a_lo.z, a.w, a_lo.w, kz.lo, kw.lo);
        mma_tf32(c, a.x, a_lo.x, a.y, a_lo.y, kx.hi, ky.hi);
        mma_tf32(c, a.z, a_lo.z, a.w, a_lo.w, kz.hi, kw.hi);
        s[sl][0][0] += c[0] + c[2];
        s[sl][0][1] += c[1] + c[3];
      }
    }
  }
}

// Adds the tile in vr, with its scores, to the running softmax.
template <typename T, int D, typename VR>
__device__ __forceinline__ void add_tile(Acc<T, D>& acc, const VR& vr,
                                         float (&s)[Tile<T, D>::kSlabs][Tile<T, D>::kNt][2],
                                         const Scale& scale, int lane) {
  using L = Tile<T, D>;
  float top = -INFINITY;
#pragma unroll
  for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
    for (int nt = 0; nt < L::kNt; ++nt) top = fmaxf(top, fmaxf(s[sl][nt][0], s[sl][nt][1]));
  if (__any_sync(0xffffffffu, top > acc.m + scale.slack)) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = fmaxf(top, acc.m);
    const float a = top == -INFINITY ? 1.f : exp2f((acc.m - top) * scale.log2);
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
        p[nt][i] = x == -INFINITY ? 0.f : sm100::ex2_approx((x - acc.m) * scale.log2);
        acc.l += p[nt][i];
      }
    if constexpr (L::kBf16) {
      // p = hi + mid + lo in three bf16 numbers of 8 bits, each cut off: exact,
      // but for parts of 0 (times an infinite value: NaN), which are filled
      uint32_t hi[2], mid[2], lo[2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float tiny[2] = {p[nt][0] * kTiny, p[nt][1] * kTiny};
        float r[2] = {};
        auto fill = [&] {
          r[0] = fmaxf(r[0], tiny[0]);
          r[1] = fmaxf(r[1], tiny[1]);
        };
        hi[nt] = bf16_parts(p[nt], r);
        fill();
        mid[nt] = bf16_parts(r, r);
        fill();
        lo[nt] = bf16_parts(r, r);
      }
      // four products side by side: each is a chain of three instructions
#pragma unroll
      for (int x = 0; x < L::kVc; ++x) {
        uint32_t a[4][4];
        float c[4][4] = {};  // added below: see score_tile
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          auto word = [&](int r) {
            const uint4& u = vr[sl][r][x];
            return w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w;
          };
          a[w][0] = __byte_perm(word(0), word(1), 0x5410);
          a[w][1] = __byte_perm(word(0), word(1), 0x7632);
          a[w][2] = __byte_perm(word(2), word(3), 0x5410);
          a[w][3] = __byte_perm(word(2), word(3), 0x7632);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) mma_bf16(c[w], a[w], lo);
#pragma unroll
        for (int w = 0; w < 4; ++w) mma_bf16(c[w], a[w], mid);
#pragma unroll
        for (int w = 0; w < 4; ++w) mma_bf16(c[w], a[w], hi);
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc.o[x * 4 + w][i] += c[w][i];
      }
    } else {
      const Split p0(__float_as_uint(p[0][0]), true), p1(__float_as_uint(p[0][1]), true);
#pragma unroll
      for (int x = 0; x < L::kVc; ++x)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint4 u0 = vr[sl][0][x], u1 = vr[sl][1][x];
          const Split a0(w ? u0.z : u0.x), a1(w ? u0.w : u0.y);
          const Split a2(w ? u1.z : u1.x), a3(w ? u1.w : u1.y);
          float c[4] = {};  // added below: see score_tile
          mma_tf32(c, a0.lo, a1.lo, a2.lo, a3.lo, p0.lo, p1.lo);
          mma_tf32(c, a0.lo, a1.lo, a2.lo, a3.lo, p0.hi, p1.hi);
          mma_tf32(c, a0.hi, a1.hi, a2.hi, a3.hi, p0.lo, p1.lo);
          mma_tf32(c, a0.hi, a1.hi, a2.hi, a3.hi, p0.hi, p1.hi);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc.o[x * 2 + w][i] += c[i];
        }
    }
  }
}

// what a partial result (maximum m, sum l) counts in one with maximum M; one
// that attended to nothing counts nothing
__device__ __forceinline__ float part_scale(float m, float l, float M, const Scale& scale) {
  return m == -INFINITY && l == 0.f ? 0.f : exp2f((m - M) * scale.log2);
}

// the final output and log-sum-exp of a sum
template <typename T>
__device__ __forceinline__ T final_out(float out, float sum) {
  return from_float<T>(sum == 0.f ? 0.f : out / sum);
}
__device__ __forceinline__ float final_lse(float M, float sum, const Scale& scale) {
  return sum == 0.f ? -INFINITY : fmaf(M, scale.score, logf(sum));
}
// what add_weights takes of a query head's maximum and sum; attended to nothing:
// no weight
__device__ __forceinline__ float2 head_stat(float M, float sum) {
  return sum == 0.f ? make_float2(0.f, 0.f) : make_float2(M, 1.f / sum);
}

// One block's share of a (sequence, KV head): its warps take the tiles of slots
// [t_lo, t_hi) in turn, acc receives each warp's result.  q: the G query rows.
// Slot t's scores go to score_out + (t / kSlots) * kSlots * G (nullptr: nowhere).
template <typename T, int D>
__device__ __forceinline__ void attend(const PagedView& cache, const int32_t* __restrict__ table,
                                       int h, const T* __restrict__ q, int G, int t_lo, int t_hi,
                                       const Scale& scale, float* score_out, Queries<T, D>& qs,
                                       Acc<T, D>& acc) {
  using L = Tile<T, D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n8 = lane >> 2, q4 = lane & 3;
  constexpr int kPer = 16 / int(sizeof(T));  // elements of a 16-byte piece
  const T* kh = static_cast<const T*>(cache.k) + (int64_t(h) << cache.page_shift) * D;
  const T* vh = static_cast<const T*>(cache.v) + (int64_t(h) << cache.page_shift) * D;

  // the G query rows, and rows of 0 up to 8 (the matrix instruction's)
  for (int i = threadIdx.x; i < kMaxG * (D / kPer); i += kThreads) {
    const int g = i / (D / kPer), e = i % (D / kPer) * kPer;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (g < G) x = *reinterpret_cast<const uint4*>(q + g * D + e);
    if constexpr (!L::kBf16) {
      const Split sx(x.x, true), sy(x.y, true), sz(x.z, true), sw(x.w, true);
      *reinterpret_cast<uint4*>(&qs.row[1][g][e]) = make_uint4(sx.lo, sy.lo, sz.lo, sw.lo);
      x = make_uint4(sx.hi, sy.hi, sz.hi, sw.hi);
    }
    *reinterpret_cast<uint4*>(&qs.row[0][g][e]) = x;
  }
  acc.m = -INFINITY;
  acc.l = 0.f;
#pragma unroll
  for (int t = 0; t < L::kMt; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc.o[t][i] = 0.f;

  // The pages of this warp's slabs, 32 slabs at a time, one per lane (the
  // next 32 on their way): a table lookup in front of every tile's loads
  // would add its latency to each.
  const int t_warp = t_lo + warp * L::kSlots;
  auto page_ids = [&](int first) {  // of slabs first .. first + 31
    const int k = first + lane;
    const int s0 = t_warp + k / L::kSlabs * L::kUnit + k % L::kSlabs * L::kSlab;
    return s0 < t_hi ? table[cache.page_of(s0)] : 0;
  };
  int ids = page_ids(0), next_ids = page_ids(32);
  // of the tile at hand: how many slots of each slab count (0 on a page
  // outside the pool), and its first row's offset
  int live[L::kSlabs];
  int64_t base[L::kSlabs];
  auto locate = [&](int tile) {
    const int t = t_warp + tile * L::kUnit, k = tile * L::kSlabs;
    if (tile > 0 && k % 32 == 0) {
      ids = next_ids;
      next_ids = page_ids(k + 32);
    }
#pragma unroll
    for (int sl = 0; sl < L::kSlabs; ++sl) {
      const int s0 = t + sl * L::kSlab;
      const int page = __shfl_sync(0xffffffffu, ids, k % 32 + sl);
      const bool ok = cache.has(page);
      if (!ok && s0 < t_hi && lane == 0) latch_status(HGA_ERR_DEVICE_CHECK);
      live[sl] = ok ? max(0, min(L::kSlab, t_hi - s0)) : 0;
      base[sl] = int64_t(page) * cache.page_stride + int64_t(cache.row_of(s0)) * D;
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

  const int tiles = t_warp < t_hi ? (t_hi - t_warp + L::kUnit - 1) / L::kUnit : 0;
  if (tiles > 0) {
    locate(0);
    load_k();
    load_v();
  }
  __syncthreads();
  const uint4* qp = reinterpret_cast<const uint4*>(&qs.row[0][n8][0]) + q4;
  for (int tile = 0; tile < tiles; ++tile) {
    asm volatile("" : "+l"(qp));  // read again for every tile
    float s[L::kSlabs][L::kNt][2];
    score_tile<T, D>(kr, qp, s);
#pragma unroll
    for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
      for (int nt = 0; nt < L::kNt; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (nt * 8 + 2 * q4 + i >= live[sl]) s[sl][nt][i] = -INFINITY;
    if (score_out && n8 < G) {
      float* dst = score_out + int64_t(t_warp + tile * L::kUnit) * G + n8 * L::kSlots + 2 * q4;
#pragma unroll
      for (int sl = 0; sl < L::kSlabs; ++sl)
#pragma unroll
        for (int nt = 0; nt < L::kNt; ++nt)
          *reinterpret_cast<float2*>(dst + sl * L::kSlab + nt * 8) =
              make_float2(s[sl][nt][0], s[sl][nt][1]);
    }
    // the next tile's K is requested before this tile's softmax, its V after
    // the product that frees the registers
    const bool more = tile + 1 < tiles;
    if (more) {
      locate(tile + 1);
      load_k();
    }
    add_tile<T, D>(acc, vr, s, scale, lane);
    if (more) load_v();
  }
}

// The warps' results into shared memory, then f(g, e, M, sum, out) for every
// query head and element: the block's maximum, sum and output (relative to the
// maximum), merged in warp order.
template <typename T, int D, typename F>
__device__ __forceinline__ void merge_warps(const Acc<T, D>& acc, float (&wo)[kWarps][kMaxG][D],
                                            float (&wm)[kWarps][kMaxG],
                                            float (&wl)[kWarps][kMaxG], int G,
                                            const Scale& scale, F&& f) {
  using L = Tile<T, D>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n8 = lane >> 2, q4 = lane & 3;
  float l = acc.l;
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (q4 == 0) {
    wm[warp][n8] = acc.m;
    wl[warp][n8] = l;
  }
  {
    constexpr int kPer = 16 / int(sizeof(T));  // elements of a 16-byte piece
#pragma unroll
    for (int x = 0; x < L::kVc; ++x)
#pragma unroll
      for (int w = 0; w < kPer / 2; ++w) {
        const float(&c)[4] = acc.o[x * (kPer / 2) + w];
        const int e = kPer * (n8 + 8 * x) + 2 * w;
        *reinterpret_cast<float2*>(&wo[warp][2 * q4][e]) = make_float2(c[0], c[2]);
        *reinterpret_cast<float2*>(&wo[warp][2 * q4 + 1][e]) = make_float2(c[1], c[3]);
      }
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += kThreads) {
    const int g = i / D, e = i % D;
    float M = -INFINITY, sum = 0.f, out = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w][g]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = part_scale(wm[w][g], wl[w][g], M, scale);
      sum = fmaf(a, wl[w][g], sum);
      out = fmaf(a, wo[w][g][e], out);
    }
    f(g, e, M, sum, out);
  }
}

// weight[slot] += sum_g p_g / (sum of head g) of slots [t_lo, t_hi), by `threads`
// threads; score: the products as attend() stored them, stat: each head's maximum and
// 1 / sum.  (By way of LSE a weight would be off by LSE's rounding, all of a head's
// the same way.)  An addition in memory, not a load and a store: two sequences
// may share a page.
template <typename T, int D>
__device__ __forceinline__ void add_weights(const PagedView& cache,
                                            const int32_t* __restrict__ table, int h, int G,
                                            int t_lo, int t_hi, const float* score,
                                            const float2* stat, const Scale& scale, int thread,
                                            int threads) {
  using L = Tile<T, D>;
  // four slots at a time: they lie on one page, and their records on 16 bytes
#pragma unroll 2
  for (int t = t_lo + 4 * thread; t < t_hi; t += 4 * threads) {
    const int page = table[cache.page_of(t)];
    if (!cache.has(page)) continue;
    const float* s = score + int64_t(t / L::kSlots) * L::kSlots * G + t % L::kSlots;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < G; ++g) {
      const float4 x = *reinterpret_cast<const float4*>(s + g * L::kSlots);
      const float2 of = stat[g];
      w.x = fmaf(sm100::ex2_approx((x.x - of.x) * scale.log2), of.y, w.x);
      w.y = fmaf(sm100::ex2_approx((x.y - of.x) * scale.log2), of.y, w.y);
      w.z = fmaf(sm100::ex2_approx((x.z - of.x) * scale.log2), of.y, w.z);
      w.w = fmaf(sm100::ex2_approx((x.w - of.x) * scale.log2), of.y, w.w);
    }
    float* dst = &cache.weight[cache.record(page, h, cache.row_of(t))];
    if (t + 4 <= t_hi) {
      atomicAdd(reinterpret_cast<float4*>(dst), w);
    } else {  // slots behind the last one stay as they are
      atomicAdd(dst, w.x);
      if (t + 1 < t_hi) atomicAdd(dst + 1, w.y);
      if (t + 2 < t_hi) atomicAdd(dst + 2, w.z);
    }
  }
}

template <typename T, int D>
struct Shared {
  Queries<T, D> q;
  float wo[kWarps][kMaxG][D];
  float wm[kWarps][kMaxG], wl[kWarps][kMaxG];
  int scan[kWarps];
  // the block's place in its run and the piece at hand: kept here rather than
  // in registers, which the tiles need
  int run_lo, u, run_hi;  // the run, and its next unit
  int seq_first;          // units before sequence `seq`
  int seq, head, t_lo, t_hi;
  int part;               // slot of the partial result; -1: the piece is whole
  int first;              // units before the head's slots
};

// grid kBlocks
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    paged_decode_kernel(PagedView cache, const T* __restrict__ q,
                        const int32_t* __restrict__ n_slots, int batch, int G, Scale scale,
                        T* __restrict__ o, float* __restrict__ lse, Work work) {
  using L = Tile<T, D>;
  __shared__ Shared<T, D> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_kv = cache.n_kv_heads;
  pdl_wait();
  pdl_launch_dependents();

  // ---- the block's run of units -------------------------------------------
  auto units_of = [&](int n) {
    return n > 0 && int64_t(n) <= cache.capacity()
               ? n_kv * ((n + L::kUnit - 1) / L::kUnit + kHeadUnits)
               : 0;
  };
  const int per = (batch + kThreads - 1) / kThreads;
  const int b_lo = min(batch, tid * per), b_hi = min(batch, b_lo + per);
  int mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int n = n_slots[b];
    mine += units_of(n);
    if (blockIdx.x == 0 && (n < 0 || int64_t(n) > cache.capacity()))
      latch_status(HGA_ERR_DEVICE_CHECK);
  }
  int incl = mine;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, w);
    if (lane >= w) incl += x;
  }
  if (lane == 31) sh.scan[warp] = incl;
  __syncthreads();
  int before = incl - mine, units = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.scan[w];
    units += sh.scan[w];
  }
  const Runs runs(units);
  // the thread whose sequences hold the run's first unit finds it there
  const int run_lo = runs.begin(blockIdx.x);
  if (int(blockIdx.x) < runs.blocks && before <= run_lo && run_lo < before + mine) {
    int at = before, b = b_lo;
    for (int x; run_lo >= at + (x = units_of(n_slots[b])); ++b) at += x;
    sh.run_lo = sh.u = run_lo;
    sh.run_hi = runs.begin(blockIdx.x + 1);
    sh.seq = b;
    sh.seq_first = at;
    work.runs[blockIdx.x] = {units, b, at, 0, 0, 0, 0, 0};
  }
  // idle sequences have no unit: nothing to attend to
  for (int b = blockIdx.x; b < batch; b += kBlocks) {
    if (n_slots[b] != 0) continue;
    const int64_t row = int64_t(b) * n_kv * G;
    for (int64_t i = tid; i < int64_t(n_kv) * G * D; i += kThreads)
      o[row * D + i] = from_float<T>(0.f);
    for (int i = tid; i < n_kv * G; i += kThreads) lse[row + i] = -INFINITY;
  }
  if (int(blockIdx.x) >= runs.blocks) {
    if (tid == 0) work.runs[blockIdx.x] = {units, -1, 0, 0, 0, 0, 0, 0};
    return;
  }

  // ---- its pieces -----------------------------------------------------------
  while (true) {
    __syncthreads();  // also: the next piece overwrites the warps' results
    if (tid == 0 && sh.u < sh.run_hi) {
      const int u = sh.u;
      int b = sh.seq, seq_first = sh.seq_first, n = n_slots[b], seq_units = units_of(n);
      while (u >= seq_first + seq_units) {
        seq_first += seq_units;
        seq_units = units_of(n = n_slots[++b]);
      }
      const int stride = seq_units / n_kv, h = (u - seq_first) / stride;
      const int first = seq_first + h * stride + kHeadUnits;  // of the head's slots
      const int end = first + stride - kHeadUnits, u_end = min(sh.run_hi, end);
      const int u_lo = max(u, first);
      const bool begins = u_lo == first, ends = u_end == end;
      if (begins && !ends && u_lo < u_end) {
        Run* run = work.runs + blockIdx.x;
        run->tail_head = b * n_kv + h;
        run->tail_first = first;
        run->tail_units = stride - kHeadUnits;
        int part, n_parts;
        Runs(units).pieces(first, stride - kHeadUnits, part, n_parts);
        run->tail_part = part;
        run->tail_n = n_parts;
      }
      sh.seq = b;
      sh.seq_first = seq_first;
      sh.head = h;
      sh.t_lo = (u_lo - first) * L::kUnit;
      sh.t_hi = min(n, (u_end - first) * L::kUnit);
      sh.part = begins && ends ? -1 : 2 * int(blockIdx.x) + (first > sh.run_lo ? 1 : 0);
      sh.first = first;
      sh.u = u_end;
    } else if (tid == 0) {
      sh.head = -1;
    }
    __syncthreads();
    if (sh.head < 0) break;
    if (sh.t_lo >= sh.t_hi) continue;  // the run ends before the head's first slot
    Acc<T, D> acc;
    {
      const int b = sh.seq, h = sh.head;
      attend<T, D>(cache, cache.table + int64_t(b) * cache.max_pages, h,
                   q + (int64_t(b) * n_kv + h) * G * D, G, sh.t_lo, sh.t_hi, scale,
                   work.scores ? work.scores + int64_t(sh.first) * L::kUnit * G : nullptr, sh.q, acc);
    }
    const int64_t row0 = (int64_t(sh.seq) * n_kv + sh.head) * G;
    merge_warps(acc, sh.wo, sh.wm, sh.wl, G, scale,
                [&](int g, int e, float M, float sum, float out) {
      if (sh.part < 0) {
        o[(row0 + g) * D + e] = final_out<T>(out, sum);
        if (e == 0) {
          lse[row0 + g] = final_lse(M, sum, scale);
          if (work.stats) work.stats[row0 + g] = make_float2(M, sum);
        }
      } else {
        float* part = work.part + int64_t(sh.part) * G * (D + 2);
        part[2 * G + g * D + e] = out;
        if (e == 0) {
          part[g] = M;
          part[G + g] = sum;
        }
      }
    });
  }
}

// ---------------------------------------------------------------------------
// Short caches in one launch: a cluster of nc blocks per (sequence, KV head),
// each with at most kFewUnits units of its slots; partial results, and the
// scores for the weights, stay in shared memory and are joined through it.
// Bound by latency: 1 x 300 slots 5.9 us (with the two kernels above and below
// 8.9), 1 x 2048 8.6 (11.0), 1 x 4096 12.7 (13.8), 8 x 1024 11.1 (14.7).
// ---------------------------------------------------------------------------
constexpr int kMaxC = 8;
// Blocks an SM is built for: with few warps on it a warp's own chain through a tile
// counts, and the registers of two blocks an SM shorten it (1 x 4096 slots 12.7
// us, 13.7 with those of three); more blocks than 2 x 148 are to run at once all
// the same (25 x 4 heads of 1000 slots, 400 blocks: 13.8 us, in two launches 18.0).
constexpr int kFewPerSm = 2;
// a float32 tile takes more instructions: 2 x 2048 slots, 8 units a block, are
// faster in two launches (18.0 us) than in one (19.6); bf16 the other way
// round, and from 12 units on two are faster there too (1 x 6144: 15.1, 17.6)
template <typename T>
constexpr int kFewUnits = sizeof(T) == 2 ? 8 : 4;

template <typename T, int D>
struct FewShared {
  Queries<T, D> q;
  float wo[kWarps][kMaxG][D];
  float wm[kWarps][kMaxG], wl[kWarps][kMaxG];
  float po[kMaxG][D], pm[kMaxG], pl[kMaxG];  // the block's partial result
  float2 stat[kMaxG];
};
// dynamic shared memory: FewShared, then (accumulate) the scores of kFewUnits units
template <typename T, int D>
__host__ __device__ constexpr size_t few_bytes(int G, bool accumulate) {
  return sizeof(FewShared<T, D>) +
         (accumulate ? size_t(kFewUnits<T>) * Tile<T, D>::kUnit * G * 4 : 0);
}

// grid (nc, n_kv_heads, batch) in clusters of (nc, 1, 1), kPerSm blocks on an SM;
// the table holds at most nc * kFewUnits units
template <typename T, int D, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm)
    paged_decode_few_kernel(PagedView cache, const T* __restrict__ q,
                            const int32_t* __restrict__ n_slots, int G, int accumulate,
                            Scale scale, T* __restrict__ o, float* __restrict__ lse) {
  using L = Tile<T, D>;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank()), nc = int(cluster.num_blocks());
  extern __shared__ __align__(16) unsigned char few_raw[];
  FewShared<T, D>& sh = *reinterpret_cast<FewShared<T, D>*>(few_raw);
  float* scores = reinterpret_cast<float*>(few_raw + sizeof(FewShared<T, D>));
  const int h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x;
  pdl_wait();
  // the whole cluster reads the same count and leaves here
  const int n = rank == 0 && h == 0 && tid == 0 ? checked_slots(cache, n_slots, b) : n_slots[b];
  if (n < 0 || int64_t(n) > cache.capacity()) return;
  const int64_t row0 = (int64_t(b) * cache.n_kv_heads + h) * G;
  const int32_t* table = cache.table + int64_t(b) * cache.max_pages;
  const int head_units = (n + L::kUnit - 1) / L::kUnit;
  const int t_lo = rank * head_units / nc * L::kUnit;
  const int t_hi = min(n, (rank + 1) * head_units / nc * L::kUnit);
  Acc<T, D> acc;
  attend<T, D>(cache, table, h, q + row0 * D, G, t_lo, t_hi, scale,
               accumulate ? scores - int64_t(t_lo) * G : nullptr, sh.q, acc);
  merge_warps(acc, sh.wo, sh.wm, sh.wl, G, scale, [&](int g, int e, float M, float sum, float out) {
    sh.po[g][e] = out;
    if (e == 0) {
      sh.pm[g] = M;
      sh.pl[g] = sum;
    }
  });
  cluster.sync();

  // every block joins its share of the output elements, in block order; a
  // thread per query head forms its maximum and sum for the weights
  auto stats = [&](int g, float& M, float& sum) {
    float m[kMaxC], l[kMaxC];
    M = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxC; ++r)
      if (r < nc) {
        const FewShared<T, D>* peer = cluster.map_shared_rank(&sh, r);
        m[r] = peer->pm[g];
        l[r] = peer->pl[g];
        M = fmaxf(M, m[r]);
      }
#pragma unroll
    for (int r = 0; r < kMaxC; ++r)
      if (r < nc) sum = fmaf(part_scale(m[r], l[r], M, scale), l[r], sum);
  };
  for (int i = rank * kThreads + tid; i < G * D; i += nc * kThreads) {
    const int g = i / D, e = i % D;
    float M, sum, out = 0.f;
    stats(g, M, sum);
    for (int r = 0; r < nc; ++r) {
      const FewShared<T, D>* peer = cluster.map_shared_rank(&sh, r);
      out = fmaf(part_scale(peer->pm[g], peer->pl[g], M, scale), peer->po[g][e], out);
    }
    o[(row0 + g) * D + e] = final_out<T>(out, sum);
    if (e == 0) lse[row0 + g] = final_lse(M, sum, scale);
  }
  if (accumulate) {
    if (tid < G) {
      float M, sum;
      stats(tid, M, sum);
      sh.stat[tid] = head_stat(M, sum);
    }
    __syncthreads();
    add_weights<T, D>(cache, table, h, G, t_lo, t_hi, scores - int64_t(t_lo) * G, sh.stat, scale,
                      tid, kThreads);
  }
  __syncthreads();
  __threadfence();  // as at the end of paged_join_kernel
  pdl_launch_dependents();
  cluster.sync();  // no block leaves while another reads its results
}

// ---------------------------------------------------------------------------
// Joins the incomplete pieces, and adds the weights.  The first `adders` blocks
// (accumulate: kBlocks, one per block of the decode kernel, over the same run;
// else 0) form the maxima and sums of the G heads and add to the weights from the
// scores that the decode kernel left, in L2 for the most part.
// At most one head goes on from each block's run to the next, so the other
// kBlocks * G blocks join: block (c, g) the pieces of query head g of the head
// that begins in block c's last piece, in block order.  Most of them have
// nothing to do; the adders come first so as not to wait for them.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

// The partial results of a (sequence, head): the first, then one in slot 0 of
// each block that follows.
struct Pieces {
  const float* first;
  const float* rest;  // of the second piece
  int step, n;
  __device__ __forceinline__ Pieces(const Work& work, int G, int d, int part, int n) : n(n) {
    const int size = G * (d + 2);
    step = 2 * size;
    first = work.part + int64_t(part) * size;
    rest = work.part + int64_t(part / 2 + 1) * step;
  }
  __device__ __forceinline__ const float* operator[](int i) const {
    return i == 0 ? first : rest + (i - 1) * step;
  }
};

// maximum and sum over the pieces for head g, by the kLanes lanes of a warp
// that share it (sub: which of them); counts[i] (if not nullptr) receives what
// piece i counts
template <int kLanes>
__device__ __forceinline__ void join_stats(const Pieces& pieces, int G, int g, int sub,
                                           const Scale& scale, float& M, float& sum,
                                           float* counts) {
  M = -INFINITY;
#pragma unroll 4
  for (int i = sub; i < pieces.n; i += kLanes) M = fmaxf(M, pieces[i][g]);
#pragma unroll
  for (int w = kLanes / 2; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  sum = 0.f;
#pragma unroll 4
  for (int i = sub; i < pieces.n; i += kLanes) {
    const float l = pieces[i][G + g], a = part_scale(pieces[i][g], l, M, scale);
    sum = fmaf(a, l, sum);
    if (counts) counts[i] = a;
  }
#pragma unroll
  for (int w = kLanes / 2; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
}

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 4)
    paged_join_kernel(PagedView cache, const int32_t* __restrict__ n_slots, int G, int adders,
                      Scale scale, T* __restrict__ o, float* __restrict__ lse, Work work) {
  using L = Tile<T, D>;
  constexpr int kRows = kJoinThreads / D;
  __shared__ float red[kRows][D];
  __shared__ float counts[kBlocks], total;
  __shared__ float2 stat[kJoinThreads / 32][kMaxG];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_kv = cache.n_kv_heads;
  pdl_wait();
  if (int(blockIdx.x) < adders) {
    const int c = int(blockIdx.x);
    const Run run = work.runs[c];
    if (run.seq < 0) return;
    const Runs runs(run.units);
    // each warp takes an eighth of the run: a piece is a chain of dependent
    // loads (counts, partial results, scores), and they then run side by side
    constexpr int kParts = kJoinThreads / 32;
    const int run_lo = runs.begin(c), run_units = runs.begin(c + 1) - run_lo;
    int u = run_lo + int(int64_t(warp) * run_units / kParts);
    const int run_hi = run_lo + int(int64_t(warp + 1) * run_units / kParts);
    int seq_first = run.seq_first, b = run.seq;
    while (u < run_hi) {
      int n, stride;
      while (true) {
        n = n_slots[b];
        stride = n > 0 && int64_t(n) <= cache.capacity()
                     ? (n + L::kUnit - 1) / L::kUnit + kHeadUnits
                     : 0;
        if (u < seq_first + stride * n_kv) break;
        seq_first += stride * n_kv;
        ++b;
      }
      const int h = (u - seq_first) / stride, head_units = stride - kHeadUnits;
      const int first = seq_first + h * stride + kHeadUnits;
      const int u_end = min(run_hi, first + head_units);
      u = max(u, first);
      if (u >= u_end) break;
      const int t_lo = (u - first) * L::kUnit, t_hi = min(n, (u_end - first) * L::kUnit);
      int part, n_parts;
      runs.pieces(first, head_units, part, n_parts);
      const Pieces pieces(work, G, D, part, n_parts);
      const int64_t row0 = (int64_t(b) * n_kv + h) * G;
      {  // four lanes per query head
        const int g = min(lane / 4, G - 1);
        float M, sum;
        if (pieces.n > 1) {
          join_stats<4>(pieces, G, g, lane % 4, scale, M, sum, nullptr);
        } else {
          const float2 whole = work.stats[row0 + g];
          M = whole.x;
          sum = whole.y;
        }
        stat[warp][g] = head_stat(M, sum);
      }
      __syncwarp();
      add_weights<T, D>(cache, cache.table + int64_t(b) * cache.max_pages, h, G, t_lo, t_hi,
                        work.scores + int64_t(first) * L::kUnit * G, stat[warp], scale, lane, 32);
      __syncwarp();
      u = u_end;
    }
  } else {
    const int g = (int(blockIdx.x) - adders) / kBlocks;
    const Run run = work.runs[(int(blockIdx.x) - adders) % kBlocks];
    if (run.tail_units == 0) return;
    const int64_t row = int64_t(run.tail_head) * G + g;
    const Pieces pieces(work, G, D, run.tail_part, run.tail_n);
    // the outputs are on their way while the maxima and sums are
    constexpr int kHeld = 8;
    const int e = tid % D, r = tid / D;
    float held[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const int i = r + k * kRows;
      held[k] = i < pieces.n ? pieces[i][2 * G + g * D + e] : 0.f;
    }
    if (warp == 0) {
      float M, sum;
      join_stats<32>(pieces, G, g, lane, scale, M, sum, counts);
      if (lane == 0) {
        total = sum;
        lse[row] = final_lse(M, sum, scale);
      }
    }
    __syncthreads();
    float out = 0.f;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const int i = r + k * kRows;
      if (i < pieces.n) out = fmaf(counts[i], held[k], out);
    }
#pragma unroll 8
    for (int i = r + kHeld * kRows; i < pieces.n; i += kRows)
      out = fmaf(counts[i], pieces[i][2 * G + g * D + e], out);
    red[r][e] = out;
    __syncthreads();
    if (r == 0) {
#pragma unroll
      for (int i = 1; i < kRows; ++i) out += red[i][e];
      o[row * D + e] = final_out<T>(out, total);
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
