// The paged key-value cache as the kernels see it (layout in hga.h): pages in
// any order of one pool, a table of pages per sequence, and per-slot records
// (accumulated attention weight, position of the token).
#pragma once

#include "hga_common.cuh"

namespace hga {

struct PagedView {
  void* k;
  void* v;
  float* weight;
  int32_t* slot_pos;
  const int32_t* table;
  int64_t n_pages;
  int64_t page_stride;  // elements
  int page_shift;       // log2(page_size)
  int max_pages;
  int n_kv_heads;
  __device__ __forceinline__ int page_of(int slot) const { return slot >> page_shift; }
  __device__ __forceinline__ int row_of(int slot) const {
    return slot & ((1 << page_shift) - 1);
  }
  __device__ __forceinline__ bool has(int page) const {
    return page >= 0 && int64_t(page) < n_pages;
  }
  __device__ __forceinline__ int64_t capacity() const {
    return int64_t(max_pages) << page_shift;
  }
  // first element of row `row` of KV head h on page `page`
  __device__ __forceinline__ int64_t elem(int page, int h, int row, int d) const {
    return int64_t(page) * page_stride + (int64_t(h) * (1 << page_shift) + row) * d;
  }
  __device__ __forceinline__ int64_t record(int page, int h, int row) const {
    return ((int64_t(page) * n_kv_heads + h) << page_shift) + row;
  }
};

// n_slots[b], or -1 (with HGA_ERR_DEVICE_CHECK latched) if it is out of range
__device__ __forceinline__ int checked_slots(const PagedView& c, const int32_t* n_slots, int b) {
  const int n = n_slots[b];
  if (n >= 0 && int64_t(n) <= c.capacity()) return n;
  latch_status(HGA_ERR_DEVICE_CHECK);
  return -1;
}

}  // namespace hga
