// Pieces shared by the operators on paged K/V caches: addressing, the checks on what
// the device reads from tables and lengths, and the split of the cached slots over CTAs.
#pragma once

#include "dd_common.cuh"
#include "dd_internal.h"

namespace dd {

// Division of a slot index (below 2^31) by the page size, as a multiplication:
// with 2^(l-1) < n <= 2^l and m = floor(2^(31+l) / n) + 1, x / n = (x m) >> (31 + l)
// for 0 <= x < 2^31, since x (m n - 2^(31+l)) <= x n < 2^(31+l).
struct FastDiv {
  uint64_t m;
  int shift;
  int n;
};
inline FastDiv make_fast_div(int n) {
  int l = 0;
  while ((1ll << l) < n) ++l;
  return FastDiv{((1ull << (31 + l)) / (uint64_t)n) + 1ull, 31 + l, n};
}
__device__ __forceinline__ int div_fast(const FastDiv& f, int x) {
  return (int)(((uint64_t)(uint32_t)x * f.m) >> f.shift);
}

// A paged cache as the kernels see it.
struct PagedView {
  char* k;
  char* v;
  int64_t layer_bytes, page_bytes, token_bytes, head_bytes;
  int layers, n_pages, Hkv;
  int cap;  // slots the table has room for (clamped to int)
  FastDiv page;
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
};

// A sequence's length as the kernels use it: values outside [0, max_len] are recorded
// and clamped, so nothing is read behind a table or a mass row.
__device__ __forceinline__ int checked_length(const int32_t* lengths, int b, int max_len) {
  const int n = lengths[b];
  if (n < 0 || n > max_len) {
    record_error(DD_ERR_BOUNDS);
    return n < 0 ? 0 : max_len;
  }
  return n;
}

// The page of a slot, or -1 for a hole; ids behind the pool are recorded and count as holes.
__device__ __forceinline__ int checked_page(int id, int n_pages) {
  if (id >= n_pages) {
    record_error(DD_ERR_BOUNDS);
    return -1;
  }
  return id < 0 ? -1 : id;
}

// Byte offset of slot j's row (head 0) of the sequence whose table row is `row`, or -1.
__device__ __forceinline__ int64_t slot_offset(const PagedView& c, const int32_t* row, int j) {
  const int p = div_fast(c.page, j);
  const int id = checked_page(row[p], c.n_pages);
  if (id < 0) return -1;
  return (int64_t)id * c.page_bytes + (int64_t)(j - p * c.page.n) * c.token_bytes;
}

PagedView make_paged_view(const dd_paged_cache& c);

}  // namespace dd
