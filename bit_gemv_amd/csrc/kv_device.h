// The paged key/value cache as kernels address it (layouts: rfp2_kv_cache in
// include/rfp2.h).  Offsets count elements of the cache's type and are 64-bit:
// a cache of a hundred million values and more passes 32 bits.
#pragma once

#include "acts_device.h"
#include "rfp2_internal.h"

namespace rfp2 {

// The page of token pos of sequence seq, or -1 where the cache has no such
// token (or the table names no page of it).
__device__ __forceinline__ int32_t kv_page(const KvView& c, int32_t seq, int32_t pos) {
  if (seq < 0 || seq >= c.seqs || (pos >> c.page_shift) >= c.max_pages) return -1;
  const int32_t p = c.table[(int64_t)seq * c.max_pages + (pos >> c.page_shift)];
  return p >= 0 && p < c.pages ? p : -1;
}

// Rows (tokens) of the pages before (page, head): the unit of every layout.
__device__ __forceinline__ int64_t kv_rows(const KvView& c, int32_t page, int head) {
  return ((int64_t)page * c.heads + head) << c.page_shift;
}

// Element `d` of row `r` (0 .. page_size - 1) after `rows` rows.
__device__ __forceinline__ int64_t k_at(const KvView& c, int64_t rows, int r, int d) {
  return (rows + r) * c.dim + d;
}
__device__ __forceinline__ int64_t v_at(const KvView& c, int64_t rows, int r, int d) {
  return (rows + (r & ~7)) * c.dim + d * 8 + (r & 7);
}
// Scale of block `b` (32 values) of row r, keys and values alike.
__device__ __forceinline__ int64_t scale_at(const KvView& c, int64_t rows, int r, int b) {
  return (rows + (r & ~7)) * (c.dim >> 5) + b * 8 + (r & 7);
}

}  // namespace rfp2
