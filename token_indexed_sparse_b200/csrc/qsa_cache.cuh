// Device view of a paged K/V cache and of a packed batch of new tokens over it.
//
// The pools hold [n_pages, page_size, G, 256] rows, so position j of sequence b
// is pool row table[b][j / page_size] * page_size + j % page_size.  Sequence b
// holds kv_len[b] tokens, the last cu_q[b + 1] - cu_q[b] of them new: packed
// row t of it sits at position kv_len[b] - (cu_q[b + 1] - t).  Everything read
// from the device arrays is checked here before it becomes an address: rows of
// no sequence, positions outside the table and page IDs outside [0, n_pages)
// name no pool row.
#pragma once

#include <stdint.h>

namespace qsa {

struct CacheView {
  const int32_t* table;   // [B, max_pages]
  const int32_t* kv_len;  // [B]
  const int32_t* cu_q;    // [B + 1]
  int B;
  int max_pages;
  int n_pages;
  int page_shift;  // log2(page_size)
};

// The sequence of packed row t (the last one that starts at or before t, so
// sequences without new tokens are passed over), or -1 for a row of none.  All
// lanes of the warp search together, 32 offsets a step (log2(B) reads one after
// another cost a decode step microseconds).
__device__ __forceinline__ int cache_seq(const CacheView& c, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = c.B;  // in [lo, hi); cu_q[lo] <= t is known only after the search
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool before = lane == 0 || (i < hi && __ldg(c.cu_q + i) <= t);
    lo += (31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, before)))) * step;
    hi = min(hi, lo + step);
  }
  return __ldg(c.cu_q + lo) <= t && t < __ldg(c.cu_q + lo + 1) ? lo : -1;
}

// Position of packed row t in its sequence b (negative when kv_len is short).
__device__ __forceinline__ int64_t cache_pos(const CacheView& c, int b, int64_t t) {
  return static_cast<int64_t>(__ldg(c.kv_len + b)) - (__ldg(c.cu_q + b + 1) - t);
}

// Pool row of position j of sequence b, or -1.
__device__ __forceinline__ int cache_row(const CacheView& c, int b, int64_t j) {
  if (j < 0 || (j >> c.page_shift) >= c.max_pages) return -1;
  const int page = __ldg(c.table + static_cast<int64_t>(b) * c.max_pages + (j >> c.page_shift));
  if (page < 0 || page >= c.n_pages) return -1;
  return (page << c.page_shift) + static_cast<int>(j & ((int64_t{1} << c.page_shift) - 1));
}

}  // namespace qsa
