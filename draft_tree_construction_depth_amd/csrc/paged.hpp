// Addressing of a paged key/value cache, shared by the append, attention and
// compaction kernels.
//
// One layer's cache is [pages][heads][page_size][head_dim]; a request's row r
// lies on page table[r / page_size] (table: the request's row of the page
// table), at row r % page_size. Page sizes are powers of two, so both are a
// shift and a mask. Without a page table the cache is contiguous per request:
// page b holds all of request b's rows and page_size is its capacity.
#pragma once

#include "common.hpp"

namespace ddt {

struct PagedRows {
  const int32_t* table;  // [batch][width], null: page b is request b's
  int64_t width;         // pages a request can have
  int64_t pages;         // pages in the pool
  int32_t page_size;
  int32_t shift;         // log2(page_size) with a table, 31 without one
  int64_t cap;           // rows a request can have: width * page_size
};

// Page of request b's row r (0 <= r < cap); -1 where the table's entry is
// outside the pool: such rows are neither read nor written.
__device__ __forceinline__ int page_of(const PagedRows& p, int64_t b, int r) {
  if (!p.table) return (int)b;
  const int page = p.table[b * p.width + (r >> p.shift)];
  return page < 0 || page >= p.pages ? -1 : page;
}

__device__ __forceinline__ int row_in_page(const PagedRows& p, int r) {
  return p.table ? r & (p.page_size - 1) : r;
}

}  // namespace ddt
