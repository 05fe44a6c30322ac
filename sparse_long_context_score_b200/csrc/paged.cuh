// paged.cuh -- a batch of new tokens over a paged compressed cache, as the append and the
// chunk attention read it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace dsa {

// Tokens [cu_q[b], cu_q[b + 1]) are sequence b's new ones; ctx_len[b] counts its cached
// tokens, the new ones among them.  Position s of sequence b is row s % page_size of page
// table[b][s / page_size].
struct PagedBatch {
  const int32_t* table;    // [B][max_pages]
  const int32_t* cu_q;     // [B + 1]
  const int32_t* ctx_len;  // [B]
  int n, B, max_pages, num_pages, page_size;
};

// Row of the pool that holds a position; -1 where there is none: a negative position, one
// behind the table, or a table entry that is no page of the pool.
__device__ __forceinline__ long long paged_row(const PagedBatch& p, int b, long long position) {
  if (position < 0) return -1;
  const long long i = position / p.page_size;
  if (i >= p.max_pages) return -1;
  const int page = p.table[(size_t)b * p.max_pages + i];
  return page >= 0 && page < p.num_pages ? (long long)page * p.page_size + (position - i * p.page_size) : -1;
}

}  // namespace dsa
