// The pages of a paged cache: who holds them (a count a page, a row of pages a sequence), and copies.
#pragma once

#include "kda_attn.cuh"

namespace kda {
namespace pages {

// refs[page]: rows that hold the page, 0 where it is free.  A row's pages come first, -1 behind them.
struct Pool {
  int32_t* refs;
  int32_t* table;
  int64_t table_stride;
  int32_t* kv_lens;
  int* status;
  int32_t num_pages, page_size, num_rows, max_blocks;
};
constexpr int kMaxRows = 16384;       // rows (pairs) that one call gives pages to

// Rows `rows` [num] wholly, or (null) every row beyond its kv_lens.
cudaError_t launch_free(const Pool& p, const int32_t* rows, int32_t num, cudaStream_t stream);
cudaError_t launch_reserve(const Pool& p, const int32_t* new_tokens, cudaStream_t stream);
cudaError_t launch_fork(const Pool& p, const int32_t* src, const int32_t* dst, int32_t num, int32_t* from,
                        int32_t* to, cudaStream_t stream);
// Keys, values and scales of pages from[i] to pages to[i]; pairs with a negative page are left out.
cudaError_t launch_copy(const attn::CacheView& c, const int32_t* from, const int32_t* to, int64_t num,
                        int* status, cudaStream_t stream);

}  // namespace pages
}  // namespace kda
