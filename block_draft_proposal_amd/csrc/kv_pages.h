// Page tables and the counts of a pool's pages, as the kernels see them.
#pragma once

#include "dflash_kv_pages.h"
#include "kv_cache.h"

namespace dflash {

struct PagesView {
  int32_t* refs;
  int32_t n_pages;
  int32_t page_size;
  FastDiv per_page;
  int32_t* table;
  int64_t table_stride;
  int32_t table_width, n_req;
  int32_t* lens;
  int32_t most;               // the longest length that a row of the table holds

  // Entries that a request of `len` positions holds, -1 for a length out of range.
  __device__ __forceinline__ int32_t entries(int32_t len) const {
    if (len < 0 || len > most) return -1;
    return len == 0 ? 0 : per_page.div(len - 1) + 1;
  }
  __device__ __forceinline__ bool in_pool(int32_t page) const { return page >= 0 && page < n_pages; }
};

size_t kv_pages_workspace(int64_t n_pages, int32_t n_req, int32_t table_width);
hipError_t launch_kv_resize(const PagesView& v, const int32_t* want, int32_t* copies, int32_t* counts, void* workspace,
                            hipStream_t stream);
hipError_t launch_kv_fork(const PagesView& v, const int32_t* parents, void* workspace, hipStream_t stream);
hipError_t launch_kv_compact(const PagesView& v, int32_t* page_map, int32_t* copies, int64_t max_copies,
                             int32_t* counts, void* workspace, hipStream_t stream);
hipError_t launch_kv_copy_pages(const KvView& c, const dflash_page_bounds* bounds, const int32_t* copies,
                                int64_t max_copies, const int32_t* counts, hipStream_t stream);

}  // namespace dflash
