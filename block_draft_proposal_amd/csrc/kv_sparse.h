// What the score reads of a pool's pages, and the launchers of the operators
// that choose pages and attend to them.
#pragma once

#include "dflash_kv_sparse.h"
#include "kv_cache.h"

namespace dflash {

struct SelectArgs {
  KvView c;                   // pages, heads and the batch; the cache's pointers are null
  const int8_t* codes;        // [n_pages][n_kv_heads][2][head_dim]
  const uint8_t* scale;       // [n_pages][n_kv_heads]
  const uint16_t* q;
  int64_t q_row, q_head;      // strides in elements
  int32_t n_q_heads, max_nodes, n_take, n_first, n_last;
  int32_t* out;
  uint32_t* keys;             // workspace [n_rows][n_kv_heads][table_width]
};

struct SparseArgs {
  KvView c;
  const uint16_t* q;
  int64_t q_row, q_head;
  int32_t n_q_heads;
  const int32_t* blocks;
  int32_t n_take;
  const uint64_t* mask;       // null: a chain
  int32_t mask_words, max_nodes;
  float scale;
  uint16_t* out;
  void* workspace;
};

// Full pages of a request's prefix.
__device__ __forceinline__ int32_t kv_blocks(const KvView& c, int32_t start) {
  return start <= 0 ? 0 : min(c.per_page.div(start), c.table_width);
}

// A row's request, its first row and the one behind its last, its start.
struct RowOf {
  int32_t req, start;
  int64_t first, end;
};
// false for padding.  Every lane of a wave has the same row.  Where all requests
// before have max_nodes rows (single tokens, blocks of one size) the request is
// known, and one round of loads has it all; else it is searched for.
__device__ __forceinline__ bool row_of(const KvView& c, int64_t row, int32_t max_nodes, RowOf& r) {
  r.req = (int32_t)min((uint32_t)row / (uint32_t)max_nodes, (uint32_t)c.n_req - 1u);
  r.first = c.offsets[r.req];
  r.end = c.offsets[r.req + 1];
  r.start = c.start[r.req];
  if (row < r.first || row >= r.end || row >= c.n_rows) {
    int64_t pos = 0;
    if (!kv_row_position(c, row, row, r.req, pos)) return false;
    r.first = c.offsets[r.req];
    r.end = c.offsets[r.req + 1];
    r.start = c.start[r.req];
  }
  r.req = __builtin_amdgcn_readfirstlane(r.req);
  return true;
}

hipError_t launch_kv_bounds(const KvView& c, int8_t* codes, uint8_t* scale, const int32_t* end, hipStream_t stream);
size_t kv_select_bytes(int64_t n_rows, int32_t n_kv_heads, int32_t table_width);
hipError_t launch_kv_select(const SelectArgs& a, hipStream_t stream);
size_t sparse_attention_bytes(const KvView& c, int64_t n_rows, int32_t n_take, int32_t max_nodes, int32_t n_q_heads);
hipError_t launch_sparse_attention(const SparseArgs& a, hipStream_t stream);

}  // namespace dflash
