// Host-side checks that the entry points on a paged KV cache share.
#pragma once

#include <algorithm>
#include <climits>

#include "api_common.h"
#include "dflash_kv_pages.h"
#include "kv_cache.h"

namespace dflash {

// The largest extent of a tensor in bytes: offsets in it stay far from 2^63.
constexpr int64_t kMaxExtent = (int64_t)1 << 60;
// The largest grid dimension in threads.
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 256;

inline int64_t code_bytes(int32_t dtype) { return dtype == DFLASH_BF16 ? 2 : 1; }

// Checks a cache and fills the view's side of it.
inline int view_cache(const dflash_kv_cache* c, KvView& v, const char* who) {
  if (!c) return fail(DFLASH_ERR_INVALID_ARG, "%s: null cache", who);
  if (c->dtype != DFLASH_BF16 && c->dtype != DFLASH_E4M3 && c->dtype != DFLASH_I8)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: unknown cache dtype %d", who, c->dtype);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128 or 256", who);
  if (c->page_size < 1 || c->page_size > 65536)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: page_size must be in 1 .. 65536", who);
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_kv_heads must be in 1 .. 1024", who);
  if (c->n_pages < 1 || c->n_pages > INT_MAX)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_pages must be in 1 .. 2^31 - 1", who);
  const int64_t rows = (int64_t)c->n_kv_heads * c->page_size, size = code_bytes(c->dtype);
  if (c->page_stride < rows * c->head_dim || c->page_stride > ((int64_t)1 << 40))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: page_stride outside n_kv_heads * page_size * head_dim .. 2^40", who);
  if (c->page_stride * size % 16) return fail(DFLASH_ERR_INVALID_ARG, "%s: page_stride must be a multiple of 16 bytes", who);
  if (c->page_stride > kMaxExtent / size / c->n_pages)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the cache is beyond 2^60 bytes", who);
  if (!c->k || !c->v) return fail(DFLASH_ERR_INVALID_ARG, "%s: null cache pointer", who);
  if (!aligned16(c->k) || !aligned16(c->v))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the cache must be 16-byte aligned", who);
  const bool scaled = c->dtype != DFLASH_BF16;
  if (scaled != (c->k_scale != nullptr) || scaled != (c->v_scale != nullptr))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: scales belong to the 8-bit caches, and both to those", who);
  if (scaled && (c->scale_page_stride < rows || c->scale_page_stride > ((int64_t)1 << 40)))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: scale_page_stride outside n_kv_heads * page_size .. 2^40", who);
  if (scaled && c->scale_page_stride > kMaxExtent / c->n_pages)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the scales are beyond 2^60 bytes", who);
  v = KvView{};
  v.k = static_cast<unsigned char*>(c->k);
  v.v = static_cast<unsigned char*>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.page_bytes = c->page_stride * size;
  v.scale_page_bytes = scaled ? c->scale_page_stride : 0;
  v.n_pages = c->n_pages;
  v.page_size = c->page_size;
  v.n_kv_heads = c->n_kv_heads;
  v.head_dim = c->head_dim;
  v.dtype = c->dtype;
  v.per_page = FastDiv::make(c->page_size);
  return DFLASH_OK;
}

// Bytes from the pool's first to its last of one tensor.
inline size_t pool_bytes(const KvView& v) {
  return (size_t)(v.n_pages - 1) * v.page_bytes +
         (size_t)v.n_kv_heads * v.page_size * v.head_dim * code_bytes(v.dtype);
}
inline bool meets_cache(const KvView& v, const void* p, size_t bytes) {
  const size_t n = pool_bytes(v);
  if (overlaps(p, bytes, v.k, n) || overlaps(p, bytes, v.v, n)) return true;
  if (!v.k_scale) return false;
  const size_t m = (size_t)(v.n_pages - 1) * v.scale_page_bytes + (size_t)v.n_kv_heads * v.page_size;
  return overlaps(p, bytes, v.k_scale, m) || overlaps(p, bytes, v.v_scale, m);
}

// Whether n rows of int32, `stride` elements apart, lie within the largest extent.
inline bool rows_reach(int64_t n, int64_t stride) { return n <= 1 || stride <= kMaxExtent / 8 / n; }

// Checks a batch and fills the view's side of it; rows: the call has dense
// rows (offsets and n_rows count).
inline int view_batch(const dflash_kv_batch* b, bool rows, KvView& v, const char* who) {
  if (!b) return fail(DFLASH_ERR_INVALID_ARG, "%s: null batch", who);
  if (b->n_req < 0 || b->n_req > (1 << 24)) return fail(DFLASH_ERR_INVALID_ARG, "%s: n_req must be in 0 .. 2^24", who);
  if (b->table_width < 1 || b->table_stride < b->table_width)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: need 1 <= table_width <= table_stride", who);
  if (!rows_reach(b->n_req, b->table_stride))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the page_table is beyond 2^60 bytes", who);
  if (rows && (b->n_rows < 0 || b->n_rows > INT_MAX))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_rows must be in 0 .. 2^31 - 1", who);
  if (b->n_req > 0 && (!b->page_table || !b->start || (rows && b->n_rows > 0 && !b->offsets)))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: null pointer in the batch", who);
  v.table = b->page_table;
  v.table_stride = b->table_stride;
  v.table_width = b->table_width;
  v.n_req = b->n_req;
  v.start = b->start;
  v.offsets = b->offsets;
  v.n_rows = rows ? b->n_rows : 0;
  return DFLASH_OK;
}

// Whether [p, p + bytes) meets one of the batch's arrays (n_req > 0).
inline bool meets_batch(const KvView& v, const void* p, size_t bytes) {
  const size_t n = (size_t)v.n_req;
  return overlaps(p, bytes, v.table, ((n - 1) * (size_t)v.table_stride + v.table_width) * 4) ||
         overlaps(p, bytes, v.start, n * 4) || overlaps(p, bytes, v.offsets, (n + 1) * 4);
}

// Strided rows [n_rows, heads, head_dim] of `size`-byte elements: alignment,
// strides within range, and their extent in bytes.
inline int check_rows(const void* p, int64_t row, int64_t head, int64_t n_rows, int32_t heads, int32_t dim, int64_t size,
               size_t& bytes, const char* name, const char* who) {
  if (!p) return fail(DFLASH_ERR_INVALID_ARG, "%s: null %s", who, name);
  if (!aligned16(p) || row * size % 16 || head * size % 16)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: %s and its strides must be multiples of 16 bytes", who, name);
  const int64_t limit = (int64_t)1 << 40;
  if (head < 0 || row < 0 || row > limit || head > limit)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: strides of %s must be in 0 .. 2^40", who, name);
  if (row > kMaxExtent / size / 2 / n_rows || head > kMaxExtent / size / 4 / heads)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: %s is beyond 2^60 bytes", who, name);
  bytes = (size_t)(((n_rows - 1) * row + (heads - 1) * head + dim) * size);
  return DFLASH_OK;
}

// Whether two arrays of n pages, `na` bytes each at a + i * sa and `nb` at
// b + i * sb, share a byte.  Pages of one stride that lie within each other's
// span are apart where those of b fit the gaps of a; of two strides, they are
// taken to meet.
inline bool pages_meet(const void* a, size_t na, int64_t sa, const void* b, size_t nb, int64_t sb, int64_t n) {
  if (!overlaps(a, (size_t)(n - 1) * sa + na, b, (size_t)(n - 1) * sb + nb)) return false;
  if (n == 1 || sa != sb) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const size_t s = (size_t)sa, gap = y >= x ? (y - x) % s : (s - (x - y) % s) % s;   // from a page of a to the next of b
  return gap < na || gap + nb > s;
}

// K, V and their scales are written side by side, in no order.
inline int check_apart(const KvView& v, const char* who) {
  const size_t rows = (size_t)v.n_kv_heads * v.page_size, codes = rows * v.head_dim * code_bytes(v.dtype);
  const int64_t n = v.n_pages;
  if (pages_meet(v.k, codes, v.page_bytes, v.v, codes, v.page_bytes, n) ||
      (v.k_scale && pages_meet(v.k_scale, rows, v.scale_page_bytes, v.v_scale, rows, v.scale_page_bytes, n)))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the cache's K and V overlap", who);
  if (!v.k_scale) return DFLASH_OK;
  for (const unsigned char* c : {v.k, v.v})
    for (const uint8_t* s : {v.k_scale, v.v_scale})
      if (pages_meet(c, codes, v.page_bytes, s, rows, v.scale_page_bytes, n))
        return fail(DFLASH_ERR_INVALID_ARG, "%s: the cache's scales overlap its K or V", who);
  return DFLASH_OK;
}

// Checks the bounds of a pool's pages; their extents in bytes.
inline int check_bounds(const dflash_page_bounds* b, size_t& code_size, size_t& scale_size, const char* who) {
  if (!b) return fail(DFLASH_ERR_INVALID_ARG, "%s: null bounds", who);
  if (b->head_dim != 64 && b->head_dim != 128 && b->head_dim != 256)
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128 or 256", who);
  if (b->page_size < 1 || b->page_size > 65536)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: page_size must be in 1 .. 65536", who);
  if (b->n_kv_heads < 1 || b->n_kv_heads > 1024)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_kv_heads must be in 1 .. 1024", who);
  if (b->n_pages < 1 || b->n_pages > INT_MAX)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_pages must be in 1 .. 2^31 - 1", who);
  if (!b->codes || !b->scale) return fail(DFLASH_ERR_INVALID_ARG, "%s: null pointer in the bounds", who);
  if (!aligned16(b->codes)) return fail(DFLASH_ERR_INVALID_ARG, "%s: the bounds' codes must be 16-byte aligned", who);
  scale_size = (size_t)b->n_pages * b->n_kv_heads;
  code_size = scale_size * 2 * b->head_dim;
  if (overlaps(b->codes, code_size, b->scale, scale_size))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the bounds' codes and scales overlap", who);
  return DFLASH_OK;
}

}  // namespace dflash
