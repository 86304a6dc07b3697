// C ABI of the page tables and the pool's counts (dflash_kv_pages.h):
// host-side validation and launches.
#include "api_kv_common.h"
#include "kv_pages.h"

namespace {

using namespace dflash;

constexpr int64_t kMaxPages = (int64_t)1 << 30;
constexpr int32_t kMaxRequests = 1 << 20;
// A request's saved entries are counted in 64 bits; their extent stays far from 2^60.
constexpr int64_t kMaxEntries = (int64_t)1 << 40;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool pool_ok(const dflash_kv_pool* p) {
  return p && p->n_pages >= 1 && p->n_pages <= kMaxPages && p->page_size >= 1 && p->page_size <= 65536;
}

// An array of the call: what it is, and whether the call writes it.
struct Array {
  const void* p;
  size_t bytes;
  const char* name;
  bool written;
};
template <int N>
int check_arrays(const Array (&a)[N], const char* who) {
  for (int i = 0; i < N; ++i) {
    if (!a[i].bytes) continue;
    if (!a[i].p) return fail(DFLASH_ERR_INVALID_ARG, "%s: null %s", who, a[i].name);
    if (!aligned4(a[i].p)) return fail(DFLASH_ERR_INVALID_ARG, "%s: %s must be 4-byte aligned", who, a[i].name);
  }
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < i; ++j)
      if (a[i].bytes && a[j].bytes && (a[i].written || a[j].written) && overlaps(a[i].p, a[i].bytes, a[j].p, a[j].bytes))
        return fail(DFLASH_ERR_INVALID_ARG, "%s: %s overlaps %s", who, a[i].name, a[j].name);
  return DFLASH_OK;
}

int view_pages(const dflash_kv_pool* pool, const dflash_kv_rows* rows, PagesView& v, const char* who) {
  if (!pool || !rows) return fail(DFLASH_ERR_INVALID_ARG, "%s: null pool or rows", who);
  if (!pool_ok(pool))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_pages must be in 1 .. 2^30 and page_size in 1 .. 65536", who);
  if (!pool->refs) return fail(DFLASH_ERR_INVALID_ARG, "%s: null refs", who);
  if (rows->n_req < 0 || rows->n_req > kMaxRequests)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_req must be in 0 .. 2^20", who);
  if (rows->table_width < 1 || rows->table_stride < rows->table_width)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: need 1 <= table_width <= table_stride", who);
  if (!rows_reach(rows->n_req, rows->table_stride))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the page_table is beyond 2^60 bytes", who);
  if ((int64_t)rows->n_req * rows->table_width > kMaxEntries)
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: n_req * table_width must be at most 2^40", who);
  v = PagesView{};
  v.refs = pool->refs;
  v.n_pages = (int32_t)pool->n_pages;
  v.page_size = pool->page_size;
  v.per_page = FastDiv::make(pool->page_size);
  v.table = rows->page_table;
  v.table_stride = rows->table_stride;
  v.table_width = rows->table_width;
  v.n_req = rows->n_req;
  v.lens = rows->lens;
  v.most = (int32_t)std::min<int64_t>((int64_t)rows->table_width * pool->page_size, INT_MAX);
  return DFLASH_OK;
}

size_t table_bytes(const PagesView& v) {
  return v.n_req ? ((size_t)(v.n_req - 1) * v.table_stride + v.table_width) * 4 : 0;
}

// The workspace's size and alignment.
int check_workspace(const PagesView& v, const void* workspace, size_t bytes, size_t& need, const char* who) {
  need = kv_pages_workspace(v.n_pages, v.n_req, v.table_width);
  if (bytes < need || !workspace)
    return fail(DFLASH_ERR_WORKSPACE, "%s: workspace of %zu bytes < %zu needed", who, bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  return DFLASH_OK;
}

}  // namespace

extern "C" {

size_t dflash_kv_pages_workspace_size(const dflash_kv_pool* pool, int32_t n_req, int32_t table_width) {
  if (!pool_ok(pool) || n_req < 0 || n_req > kMaxRequests || table_width < 1 ||
      (int64_t)n_req * table_width > kMaxEntries)
    return 0;
  return kv_pages_workspace(pool->n_pages, n_req, table_width);
}

int dflash_kv_resize(const dflash_kv_pool* pool, const dflash_kv_rows* rows, const int32_t* want, int32_t* copies,
                     int32_t* counts, void* workspace, size_t workspace_bytes, dflash_stream_t stream) {
  const char* who = "dflash_kv_resize";
  PagesView v;
  int st = view_pages(pool, rows, v, who);
  if (st != DFLASH_OK) return st;
  size_t need = 0;
  if ((st = check_workspace(v, workspace, workspace_bytes, need, who)) != DFLASH_OK) return st;
  const size_t n = (size_t)v.n_req;
  const Array arrays[] = {{v.refs, (size_t)v.n_pages * 4, "refs", true}, {v.table, table_bytes(v), "page_table", true},
                          {v.lens, n * 4, "lens", true}, {want, n * 4, "want", false}, {copies, n * 8, "copies", true},
                          {counts, 8, "counts", true}, {workspace, need, "the workspace", true}};
  if ((st = check_arrays(arrays, who)) != DFLASH_OK) return st;
  st = launch_status(launch_kv_resize(v, want, copies, counts, workspace, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

int dflash_kv_fork(const dflash_kv_pool* pool, const dflash_kv_rows* rows, const int32_t* parents, void* workspace,
                   size_t workspace_bytes, dflash_stream_t stream) {
  const char* who = "dflash_kv_fork";
  PagesView v;
  int st = view_pages(pool, rows, v, who);
  if (st != DFLASH_OK) return st;
  if (v.n_req == 0) return ok();
  size_t need = 0;
  if ((st = check_workspace(v, workspace, workspace_bytes, need, who)) != DFLASH_OK) return st;
  const size_t n = (size_t)v.n_req;
  const Array arrays[] = {{v.refs, (size_t)v.n_pages * 4, "refs", true}, {v.table, table_bytes(v), "page_table", true},
                          {v.lens, n * 4, "lens", true}, {parents, n * 4, "parents", false},
                          {workspace, need, "the workspace", true}};
  if ((st = check_arrays(arrays, who)) != DFLASH_OK) return st;
  st = launch_status(launch_kv_fork(v, parents, workspace, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

int dflash_kv_compact(const dflash_kv_pool* pool, const dflash_kv_rows* rows, int32_t* page_map, int32_t* copies,
                      int64_t max_copies, int32_t* counts, void* workspace, size_t workspace_bytes,
                      dflash_stream_t stream) {
  const char* who = "dflash_kv_compact";
  PagesView v;
  int st = view_pages(pool, rows, v, who);
  if (st != DFLASH_OK) return st;
  if (max_copies < 0 || max_copies > kMaxPages)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: max_copies must be in 0 .. 2^30", who);
  size_t need = 0;
  if ((st = check_workspace(v, workspace, workspace_bytes, need, who)) != DFLASH_OK) return st;
  const size_t n = (size_t)v.n_req;
  const Array arrays[] = {{v.refs, (size_t)v.n_pages * 4, "refs", true}, {v.table, table_bytes(v), "page_table", true},
                          {v.lens, n * 4, "lens", false}, {page_map, (size_t)v.n_pages * 4, "page_map", true},
                          {copies, (size_t)max_copies * 8, "copies", true}, {counts, 8, "counts", true},
                          {workspace, need, "the workspace", true}};
  if ((st = check_arrays(arrays, who)) != DFLASH_OK) return st;
  st = launch_status(launch_kv_compact(v, page_map, copies, max_copies, counts, workspace, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

int dflash_kv_copy_pages(const dflash_kv_cache* cache, const dflash_page_bounds* bounds, const int32_t* copies,
                         int64_t max_copies, const int32_t* counts, dflash_stream_t stream) {
  const char* who = "dflash_kv_copy_pages";
  KvView c;
  int st = view_cache(cache, c, who);
  if (st != DFLASH_OK) return st;
  if (max_copies < 0 || max_copies > kMaxPages)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: max_copies must be in 0 .. 2^30", who);
  if ((st = check_apart(c, who)) != DFLASH_OK) return st;
  size_t code_size = 0, scale_size = 0;
  if (bounds) {
    if ((st = check_bounds(bounds, code_size, scale_size, who)) != DFLASH_OK) return st;
    if (bounds->n_pages != c.n_pages || bounds->page_size != c.page_size || bounds->n_kv_heads != c.n_kv_heads ||
        bounds->head_dim != c.head_dim)
      return fail(DFLASH_ERR_INVALID_ARG, "%s: the bounds are not of the cache's pages and heads", who);
    if (meets_cache(c, bounds->codes, code_size) || meets_cache(c, bounds->scale, scale_size))
      return fail(DFLASH_ERR_INVALID_ARG, "%s: the bounds overlap the cache", who);
  }
  if (max_copies == 0) return ok();
  const size_t list = (size_t)max_copies * 8;
  const Array arrays[] = {{copies, list, "copies", false}, {counts, counts ? 8u : 0u, "counts", false}};
  if ((st = check_arrays(arrays, who)) != DFLASH_OK) return st;
  if (meets_cache(c, copies, list) || (counts && meets_cache(c, counts, 8)))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: copies or counts overlaps the cache", who);
  if (bounds)
    for (const Array& a : arrays)
      if (a.bytes && (overlaps(a.p, a.bytes, bounds->codes, code_size) || overlaps(a.p, a.bytes, bounds->scale, scale_size)))
        return fail(DFLASH_ERR_INVALID_ARG, "%s: copies or counts overlaps the bounds", who);
  st = launch_status(launch_kv_copy_pages(c, bounds, copies, max_copies, counts, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

}  // extern "C"
