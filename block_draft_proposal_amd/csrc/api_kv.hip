// C ABI of the paged KV cache and the draft-tree attention (dflash_kv.h):
// host-side validation and launches.
#include <climits>
#include <cmath>

#include "api_common.h"
#include "dflash_kv.h"
#include "kv_cache.h"

namespace {

using namespace dflash;

constexpr int kMaxGroup = 64, kMaxNodes = 4096;

// The largest extent of a tensor in bytes: offsets in it stay far from 2^63.
constexpr int64_t kMaxExtent = (int64_t)1 << 60;
// The largest grid dimension in threads.
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 256;

int64_t code_bytes(int32_t dtype) { return dtype == DFLASH_BF16 ? 2 : 1; }

// Checks a cache and fills the view's side of it.
int view_cache(const dflash_kv_cache* c, KvView& v, const char* who) {
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
size_t pool_bytes(const KvView& v) {
  return (size_t)(v.n_pages - 1) * v.page_bytes +
         (size_t)v.n_kv_heads * v.page_size * v.head_dim * code_bytes(v.dtype);
}
bool meets_cache(const KvView& v, const void* p, size_t bytes) {
  const size_t n = pool_bytes(v);
  if (overlaps(p, bytes, v.k, n) || overlaps(p, bytes, v.v, n)) return true;
  if (!v.k_scale) return false;
  const size_t m = (size_t)(v.n_pages - 1) * v.scale_page_bytes + (size_t)v.n_kv_heads * v.page_size;
  return overlaps(p, bytes, v.k_scale, m) || overlaps(p, bytes, v.v_scale, m);
}

// Whether n rows of int32, `stride` elements apart, lie within the largest extent.
bool rows_reach(int64_t n, int64_t stride) { return n <= 1 || stride <= kMaxExtent / 8 / n; }

// Checks a batch and fills the view's side of it; rows: the call has dense
// rows (offsets and n_rows count).
int view_batch(const dflash_kv_batch* b, bool rows, KvView& v, const char* who) {
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
bool meets_batch(const KvView& v, const void* p, size_t bytes) {
  const size_t n = (size_t)v.n_req;
  return overlaps(p, bytes, v.table, ((n - 1) * (size_t)v.table_stride + v.table_width) * 4) ||
         overlaps(p, bytes, v.start, n * 4) || overlaps(p, bytes, v.offsets, (n + 1) * 4);
}

// Strided rows [n_rows, heads, head_dim] of `size`-byte elements: alignment,
// strides within range, and their extent in bytes.
int check_rows(const void* p, int64_t row, int64_t head, int64_t n_rows, int32_t heads, int32_t dim, int64_t size,
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

// A thread holds 8 elements of a row in the write and the read.
int check_stream(const KvView& v, const char* who) {
  if (v.n_rows > kMaxThreads / (v.head_dim / 8))
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: n_rows * head_dim must be below 2^35", who);
  return DFLASH_OK;
}

// Whether two arrays of n pages, `na` bytes each at a + i * sa and `nb` at
// b + i * sb, share a byte.  Pages of one stride that lie within each other's
// span are apart where those of b fit the gaps of a; of two strides, they are
// taken to meet.
bool pages_meet(const void* a, size_t na, int64_t sa, const void* b, size_t nb, int64_t sb, int64_t n) {
  if (!overlaps(a, (size_t)(n - 1) * sa + na, b, (size_t)(n - 1) * sb + nb)) return false;
  if (n == 1 || sa != sb) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const size_t s = (size_t)sa, gap = y >= x ? (y - x) % s : (s - (x - y) % s) % s;   // from a page of a to the next of b
  return gap < na || gap + nb > s;
}

// K, V and their scales are written side by side, in no order.
int check_apart(const KvView& v, const char* who) {
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

bool tree_shape_ok(int32_t n_kv_heads, int32_t n_q_heads, int32_t max_nodes) {
  return n_q_heads >= 1 && n_q_heads % n_kv_heads == 0 && n_q_heads / n_kv_heads <= kMaxGroup && max_nodes >= 1 &&
         max_nodes <= kMaxNodes;
}

}  // namespace

extern "C" {

int dflash_kv_write(const dflash_kv_cache* cache, const dflash_kv_batch* batch, const void* k, int64_t k_row_stride,
                    int64_t k_head_stride, const void* v, int64_t v_row_stride, int64_t v_head_stride, int32_t dtype,
                    dflash_stream_t stream) {
  const char* who = "dflash_kv_write";
  KvView c;
  int st = view_cache(cache, c, who);
  if (st != DFLASH_OK) return st;
  if ((st = view_batch(batch, true, c, who)) != DFLASH_OK) return st;
  if (!dtype_ok(dtype)) return fail(DFLASH_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
  if (c.n_req == 0 || c.n_rows == 0) return ok();
  if ((st = check_stream(c, who)) != DFLASH_OK) return st;
  if ((st = check_apart(c, who)) != DFLASH_OK) return st;
  size_t kb = 0, vb = 0;
  if ((st = check_rows(k, k_row_stride, k_head_stride, c.n_rows, c.n_kv_heads, c.head_dim, elem_bytes(dtype), kb, "k",
                       who)) != DFLASH_OK ||
      (st = check_rows(v, v_row_stride, v_head_stride, c.n_rows, c.n_kv_heads, c.head_dim, elem_bytes(dtype), vb, "v",
                       who)) != DFLASH_OK)
    return st;
  if (meets_cache(c, k, kb) || meets_cache(c, v, vb))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: k or v overlaps the cache", who);
  const KvRows in{k, v, k_row_stride, k_head_stride, v_row_stride, v_head_stride, dtype};
  st = launch_status(launch_kv_write(c, in, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

int dflash_kv_read(const dflash_kv_cache* cache, const dflash_kv_batch* batch, void* k_out, void* v_out,
                   int32_t dtype, dflash_stream_t stream) {
  const char* who = "dflash_kv_read";
  KvView c;
  int st = view_cache(cache, c, who);
  if (st != DFLASH_OK) return st;
  if ((st = view_batch(batch, true, c, who)) != DFLASH_OK) return st;
  if (!dtype_ok(dtype)) return fail(DFLASH_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
  if (c.n_req == 0 || c.n_rows == 0) return ok();
  if ((st = check_stream(c, who)) != DFLASH_OK) return st;
  if (!k_out || !v_out) return fail(DFLASH_ERR_INVALID_ARG, "%s: null output", who);
  if (!aligned16(k_out) || !aligned16(v_out))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: k_out and v_out must be 16-byte aligned", who);
  const size_t n = (size_t)c.n_rows * c.n_kv_heads * c.head_dim * elem_bytes(dtype);
  if (overlaps(k_out, n, v_out, n) || meets_cache(c, k_out, n) || meets_cache(c, v_out, n))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: k_out and v_out overlap each other or the cache", who);
  if (meets_batch(c, k_out, n) || meets_batch(c, v_out, n))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: k_out or v_out overlaps the batch's arrays", who);
  st = launch_status(launch_kv_read(c, k_out, v_out, dtype, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

int dflash_kv_commit(const dflash_kv_cache* cache, const dflash_kv_batch* batch, const int32_t* paths,
                     int64_t path_stride, int32_t path_width, const int32_t* path_lens, dflash_stream_t stream) {
  const char* who = "dflash_kv_commit";
  KvView c;
  int st = view_cache(cache, c, who);
  if (st != DFLASH_OK) return st;
  if ((st = view_batch(batch, false, c, who)) != DFLASH_OK) return st;
  if (path_width < 0 || path_stride < path_width)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: need 0 <= path_width <= path_stride", who);
  if (c.n_req == 0 || path_width == 0) return ok();
  if (!rows_reach(c.n_req, path_stride)) return fail(DFLASH_ERR_INVALID_ARG, "%s: paths is beyond 2^60 bytes", who);
  if ((int64_t)c.n_req * c.n_kv_heads > kMaxThreads / 128)
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: n_req * n_kv_heads must be below 2^25", who);
  if ((st = check_apart(c, who)) != DFLASH_OK) return st;
  if (!paths || !path_lens) return fail(DFLASH_ERR_INVALID_ARG, "%s: null pointer", who);
  st = launch_status(launch_kv_commit(c, paths, path_stride, path_width, path_lens, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

size_t dflash_tree_attention_workspace_size(const dflash_kv_cache* cache, int32_t n_req, int32_t max_nodes,
                                            int32_t n_q_heads) {
  KvView c;
  if (view_cache(cache, c, "dflash_tree_attention_workspace_size") != DFLASH_OK) return 0;
  ok();
  if (n_req <= 0 || !tree_shape_ok(c.n_kv_heads, n_q_heads, max_nodes)) return 0;
  return tree_attention_bytes(c, n_req, max_nodes, n_q_heads);
}

int dflash_tree_attention(const dflash_kv_cache* cache, const dflash_kv_batch* batch, const void* q,
                          int64_t q_row_stride, int64_t q_head_stride, int32_t n_q_heads, const uint64_t* mask,
                          int32_t mask_words, int32_t max_nodes, float scale, int32_t dtype, void* out,
                          void* workspace, size_t workspace_bytes, dflash_stream_t stream) {
  const char* who = "dflash_tree_attention";
  TreeArgs a{};
  int st = view_cache(cache, a.c, who);
  if (st != DFLASH_OK) return st;
  if ((st = view_batch(batch, true, a.c, who)) != DFLASH_OK) return st;
  if (!dtype_ok(dtype)) return fail(DFLASH_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
  if (dtype != DFLASH_BF16) return fail(DFLASH_ERR_UNSUPPORTED, "%s: bf16 queries only", who);
  if (n_q_heads < 1 || n_q_heads % a.c.n_kv_heads)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_q_heads must be a positive multiple of n_kv_heads", who);
  if (n_q_heads / a.c.n_kv_heads > kMaxGroup)
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: more than %d query heads to a kv head", who, kMaxGroup);
  if (max_nodes < 1) return fail(DFLASH_ERR_INVALID_ARG, "%s: max_nodes must be >= 1", who);
  if (max_nodes > kMaxNodes) return fail(DFLASH_ERR_UNSUPPORTED, "%s: max_nodes > %d", who, kMaxNodes);
  if (!std::isfinite(scale) || scale <= 0.f || scale > 0x1p100f)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: scale must be > 0 and at most 2^100", who);
  if (a.c.n_req == 0 || a.c.n_rows == 0) return ok();   // a mask of no rows may be null
  if (mask ? mask_words < (max_nodes + 63) / 64 : mask_words != 0)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: mask_words must be >= ceil(max_nodes / 64) with a mask, 0 without", who);
  if (reinterpret_cast<uintptr_t>(mask) & 7) return fail(DFLASH_ERR_INVALID_ARG, "%s: mask must be 8-byte aligned", who);
  size_t qb = 0;
  if ((st = check_rows(q, q_row_stride, q_head_stride, a.c.n_rows, n_q_heads, a.c.head_dim, 2, qb, "q", who)) != DFLASH_OK)
    return st;
  if (!out || !aligned16(out)) return fail(DFLASH_ERR_INVALID_ARG, "%s: out must be a 16-byte aligned pointer", who);
  const size_t ob = (size_t)a.c.n_rows * n_q_heads * a.c.head_dim * 2;
  if (overlaps(out, ob, q, qb) || meets_cache(a.c, out, ob))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: out overlaps q or the cache", who);
  const size_t mb = mask ? (size_t)a.c.n_rows * mask_words * 8 : 0;
  if (meets_batch(a.c, out, ob) || overlaps(out, ob, mask, mb))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: out overlaps the batch's arrays or the mask", who);
  const size_t need = tree_attention_bytes(a.c, a.c.n_req, max_nodes, n_q_heads);
  if (workspace_bytes < need || (need && !workspace))
    return fail(DFLASH_ERR_WORKSPACE, "%s: workspace of %zu bytes < %zu needed", who, workspace_bytes, need);
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  if (overlaps(workspace, need, out, ob) || overlaps(workspace, need, q, qb) || meets_cache(a.c, workspace, need))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the workspace overlaps q, out or the cache", who);
  if (meets_batch(a.c, workspace, need) || overlaps(workspace, need, mask, mb))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the workspace overlaps the batch's arrays or the mask", who);
  a.q = static_cast<const uint16_t*>(q);
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.n_q_heads = n_q_heads;
  a.mask = mask;
  a.mask_words = mask_words;
  a.max_nodes = max_nodes;
  a.scale = scale;
  a.out = static_cast<uint16_t*>(out);
  a.workspace = workspace;
  st = launch_status(launch_tree_attention(a, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

}  // extern "C"
