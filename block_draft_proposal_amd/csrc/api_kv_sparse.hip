// C ABI of the choice of pages and of the attention over them
// (dflash_kv_sparse.h): host-side validation and launches.
#include <cmath>

#include "api_kv_common.h"
#include "kv_sparse.h"

namespace {

using namespace dflash;

constexpr int kMaxGroup = 64, kMaxNodes = 4096, kMaxTake = 65536;
// Rows times kv heads of a call: up to 1024 threads each, in one launch.
constexpr int64_t kMaxItems = (int64_t)1 << 21;
// Requests whose pages' bounds one call makes: a workgroup each.
constexpr int32_t kMaxRequests = 1 << 20;
// Blocks of a request that keys are kept of.
constexpr int32_t kMaxBlocks = 1 << 24;

// Query heads of a call with n_kv_heads.
int check_heads(int32_t n_kv_heads, int32_t n_q_heads, const char* who) {
  if (n_q_heads < 1 || n_q_heads % n_kv_heads)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_q_heads must be a positive multiple of n_kv_heads", who);
  if (n_q_heads / n_kv_heads > kMaxGroup)
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: more than %d query heads to a kv head", who, kMaxGroup);
  return DFLASH_OK;
}
int check_nodes(int32_t max_nodes, const char* who) {
  if (max_nodes < 1) return fail(DFLASH_ERR_INVALID_ARG, "%s: max_nodes must be >= 1", who);
  if (max_nodes > kMaxNodes) return fail(DFLASH_ERR_UNSUPPORTED, "%s: max_nodes > %d", who, kMaxNodes);
  return DFLASH_OK;
}
int check_dtype(int32_t dtype, const char* who) {
  if (!dtype_ok(dtype)) return fail(DFLASH_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
  if (dtype != DFLASH_BF16) return fail(DFLASH_ERR_UNSUPPORTED, "%s: bf16 queries only", who);
  return DFLASH_OK;
}
int check_workspace(const void* workspace, size_t bytes, size_t need, const char* who) {
  if (bytes < need || (need && !workspace))
    return fail(DFLASH_ERR_WORKSPACE, "%s: workspace of %zu bytes < %zu needed", who, bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  return DFLASH_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

int dflash_kv_bounds(const dflash_kv_cache* cache, const dflash_page_bounds* bounds, const dflash_kv_batch* batch,
                     const int32_t* end, dflash_stream_t stream) {
  const char* who = "dflash_kv_bounds";
  KvView c;
  int st = view_cache(cache, c, who);
  if (st != DFLASH_OK) return st;
  if ((st = view_batch(batch, false, c, who)) != DFLASH_OK) return st;
  size_t code_size = 0, scale_size = 0;
  if ((st = check_bounds(bounds, code_size, scale_size, who)) != DFLASH_OK) return st;
  if (bounds->n_pages != c.n_pages || bounds->page_size != c.page_size || bounds->n_kv_heads != c.n_kv_heads ||
      bounds->head_dim != c.head_dim)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the bounds are not of the cache's pages and heads", who);
  if (meets_cache(c, bounds->codes, code_size) || meets_cache(c, bounds->scale, scale_size))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: the bounds overlap the cache", who);
  if (c.n_req == 0) return ok();
  if (c.n_req > kMaxRequests) return fail(DFLASH_ERR_UNSUPPORTED, "%s: n_req > 2^20", who);
  if (!end) return fail(DFLASH_ERR_INVALID_ARG, "%s: null end", who);
  const size_t n = (size_t)c.n_req * 4, table = ((size_t)(c.n_req - 1) * c.table_stride + c.table_width) * 4;
  const struct { const void* p; size_t bytes; } arrays[] = {{c.table, table}, {c.start, n}, {end, n}};
  for (const auto& a : arrays)
    if (overlaps(a.p, a.bytes, bounds->codes, code_size) || overlaps(a.p, a.bytes, bounds->scale, scale_size))
      return fail(DFLASH_ERR_INVALID_ARG, "%s: the bounds overlap the batch's arrays", who);
  st = launch_status(launch_kv_bounds(c, bounds->codes, bounds->scale, end, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

size_t dflash_kv_select_workspace_size(const dflash_page_bounds* bounds, int64_t n_rows, int32_t table_width) {
  size_t code_size = 0, scale_size = 0;
  if (check_bounds(bounds, code_size, scale_size, "dflash_kv_select_workspace_size") != DFLASH_OK) return 0;
  ok();
  if (n_rows <= 0 || n_rows > kMaxItems / bounds->n_kv_heads || table_width < 1 || table_width > kMaxBlocks) return 0;
  return kv_select_bytes(n_rows, bounds->n_kv_heads, table_width);
}

int dflash_kv_select(const dflash_page_bounds* bounds, const dflash_kv_batch* batch, const void* q,
                     int64_t q_row_stride, int64_t q_head_stride, int32_t n_q_heads, int32_t max_nodes, int32_t n_take,
                     int32_t n_first, int32_t n_last, int32_t dtype, int32_t* out, void* workspace,
                     size_t workspace_bytes, dflash_stream_t stream) {
  const char* who = "dflash_kv_select";
  SelectArgs a{};
  size_t code_size = 0, scale_size = 0;
  int st = check_bounds(bounds, code_size, scale_size, who);
  if (st != DFLASH_OK) return st;
  if ((st = view_batch(batch, true, a.c, who)) != DFLASH_OK) return st;
  if ((st = check_dtype(dtype, who)) != DFLASH_OK || (st = check_heads(bounds->n_kv_heads, n_q_heads, who)) != DFLASH_OK ||
      (st = check_nodes(max_nodes, who)) != DFLASH_OK)
    return st;
  if (n_take < 1 || n_take > kMaxTake)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: n_take must be in 1 .. %d", who, kMaxTake);
  if (n_first < 0 || n_last < 0 || (int64_t)n_first + n_last > n_take)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: need n_first, n_last >= 0 and n_first + n_last <= n_take", who);
  if (a.c.n_req == 0 || a.c.n_rows == 0) return ok();
  if (a.c.n_rows > kMaxItems / bounds->n_kv_heads)
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: n_rows * n_kv_heads must be at most 2^21", who);
  if (a.c.table_width > kMaxBlocks) return fail(DFLASH_ERR_UNSUPPORTED, "%s: table_width > 2^24", who);
  size_t qb = 0;
  if ((st = check_rows(q, q_row_stride, q_head_stride, a.c.n_rows, n_q_heads, bounds->head_dim, 2, qb, "q", who)) != DFLASH_OK)
    return st;
  if (!out || !aligned4(out)) return fail(DFLASH_ERR_INVALID_ARG, "%s: out must be a 4-byte aligned pointer", who);
  const size_t ob = (size_t)a.c.n_rows * bounds->n_kv_heads * n_take * 4;
  const size_t need = kv_select_bytes(a.c.n_rows, bounds->n_kv_heads, a.c.table_width);
  if ((st = check_workspace(workspace, workspace_bytes, need, who)) != DFLASH_OK) return st;
  const struct { const void* p; size_t bytes; } written[] = {{out, ob}, {workspace, need}};
  for (const auto& x : written)
    if (overlaps(x.p, x.bytes, q, qb) || overlaps(x.p, x.bytes, bounds->codes, code_size) ||
        overlaps(x.p, x.bytes, bounds->scale, scale_size) || meets_batch(a.c, x.p, x.bytes))
      return fail(DFLASH_ERR_INVALID_ARG, "%s: out or the workspace overlaps q, the bounds or the batch's arrays", who);
  if (overlaps(out, ob, workspace, need)) return fail(DFLASH_ERR_INVALID_ARG, "%s: out overlaps the workspace", who);
  a.c.n_pages = bounds->n_pages;
  a.c.page_size = bounds->page_size;
  a.c.n_kv_heads = bounds->n_kv_heads;
  a.c.head_dim = bounds->head_dim;
  a.c.per_page = FastDiv::make(bounds->page_size);
  a.codes = bounds->codes;
  a.scale = bounds->scale;
  a.q = static_cast<const uint16_t*>(q);
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.n_q_heads = n_q_heads;
  a.max_nodes = max_nodes;
  a.n_take = n_take;
  a.n_first = n_first;
  a.n_last = n_last;
  a.out = out;
  a.keys = static_cast<uint32_t*>(workspace);
  st = launch_status(launch_kv_select(a, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

size_t dflash_sparse_attention_workspace_size(const dflash_kv_cache* cache, int64_t n_rows, int32_t n_take,
                                              int32_t max_nodes, int32_t n_q_heads) {
  KvView c;
  if (view_cache(cache, c, "dflash_sparse_attention_workspace_size") != DFLASH_OK) return 0;
  ok();
  if (n_rows <= 0 || n_rows > kMaxItems / c.n_kv_heads || n_take < 0 || n_take > kMaxTake || n_q_heads < 1 ||
      n_q_heads % c.n_kv_heads || n_q_heads / c.n_kv_heads > kMaxGroup || max_nodes < 1 || max_nodes > kMaxNodes)
    return 0;
  return sparse_attention_bytes(c, n_rows, n_take, max_nodes, n_q_heads);
}

int dflash_sparse_attention(const dflash_kv_cache* cache, const dflash_kv_batch* batch, const void* q,
                            int64_t q_row_stride, int64_t q_head_stride, int32_t n_q_heads, const int32_t* blocks,
                            int32_t n_take, const uint64_t* mask, int32_t mask_words, int32_t max_nodes, float scale,
                            int32_t dtype, void* out, void* workspace, size_t workspace_bytes,
                            dflash_stream_t stream) {
  const char* who = "dflash_sparse_attention";
  SparseArgs a{};
  int st = view_cache(cache, a.c, who);
  if (st != DFLASH_OK) return st;
  if ((st = view_batch(batch, true, a.c, who)) != DFLASH_OK) return st;
  if ((st = check_dtype(dtype, who)) != DFLASH_OK || (st = check_heads(a.c.n_kv_heads, n_q_heads, who)) != DFLASH_OK ||
      (st = check_nodes(max_nodes, who)) != DFLASH_OK)
    return st;
  if (!std::isfinite(scale) || scale <= 0.f || scale > 0x1p100f)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: scale must be > 0 and at most 2^100", who);
  if (n_take < 0 || n_take > kMaxTake) return fail(DFLASH_ERR_INVALID_ARG, "%s: n_take must be in 0 .. %d", who, kMaxTake);
  if ((int64_t)n_take * a.c.page_size > (1 << 30))
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: n_take * page_size must be at most 2^30", who);
  if (a.c.n_req == 0 || a.c.n_rows == 0) return ok();   // a mask of no rows may be null
  if (a.c.n_rows > kMaxItems / a.c.n_kv_heads)
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: n_rows * n_kv_heads must be at most 2^21", who);
  if (mask ? mask_words < (max_nodes + 63) / 64 : mask_words != 0)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: mask_words must be >= ceil(max_nodes / 64) with a mask, 0 without", who);
  if (reinterpret_cast<uintptr_t>(mask) & 7) return fail(DFLASH_ERR_INVALID_ARG, "%s: mask must be 8-byte aligned", who);
  if (n_take > 0 && (!blocks || !aligned4(blocks)))
    return fail(DFLASH_ERR_INVALID_ARG, "%s: blocks must be a 4-byte aligned pointer", who);
  size_t qb = 0;
  if ((st = check_rows(q, q_row_stride, q_head_stride, a.c.n_rows, n_q_heads, a.c.head_dim, 2, qb, "q", who)) != DFLASH_OK)
    return st;
  if (!out || !aligned16(out)) return fail(DFLASH_ERR_INVALID_ARG, "%s: out must be a 16-byte aligned pointer", who);
  const size_t need = sparse_attention_bytes(a.c, a.c.n_rows, n_take, max_nodes, n_q_heads);
  if ((st = check_workspace(workspace, workspace_bytes, need, who)) != DFLASH_OK) return st;
  const size_t ob = (size_t)a.c.n_rows * n_q_heads * a.c.head_dim * 2, mb = mask ? (size_t)a.c.n_rows * mask_words * 8 : 0;
  const size_t bb = (size_t)a.c.n_rows * a.c.n_kv_heads * n_take * 4;
  const struct { const void* p; size_t bytes; const char* name; } written[] = {{out, ob, "out"}, {workspace, need, "the workspace"}};
  for (const auto& x : written)
    if (overlaps(x.p, x.bytes, q, qb) || meets_cache(a.c, x.p, x.bytes) || meets_batch(a.c, x.p, x.bytes) ||
        (mb && overlaps(x.p, x.bytes, mask, mb)) || (bb && overlaps(x.p, x.bytes, blocks, bb)))
      return fail(DFLASH_ERR_INVALID_ARG, "%s: %s overlaps q, the cache, the batch's arrays, the mask or the blocks", who, x.name);
  if (overlaps(out, ob, workspace, need)) return fail(DFLASH_ERR_INVALID_ARG, "%s: out overlaps the workspace", who);
  a.q = static_cast<const uint16_t*>(q);
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.n_q_heads = n_q_heads;
  a.blocks = blocks;
  a.n_take = n_take;
  a.mask = mask;
  a.mask_words = mask_words;
  a.max_nodes = max_nodes;
  a.scale = scale;
  a.out = static_cast<uint16_t*>(out);
  a.workspace = workspace;
  st = launch_status(launch_sparse_attention(a, as_hip(stream)), who);
  return st == DFLASH_OK ? ok() : st;
}

}  // extern "C"
