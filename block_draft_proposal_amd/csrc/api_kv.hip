// C ABI of the paged KV cache and the draft-tree attention (dflash_kv.h):
// host-side validation and launches.
#include <cmath>

#include "api_kv_common.h"

namespace {

using namespace dflash;

constexpr int kMaxGroup = 64, kMaxNodes = 4096;

// A thread holds 8 elements of a row in the write and the read.
int check_stream(const KvView& v, const char* who) {
  if (v.n_rows > kMaxThreads / (v.head_dim / 8))
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: n_rows * head_dim must be below 2^35", who);
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
