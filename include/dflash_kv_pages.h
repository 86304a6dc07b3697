/*
 * dflash_kv_pages.h -- who holds which pages of a paged KV cache
 * (dflash_kv.h): requests that grow, shrink, end, share a prefix and part
 * again, and a pool that is packed.
 *
 *   dflash_kv_resize      requests take free pages or let theirs go
 *   dflash_kv_fork        requests become copies of others, sharing their pages
 *   dflash_kv_compact     the pool's top pages move to the free ones below
 *   dflash_kv_copy_pages  the contents of the pages that the others name
 *
 * The first three are planning: they read and write tables, lengths and
 * counts, which all layers' caches share, and name the pages whose contents
 * have to move; dflash_kv_copy_pages then does that for each layer's cache,
 * on the same stream, before its pages are written again.
 *
 * The conventions of dflash_kv.h hold: device pointers, no allocation and no
 * host synchronisation inside a call, everything that the host can see
 * checked before anything is enqueued, and the device of `stream` current.
 * Results do not depend on the order in which anything runs.
 *
 * A page p is free where refs[p] is 0, held by refs[p] requests where it is
 * above, and never given or moved where it is below.  The counts are the
 * caller's to begin with (zeros, and empty rows) and have to fit the tables; a
 * call keeps them so.  Request r holds the
 * first ceil(lens[r] / page_size) entries of its row of page_table.  What lies
 * behind them is not read (resize, fork: entries that a call adds are written,
 * those that it takes off become -1).  Entries outside [0, n_pages) hold
 * nothing; a request may hold a page once.  A request whose length is below 0
 * or beyond the table is left alone.
 *
 * Pages whose holder is no request of the call (a cache of prompts) are kept
 * by a count of their own: refs[p] raised by one.
 */
#ifndef DFLASH_KV_PAGES_H
#define DFLASH_KV_PAGES_H

#include "dflash_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t* refs;        /* [n_pages] */
  int64_t n_pages;      /* 1 .. 2^30 */
  int32_t page_size;    /* 1 .. 65536 */
} dflash_kv_pool;

/* What dflash_kv_sparse.h keeps of each full page; it moves with the page. */
typedef struct {
  int8_t* codes;        /* [n_pages][n_kv_heads][2][head_dim], 16-byte aligned */
  uint8_t* scale;       /* [n_pages][n_kv_heads] */
  int64_t n_pages;
  int32_t page_size, n_kv_heads, head_dim;
} dflash_page_bounds;

/* All requests that hold pages of the pool. */
typedef struct {
  int32_t* page_table;  /* row r at page_table + r * table_stride, table_width entries */
  int64_t table_stride; /* elements, >= table_width */
  int32_t table_width;  /* >= 1 */
  int32_t n_req;        /* 0 .. 2^20 */
  int32_t* lens;        /* [n_req] positions that each request has */
} dflash_kv_rows;

/* Scratch of dflash_kv_resize, dflash_kv_fork and dflash_kv_compact alike, at
 * a 256-byte aligned address.  It never falls with n_req or table_width.  One
 * serves calls that follow one another; calls that may run at the same time
 * need one each.  0 for sizes that the calls refuse. */
size_t dflash_kv_pages_workspace_size(const dflash_kv_pool* pool, int32_t n_req, int32_t table_width);

/* ---------------------------------------------------------------------------
 * dflash_kv_resize -- lens[r] becomes want[r].
 *   A request that shrinks lets its last pages go: their counts fall by one,
 *   their entries become -1.
 *   One that grows takes a free page (count 1) for each entry that it lacks.
 *   Where its last page is partly filled (lens[r] is no multiple of page_size)
 *   and has other holders, it takes one more page, which takes that entry, and
 *   the old page's count falls by one: the copy that it can write to.  Should
 *   all holders of such a page grow in one call, the first of them keeps it.
 *   copies[i] = (old page, new page), in the order of the requests.
 * Pages let go by a call are free within it.  Free pages are given lowest
 * first, to the requests in order, the copy's before the rest.  If there are
 * too few of them, nobody grows (what shrinks, shrinks) and lens shows it.
 *   want    [n_req]; a request whose want is below 0 or beyond
 *           table_width * page_size (or 2^31 - 1) is left alone
 *   copies  [n_req][2]; entries from counts[0] on are left as they were
 *   counts  [2]: the number of copies, and of free pages that were missing */
int dflash_kv_resize(const dflash_kv_pool* pool, const dflash_kv_rows* rows, const int32_t* want, int32_t* copies,
                     int32_t* counts, void* workspace, size_t workspace_bytes, dflash_stream_t stream);

/* ---------------------------------------------------------------------------
 * dflash_kv_fork -- all at once, row r of page_table and lens[r] become what
 * row parents[r] and its length were.  The pages that r held are let go, those
 * that it holds now are counted once more: a prompt's samples, or the beams
 * that a step of beam search goes on with.  parents[r] == r changes nothing,
 * parents[r] < 0 empties the row, and rows with parents[r] >= n_req, or whose
 * parent's length is out of range, are left as they were.
 * A row of a length out of range that gets a parent is taken to hold nothing.
 * No contents move: a partly filled page that two requests now hold is copied
 * by the dflash_kv_resize that lets one of them grow. */
int dflash_kv_fork(const dflash_kv_pool* pool, const dflash_kv_rows* rows, const int32_t* parents, void* workspace,
                   size_t workspace_bytes, dflash_stream_t stream);

/* ---------------------------------------------------------------------------
 * dflash_kv_compact -- the highest held page (count above 0) moves to the
 * lowest free one, the next to the next, while the held page lies above the
 * free one and at most max_copies times: with max_copies >= n_pages / 2 the
 * held pages end up packed at the bottom (but for pages with counts below 0,
 * which stay), with less the call takes a bounded time and the next goes on.
 *   page_map  [n_pages]: the page that page p's holders find it at now (p where
 *             it did not move, -1 where it was free): for holders that are no
 *             request of the call.  The call rewrites its own tables.
 *   copies    [max_copies][2] = (old page, new page); entries from counts[0] on
 *             are left as they were
 *   counts    [2]: the number of copies, and of held pages */
int dflash_kv_compact(const dflash_kv_pool* pool, const dflash_kv_rows* rows, int32_t* page_map, int32_t* copies,
                      int64_t max_copies, int32_t* counts, void* workspace, size_t workspace_bytes,
                      dflash_stream_t stream);

/* ---------------------------------------------------------------------------
 * dflash_kv_copy_pages -- page copies[i][1] of the cache becomes a copy of page
 * copies[i][0] (codes and scales as they are) for i < n, n = counts[0], at most
 * max_copies (counts NULL: n = max_copies).  Pairs with a page outside
 * [0, n_pages), or of a page with itself, are skipped.  No page may be the
 * target of two pairs, or target and source; the lists of dflash_kv_resize and
 * dflash_kv_compact have none such.
 * bounds: NULL, or of the same pages and heads as the cache, copied along.
 * No two of the cache's k, v, k_scale and v_scale and the bounds may share
 * memory, nor may copies or counts with them. */
int dflash_kv_copy_pages(const dflash_kv_cache* cache, const dflash_page_bounds* bounds, const int32_t* copies,
                         int64_t max_copies, const int32_t* counts, dflash_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_KV_PAGES_H */
