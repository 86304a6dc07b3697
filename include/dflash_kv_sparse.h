/*
 * dflash_kv_sparse.h -- attention over a few pages of a long paged KV cache
 * (dflash_kv.h), which a cheap score chooses for each query.
 *
 *   dflash_kv_bounds        what the score reads of each page that is full
 *   dflash_kv_select        the pages of each query row and kv head
 *   dflash_sparse_attention attention over these, the rest of the prefix
 *                           behind the last full page, and the row's tree
 *
 * The conventions of dflash_kv.h hold, its caches, batches and page tables
 * too.  Request r has a prefix of start[r] positions, of which
 * B = floor(start[r] / page_size) pages are full: blocks 0 .. B - 1, block b in
 * page page_table[r][b].  The batch's rows are the nodes behind the prefix, as
 * in dflash_tree_attention: a block of drafted tokens, or one new token.
 */
#ifndef DFLASH_KV_SPARSE_H
#define DFLASH_KV_SPARSE_H

#include "dflash_kv.h"
#include "dflash_kv_pages.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * dflash_kv_bounds -- for every page that positions start[r] .. end[r] - 1 fill
 * up (blocks floor(start / page_size) .. floor(end / page_size) - 1) and every
 * kv head: the least and the greatest key of each channel, as the cache holds
 * them (codes times scales), rounded outwards to 8 bits:
 *   e = the smallest integer >= -100 with max |k| * 2^-e <= 127;
 *   scale byte = e + 127;  codes[0] = floor(least * 2^-e);
 *   codes[1] = ceil(greatest * 2^-e).
 * Every step is exact, so the bounds are a function of the keys alone.  A page
 * head with a key that is an infinity or a NaN gets scale byte 255, codes 0.
 * Call it once the positions are final: after dflash_kv_write of a prompt,
 * after dflash_kv_commit of accepted nodes (start: the length before, end:
 * after).
 *   start, end   [n_req]; of the batch page_table, table_stride, table_width,
 *                n_req and start are used.  Requests with end <= start, and
 *                blocks beyond the table or with pages outside the pool, have
 *                nothing done for them.
 *   bounds       of the cache's pages and heads; may not overlap the cache or
 *                the batch's arrays
 *   n_req        at most 2^20
 * Pages that two requests share may be given by both: they write the same. */
int dflash_kv_bounds(const dflash_kv_cache* cache, const dflash_page_bounds* bounds, const dflash_kv_batch* batch,
                     const int32_t* end, dflash_stream_t stream);

/* ---------------------------------------------------------------------------
 * dflash_kv_select -- for every row i and kv head g the blocks that may matter
 * most to it.  With the row's queries of the group's heads in 8 bits,
 *   e_q = the smallest integer >= -100 with max |q| * 2^-e_q <= 127 over the
 *   group,  c = q * 2^-e_q rounded to the nearest integer, ties to even
 * (all 0 where one of them is an infinity or a NaN), block b's score is
 *   2^(scale byte - 127) * max over the group's heads of
 *       sum over d of c_d * (c_d > 0 ? codes[1][d] : codes[0][d]):
 * no product of c with a key of the block is above it.  The sums are whole
 * numbers and the score is exact, so that the choice does not depend on how it
 * was computed.
 * The first n_first blocks and the last n_last are taken always (a block in
 * both once), then blocks with scale byte 255 or without a page in the pool
 * (attention has to see what is wrong there), then the highest scores; ties go
 * to the lower block.
 *   q     bf16, row i, head h at q + i * q_row_stride + h * q_head_stride
 *         (elements); pointer and strides multiples of 16 bytes
 *   out   int32 [n_rows, n_kv_heads, n_take]: the blocks in ascending order,
 *         -1 behind them where there are fewer than n_take.  Rows of the
 *         padding, and of a request beyond max_nodes, are left as they were.
 *         May not overlap q, the bounds, the batch's arrays or the workspace.
 *   n_take  1 .. 65536, n_first and n_last >= 0 with n_first + n_last <= n_take
 *   max_nodes  1 .. 4096: no request has more rows
 *   n_q_heads  a multiple of n_kv_heads, up to 64 query heads to a kv head
 * A request whose start is below 0 has no blocks, one whose start is beyond the
 * table's positions as many as the table holds.  Scale bytes below 25, which
 * dflash_kv_bounds does not write, count as 25.
 * n_rows * n_kv_heads is at most 2^21, table_width at most 2^24.
 * Scratch: dflash_kv_select_workspace_size() bytes, 256-byte aligned; it never
 * falls with n_rows or table_width; calls that may run at the same time need
 * one each. */
size_t dflash_kv_select_workspace_size(const dflash_page_bounds* bounds, int64_t n_rows, int32_t table_width);
int dflash_kv_select(const dflash_page_bounds* bounds, const dflash_kv_batch* batch, const void* q,
                     int64_t q_row_stride, int64_t q_head_stride, int32_t n_q_heads, int32_t max_nodes, int32_t n_take,
                     int32_t n_first, int32_t n_last, int32_t dtype, int32_t* out, void* workspace,
                     size_t workspace_bytes, dflash_stream_t stream);

/* ---------------------------------------------------------------------------
 * dflash_sparse_attention -- dflash_tree_attention over part of the prefix: row
 * i sees, for the heads of kv head g, the positions of the blocks
 * blocks[i][g][0 .. n_take), the prefix's positions from B * page_size on, and
 * the nodes of its request that its mask names (mask NULL: a chain).  With all
 * blocks 0 .. B - 1 it is dflash_tree_attention.
 *   blocks  int32 [n_rows, n_kv_heads, n_take], 4-byte aligned, in ascending
 *           order as dflash_kv_select leaves them: an entry below 0 or from B
 *           on, or not above the entry before it, names nothing (so that a list
 *           that falls and rises again may not name a block twice: it may then
 *           count once or twice).  n_take 0 .. 65536 (0: blocks is not looked at)
 *   q, mask, out, max_nodes, scale   as for dflash_tree_attention
 * A row that sees nothing gets zeros.  What a row does not see has no effect on
 * it, whatever values the cache holds there, but for the last bits: the nodes of
 * a request are taken together.  Positions without a page in the pool make the
 * rows that see them NaN; a length (start plus nodes) beyond the table makes all
 * rows of its request NaN that see anything.
 * Arithmetic: as for dflash_tree_attention.  A NaN among the keys that a row sees
 * makes its result NaN; an infinity or a NaN among the values makes it an
 * infinity or a NaN in that channel.  A key with an infinity has the score that
 * the product gives it: at -infinity its weight is 0 (a row whose keys all have
 * that is NaN), at +infinity the row is NaN.  A call's result is the same every
 * time; its sums are split by the whole batch, so a request may differ in the
 * last bits from one batch to another.
 *   max_nodes also decides whether the nodes of a request are taken together:
 *           give the batch's own largest number, 1 for plain decoding.
 * n_rows * n_kv_heads is at most 2^21, n_take * page_size at most 2^30.
 * Scratch: dflash_sparse_attention_workspace_size() bytes, 256-byte aligned; it
 * never falls with n_rows, n_take, max_nodes or n_q_heads; it may not overlap
 * anything else of the call, and calls that may run at the same time need one
 * each. */
size_t dflash_sparse_attention_workspace_size(const dflash_kv_cache* cache, int64_t n_rows, int32_t n_take,
                                              int32_t max_nodes, int32_t n_q_heads);
int dflash_sparse_attention(const dflash_kv_cache* cache, const dflash_kv_batch* batch, const void* q,
                            int64_t q_row_stride, int64_t q_head_stride, int32_t n_q_heads, const int32_t* blocks,
                            int32_t n_take, const uint64_t* mask, int32_t mask_words, int32_t max_nodes, float scale,
                            int32_t dtype, void* out, void* workspace, size_t workspace_bytes,
                            dflash_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_KV_SPARSE_H */
