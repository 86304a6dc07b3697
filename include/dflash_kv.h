/*
 * dflash_kv.h -- the paged KV cache beside the draft-block path and the
 * attention of drafted nodes over it: what the target's (or the drafter's)
 * pass over a drafted block needs between dflash_propose_block and
 * dflash_verify.
 *
 *   dflash_kv_write       rows of K and V into the cache, quantised on the way
 *   dflash_kv_read        ranges of positions back in bf16 or fp32
 *   dflash_tree_attention every drafted node over the prefix and its tree
 *   dflash_kv_commit      the accepted path's rows moved behind the prefix
 *
 * The conventions of dflash.h hold: device pointers unless marked "host",
 * caller-owned buffers, no allocation and no host synchronisation inside a
 * call, everything checked on the host before anything is enqueued, status
 * codes and dflash_last_error().  The device of `stream` must be current.
 * The structs below are host structs; they are read before the call returns.
 *
 * The cache.  n_pages pages; page p holds, for each kv head, page_size rows
 * of head_dim elements of K at
 *     k + p * page_stride + (head * page_size + slot) * head_dim
 * and of V likewise.  A row is bf16, or 8 bits an element with one scale byte
 * per (token, kv head) at
 *     k_scale + p * scale_page_stride + head * page_size + slot.
 * A scale byte b stands for 2^(b - 127) (b = 255: NaN).  Powers of two make
 * the scaling exact: an element is rounded once, to its 8-bit code, and
 * code * scale is exact in bf16 and fp32.  Position t of request r lies in
 * page page_table[r][t / page_size], slot t % page_size.
 *
 * Page tables, lengths and offsets are device data and cannot be checked on
 * the host.  A position whose page index lies outside the table's width, or
 * whose page lies outside [0, n_pages), touches no memory: it is not written,
 * reads as NaN, and makes the attention rows of its request NaN (but for rows
 * that see nothing, which are zeros).  So do lengths beyond 2^31 - 2^17.
 */
#ifndef DFLASH_KV_H
#define DFLASH_KV_H

#include "dflash.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit element types of a cache, beside DFLASH_BF16: OCP e4m3 (finite up to
 * 448, no infinities) and signed integers in [-127, 127]. */
enum { DFLASH_E4M3 = 2, DFLASH_I8 = 3 };

typedef struct {
  void* k;                    /* 16-byte aligned */
  void* v;                    /* 16-byte aligned */
  uint8_t* k_scale;           /* NULL for DFLASH_BF16 */
  uint8_t* v_scale;           /* NULL for DFLASH_BF16 */
  int64_t page_stride;        /* elements from a page to the next, K and V alike; >= n_kv_heads * page_size *
                                 head_dim, a multiple of 16 bytes */
  int64_t scale_page_stride;  /* bytes; >= n_kv_heads * page_size (8-bit caches) */
  int64_t n_pages;            /* 1 .. 2^31 - 1 */
  int32_t page_size;          /* 1 .. 65536, a power of two or not */
  int32_t n_kv_heads;         /* 1 .. 1024 */
  int32_t head_dim;           /* 64, 128 or 256 */
  int32_t dtype;              /* DFLASH_BF16, DFLASH_E4M3 or DFLASH_I8 */
} dflash_kv_cache;

/* A ragged batch: rows offsets[r] .. offsets[r+1]-1 of the call's tensors
 * belong to request r, and row offsets[r] + i is its position start[r] + i.
 * offsets ascend; rows from offsets[n_req] up to n_rows (padding) are neither
 * read nor written.  A request without rows costs a step of a walk from its
 * neighbours: long runs of them (tens of thousands) are better left out. */
typedef struct {
  const int32_t* page_table;  /* row r at page_table + r * table_stride, table_width entries */
  int64_t table_stride;       /* elements, >= table_width */
  int32_t table_width;        /* >= 1 */
  int32_t n_req;              /* >= 0 */
  const int32_t* start;       /* [n_req], >= 0: positions in the cache before the batch's rows */
  const int32_t* offsets;     /* [n_req + 1] */
  int64_t n_rows;             /* rows of the call's tensors, < 2^31 */
} dflash_kv_batch;

/* ---------------------------------------------------------------------------
 * dflash_kv_write -- stores K and V rows at their positions.
 *   bf16 cache:  the element rounded to bf16 (nearest, ties to even).
 *   8-bit cache: per (row, kv head), amax = max |x| over head_dim;
 *     e = the smallest integer >= -100 with amax * 2^-e <= top
 *     (448 for e4m3, 127 for int8);  scale byte = e + 127;
 *     code = x * 2^-e rounded once (nearest, ties to even).
 *     A row that holds an infinity or a NaN gets scale byte 255 and codes 0,
 *     so that it reads back as NaN.
 *     Above 2^127 a row's largest values may round to a code that reads back
 *     beyond the range, as an infinity.
 *   k, v  row i, kv head h at k + i * k_row_stride + h * k_head_stride (strides
 *         in elements), head_dim contiguous elements of `dtype` (DFLASH_BF16
 *         or DFLASH_F32); pointers and strides multiples of 16 bytes; they may
 *         not overlap the cache.
 * n_rows * head_dim is below 2^35 (here and in dflash_kv_read).
 * No two of the cache's k, v, k_scale and v_scale may share memory (here and
 * in dflash_kv_commit; the read and the attention take it).  They may lie in
 * each other's gaps, as in one pool whose pages hold all four, if they then
 * have one page stride in bytes.
 * Positions written by one call must be distinct rows of the cache: requests
 * may share pages that they only read, not pages that they write. */
int dflash_kv_write(const dflash_kv_cache* cache, const dflash_kv_batch* batch, const void* k, int64_t k_row_stride,
                    int64_t k_head_stride, const void* v, int64_t v_row_stride, int64_t v_head_stride, int32_t dtype,
                    dflash_stream_t stream);

/* ---------------------------------------------------------------------------
 * dflash_kv_read -- the inverse: row offsets[r] + i of k_out and v_out takes
 * the values at position start[r] + i (bf16 and fp32 alike exact, except that
 * a bf16 result of magnitude below 2^-126 is rounded).
 *   k_out, v_out  [n_rows, n_kv_heads, head_dim] contiguous, dtype DFLASH_BF16
 *                 or DFLASH_F32, 16-byte aligned; they may not overlap the
 *                 cache, each other or the batch's arrays. */
int dflash_kv_read(const dflash_kv_cache* cache, const dflash_kv_batch* batch, void* k_out, void* v_out,
                   int32_t dtype, dflash_stream_t stream);

/* ---------------------------------------------------------------------------
 * dflash_kv_commit -- moves the accepted nodes of each request's tree behind
 * its prefix:
 *   for i < path_lens[r]:  position start[r] + paths[r][i]  ->  start[r] + i
 * Codes and scales are copied as they are.  A path ascends (a node is drafted
 * after its parent), paths[r][i] >= i, so the move works in place.  An entry
 * below i is skipped, and so is one whose source or destination position lies
 * outside the table or the pool.
 *   paths      row r at paths + r * path_stride, path_width entries
 *   path_lens  [n_req]; lengths beyond path_width count as path_width
 * Only page_table, table_stride, table_width, start and n_req of the batch
 * are used; n_req * n_kv_heads is below 2^25.  Pages moved by one call may not
 * be shared between requests. */
int dflash_kv_commit(const dflash_kv_cache* cache, const dflash_kv_batch* batch, const int32_t* paths,
                     int64_t path_stride, int32_t path_width, const int32_t* path_lens, dflash_stream_t stream);

/* ---------------------------------------------------------------------------
 * dflash_tree_attention -- attention of the drafted nodes.  Request r has a
 * prefix of start[r] positions and n = offsets[r+1] - offsets[r] nodes, whose
 * K and V are in the cache at positions start[r] .. start[r] + n - 1
 * (dflash_kv_write puts them there).  For node i and query head h, with kv
 * head g = h / (n_q_heads / n_kv_heads):
 *   out[i,h] = sum_j w_j v[j,g],  w = softmax_j( scale * <q[i,h], k[j,g]> )
 * over the positions j that node i sees: the whole prefix, and node j when bit
 * j % 64 of mask[i][j / 64] is set (mask NULL: a chain, every node j <= i).
 * Bits from n on are ignored.  A node that sees nothing gets zeros.  What it
 * does not see has no effect on it, whatever values the cache holds there.
 *   q     row i, head h at q + i * q_row_stride + h * q_head_stride (elements),
 *         bf16; pointer and strides multiples of 16 bytes
 *   mask  uint64 [n_rows, mask_words], bit j of word w is node 64 w + j;
 *         mask_words >= ceil(max_nodes / 64); or NULL with mask_words 0
 *         (neither is looked at in a call without rows or requests)
 *   out   bf16 [n_rows, n_q_heads, head_dim] contiguous, 16-byte aligned; may
 *         not overlap q, mask, the batch's arrays or the cache
 *   max_nodes  1 .. 4096: no request has more nodes (rows of a request beyond
 *         it are left as they were).  It also chooses how many of a kv head's
 *         rows a workgroup takes: give the batch's own largest number, not the
 *         largest ever.  32 rows in a form for 256 take 1.8 times their time.
 *   scale > 0, at most 2^100
 * n_q_heads is a multiple of n_kv_heads, up to 64 query heads to a kv head.
 * Arithmetic: products exact in fp32, sums, maximum and softmax in fp32; the
 * weights are rounded to bf16 for the product with V, the result once to bf16.
 * The sums keep weights up to 2^8, so |v| * positions, and the scale of any V
 * row, have to stay below 2^119, and scale * |<q, k>|, and scale times the scale
 * of any K row, below 2^126: beyond, a result may be an infinity or a NaN.  So
 * may one that an infinity of the prefix has a part in.  A call's result is the same every
 * time; its sums are split by the lengths of the whole batch, so a request
 * may differ in the last bits from one batch to another.
 * Scratch: dflash_tree_attention_workspace_size() bytes, 256-byte aligned; it
 * does not depend on the lengths, so one workspace serves a growing cache, and
 * never falls with max_nodes, n_req or n_q_heads, so one for the largest values
 * serves every call on the cache.
 * It may not overlap q, out, mask, the batch's arrays or the cache, and calls
 * that may run at the same time need one each. */
size_t dflash_tree_attention_workspace_size(const dflash_kv_cache* cache, int32_t n_req, int32_t max_nodes,
                                            int32_t n_q_heads);
int dflash_tree_attention(const dflash_kv_cache* cache, const dflash_kv_batch* batch, const void* q,
                          int64_t q_row_stride, int64_t q_head_stride, int32_t n_q_heads, const uint64_t* mask,
                          int32_t mask_words, int32_t max_nodes, float scale, int32_t dtype, void* out,
                          void* workspace, size_t workspace_bytes, dflash_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_KV_H */
