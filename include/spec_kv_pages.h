/*
 * spec_kv_pages.h -- who holds the pages of the paged key/value cache of spec_kv.h
 * (libspecverify.so, CUDA kernels for sm_103a).
 *
 * The lengths of the sequences are known on the device: verification says how many
 * tokens it kept.  So that pages can follow them without the host, each page has a
 * count of the table entries that hold it:
 *
 *   spec_kv_hold  gives every sequence the pages that its tokens need and takes away
 *                 the others: before a round (for the tokens that come, and with what
 *                 left a window), after one (what was rejected), at a sequence's
 *                 end (everything).
 *   spec_kv_fork  makes some sequences copies of others: whole pages are shared, the
 *                 last, partly filled one is copied.
 *
 * Conventions: those of spec_verify.h, without a workspace.  What one call does goes by
 * the inputs alone, not by timing.  Calls that share counts must not overlap in time on
 * the GPU.  The table's entries (rows count up to the next 128, those of more than 128 up
 * to the next 512) and the pool's pages are tracked in one cluster's shared memory, a bit
 * each: beyond some 14 million together (7 million where the device has no room for a
 * cluster of 16 CTAs) a call is SPEC_ERR_UNSUPPORTED.  Tables of that size are held by the
 * host.
 *
 * Counts.  refs[p] is the number of table entries that hold page p; 0 (or less): the
 * page is free.  All zero, with a table of -1, is an empty pool.  A caller may count
 * entries of his own, to keep pages out of use.  An entry of the table is a page or
 * negative: none.  A sequence writes to the page of its last token only where it alone
 * holds it, which spec_kv_fork sees to: a sequence is not cut back to fewer tokens than
 * it had when it was forked, or became a fork, and then appended to.
 */
#ifndef SPEC_KV_PAGES_H
#define SPEC_KV_PAGES_H

#include "spec_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t num_pages;         /* pages of the pool, >= 1 */
  int32_t page_size;         /* token slots a page: 16, 32, 64 or 128 */
  int32_t B;                 /* sequences, >= 0 */
  int32_t max_pages;         /* columns of the page table, >= 1 */
  int32_t* refs;             /* device [num_pages] */
  int32_t* page_table;       /* device [B, max_pages], rows table_stride (>= max_pages) apart */
  int64_t table_stride;
  int32_t* free_pages;       /* optional device int32[1]: free pages after the call */
  void* stream;              /* cudaStream_t */
  int32_t* status;           /* optional device int32[1]: first device-detected error */
} spec_kv_pages;

/* Give each sequence exactly the pages that it needs.
 *   seq_lens  device [B]: tokens stored, >= 0
 *   new_lens  device [B]: tokens to come, >= 0; NULL = T each
 *   window    > 0: queries of the tokens to come see that many tokens, their own
 *             included; 0: all before them
 *   sinks     first tokens that they see beside the window
 * A sequence of L tokens with n to come needs the pages of positions below L + n, of
 * those before L + 1 - window only where a position below `sinks` lies in them.  Other
 * entries of its row become -1 and what they held is counted down; then the entries that
 * it needs and that are negative, sequence by sequence and page by page, get the
 * lowest-numbered free pages, each counted once (the pages released by this call among
 * them).  What a page holds stays as it is.
 * Device errors: a sequence whose lengths are out of range (negative, or beyond
 * max_pages pages) is left as it is, and so is an entry that it needs and that is no
 * page of the pool: SPEC_ERR_CACHE_RANGE.  Where free pages run out, the entries that
 * come last stay negative: SPEC_ERR_CACHE_FULL. */
spec_status spec_kv_hold(const spec_kv_pages* pages, const int32_t* seq_lens, const int32_t* new_lens, int32_t T,
                         int32_t window, int32_t sinks);

/* Make sequences copies of others.
 *   cache     the pool, of as many pages of the same size
 *   seq_lens  device [B]: tokens stored; a copy gets its parent's
 *   parents   device [B]: the sequence that b becomes a copy of; -1 or b: it stays
 * A parent is a sequence that stays.  The row of a copy becomes its parent's: entries of
 * pages that the parent's tokens fill are shared and counted, the last one that they do
 * not fill is replaced by a free page, to which the filled slots and the scales are
 * copied (free pages are taken as by spec_kv_hold, sequence by sequence), and the others
 * are -1.  What the row held is counted down, and may be taken by the same call.
 * Device errors: a copy whose parent is none of the sequences, does not stay or has a
 * length out of range stays as it is; an entry of a parent that is beyond the pool, and
 * one of its last page that is negative, becomes -1 in the copy (negative ones of whole
 * pages do without an error): SPEC_ERR_CACHE_RANGE.  Where free pages run out, the entry
 * of the last page is -1: SPEC_ERR_CACHE_FULL. */
spec_status spec_kv_fork(const spec_kv_pages* pages, const spec_kv_cache* cache, int32_t* seq_lens,
                         const int32_t* parents);

#ifdef __cplusplus
}
#endif

#endif
