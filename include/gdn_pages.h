/*
 * gdn_pages.h -- C ABI of the page operators of a cache on one GB300 GPU:
 * giving pages to sequences, forking and freeing sequences, closing the holes
 * between live pages, and copying pages.  A page is one row of every buffer
 * of the cache: a state pool's row (gdn_prefill.h, gdn_linear.h), or a block
 * of a key/value cache's tokens, the same index in each layer's buffer.
 *
 * The bookkeeping (device memory, owned by the caller, dense):
 *   table      [max_seqs, max_pages] int32: the pages of a sequence, in
 *              order; -1 where it has none.  With max_pages = 1 a column of
 *              state indices.
 *   refcounts  [n_pages] int32: how many table entries name the page; 0: free
 *   lengths    [max_seqs] int32: tokens of a sequence (optional, see fork)
 * Lists of sequences are device memory too (int32); nothing is read on the
 * host, and nothing synchronises.
 *
 * Every choice is fixed: free pages are given out lowest first, in the order
 * of the list of sequences and then of the table's entries.
 *
 * Errors: host-checkable conditions are refused and nothing is launched.
 * What depends on device data sets bits of *device_status (optional), and the
 * entry at fault is skipped; the others are served as if it were not there:
 *   GDN_PAGES_ERR_SEQ        a sequence outside [0, max_seqs) or, in fork, a
 *                            parent that is its own child, or named twice in
 *                            a list whose entries have to differ (the first
 *                            is served)
 *   GDN_PAGES_ERR_CHILD      fork: the child still has pages
 *   GDN_PAGES_ERR_PAGE       a page outside [0, n_pages), a page that a
 *                            length calls for and the table lacks, a count
 *                            outside [0, max_pages], a page of refcount 0 freed
 *   GDN_PAGES_ERR_NO_PAGES   not enough free pages: the first sequence of the
 *                            list that does not fit and all after it get
 *                            nothing
 */
#ifndef GDN_PAGES_H
#define GDN_PAGES_H

#include "gdn_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    GDN_PAGES_ERR_SEQ = 1u << 8,
    GDN_PAGES_ERR_CHILD = 1u << 9,
    GDN_PAGES_ERR_PAGE = 1u << 10,
    GDN_PAGES_ERR_NO_PAGES = 1u << 11
};

#define GDN_PAGES_MAX_BUFFERS 128

/* One buffer: n_pages rows of row_bytes bytes, row_stride bytes apart. */
typedef struct gdn_pages_buffer {
    void *base;
    int64_t row_stride; /* >= row_bytes */
    int64_t row_bytes;  /* >= 0 */
} gdn_pages_buffer;

typedef struct gdn_pages_book {
    int32_t *table, *refcounts, *lengths; /* lengths may be NULL where it is not needed */
    int32_t max_seqs, max_pages, n_pages;
} gdn_pages_book;

/* Workspace (16-byte aligned device memory) that runs with these bounds need:
 * `list` sequences in a list.  A workspace serves one run at a time. */
size_t gdn_pages_workspace_bytes(int32_t max_seqs, int32_t max_pages, int32_t n_pages, int32_t list);

/* Entries 0 .. counts[k] - 1 of sequence seqs[k] that have no page get one.
 * rows [n, max_pages] (optional) receives the table rows of the list's
 * sequences (-1 for an entry at fault). */
gdn_status gdn_pages_reserve_run(const gdn_pages_book *book, const int32_t *seqs, const int32_t *counts, int32_t n,
                                 int32_t *rows, int32_t *device_status, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* children[k], which has no pages, becomes a copy of parents[k].
 *   page_tokens > 0: a page holds page_tokens tokens that do not change once
 *     written.  The ceil(lengths[parent] / page_tokens) pages in use are shared
 *     (refcount + 1), except a last page that is partly filled: the child gets
 *     a page of its own with a copy of it.  lengths is required.
 *   page_tokens = 0: pages are states that every step overwrites.  Each of
 *     the parent's pages is copied.
 * lengths[child] becomes lengths[parent] (0 when the child got nothing).
 * Parents are taken as they are before the call; a parent may be named more
 * than once. */
gdn_status gdn_pages_fork_run(const gdn_pages_book *book, const gdn_pages_buffer *buffers, int32_t n_buffers,
                              const int32_t *parents, const int32_t *children, int32_t n, int32_t page_tokens,
                              int32_t *rows, int32_t *device_status, void *workspace, size_t workspace_bytes,
                              void *stream);

/* The sequences' pages lose a reference each; their table entries become -1,
 * their lengths 0.  A sequence named twice is freed once. */
gdn_status gdn_pages_free_run(const gdn_pages_book *book, const int32_t *seqs, int32_t n, int32_t *device_status,
                              void *stream);

/* With L live pages (refcount > 0), the live pages at or past L move, in
 * order, into the free pages below L, in order.  remap [n_pages] receives each
 * page's new index (-1 for a free page), n_live [1] receives L.  table_out and
 * refcounts_out receive the new bookkeeping and may be the book's own: with
 * other buffers the old bookkeeping stays valid until the caller changes over,
 * since only pages that were free are written.  Table entries outside
 * [0, n_pages), or naming a free page, become -1 (the former but -1 with
 * GDN_PAGES_ERR_PAGE). */
gdn_status gdn_pages_compact_run(const gdn_pages_book *book, const gdn_pages_buffer *buffers, int32_t n_buffers,
                                 int32_t *table_out, int32_t *refcounts_out, int32_t *remap, int32_t *n_live,
                                 int32_t *device_status, void *workspace, size_t workspace_bytes, void *stream);

/* Row src[i] of every source buffer to row dst[i] of the destination buffer
 * of the same place, for the n pairs of the lists; pairs with a negative
 * index are skipped, pairs out of range set GDN_PAGES_ERR_PAGE.  No row is
 * named twice in dst, and no row is both read and written (rows that are race
 * on their content). */
gdn_status gdn_pages_copy_run(const gdn_pages_buffer *src_buffers, int32_t src_pages, const gdn_pages_buffer *dst_buffers,
                              int32_t dst_pages, int32_t n_buffers, const int32_t *src, const int32_t *dst, int32_t n,
                              int32_t *device_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_PAGES_H */
