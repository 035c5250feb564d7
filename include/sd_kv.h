/*
 * sd_kv.h — C ABI of the pages of a paged KV cache that rows share: forking
 * and extending block tables, giving pages back, copying pages, and moving
 * the pages in use to the front of the pool.  sd_kv_rollback of sd_verify.h
 * truncates the same tables.
 *
 * A pool has N pages of page_size entries.  refs [N] counts the table entries
 * (of whatever tables) that hold each page; a page of count 0 is free.  A
 * block table [rows][max_pages] lists the pages of each row (int32 ids, -1:
 * none), kv_len [rows] how many entries it holds (taken into
 * [0, max_pages page_size]).  Rows share full pages; a row that is to be
 * written must hold its last, partly filled page alone, which sd_kv_fork sees
 * to.  No call reads or writes a page's contents but sd_kv_copy.
 *
 * Conventions are those of sd_verify.h: every call is stream-ordered and
 * asynchronous, checks its arguments on the host, allocates nothing and keeps
 * no pointer; pointers are device pointers owned by the caller unless marked
 * "host"; data errors set bits in the optional *status word.  Results do not
 * depend on the order in which the GPU's threads run.
 */
#ifndef SD_KV_H_
#define SD_KV_H_

#include "sd_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of *status. */
#define SD_STATUS_BAD_PARENT 0x10u /* a parent outside the rows it may name   */
#define SD_STATUS_BAD_PAGE 0x20u /* a page id outside [0, N), none where a row
                                    needs one, or a page given back that
                                    nobody holds                              */
#define SD_STATUS_NO_PAGE 0x40u  /* a page was needed and none was free, or a
                                    row is longer than its table              */

#define SD_MAX_ROWS 16384     /* rows of a block table in sd_kv_fork          */
#define SD_MAX_PAGES (1 << 24) /* pages of a pool                             */
#define SD_MAX_CACHES 256     /* cache tensors of one sd_kv_copy call         */

/*
 * New rows from old ones: new row r holds the entries of old row p =
 * parents[r] (n = kv_len[p] of them) and room for `append` more.
 *   Full pages of p are shared.  A partly filled last page goes to r in one
 * of two ways: r's own page (and a pair in src, dst, fill: page src's first
 * `fill` entries are to be copied to page dst), or p's page itself where r is
 * p's heir and refs of that page is 1.  The heir of p, where the old rows end
 * with the call (keep = 0), is the lowest r whose parent it is: it takes p's
 * row over as it is, pages beyond its length included.  The other slots up to
 * ceil((n + append) / page_size) get pages, the ones beyond are -1.
 *   Pages are taken in the order of rows, then slots: the i-th that is needed
 * is the i-th free page by id, as refs were before the call.  Where none is
 * left the slot becomes -1 and SD_STATUS_NO_PAGE is set (the pair of such a
 * copy is -1, -1), but an heir keeps the page that it could not copy, shared as
 * it was: no row that goes on loses entries.  A later call in place
 * (sd_kv_extend) takes the pages that were missing, that copy's among them;
 * until then such a row must not be written.  Other rows whose last page
 * could not be copied are to be forked again.  NO_PAGE is set too where
 * n + append passes the table, which then bounds it.
 *   refs: + 1 for each slot that holds a page anew; old rows that end without
 * an heir give their pages back, and an heir gives back a page that it
 * copied.  Ids outside [0, N), pages that were free before the call (rows
 * that were given back and not cleared name such), and pages given back more
 * often than they are then held set SD_STATUS_BAD_PAGE; counts end at 0, and a
 * page that the call handed out stays held.
 *   A parent of -1 (or, with SD_STATUS_BAD_PARENT, one outside the rows) makes
 * an empty row.  Slots within a row's length that hold no page id are passed
 * on and set SD_STATUS_BAD_PAGE.
 *   groups > 0: parents are relative to their group; R and rows_in are
 * multiples of it, and row r's group starts at old row
 * (r / (R / groups)) (rows_in / groups).
 *   src, dst, fill [R]: the pairs in the order of rows, -1, -1, 0 after the
 * last; count [1]: how many.
 *   parents null (R = rows_in, table_out = table, len_out null, keep = 0):
 * the rows go on in place, each as its own heir: sd_kv_extend.
 * Otherwise table_out and len_out must not overlap table and kv_len.
 * R, rows_in <= SD_MAX_ROWS; N <= SD_MAX_PAGES; max_pages page_size and
 * max_pages R below 2^31.  workspace: at least
 * sd_kv_fork_workspace_size bytes, 16-byte aligned; nothing in it needs
 * clearing, and calls that share it must not overlap on the GPU.
 */
typedef struct sd_kv_fork_args {
  int32_t rows_in, R, groups, max_pages, page_size, append, keep, N;
  const int32_t *parents;    /* [R] or null                                   */
  const int32_t *table;      /* [rows_in][max_pages]                          */
  const int32_t *kv_len;     /* [rows_in]                                     */
  int32_t *refs;             /* [N], in and out                               */
  int32_t *table_out;        /* [R][max_pages]                                */
  int32_t *len_out;          /* [R]                                           */
  int32_t *src, *dst, *fill; /* [R]                                           */
  int32_t *count;            /* [1]                                           */
  int32_t *status;           /* one int32 or null                             */
  void *workspace;
  size_t workspace_bytes;
} sd_kv_fork_args;

/* 0 for arguments out of range. */
size_t sd_kv_fork_workspace_size(int32_t rows_in, int32_t R, int32_t N);

sd_status_t sd_kv_fork(const sd_kv_fork_args *args, void *stream);

/*
 * Gives pages back: refs[p] - 1 for the ids p = pages[b][i] of pages
 * [rows][cols] with which[b] != 0 (any b without which) and b cols + i <
 * *count (any place without count): the rows of requests that end, or the
 * freed list and total of sd_kv_rollback.  -1 is passed over.  Ids outside [0, N), and pages
 * given back more often than they are held, set SD_STATUS_BAD_PAGE; counts
 * end at 0.  clear != 0: the entries that are taken become -1.
 */
sd_status_t sd_kv_free(int64_t rows, int64_t cols, int32_t *pages, const uint8_t *which,
                       const int32_t *count, int32_t clear, int32_t N, int32_t *refs,
                       int32_t *status, void *stream);

/*
 * Moves the pages in use to the front: with L pages of refs > 0, the i-th
 * such page with an id >= L (by id) takes the place of the i-th free page
 * with an id < L.  src, dst [N / 2]: the pairs in that order, -1, -1 after
 * the last; count [1]: how many; live [1]: L; new_ids [N]: where each page in
 * use is afterwards, -1 for a free one.  refs is brought up to date, and so
 * are the entries of table [n_table] (optional; any number of block tables
 * laid side by side): -1 is passed over, an id outside [0, N) or of a free
 * page is left and sets SD_STATUS_BAD_PAGE.  The contents follow by
 * sd_kv_copy.  workspace: at least sd_kv_compact_workspace_size bytes,
 * 16-byte aligned; nothing in it needs clearing, and calls that share it must
 * not overlap on the GPU.
 */
size_t sd_kv_compact_workspace_size(int32_t N);

sd_status_t sd_kv_compact(int32_t N, int32_t *refs, int64_t n_table, int32_t *table, int32_t *src,
                          int32_t *dst, int32_t *count, int32_t *live, int32_t *new_ids,
                          int32_t *status, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Copies pages inside caches: for the first *count pairs (all `pairs` of them
 * without count) page src[i] to page dst[i], in every one of n_caches arrays
 * of `layers` layers of N pages.  A page is `parts` parts, each of page_size
 * entries of entry_bytes bytes, contiguous; of each part the first fill[i]
 * entries are copied (all of them without fill; fill is taken into
 * [0, page_size]).  Entries first in a page: parts = 1; heads first: parts =
 * heads.  A pair of -1, -1 is passed over; any other id outside [0, N) sets
 * SD_STATUS_BAD_PAGE and the pair is left out.  No page may be both a source
 * and a destination, and none twice a destination.
 */
typedef struct sd_kv_copy_args {
  int32_t n_caches, layers, N, parts, page_size;
  int64_t entry_bytes;
  int64_t layer_stride, page_stride; /* bytes                                 */
  void *const *caches;       /* host array of n_caches device pointers        */
  int32_t pairs;
  const int32_t *src, *dst;  /* [pairs]                                       */
  const int32_t *fill;       /* [pairs] or null                               */
  const int32_t *count;      /* [1] or null                                   */
  int32_t *status;           /* one int32 or null                             */
} sd_kv_copy_args;

sd_status_t sd_kv_copy(const sd_kv_copy_args *args, void *stream);

/* Sizes of the argument structs as compiled into the library. */
size_t sd_kv_fork_args_size(void);
size_t sd_kv_copy_args_size(void);

#ifdef __cplusplus
}
#endif

#endif /* SD_KV_H_ */
