/*
 * mla_kv_tables.h -- C ABI of a serving step's page tables: built on the device
 * from the requests' lengths, so that a decoding loop needs no host round trip
 * between accepting tokens and the next verify call.
 *
 * A pool of num_pages pages of page_size slots is shared by the requests.  Row b
 * of block_table names the pages of request b, pages_held[b] of them; the pages
 * that nobody holds wait in a ring in the order in which they came free.  One
 * call brings all of it to this step's lengths and writes what the step's other
 * calls read: the block table and the page-size-1 tables of the attention calls,
 * and the slots of the new tokens for the writes.
 *
 * Conventions as in mla_verify.h: DEVICE pointers owned by the caller, nothing
 * allocated, asynchronous on `stream` (whose device must be the current one),
 * host-visible argument errors returned before any launch.  A workspace is used
 * by one call at a time; it needs no clearing.  Two calls on the same tables must
 * be ordered.  Errors found on the device are read with mla_kv8_check.
 */
#ifndef MLA_KV_TABLES_H
#define MLA_KV_TABLES_H

#include "mla_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_KV_TABLES_WORKSPACE_BYTES 16384u

typedef struct {
    int B;                      /* requests, 0..MLA_KV_TABLES_MAX_B (0 = no-op) */
    int Q;                      /* new tokens of each request, >= 0; not used with new_lens */
    int page_size;              /* slots per page, >= 1 */
    int max_pages;              /* columns of block_table, >= 1; max_pages * page_size <= INT32_MAX */
    int num_pages;              /* pages of the pool, >= 1; num_pages * page_size <= INT32_MAX */
    const int32_t *prefix_lens; /* [B] tokens before the new ones, >= 0; -1: an unused row, which holds no pages
                                   after the call */
    const int32_t *new_lens;    /* [B] new tokens, >= 0 (not read where prefix_lens is -1); NULL: Q each */
    int32_t *block_table;       /* in/out [B][max_pages] */
    int32_t *pages_held;        /* in/out [B], 0..max_pages */
    int32_t *free_ring;         /* in/out [ring]: entry i % ring for head <= i < tail names a free page */
    int64_t *free_state;        /* in/out [3]: head, tail; 0 <= head <= tail <= head + ring; and a word of the
                                   library's that is 0 between calls */
    int ring;                   /* entries of free_ring, >= 1; num_pages are always enough */
    int32_t *slots;             /* out, may be NULL: slots of the new tokens.  Without new_lens [B][Q], -1 for unused
                                   rows; with new_lens the requests' tokens one after the other, -1 behind the last */
    int64_t slots_len;          /* entries of slots; B * Q without new_lens */
    int32_t *kv_indptr;         /* out [B+1], may be NULL: sums of prefix_lens + new tokens, 0 for unused rows */
    int32_t *kv_indices;        /* out, may be NULL: the slots of all positions, request after request; entries
                                   behind the last are left as they were */
    int64_t indices_len;        /* entries of kv_indices */
    int32_t *scales;            /* in/out, may be NULL: an 8-bit cache's scale words; those of blocks all of whose
                                   slots lie in one page that the call hands out become 0 (a block over several
                                   pages, or over the last page's end, keeps its scale: let `block` divide
                                   page_size) */
    int block;                  /* slots per block of that cache, >= 1; not used without scales */
} mla_kv_tables_args;

#define MLA_KV_TABLES_MAX_B 4096

/* With need = ceil((prefix_lens[b] + new tokens) / page_size), 0 for an unused
 * row, every request gets
 *   need - held pages from the ring's head on, requests in order, where it holds
 *     too few: entries held .. need - 1 of its row;
 *   or its entries need .. held - 1 go behind the ring's tail, requests in order,
 *     and become -1 in its row.  They can be handed out by the next call.
 * Other entries of block_table are left as they were.  The slot of position p is
 * block_table[b][p / page_size] * page_size + p % page_size.  Every entry below
 * need names a page: those that a window has passed stay held until the request
 * ends, and must not be cleared in between.
 *
 * Nothing is written when the tables cannot be built: a prefix length below -1
 * or a negative new length (MLA_DEVERR_PREFIX), a request of more than max_pages
 * pages, a held count outside 0..max_pages or a ring state outside its bounds
 * (MLA_DEVERR_PAGES), too few free pages, a ring too small for the pages that
 * come back, or more positions or new tokens than kv_indices, slots or 32 bits
 * hold (MLA_DEVERR_CAPACITY).  A page id outside [0, num_pages) in a held entry
 * or in the ring records MLA_DEVERR_SLOT; its slots are written as -1, and where
 * its entry comes back it goes into the ring as it is. */
mla_status mla_kv_tables(const mla_kv_tables_args *args, void *workspace, size_t ws_bytes, mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_KV_TABLES_H */
