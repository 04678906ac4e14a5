/*
 * mla_kv8.h -- C ABI of the paged 8-bit latent KV cache: rows quantised as they
 * are written under one scale per block of pool slots, read back, and attended
 * over by the DDTree verify attention of mla_verify.h, with an optional sliding
 * window and first tokens that stay visible.
 *
 * The cache row.  A pool row of MLA_KV8_ROW_BYTES holds one token:
 *
 *   bytes   0..511  the latent kv_c: 512 e4m3 codes (bias 7, subnormals, largest
 *                   448; 0x7f and 0xff are NaN, which a write never stores)
 *   bytes 512..639  the rope key k_pe, 64 bf16 values
 *
 * both in units of 2^(exponent + k).  Slot s belongs to block s / block; the
 * scale word scales[s / block] is 0 while the block holds no rows, and k + 1,
 * with k in 0..MLA_KV8_MAX_SCALE, once it does.  MLA has one key head, so one
 * scale per block is one per block and head.  `block` is any number of slots,
 * the page size of the tables in most servers; a zeroed array of words is an
 * empty cache, and mla_kv_tables (mla_kv_tables.h) empties the blocks inside the
 * pages it hands out.  A block that is larger than a page is never emptied, so its
 * scale never falls; at page_size 1 that leaves blocks of one slot.
 *
 * `exponent` is one number per cache: e4m3 codes lose precision below 2^-6 and
 * stop at 448, and k only makes units larger, so it should put the largest
 * magnitudes of quiet blocks at about 448 * 2^exponent.  -7 suits latents of
 * about unit size.
 *
 * Conventions as in mla_verify.h: DEVICE pointers owned by the caller, nothing
 * allocated, asynchronous on `stream` (whose device must be the current one),
 * host-visible argument errors returned before any launch.  A workspace is
 * used by one call at a time; it needs no clearing.  Errors found on the
 * device are read with mla_kv8_check.
 */
#ifndef MLA_KV8_H
#define MLA_KV8_H

#include "mla_kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_KV8_ROW_BYTES 640
#define MLA_KV8_MAX_SCALE 15
#define MLA_KV8_MAX_EXPONENT 32
#define MLA_KV8_WORKSPACE_BYTES 16384u /* for mla_kv8_write and mla_kv8_read */

typedef struct {
    void *rows;         /* pool row r at byte offset r * row_stride; 32-byte aligned */
    int64_t row_stride; /* bytes; >= MLA_KV8_ROW_BYTES, a multiple of 32 */
    int64_t slots;      /* pool rows, 1..INT32_MAX */
    int32_t *scales;    /* [ceil(slots / block)] scale words */
    int block;          /* slots per block, >= 1 */
    int exponent;       /* -MLA_KV8_MAX_EXPONENT..MLA_KV8_MAX_EXPONENT */
} mla_kv8_cache;

/* Quantises row i of kv_c and k_pe into pool slot slots[i], for every i with
 * slots[i] >= 0 (mla_kvq_rows as in mla_kvq.h).  A row of largest latent
 * magnitude a needs k(a), the least k >= 0 with a <= 448 * 2^(exponent + k), or
 * 15 where there is none.  Each block that a row goes to gets
 *     k = max(its k, k(a) of the rows that go there),
 * an empty one what its rows need.  A latent x is stored as the e4m3 number
 * nearest x / 2^(exponent + k) (ties to even, at most 448), a rope value as the
 * nearest bf16 number.  Rows that a block held before keep their values: where
 * its k grew by d, codes become the e4m3 numbers nearest code / 2^d, which is
 * exact for codes of at least 2^(d-6), and rope values are divided by 2^d.  (The
 * bytes of rows that were never written may change with them; those of a block
 * that was empty stay as they were.)  One thread block moves a grown block: blocks of
 * many thousand slots make such a write slow.
 *
 * An infinite latent is stored as the largest magnitude with its sign and does
 * not count for k, NaN is stored as 0, and MLA_DEVERR_NONFINITE is recorded.  A
 * slot outside [-1, slots) writes nothing and records MLA_DEVERR_SLOT; the other
 * rows are written.  The slots >= 0 must differ from each other.  Two calls that write the same block
 * must be ordered, and so must a write and anything that reads the block's rows.
 * kv_c and k_pe must not overlap the cache.  Equal arguments and cache give
 * equal bytes. */
mla_status mla_kv8_write(const mla_kv8_cache *cache, const mla_kvq_rows *src, void *workspace, size_t ws_bytes,
                         mla_stream_t stream);

/* Reads pool slot slots[i] back into row i of kv_c and k_pe, for every i with
 * slots[i] >= 0: the values that the row stands for.  Nothing is rounded unless
 * a value leaves the range of the element type.  Rows with slot -1 are left as
 * they were.  A slot outside [-1, slots) leaves its row as it was and records
 * MLA_DEVERR_SLOT.  A slot may be named any number of times; rows of an empty
 * block are read in units of 2^exponent. */
mla_status mla_kv8_read(const mla_kv8_cache *cache, const mla_kvq_rows *dst, void *workspace, size_t ws_bytes,
                        mla_stream_t stream);

/* The attention.  Rows, positions and tables as in mla_kvq_attn: sequence b has
 * positions 0 .. prefix_lens[b] + Q - 1, the prefix first, then node t at
 * position prefix_lens[b] + t, and the pool rows of all of them have been
 * written.  Single-token decoding is Q = 1. */
typedef struct {
    int B;                      /* sequences, >= 0 (0 = no-op) */
    int Q;                      /* nodes per sequence, 0..64 (0 = no-op) */
    int H;                      /* heads, >= 1; Q * H up to 2^24 and B * Q * H up to INT32_MAX */
    mla_kv8_cache cache;
    const void *q_lat;          /* bf16 [B][Q][H][512], contiguous, 16-byte aligned */
    const void *q_pe;           /* bf16 [B][Q][H][64], contiguous, 16-byte aligned */
    int page_size;              /* 1: kv_indptr/kv_indices;  > 1: block_table */
    const int32_t *kv_indptr;   /* [B+1]; kv_indptr[0] == 0, spans prefix_lens[b]+Q (0 for an unused sequence) */
    const int32_t *kv_indices;  /* [kv_indptr[B]] pool slots; not NULL, even when that is 0 */
    const int32_t *block_table; /* [B][max_pages] page ids */
    int max_pages;              /* columns of block_table */
    const int32_t *prefix_lens; /* [B], >= 0; -1 marks an unused sequence of a padded batch: nothing of it is
                                   read, its rows of out and lse are left as they were */
    const int32_t *tree_parent; /* [B][Q], parent[i] in [-1, i-1]; NULL: each node's parent is the node before */
    int window;                 /* 0: none; W > 0: node i sees place p when p < sinks or place(i) - p < W, as in */
    int sinks;                  /* mla_kvq_attn; sinks >= 0, 0 without a window */
    float scale;                /* score scale, > 0; scale * 2^exponent * log2(e) must be a normal fp32 number */
    void *out;                  /* bf16 [B][Q][H][512], 16-byte aligned */
    float *lse;                 /* [B][Q][H], natural log; may be NULL */
} mla_kv8_attn_args;

/* Both products take the cache's codes as they are and accumulate in fp32.  A
 * query enters as two e4m3 terms in units of a power of two of its row: exact for
 * elements of at least 2^-9 of the row's largest magnitude, else off by at most
 * 2^-16 of that.  A softmax weight enters as three e5m2 terms, off by at most 2^-9
 * of its rounding to 11 bits, as a bf16 number would be.  Beside that the small ones
 * among the weights of a tile are together off by at most 2^-8.6 of its largest, and
 * none by more than itself, however small the tile's weights are beside others' and
 * however the scales of its blocks differ; a tile is 64 positions from a multiple of
 * 64 on, 128 where Q * H is at most 64.  (2^40 below the largest weight times 2^k
 * that came before, a weight times 2^k may be off by 2^-64 of that.)
 * lse is natural-log, -infinity with a row of zeros in out where every visible
 * score is -infinity; a row whose queries hold an infinity or NaN is NaN.  Equal
 * arguments give equal bytes.
 *
 * Table entries of prefix positions that no node of a sequence sees are not
 * read.  A bad table (MLA_DEVERR_PREFIX, _INDPTR, _PAGES: found before any work)
 * leaves out and lse as they were; a slot outside the pool or a parent outside
 * [-1, i-1] (MLA_DEVERR_SLOT, _PARENT) is read as no token or -1 and leaves that
 * sequence's outputs unspecified.  No access leaves the pool.  A wait that
 * outlasts two seconds ends the kernel with MLA_DEVERR_TIMEOUT; the outputs are
 * then unspecified. */
mla_status mla_kv8_attn(const mla_kv8_attn_args *args, void *workspace, size_t ws_bytes, mla_stream_t stream);

/* Bytes of workspace that mla_kv8_attn needs on the current device, 256-byte
 * aligned.  0 when the arguments are invalid or no CUDA device can be queried. */
size_t mla_kv8_attn_workspace_size(const mla_kv8_attn_args *args);

/* Failure-detection self-test, as mla_kvq_selftest_timeout: mla_kv8_attn with
 * every device wait limited to hold_ns (0 < hold_ns <= 1e9) and its products held
 * back on a barrier that nothing completes. */
mla_status mla_kv8_selftest_timeout(const mla_kv8_attn_args *args, void *workspace, size_t ws_bytes,
                                    uint64_t hold_ns, mla_stream_t stream);

/* Synchronises `stream`, then reads the error bits that the last call of this
 * header on this workspace left; as mla_kvq_check. */
mla_status mla_kv8_check(const void *workspace, mla_stream_t stream, uint32_t *bits);

#ifdef __cplusplus
}
#endif

/* the page tables of a step, which can empty the blocks of a cache as above */
#include "mla_kv_tables.h"

#endif /* MLA_KV8_H */
