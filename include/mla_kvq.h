/*
 * mla_kvq.h -- C ABI of the 4-bit latent KV cache: rows quantised as they are
 * written, read back, and attended over by the DDTree verify attention of
 * mla_verify.h, with an optional sliding window and first tokens that stay
 * visible.
 *
 * The cache row.  A pool row of MLA_KVQ_ROW_BYTES holds one token:
 *
 *   bytes   0..255  512 codes of 4 bits.  The 32-bit little-endian word w
 *                   holds elements 8w .. 8w+7 of the latent kv_c: element
 *                   8w + 2t + j is nibble t + 4j (bits 4t+16j .. 4t+16j+3).
 *   bytes 256..287  32 scales of 8 bits; scale i belongs to elements
 *                   16i .. 16i+15.  Bits 0-6 are an e4m3 magnitude (bias 7,
 *                   subnormals, 0x7f = 480: there is no NaN); bit 7 is
 *                   ignored.
 *   bytes 288..415  the rope key k_pe, 64 bf16 values.
 *
 * Element e stands for  (code_e - 8) * scale_{e/16} * 2^exponent,  a number
 * that bf16 and fp32 hold exactly (at most 4 + 4 significant bits).  Any bytes
 * stand for finite latents, so a row that a query does not see cannot reach
 * its output, whatever was in the memory.  The rope key stays in bf16: it is a
 * ninth of the elements, and its errors move the scores directly.
 *
 * `exponent` is one number per cache, for latents whose norm weights put them
 * far from 1: scales below 2^-6 lose precision and scales stop at 448, so the
 * largest magnitude of 16 neighbouring latents should lie in about
 * [2^-3, 2^11] * 2^exponent.  0 suits latents of about unit size.
 *
 * Conventions as in mla_verify.h: DEVICE pointers owned by the caller, nothing
 * allocated, asynchronous on `stream` (whose device must be the current one),
 * host-visible argument errors returned before any launch.  A workspace is
 * used by one call at a time; it needs no clearing.  Errors found on the
 * device are read with mla_kvq_check.
 */
#ifndef MLA_KVQ_H
#define MLA_KVQ_H

#include "mla_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_KVQ_ROW_BYTES 416
#define MLA_KVQ_MAX_EXPONENT 32
#define MLA_KVQ_WORKSPACE_BYTES 16384u /* for mla_kvq_write and mla_kvq_read */

#define MLA_DEVERR_NONFINITE 0x200u /* mla_kvq_write: a latent was infinite or NaN */

typedef struct {
    void *rows;         /* pool row r at byte offset r * row_stride; 32-byte aligned */
    int64_t row_stride; /* bytes; >= MLA_KVQ_ROW_BYTES, a multiple of 32 */
    int64_t slots;      /* pool rows, 1..INT32_MAX */
    int exponent;       /* -MLA_KVQ_MAX_EXPONENT..MLA_KVQ_MAX_EXPONENT */
} mla_kvq_cache;

/* The rows a write takes or a read fills. */
typedef struct {
    int64_t n;              /* rows, >= 0 (0 = no-op), <= INT32_MAX */
    mla_dtype dtype;        /* element type of kv_c and k_pe */
    void *kv_c;             /* row i at element offset i * kv_c_stride (512 used); read only for a write */
    void *k_pe;             /* row i at element offset i * k_pe_stride (64 used); read only for a write */
    int64_t kv_c_stride;    /* elements; >= 512, row bytes a multiple of 16 */
    int64_t k_pe_stride;    /* elements; >= 64,  row bytes a multiple of 16 */
    const int32_t *slots;   /* [n] pool slot of each row; -1 skips the row */
} mla_kvq_rows;

/* Quantises row i of kv_c and k_pe into pool slot slots[i], for every i with
 * slots[i] >= 0.  Of 16 neighbouring latents x, with x' = x / 2^exponent:
 *     scale = the e4m3 number nearest max|x'| / 7 (ties to even, at most 448)
 *     code  = 8 + the integer nearest x' / scale (ties to even), within 1..15;
 *             8 where the scale is 0
 * both as if computed without rounding in between.  fp32 rope keys are rounded
 * to bf16.  An infinite latent is stored as the largest magnitude a block can
 * hold with its sign, NaN as 0, and MLA_DEVERR_NONFINITE is recorded (rope
 * keys are stored as they are).  A slot outside [-1, slots) writes nothing and
 * records MLA_DEVERR_SLOT; the other rows are written.  The slots >= 0 must
 * differ from each other: of two rows for one slot, which row's bytes end up
 * in which part of it is not defined.  kv_c and k_pe must not overlap the
 * cache. */
mla_status mla_kvq_write(const mla_kvq_cache *cache, const mla_kvq_rows *src, void *workspace, size_t ws_bytes,
                         mla_stream_t stream);

/* Reads pool slot slots[i] back into row i of kv_c and k_pe, for every i with
 * slots[i] >= 0: the values that the row stands for, without rounding.  Rows
 * with slot -1 are left as they were.  A slot outside [-1, slots) leaves its
 * row as it was and records MLA_DEVERR_SLOT.  A slot may be named any number
 * of times. */
mla_status mla_kvq_read(const mla_kvq_cache *cache, const mla_kvq_rows *dst, void *workspace, size_t ws_bytes,
                        mla_stream_t stream);

/* The attention.  Rows, positions and tables as in mla_verify_attn: sequence b
 * has positions 0 .. prefix_lens[b] + Q - 1, the prefix first, then node t at
 * position prefix_lens[b] + t, and the pool rows of all of them have been
 * written.  Single-token decoding is Q = 1. */
typedef struct {
    int B;                      /* sequences, >= 0 (0 = no-op) */
    int Q;                      /* nodes per sequence, 0..64 (0 = no-op) */
    int H;                      /* heads, >= 1; Q * H up to 2^24 and B * Q * H up to INT32_MAX */
    mla_kvq_cache cache;
    const void *q_lat;          /* bf16 [B][Q][H][512], contiguous */
    const void *q_pe;           /* bf16 [B][Q][H][64], contiguous; times 2^-exponent in bf16, which is exact
                                   for magnitudes 2^-94 .. 2^95 (and for any with exponent 0) */
    int page_size;              /* 1: kv_indptr/kv_indices;  > 1: block_table */
    const int32_t *kv_indptr;   /* [B+1]; kv_indptr[0] == 0, spans prefix_lens[b]+Q (0 for an unused sequence) */
    const int32_t *kv_indices;  /* [kv_indptr[B]] pool slots; not NULL, even when that is 0 */
    const int32_t *block_table; /* [B][max_pages] page ids */
    int max_pages;              /* columns of block_table */
    const int32_t *prefix_lens; /* [B], >= 0; -1 marks an unused sequence of a padded batch: nothing of it is
                                   read, its rows of out and lse are left as they were */
    const int32_t *tree_parent; /* [B][Q], parent[i] in [-1, i-1]; NULL: each node's parent is the node before */
    int window;                 /* 0: none; W > 0: see below */
    int sinks;                  /* first tokens that stay visible under a window, >= 0; 0 without a window */
    float scale;                /* score scale, > 0; scale * 2^exponent * log2(e) must be a normal fp32 number */
    void *out;                  /* bf16 [B][Q][H][512] */
    float *lse;                 /* [B][Q][H], natural log; may be NULL */
} mla_kvq_attn_args;

/* Node i sees the prefix, itself and its ancestors.  A window W > 0
 * (mla_verify_attn, over the bf16 and fp32 caches, has none) keeps of those the
 * tokens less than W places back and the first `sinks` tokens: with
 * a prefix token's place its position and a node's place prefix_lens[b] + its
 * depth (0 for a node without parent), node i sees place p when
 *     p < sinks  or  place(i) - p < W.
 * Table entries of prefix positions that no node of a sequence sees are not
 * read, so their pages may have been freed.
 *
 * The softmax statistics and both products accumulate in fp32; keys and values
 * enter the products exactly, the softmax weights rounded to 11 bits.  lse is
 * natural-log, -infinity with a row of zeros in out where every visible score
 * is -infinity; equal arguments give equal bytes.  Enqueues the attention
 * kernel and a kernel that merges the pieces of rows that several clusters
 * shared.  A bad table (MLA_DEVERR_PREFIX, _INDPTR, _PAGES: found before any
 * work) leaves out and lse as they were; a slot outside the pool or a parent
 * outside [-1, i-1] (MLA_DEVERR_SLOT, _PARENT) is read as slot 0 or -1 and
 * leaves that sequence's outputs unspecified. No access leaves the pool. A wait
 * that outlasts two seconds ends the kernel with MLA_DEVERR_TIMEOUT; the
 * outputs are then unspecified. */
mla_status mla_kvq_attn(const mla_kvq_attn_args *args, void *workspace, size_t ws_bytes, mla_stream_t stream);

/* Bytes of workspace that mla_kvq_attn needs on the current device, 256-byte
 * aligned: the partial results of rows shared between clusters.  0 when the
 * arguments are invalid or no CUDA device can be queried. */
size_t mla_kvq_attn_workspace_size(const mla_kvq_attn_args *args);

/* Failure-detection self-test, as mla_verify_selftest_timeout.  Runs mla_kvq_attn
 * with every device wait limited to hold_ns (0 < hold_ns <= 1e9) and the value
 * product held back on a barrier that nothing completes: the parts of the
 * kernel before it fill their buffers, wait for it, give up, drain what they
 * issued and free their Tensor Memory, and the call completes with
 * MLA_DEVERR_TIMEOUT; out and lse are unspecified.  The context stays usable:
 * the next call on the same workspace runs normally.  Returns
 * MLA_ERR_INVALID_ARG for a zero or larger hold_ns or an empty problem,
 * otherwise as mla_kvq_attn. */
mla_status mla_kvq_selftest_timeout(const mla_kvq_attn_args *args, void *workspace, size_t ws_bytes,
                                    uint64_t hold_ns, mla_stream_t stream);

/* Synchronises `stream`, then reads the error bits that the last call of this
 * header on this workspace left (a call with nothing to do launches nothing
 * and leaves them as they were).  Returns MLA_OK or MLA_ERR_DEVICE_CHECK (or
 * MLA_ERR_CUDA); *bits (may be NULL) receives the MLA_DEVERR_* bits. */
mla_status mla_kvq_check(const void *workspace, mla_stream_t stream, uint32_t *bits);

#ifdef __cplusplus
}
#endif

/* the paged 8-bit latent cache, whose calls use the types above */
#include "mla_kv8.h"

#endif /* MLA_KVQ_H */
