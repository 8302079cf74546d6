/*
 * lora_kv.h -- C ABI of the paged key/value cache and the attention over it (GB300, sm_103a):
 * what a served decoder layer runs between the q/k/v projections and o_proj
 * (lora_linear_grouped, lora_linear of lora_linear.h).
 *
 * The cache. P pages of p tokens (p a power of two, 16..256) for H_kv heads of D values
 * (D 64 or 128). The arenas belong to the caller:
 *   k_pages, v_pages    [P][H_kv][p][D]  bf16 (LORA_KV_BF16) or int8 codes (LORA_KV_INT8)
 *   k_scales, v_scales  [P][H_kv][p]     bf16 (LORA_KV_INT8; NULL for LORA_KV_BF16)
 * Row (page, head, r) of an int8 cache stands for the D values scale * code.
 *
 * The batch (lora_kv_batch). Sequence b holds kv_len[b] tokens; its token j sits in page
 * page_table[b][j / p], row j % p. Rows start[b] .. start[b+1] - 1 of a call's token tensors
 * are the LAST n_b = start[b+1] - start[b] tokens of the sequence: row start[b] + i is the token
 * at position kv_len[b] - n_b + i. kv_len counts them: a step sets kv_len to the length after
 * its new tokens, writes them, then attends. n_b may be 0, and rows whose position would be
 * negative (kv_len < n_b) are skipped by the write and come back as zeros from the others.
 *
 * Conventions, besides those of lora_linear.h:
 *  - page_table, start and kv_len are DEVICE arrays, read in stream order: lengths may change
 *    between replays of a captured CUDA graph (T, n_seqs and max_new are what it was captured
 *    with).
 *  - Token tensors (K, V, Q, O) are bf16, [T][heads][D] with the heads of a token contiguous
 *    and token_stride elements from one token to the next (slices of a fused projection's
 *    output are fine): token_stride a multiple of 8 and at least heads * D, pointers 16-byte
 *    aligned. Rows at and after start[n_seqs] are not written, and what they hold does not matter
 *    (they have to exist: the write loads all T rows).
 *  - A table entry outside 0..P-1, a kv_len beyond table_stride * p or a start outside 0..T
 *    sets the cache's error word and is not followed; lora_kv_check_errors then returns
 *    LORA_ERR_RANGE, the rows of that sequence are unspecified, other rows stay correct.
 *    Table entries past a sequence's last page are not read.
 *  - Cache rows that hold no token of a sequence may hold anything (inf and NaN included). An
 *    infinity or a NaN in a token's K or V reaches the rows that see that token, no others. One of
 *    V in a bf16 cache makes that value of O that infinity, whatever weight the token has, and NaN
 *    where the row also sees a NaN or the other infinity there.
 *  - T and table_stride * p are at most 2^30, T * n_heads below 2^31 (else LORA_ERR_ARG).
 *  - Calls are made with the device current that the cache was created on (else LORA_ERR_ARG).
 *  - A cache is not thread-safe: use it from one host thread at a time. Calls on several
 *    streams are allowed: attention calls (which share scratch) are ordered by the library,
 *    those captured in a graph by whoever replays it (no other attention call of the cache beside
 *    the replay); the order of a write and the calls that use what it wrote is the caller's, as
 *    for any two kernels.
 */
#ifndef LORA_KV_H
#define LORA_KV_H

#include "lora_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque cache handle: the arenas' addresses, the error word and the attention's scratch. */
typedef struct lora_kv lora_kv;
typedef lora_kv *lora_kv_t;

typedef enum { LORA_KV_BF16 = 0, LORA_KV_INT8 = 1 } lora_kv_format;

typedef struct lora_kv_batch {
    const int32_t *page_table;  /* device [n_seqs][table_stride]                        */
    const int32_t *start;       /* device [n_seqs + 1], from 0, not decreasing          */
    const int32_t *kv_len;      /* device [n_seqs]                                      */
    int32_t table_stride;       /* entries per sequence                                 */
    int32_t n_seqs;
    int32_t T;                  /* rows of the token tensors, >= start[n_seqs]          */
    int32_t max_new;            /* a bound on n_b: only chooses between kernels, a wrong
                                   one costs time                                       */
} lora_kv_batch;

/*
 * Create a cache over the caller's arenas (device memory of the current device, 16-byte
 * aligned, valid until the cache is destroyed). Nothing is written to them.
 * Errors: SHAPE (page_tokens, head_dim, n_kv_heads outside 1..256, num_pages < 1 or more than
 * 2^31 - 1 cache rows of one head), ARG (unknown format, null or misaligned arenas, scales
 * given for a bf16 cache, out == NULL), UNSUPPORTED, OOM, CUDA.
 */
lora_status lora_kv_create(int num_pages, int page_tokens, int n_kv_heads, int head_dim, int format,
                           void *k_pages, void *v_pages, void *k_scales, void *v_scales,
                           lora_kv_t *out);

/* Wait for the device, then free the handle and its scratch (not the arenas). */
lora_status lora_kv_destroy(lora_kv_t kv);

/* Make sure of the attention's scratch for calls of up to max_tokens rows, n_heads query heads
 * and max_seqs sequences, whatever rows each has and whatever max_new they give. The first call
 * that needs scratch beyond the handle's own allocates it (40 MB): call this first when
 * lora_kv_attention will run inside a CUDA graph capture. */
lora_status lora_kv_reserve(lora_kv_t kv, int max_tokens, int n_heads, int max_seqs);

/*
 * Write the batch's tokens into their pages. K and V: [T][H_kv][D]. bf16 caches take the values
 * as they are. int8 caches quantise each row x (one token, one head) by itself:
 *     s = max(bf16(max_d |x_d| / 127), 2^-126),  code_d = clamp(rint(x_d / s), -127, 127)
 * (ties to even). s is rounded to bf16 before the division; x_d and s then have 8 significant
 * bits each, so x_d / s is a tie exactly or by a margin that fp32 resolves, and the codes are
 * those of exact arithmetic. A row with an infinity or a NaN is stored as code 0 and scale
 * NaN: it reads back as NaN.
 * Two tokens of one call must not share a cache row (sequences that share a prefix page may,
 * for the tokens they do not write). Asynchronous on `stream`. Errors: ARG, CUDA.
 */
lora_status lora_kv_write(lora_kv_t kv, const void *K, int64_t k_stride, const void *V, int64_t v_stride,
                          const lora_kv_batch *batch, lora_stream_t stream);

/*
 * Read the batch's tokens back: K and V [T][H_kv][D] bf16, an int8 cache's values as
 * bf16(scale * code), the exact product rounded once. start = prefix sums of kv_len reads
 * whole sequences. Asynchronous on `stream`. Errors: ARG, CUDA.
 */
lora_status lora_kv_read(lora_kv_t kv, void *K, int64_t k_stride, void *V, int64_t v_stride,
                         const lora_kv_batch *batch, lora_stream_t stream);

/*
 * Attention of the batch's tokens over the cache (which already holds them): for row t at
 * position pos of sequence b, query head h and kv head h / (n_heads / H_kv),
 *     z_j = scale * <Q[t,h], K_j>,  j <= pos, and j > pos - window if window > 0,
 *     lse[t,h] = log sum_j exp(z_j),   O[t,h] = sum_j exp(z_j - lse) V_j
 * and O = 0, lse = -inf for a row that sees no token. Scores, maxima, sums and O are held in
 * fp32, and O is rounded to bf16 once. On its way into the product with V a weight is the sum of
 * two bf16 numbers (off by 2^-16 of it) in sequences of up to 24 rows of a kv head (n_b * n_heads /
 * H_kv) and, in longer ones, where a key may hold more than a quarter of what its row has so far;
 * elsewhere it is rounded to bf16 (2^-8 of it). lse (fp32 [T][n_heads]) may be NULL.
 *   n_heads: a multiple of H_kv, at most 1024. O must not alias Q or the cache.
 * Asynchronous on `stream`. Errors: ARG, SHAPE (n_heads), OOM (scratch), CUDA.
 */
lora_status lora_kv_attention(lora_kv_t kv, const void *Q, int64_t q_stride, int n_heads,
                              const lora_kv_batch *batch, float scale, int window, void *O,
                              int64_t o_stride, float *lse, lora_stream_t stream);

/* Wait for the calls enqueued on the cache, then read and clear its error word: LORA_OK,
 * LORA_ERR_RANGE or LORA_ERR_TIMEOUT, LORA_ERR_CUDA if the device reported an error. After
 * LORA_ERR_TIMEOUT (a kernel's bounded wait ran out) the outputs of the attention calls since the
 * last check are unspecified; the cache is ready for new calls. (Graph replays are not tracked:
 * synchronise their stream first.) */
lora_status lora_kv_check_errors(lora_kv_t kv);

/* Test hook: leave the cache as attention calls do whose bounded waits ran out (the error word, and
 * pieces of a split sequence that others wait to join). Nothing waits or fails on the device. */
lora_status lora_kv_selftest_timeout(lora_kv_t kv, lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_KV_H */
