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
#include "lora_rotary.h"

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
 * The write with rotary positions (lora_rotary.h) on the way: K's rows are rotated by their tokens' positions
 * in fp32 and written (rounded once to bf16, or quantised from fp32 as above), V's are written as they are,
 * and, where n_heads > 0, Q ([T][n_heads][D]) is rotated into Q_out (rounded once), in one pass.
 * Scales and codes of V are those of lora_kv_write. K's come from fp32 values that are off by their
 * arithmetic (2^-21 of the pair's length, factor included): a code is within 1/2 + 2^-13 of a step of the exact
 * value. A rotated value beyond fp32 is an infinity, in a bf16 cache and in Q_out also one that rounds beyond bf16.
 * Q_out == Q (and its stride) rotates in place; otherwise the two do not overlap. Rows of Q_out at positions below zero become zeros; those at
 * and after start[n_seqs] and those of a bad sequence are not written (Q's and K's are loaded).
 * rotary: HOST, rotary_dim at most the cache's head_dim. n_heads: 0..1024.
 * Asynchronous on `stream`. Errors: ARG, SHAPE (rotary_dim, n_heads), CUDA.
 */
lora_status lora_kv_write_rotary(lora_kv_t kv, const lora_rotary *rotary, const void *K, int64_t k_stride,
                                 const void *V, int64_t v_stride, const void *Q, int64_t q_stride, int n_heads,
                                 void *Q_out, int64_t qo_stride, const lora_kv_batch *batch, lora_stream_t stream);

/*
 * Read the batch's tokens back: K and V [T][H_kv][D] bf16, an int8 cache's values as
 * bf16(scale * code), the exact product rounded once. start = prefix sums of kv_len reads
 * whole sequences. Asynchronous on `stream`. Errors: ARG, CUDA.
 */
lora_status lora_kv_read(lora_kv_t kv, void *K, int64_t k_stride, void *V, int64_t v_stride,
                         const lora_kv_batch *batch, lora_stream_t stream);

/*
 * The page tables of sequences that come, fork, grow, shrink and go. A lora_kv_pages keeps, over the caller's
 * device arrays (valid until it is destroyed; a lora_kv_batch may name them),
 *   page_table [max_seqs][table_stride], kv_len [max_seqs]    as a batch has them, a row a slot
 *   refs [num_pages]                                           table entries that name each page
 * where slot s holds kv_len[s] tokens (0: it is empty) in its first ceil(kv_len[s] / p) entries. A new
 * one: lengths and refs 0. Only these calls change the arrays, or the caller, who keeps refs true. The
 * tables serve any number of caches (one a layer) of num_pages pages or more: the calls below change the
 * tables, and lora_kv_copy makes the copies of pages that the last of them asks for in one cache.
 * Calls are ordered by the library, on whatever streams (captured ones by whoever replays the graph); nothing is
 * allocated after the creation. Not thread-safe. Limits: max_seqs 65536, max_seqs * table_stride below 2^31,
 * table_stride * p at most 2^30.
 */
typedef struct lora_kv_pages lora_kv_pages;
typedef lora_kv_pages *lora_kv_pages_t;

/* Create on the current device; nothing is written to the arrays. Errors: SHAPE (num_pages outside 1..2^27,
 * page_tokens, max_seqs, table_stride), ARG (null or misaligned (4 bytes) arrays, out == NULL), UNSUPPORTED,
 * OOM, CUDA. */
lora_status lora_kv_pages_create(int num_pages, int page_tokens, int max_seqs, int table_stride,
                                 int32_t *page_table, int32_t *kv_len, int32_t *refs, lora_kv_pages_t *out);

/* Wait for the device, then free the handle and its scratch (not the arrays). */
lora_status lora_kv_pages_destroy(lora_kv_pages_t pages);

/*
 * Every slot i becomes the first n_i = min(keep[i], kv_len[parent[i]]) tokens of what slot parent[i] holds now
 * (parent -1: nothing), and room[i] tokens behind them: kv_len[i] = n_i + room[i]. parent, keep, room: device
 * int32 [max_seqs]; NULL: the slot itself, all its tokens, 0. So a step that extends its sequences
 * gives room; parent copies, reorders (all at once: beams) and frees; keep trims.
 *
 * Pages that n_i fills are shared. The page that n_i ends inside belongs to one slot alone, which may write
 * its other rows: it stays with the slot that ends inside it (first those with parent[i] = i, then the
 * lowest i) if no slot has all of it; the others get a page of their own and a copy of its rows (lora_kv_copy).
 * New pages are the lowest that no slot names afterwards, slot by slot, entry by entry. Entries that a slot no
 * longer uses become -1.
 *
 * Where the pages do not suffice (LORA_ERR_OOM from lora_kv_pages_check_errors), or a parent, a room, a length or
 * an entry is out of range (LORA_ERR_RANGE), nothing changes and nothing is to be copied. With room alone
 * (parent and keep NULL) the call takes refs at its word, and a page that a slot ends inside and refs does not
 * count once (these calls make no such tables) is LORA_ERR_RANGE, too.
 * Asynchronous on `stream`. Errors: ARG, CUDA.
 */
lora_status lora_kv_pages_update(lora_kv_pages_t pages, const int32_t *parent, const int32_t *keep, const int32_t *room,
                                 lora_stream_t stream);

/*
 * With n pages in use, moves those numbered n and above, in order, to the free pages below n, in order: afterwards
 * pages 0..n-1 are used, and the arenas' rest may serve others. table_out, refs_out: device arrays like
 * page_table and refs that get the new state (the handle's own keep the old one, for steps that still run on
 * it); both NULL: in place. kv_len does not change. lora_kv_copy then moves the pages, in each cache.
 * Entries out of range are left as they are (LORA_ERR_RANGE).
 * Asynchronous on `stream`. Errors: ARG, CUDA.
 */
lora_status lora_kv_pages_compact(lora_kv_pages_t pages, int32_t *table_out, int32_t *refs_out, lora_stream_t stream);

/* Wait for the calls enqueued on the handle, then HOST *used = pages that refs names. Errors: ARG, CUDA. */
lora_status lora_kv_pages_used(lora_kv_pages_t pages, int *used);

/* Wait for the calls enqueued on the handle, then read and clear its error word: LORA_OK, LORA_ERR_OOM,
 * LORA_ERR_RANGE, LORA_ERR_CUDA. (Graph replays are not tracked: synchronise their stream first.) */
lora_status lora_kv_pages_check_errors(lora_kv_pages_t pages);

/* Make the copies that the last update or compaction of `pages` asks for in the cache (K, V and scales; the rows
 * in use of an update's pages, whole pages of a compaction's). Follows that call; a later call on `pages` follows
 * this one. Asynchronous on `stream`. Errors: ARG (null, another device, page_tokens that differ, a cache of
 * fewer pages), CUDA. */
lora_status lora_kv_copy(lora_kv_t kv, lora_kv_pages_t pages, lora_stream_t stream);

/* Copy the first rows[i] (NULL: all) tokens of page src[i] to page dst[i], i < n (device int32 arrays). Pairs with a
 * negative page are left out; one with a page or a row count out of range sets the error word (LORA_ERR_RANGE).
 * No page is a destination twice, or a destination and a source (of another pair).
 * Asynchronous on `stream`. Errors: ARG (also n < 0), CUDA. */
lora_status lora_kv_copy_pages(lora_kv_t kv, const int32_t *src, const int32_t *dst, const int32_t *rows, int n,
                               lora_stream_t stream);

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

/* The batch's groups of sequences that share a prefix. Sequences seq_start[g] .. seq_start[g+1] - 1 of the batch
 * (no group: those before the first and behind the last) hold the same first prefix_len[g] tokens, in the same
 * pages as far as these are whole: lora_kv_pages_update makes such tables. */
typedef struct lora_kv_groups {
    const int32_t *seq_start;   /* device [n_groups + 1], not decreasing                */
    const int32_t *prefix_len;  /* device [n_groups]                                    */
    int32_t n_groups;           /* at most the batch's n_seqs                           */
    int32_t max_tokens;         /* a bound on the rows of one group (the sum of its n_b): only chooses
                                   between kernels                                      */
} lora_kv_groups;

/* As lora_kv_reserve, for lora_kv_attention_shared: 50 MB, T * n_heads * (D + 3) floats and lora_kv_reserve's. A call
 * that needs more than the handle has allocates it, and twice what the handle had where that is more and there is room;
 * this allocates no more than its size needs. What a larger block replaces is freed with the handle (a captured
 * graph may name it). */
lora_status lora_kv_reserve_shared(lora_kv_t kv, int max_tokens, int n_heads, int max_seqs);

/*
 * lora_kv_attention without a window, for a batch whose sequences share prefixes: every group's prefix is read
 * once, through the pages of its first sequence with rows. Same O and lse, but for the order of the sums: O of
 * the two parts is joined in fp32, and where the batch has sequences of up to 24 rows of a kv head (or max_new and T
 * leave room for them) every weight of a prefix is the sum of two bf16 numbers. What is shared is the largest number
 * of whole pages that holds at most prefix_len[g] tokens and, for each of the group's sequences with rows, none of its new
 * tokens; the rest is read per sequence. It pays for many short chunks over a long prefix (one group of single tokens, 32
 * heads on 8: from 16 sequences over 4000 tokens, or 8 over 16000; 64 over 1000 gain a tenth); for few rows, short
 * prefixes and chunks of more than 24 rows a kv head lora_kv_attention is quicker (kv_shared.cu has both
 * times). A group of one sequence shares nothing. seq_start out of order or outside 0..n_seqs sets
 * the error word (LORA_ERR_RANGE), and nothing is shared. groups may be NULL (nothing is shared).
 * Asynchronous on `stream`. Errors: ARG, SHAPE (n_heads), OOM (scratch), CUDA.
 */
lora_status lora_kv_attention_shared(lora_kv_t kv, const void *Q, int64_t q_stride, int n_heads,
                                     const lora_kv_batch *batch, const lora_kv_groups *groups, float scale, void *O,
                                     int64_t o_stride, float *lse, lora_stream_t stream);

/* Wait for the calls enqueued on the cache, then read and clear its error word: LORA_OK,
 * LORA_ERR_RANGE or LORA_ERR_TIMEOUT, LORA_ERR_CUDA if the device reported an error. After
 * LORA_ERR_TIMEOUT (a kernel's bounded wait ran out) the outputs of the attention calls since the
 * last check are unspecified; the cache is ready for new calls. (Graph replays are not tracked:
 * synchronise their stream first.) */
lora_status lora_kv_check_errors(lora_kv_t kv);

/* Test hook: leave the cache as attention calls do whose bounded waits ran out (the error word, pieces of a
 * split sequence that others wait to join, and anything in the scratch of shared prefixes). Nothing waits or fails on
 * the device. Not inside a capture. */
lora_status lora_kv_selftest_timeout(lora_kv_t kv, lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_KV_H */
