/*
 * qbn_kv.h - C ABI of the qbn library's paged key-value cache: appending new
 * tokens, attention over the cache (one new token per sequence, or chunks of
 * new tokens with a sliding window and sink tokens), and the page
 * bookkeeping between steps, for AMD Instinct MI355X (gfx950).
 *
 * The conventions of qbn.h hold here too: caller-owned DEVICE pointers, calls
 * asynchronous on `stream`, nothing allocated, nothing retained, every
 * argument checked on the host before anything is enqueued (a rejected call
 * returns a nonzero qbn_status and enqueues nothing). What the host cannot
 * see (table entries, lengths, row lists) is checked on the device, as stated
 * with each call; no content of those arrays makes a kernel read or write
 * outside the buffers it was given. All calls can be captured into a HIP
 * graph.
 *
 * The cache. `layers` x `pages` pages of `page_size` tokens each. A page holds
 * the keys and the values of `heads` key-value heads:
 *   k, v               [layers][pages][heads][page_size][head_dim] elements
 *   k_scales, v_scales [layers][pages][heads][head_dim / 32][page_size] u8
 * Element formats:
 *   QBN_KV_BF16  bfloat16; no scales (NULL).
 *   QBN_MXFP8    E4M3FN bytes, one E8M0 scale per 32 elements of a token.
 *   QBN_MXFP4    E2M1 codes, two per byte, low nibble = even element, the
 *                same scales. 4.25 bits per element.
 * The scales are stored token-minor: eight consecutive tokens' scales of one
 * block of 32 are one 8-byte word, which is how attention reads them.
 * page_size is 16, 32, 64, 128 or 256; head_dim 64, 96, 128, 192 or 256.
 *
 * The batch. Row b of `table` lists the pages of sequence b: token t sits in
 * page table[b][t / page_size] at t % page_size. lens[b] counts the tokens
 * of sequence b INCLUDING the new ones of this step: of its new tokens, the
 * last one is at position lens[b] - 1. cu (int32 [seqs + 1], ascending, in
 * 0 .. tokens) says which rows of q / k / v are the new tokens of sequence b:
 * cu[b] .. cu[b + 1] - 1. Rows before cu[0] and from cu[seqs] on belong to no
 * sequence (padding). cu = NULL stands for one new token per sequence.
 */
#ifndef QBN_KV_H
#define QBN_KV_H

#include "qbn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element format of an unquantized cache; QBN_MXFP8 and QBN_MXFP4 are the
 * others. */
#define QBN_KV_BF16 16

typedef struct qbn_kv_cache {
    int32_t format;    /* QBN_KV_BF16, QBN_MXFP8 or QBN_MXFP4 */
    int32_t heads;     /* key-value heads */
    int32_t head_dim;  /* elements per head of K and of V */
    int32_t page_size; /* tokens per page */
    int64_t layers;
    int64_t pages;     /* pages per layer */
    void *k, *v;                 /* 16-byte aligned */
    void *k_scales, *v_scales;   /* 16-byte aligned; NULL for QBN_KV_BF16 */
} qbn_kv_cache;

typedef struct qbn_kv_batch {
    int64_t seqs;         /* sequences of the batch */
    int64_t tokens;       /* new tokens of all of them (== seqs where cu is NULL) */
    int64_t row;          /* table entries per sequence */
    int64_t row_stride;   /* entries from one table row to the next, >= row */
    const int32_t *table;
    const int32_t *lens;  /* [seqs] */
    const int32_t *cu;    /* [seqs + 1] or NULL */
} qbn_kv_batch;

/* The pool's bookkeeping: one table row per sequence slot, and how many table
 * entries name each page (0: the page is free). An entry is a page or -1. */
typedef struct qbn_kv_pool {
    int64_t seqs;     /* sequence slots */
    int64_t row;      /* table entries per slot */
    int64_t pages;
    int32_t page_size;
    int32_t reserved; /* must be 0 */
    int32_t *table;   /* [seqs][row] */
    int32_t *lens;    /* [seqs] */
    int32_t *refs;    /* [pages] */
} qbn_kv_pool;

/* sizeof of the three structs above, for bindings: which = 0, 1, 2. */
QBN_API size_t qbn_kv_struct_size(int32_t which);

/* Bytes of K's (equally V's) elements (part 0) or scales (part 1) of a cache
 * of this shape; -1 if the format, part or shape is invalid. */
QBN_API int64_t qbn_kv_bytes(int32_t format, int64_t layers, int64_t pages, int32_t heads, int32_t page_size,
                             int32_t head_dim, int32_t part);

/* Write the new tokens' keys and values into their pages of one layer.
 * k, v: QBN_F32 or QBN_BF16, element [token][head][i] at
 * token * token_stride + head * head_stride + i (strides in elements; views of
 * a fused projection are taken as they are). Base pointers and strides are
 * 16-byte multiples. QBN_KV_BF16 rounds to nearest even; the MX formats follow
 * the rule of qbn_quantize_mx (exponent floor(log2 max|x|) - emax per 32,
 * elements rounded to nearest even and saturated; finite values). A token
 * whose table entry is not a page of the cache, or whose position is negative
 * or beyond the row, is not written (attention over it gives NaN), nor is a row
 * that no sequence has (before cu[0], or from cu[seqs] on). */
QBN_API int32_t qbn_kv_append(const qbn_kv_cache *cache, int64_t layer, const qbn_kv_batch *batch, const void *k,
                              int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                              int64_t v_head_stride, int32_t dtype, void *stream);

/* Attention. For the query of position p of sequence b, head h, with
 * key-value head h / (q_heads / heads):
 *   s_j = scale * q . k_j over the visible j,
 *   out = sum_j softmax(s)_j v_j,   lse = log sum_j exp(s_j)   (natural log).
 * Token j is visible if j <= p, j < lens[b], and (window == 0, or
 * j > p - window, or j < sinks): the last `window` tokens up to p itself, and
 * the first `sinks` ones. A query that sees nothing (lens[b] == 0, more new
 * tokens than lens[b], or a row of no sequence) gives out = 0, lse = -inf.
 * So does one whose visible scores are all -inf (no softmax of theirs exists);
 * a visible score of +inf or NaN gives NaN in out and lse, and an infinity of a
 * visible v_j whose weight is below binary32 gives an infinity or NaN.
 * What is stored in tokens that a query does not see, infinities and NaN
 * included, never reaches its output. If a visible token's table entry is not
 * a page of the cache, or lens[b] is negative or beyond the row, the outputs
 * concerned are NaN (the queries of that sequence's tile). If cu does not
 * ascend or leaves 0 .. tokens, all outputs are NaN.
 * q: QBN_BF16 with strides as in qbn_kv_append; out: bfloat16
 * [tokens][q_heads][head_dim], lse: binary32 [tokens][q_heads] or NULL.
 * q_heads % heads == 0; scale * log2 e is finite.
 * Elements times their scales enter as bfloat16, which holds them exactly but
 * for two ends: E4M3 values with scale bytes 0 to 2 may lie below its smallest
 * (rounded to nearest), and E4M3 with bytes from 247 and E2M1 with bytes from
 * 253 on may pass its largest (infinite). qbn_kv_append writes those bytes only
 * for magnitudes below 2^-116, and for infinities. Products are exact; sums,
 * softmax statistics and accumulators are binary32. The softmax weights are
 * rounded to bfloat16 for the product with V (by 2^-8 of each at most, as much
 * as the output's own rounding), their sum is not. The sums are divided at the
 * end: they hold a |v_j| times the number of tokens of 2^100 (of 2^40 where
 * scores pass 10^7). No atomics: repeated calls give bit-identical results.
 * The work is split over a sequence's length where there are few sequences;
 * the pieces go through `workspace` (device, 16-byte aligned, at least
 * qbn_kv_attention_workspace bytes, not kept: it may be shared by calls that
 * follow each other on a stream). That function gives -1, and the calls
 * QBN_ERR_SHAPE, also where a launch would have 2^32 threads or more (from
 * about 2^24 pairs of a sequence and 16 query heads of a key-value head on). */
QBN_API int64_t qbn_kv_attention_workspace(const qbn_kv_cache *cache, const qbn_kv_batch *batch, int32_t q_heads,
                                           int32_t window, int32_t sinks, int32_t decode);

/* One new token per sequence: batch->cu must be NULL. */
QBN_API int32_t qbn_kv_attention_decode(const qbn_kv_cache *cache, int64_t layer, const qbn_kv_batch *batch,
                                        int32_t q_heads, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                        float scale, int32_t window, int32_t sinks, void *out, float *lse,
                                        void *workspace, int64_t workspace_bytes, void *stream);

/* Chunks of new tokens, causal. */
QBN_API int32_t qbn_kv_attention_prefill(const qbn_kv_cache *cache, int64_t layer, const qbn_kv_batch *batch,
                                         int32_t q_heads, const void *q, int64_t q_token_stride,
                                         int64_t q_head_stride, float scale, int32_t window, int32_t sinks, void *out,
                                         float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/* Page bookkeeping, all on the device. Each call reads the pool `in` and
 * writes the pool `out`, which has the same sizes and is either in itself
 * (the same three pointers) or wholly separate from it (tables that another
 * stream still reads stay as they are). Pages are taken in a fixed order (the
 * lowest-numbered free pages, in the order of the requests), so results do
 * not depend on scheduling. status (device int32) receives -1, or the index
 * of the first request that cannot be met; then nothing changes (out receives
 * in). workspace: device, 16-byte aligned, qbn_kv_pool_workspace(out, count)
 * bytes. At most 2^20 pages and 2^20 slots. */
QBN_API int64_t qbn_kv_pool_workspace(const qbn_kv_pool *pool, int64_t count);

/* Room for tokens[i] >= 0 more tokens in slot rows[i], i < count: the slot's
 * length grows by tokens[i], and the pages it then needs beyond those it has
 * are taken. Request i fails if its slot is out of range or named before,
 * tokens[i] < 0, the row is too short, or the free pages run out. */
QBN_API int32_t qbn_kv_reserve(const qbn_kv_pool *in, const qbn_kv_pool *out, int64_t count, const int32_t *rows,
                               const int32_t *tokens, int32_t *status, void *workspace, int64_t workspace_bytes,
                               void *stream);

/* Slot children[i] (of length 0) becomes a copy of slot parents[i]: full
 * pages are shared, a last page that is not full is copied, in every layer,
 * to a page taken for it, so that both can append. Request i fails if a slot
 * is out of range, the child is named before, is its own parent or has a
 * length, the parent's length is outside its row, the page to copy is not a
 * page of the pool, or the free pages run out. */
QBN_API int32_t qbn_kv_fork(const qbn_kv_cache *cache, const qbn_kv_pool *in, const qbn_kv_pool *out, int64_t count,
                            const int32_t *parents, const int32_t *children, int32_t *status, void *workspace,
                            int64_t workspace_bytes, void *stream);

/* Give back the pages of slots rows[i]. window == 0: every page; the slot's
 * entries become -1 and its length 0. window > 0: only pages all of whose
 * tokens lie at or beyond `sinks` and more than `window` before the slot's
 * length (no later query of that window sees them); the length stays. A page
 * is free once nothing names it. Slots out of range are passed over, one
 * named twice counts once. */
QBN_API int32_t qbn_kv_free(const qbn_kv_pool *in, const qbn_kv_pool *out, int64_t count, const int32_t *rows,
                            int32_t window, int32_t sinks, void *stream);

/* Pack the pool: with L pages in use, those at or beyond L move, in order,
 * into the free pages below L (in every layer), and the tables follow. *live
 * (device int32) receives L. Afterwards pages L and up are free. */
QBN_API int32_t qbn_kv_compact(const qbn_kv_cache *cache, const qbn_kv_pool *in, const qbn_kv_pool *out,
                               int32_t *live, void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QBN_KV_H */
