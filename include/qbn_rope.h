/*
 * qbn_rope.h - C ABI of the qbn library's rotary positions: turning queries
 * and keys by their positions, alone or on the way into the paged key-value
 * cache, for AMD Instinct MI355X (gfx950).
 *
 * The conventions of qbn.h and qbn_kv.h hold here too: caller-owned DEVICE
 * pointers, calls asynchronous on `stream`, nothing allocated, nothing
 * retained, every argument checked on the host before anything is enqueued.
 * All calls can be captured into a HIP graph.
 *
 * The rotation. Of a vector x of `dim` elements at position p, the first
 * `rot` are `rot / 2` pairs (a, b); pair i becomes
 *   a' = factor (a cos(p f_i) - b sin(p f_i)),
 *   b' = factor (b cos(p f_i) + a sin(p f_i)).
 * QBN_ROPE_HALF: pair i is (x[i], x[i + rot / 2]); QBN_ROPE_INTERLEAVED:
 * (x[2 i], x[2 i + 1]). Elements from rot on stay as they are. The frequencies
 * are given as fractions of a turn in units of 2^-64:
 *   turns[i] = round(f_i / (2 pi) * 2^64) mod 2^64,
 * so that p * turns[i] in 64-bit arithmetic that wraps is the angle without
 * its whole turns, off by |p| 2^-65 turns at most at any position. The angle
 * then enters with 32 bits after the point (1.5e-9 rad); cosine and sine are
 * within 1.5 units in the last place of binary32 of 1, products and sums are
 * binary32, the result is rounded to nearest even once. A position is any
 * int32, negative ones included.
 */
#ifndef QBN_ROPE_H
#define QBN_ROPE_H

#include "qbn_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QBN_ROPE_HALF 0
#define QBN_ROPE_INTERLEAVED 1

typedef struct qbn_rotation {
    int32_t layout;        /* QBN_ROPE_HALF or QBN_ROPE_INTERLEAVED */
    int32_t rot;           /* elements that turn: a multiple of 16, at most dim */
    float factor;          /* on cosine and sine; finite */
    int32_t reserved;      /* must be 0 */
    const uint64_t *turns; /* [rot / 2], 16-byte aligned */
} qbn_rotation;

QBN_API size_t qbn_rotation_struct_size(void);

/* out[token][head] = x[token][head] turned by positions[token] (int32
 * [tokens], on the device). x, out: `dtype` QBN_F32 or QBN_BF16, element
 * [token][head][i] at token * token_stride + head * head_stride + i (strides in
 * elements). dim is a multiple of 16 up to 1024; base pointers and strides are
 * 16-byte multiples. out is x itself (the same pointer and strides; what does
 * not turn is then not touched) or shares no byte with its range. */
QBN_API int32_t qbn_rope(const qbn_rotation *rope, int64_t tokens, int32_t heads, int32_t dim,
                         const int32_t *positions, const void *x, int64_t x_token_stride, int64_t x_head_stride,
                         void *out, int64_t out_token_stride, int64_t out_head_stride, int32_t dtype, void *stream);

/* qbn_kv_append with keys turned by their positions in their sequences (lens
 * counts the new tokens, the last is at lens - 1) before they are stored: from
 * binary32, with one rounding to the cache's format. With q_heads > 0 the
 * queries of the same rows (q, of `dtype` too) are turned alike and written to
 * q_out, bfloat16. A row that no sequence has, or whose position is negative, is
 * not stored, and its queries are copied as they are; so q_out, which may be q
 * itself (the same pointer and strides, QBN_BF16), is written in every row.
 * Otherwise it shares no byte with the ranges of q, k and v; in q's place it
 * shares no element with k and v. rope->rot is at most the cache's head_dim. */
QBN_API int32_t qbn_kv_append_rope(const qbn_kv_cache *cache, int64_t layer, const qbn_kv_batch *batch,
                                   const qbn_rotation *rope, int32_t q_heads, const void *q, int64_t q_token_stride,
                                   int64_t q_head_stride, void *q_out, int64_t out_token_stride,
                                   int64_t out_head_stride, const void *k, int64_t k_token_stride,
                                   int64_t k_head_stride, const void *v, int64_t v_token_stride,
                                   int64_t v_head_stride, int32_t dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QBN_ROPE_H */
