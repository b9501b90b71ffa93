/*
 * qbn_moe.h - C ABI of the qbn library's mixture-of-experts layer over 4-bit
 * weights: choosing a few experts for each token, and the experts' products,
 * for AMD Instinct MI355X (gfx950).
 *
 * The conventions of qbn.h hold here too: caller-owned DEVICE pointers, calls
 * asynchronous on `stream`, nothing allocated, nothing retained, every
 * argument checked on the host before anything is enqueued. What the host
 * cannot see (the chosen experts) is checked on the device. No atomics whose
 * order could change a result: repeated calls give bit-identical results. All
 * calls can be captured into a HIP graph.
 *
 * The choice. logit[t][e] = sum_i x[t][i] router[e][i] (+ bias[e]), summed in
 * binary64 (the products are exact). The top_k largest of each token are its
 * experts, in falling order, equal ones by their number. Their weights are the
 * softmax over the chosen logits (normalize != 0) or over all experts'
 * (normalize == 0), in binary64, rounded to binary32. NaN ranks as -inf
 * does, below every finite number, and a token with a logit of NaN or +inf, or with none above -inf,
 * has weights of NaN; ids are valid and distinct in any case.
 *
 * The experts. For token t with experts e_j and weights w_j:
 *   h_j = silu(gate_j) * up_j,  gate_j = W13[e_j][0 .. inter) x,
 *   up_j = W13[e_j][inter .. 2 inter) x,   silu(a) = a / (1 + exp(-a)),
 *   out = sum_j w_j W2[e_j] h_j   (in the order of j, rounded once).
 * An id that is no expert's stands for none: it adds nothing, whatever its
 * weight. A token without experts gives 0. The same expert twice counts twice.
 * Weights enter the products as bfloat16, which holds every E2M1 value times
 * its scale exactly (scale byte 0 with code 1 or 9 as a subnormal) but for
 * those that pass its largest, with MXFP4 scale bytes 253 and 254: they are
 * infinite, and every sum that one enters is infinite or NaN. (Of the products
 * of such a block some may be with zeros that pad x or h, or with a part of h
 * that is 0.) Products are exact and sums binary32. h is held as the sum of two
 * bfloat16 values (2^-17 relative), and silu(a) for a < -87 may be 0 instead of
 * less than 2^-119. NVFP4's factor per expert is applied to the
 * sums.
 */
#ifndef QBN_MOE_H
#define QBN_MOE_H

#include "qbn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qbn_moe_router {
    int32_t experts;     /* 1 .. 1024 */
    int32_t top_k;       /* 1 .. min(experts, 32) */
    int32_t hidden;      /* a multiple of 32, at most 2^16 */
    int32_t normalize;   /* 0 or 1 */
    const void *weight;  /* bfloat16 [experts][hidden], 16-byte aligned */
    const float *bias;   /* [experts] or NULL */
} qbn_moe_router;

typedef struct qbn_moe_weights {
    int32_t format;    /* QBN_MXFP4 or QBN_NVFP4 */
    int32_t experts;   /* 1 .. 1024 */
    int32_t hidden;    /* a multiple of 32, at most 2^16 */
    int32_t inter;     /* a multiple of 32, at most 2^16 */
    const void *w13;        /* u8 [experts][2 inter][hidden / 2], 16-byte aligned */
    const void *w13_scales; /* u8 [experts][2 inter][hidden / 32], NVFP4: hidden / 16; 16-byte aligned */
    const void *w2;         /* u8 [experts][hidden][inter / 2], 16-byte aligned */
    const void *w2_scales;  /* u8 [experts][hidden][inter / 32], NVFP4: inter / 16; 16-byte aligned */
    const float *w13_scale2, *w2_scale2; /* NVFP4: [experts]; MXFP4: NULL */
} qbn_moe_weights;

/* sizeof of the two structs above, for bindings: which = 0, 1. */
QBN_API size_t qbn_moe_struct_size(int32_t which);

/* Tokens whose work goes through a workspace at a time; more are done in so
 * many portions, each reading the weights that it needs. */
#define QBN_MOE_PORTION 256

/* Bytes of workspace that the calls below need for `tokens` tokens of top_k
 * experts each: for the choice (experts NULL), for the experts' products
 * (router NULL), or for both; -1 where an argument is not valid. Device,
 * 16-byte aligned, any content; not kept: calls that follow each other on a
 * stream may share it, and one that serves a number of tokens serves every
 * smaller one. What a call writes (ids, weights, out, the workspace) shares
 * no byte with anything else that it is given. */
QBN_API int64_t qbn_moe_workspace(const qbn_moe_router *router, const qbn_moe_weights *experts, int64_t tokens,
                                  int32_t top_k);

/* ids int32 [tokens][top_k], weights binary32 [tokens][top_k]. x: bfloat16
 * [tokens][x_stride], 16-byte aligned, x_stride (elements) >= hidden and a
 * multiple of 8. */
QBN_API int32_t qbn_moe_route(const qbn_moe_router *router, int64_t tokens, const void *x, int64_t x_stride,
                              int32_t *ids, float *weights, void *workspace, int64_t workspace_bytes, void *stream);

/* out: bfloat16 [tokens][out_stride], out_stride >= hidden; it shares no byte
 * with x's rows (from the first to the last). */
QBN_API int32_t qbn_moe_experts(const qbn_moe_weights *experts, int64_t tokens, int32_t top_k, const void *x,
                                int64_t x_stride, const int32_t *ids, const float *weights, void *out,
                                int64_t out_stride, void *workspace, int64_t workspace_bytes, void *stream);

/* Both in one call; ids and weights receive the choice. */
QBN_API int32_t qbn_moe(const qbn_moe_router *router, const qbn_moe_weights *experts, int64_t tokens, const void *x,
                        int64_t x_stride, int32_t *ids, float *weights, void *out, int64_t out_stride,
                        void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QBN_MOE_H */
