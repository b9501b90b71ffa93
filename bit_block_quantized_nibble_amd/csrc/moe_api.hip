// C-ABI entry points of the experts' layer: host-side argument checks, then
// dispatch to the launchers. Nothing is enqueued by a rejected call.
#include "moe_launch.h"
#include "qbn_launch.h"

namespace {

using qbn::hip_status;

constexpr int64_t kMaxTokens = (int64_t)1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 30;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool known_width(int32_t w) { return w > 0 && w % 32 == 0 && w <= (1 << 16); }
bool known_top(int32_t k) { return k > 0 && k <= 32; }

int32_t check_router_shape(const qbn_moe_router *r) {
    if (!r) return QBN_ERR_NULL;
    if (r->experts <= 0 || r->experts > 1024 || !known_top(r->top_k) || r->top_k > r->experts || !known_width(r->hidden))
        return QBN_ERR_SHAPE;
    return r->normalize == 0 || r->normalize == 1 ? QBN_OK : QBN_ERR_FORMAT;
}
int32_t check_router(const qbn_moe_router *r) {
    const int32_t st = check_router_shape(r);
    if (st) return st;
    if (!r->weight) return QBN_ERR_NULL;
    return aligned(r->weight, 16) && aligned(r->bias, 4) ? QBN_OK : QBN_ERR_ALIGN;
}

int32_t check_experts_shape(const qbn_moe_weights *e) {
    if (!e) return QBN_ERR_NULL;
    if (e->format != QBN_MXFP4 && e->format != QBN_NVFP4)
        return e->format >= QBN_MXFP4 && e->format <= QBN_NVFP4_CKE ? QBN_ERR_UNSUPPORTED : QBN_ERR_FORMAT;
    if (e->experts <= 0 || e->experts > 1024 || !known_width(e->hidden) || !known_width(e->inter)) return QBN_ERR_SHAPE;
    return QBN_OK;
}
int32_t check_experts(const qbn_moe_weights *e) {
    const int32_t st = check_experts_shape(e);
    if (st) return st;
    if (!e->w13 || !e->w13_scales || !e->w2 || !e->w2_scales) return QBN_ERR_NULL;
    if (!aligned(e->w13, 16) || !aligned(e->w13_scales, 16) || !aligned(e->w2, 16) || !aligned(e->w2_scales, 16))
        return QBN_ERR_ALIGN;
    if (e->format == QBN_MXFP4) return e->w13_scale2 || e->w2_scale2 ? QBN_ERR_SCALE2 : QBN_OK;
    if (!e->w13_scale2 || !e->w2_scale2) return QBN_ERR_NULL;
    return aligned(e->w13_scale2, 4) && aligned(e->w2_scale2, 4) ? QBN_OK : QBN_ERR_ALIGN;
}

// Rows of `hidden` bfloat16 values: 16-byte pieces.
int32_t check_rows(const void *p, int64_t stride, int64_t tokens, int64_t hidden) {
    if (!p) return QBN_ERR_NULL;
    if ((tokens > 1 && stride < hidden) || stride > kMaxStride) return QBN_ERR_SHAPE;
    return aligned(p, 16) && (tokens == 1 || stride % 8 == 0) ? QBN_OK : QBN_ERR_ALIGN;
}

int32_t check_choice(const int32_t *ids, const float *weights) {
    if (!ids || !weights) return QBN_ERR_NULL;
    return aligned(ids, 4) && aligned(weights, 4) ? QBN_OK : QBN_ERR_ALIGN;
}

int32_t check_workspace(const void *ws, int64_t have, int64_t need) {
    if (!ws) return QBN_ERR_NULL;
    if (!aligned(ws, 16)) return QBN_ERR_ALIGN;
    return have < need ? QBN_ERR_SHAPE : QBN_OK;
}

bool apart(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x + (uintptr_t)na <= y || y + (uintptr_t)nb <= x;
}

int32_t check_out(const void *x, int64_t xs, const void *out, int64_t os, int64_t tokens, int64_t hidden) {
    const int32_t st = check_rows(out, os, tokens, hidden);
    if (st) return st;
    const int64_t n = tokens - 1;
    return apart(x, (n * xs + hidden) * 2, out, (n * os + hidden) * 2) ? QBN_OK : QBN_ERR_UNSUPPORTED;
}

int64_t rounded(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace

extern "C" {

size_t qbn_moe_struct_size(int32_t which) {
    return which == 0 ? sizeof(qbn_moe_router) : which == 1 ? sizeof(qbn_moe_weights) : 0;
}

int64_t qbn_moe_workspace(const qbn_moe_router *router, const qbn_moe_weights *experts, int64_t tokens, int32_t top_k) {
    if ((!router && !experts) || tokens < 0 || tokens > kMaxTokens || !known_top(top_k)) return -1;
    if ((router && check_router_shape(router)) || (experts && check_experts_shape(experts))) return -1;
    int64_t n = 0;
    if (router) n += rounded(qbn::moe_route_workspace(*router, tokens));
    if (experts) n += rounded(qbn::moe_experts_workspace(*experts, tokens, top_k));
    return n;
}

int32_t qbn_moe_route(const qbn_moe_router *router, int64_t tokens, const void *x, int64_t x_stride, int32_t *ids,
                      float *weights, void *workspace, int64_t workspace_bytes, void *stream) {
    int32_t st = check_router(router);
    if (st) return st;
    if (tokens < 0 || tokens > kMaxTokens) return QBN_ERR_SHAPE;
    if (tokens == 0) return QBN_OK;
    st = check_rows(x, x_stride, tokens, router->hidden);
    if (!st) st = check_choice(ids, weights);
    if (!st) st = check_workspace(workspace, workspace_bytes, qbn_moe_workspace(router, nullptr, tokens, router->top_k));
    if (st) return st;
    return hip_status(qbn::launch_moe_route(*router, tokens, x, x_stride, ids, weights, workspace, (hipStream_t)stream));
}

int32_t qbn_moe_experts(const qbn_moe_weights *experts, int64_t tokens, int32_t top_k, const void *x, int64_t x_stride,
                        const int32_t *ids, const float *weights, void *out, int64_t out_stride, void *workspace,
                        int64_t workspace_bytes, void *stream) {
    int32_t st = check_experts(experts);
    if (st) return st;
    if (tokens < 0 || tokens > kMaxTokens || !known_top(top_k)) return QBN_ERR_SHAPE;
    if (tokens == 0) return QBN_OK;
    st = check_rows(x, x_stride, tokens, experts->hidden);
    if (!st) st = check_choice(ids, weights);
    if (!st) st = check_out(x, x_stride, out, out_stride, tokens, experts->hidden);
    if (!st) st = check_workspace(workspace, workspace_bytes, qbn_moe_workspace(nullptr, experts, tokens, top_k));
    if (st) return st;
    return hip_status(qbn::launch_moe_experts(*experts, tokens, top_k, x, x_stride, ids, weights, out, out_stride,
                                              workspace, (hipStream_t)stream));
}

int32_t qbn_moe(const qbn_moe_router *router, const qbn_moe_weights *experts, int64_t tokens, const void *x,
                int64_t x_stride, int32_t *ids, float *weights, void *out, int64_t out_stride, void *workspace,
                int64_t workspace_bytes, void *stream) {
    int32_t st = check_router(router);
    if (!st) st = check_experts(experts);
    if (st) return st;
    if (router->hidden != experts->hidden || router->experts != experts->experts) return QBN_ERR_SHAPE;
    if (tokens < 0 || tokens > kMaxTokens) return QBN_ERR_SHAPE;
    if (tokens == 0) return QBN_OK;
    st = check_rows(x, x_stride, tokens, experts->hidden);
    if (!st) st = check_choice(ids, weights);
    if (!st) st = check_out(x, x_stride, out, out_stride, tokens, experts->hidden);
    if (!st) st = check_workspace(workspace, workspace_bytes, qbn_moe_workspace(router, experts, tokens, router->top_k));
    if (st) return st;
    uint8_t *ws = (uint8_t *)workspace;
    st = hip_status(qbn::launch_moe_route(*router, tokens, x, x_stride, ids, weights, ws, (hipStream_t)stream));
    if (st) return st;
    return hip_status(qbn::launch_moe_experts(*experts, tokens, router->top_k, x, x_stride, ids, weights, out, out_stride,
                                              ws + rounded(qbn::moe_route_workspace(*router, tokens)),
                                              (hipStream_t)stream));
}

}  // extern "C"
