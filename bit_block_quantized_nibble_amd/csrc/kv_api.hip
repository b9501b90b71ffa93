// C-ABI entry points of the paged key-value cache and of the rotation by
// positions: host-side argument checks, then dispatch to the launchers. Nothing
// is enqueued by a rejected call.
#include <math.h>

#include "kv_launch.h"
#include "qbn_launch.h"
#include "rope_launch.h"

namespace {

using qbn::hip_status;

constexpr int64_t kMaxElems = (int64_t)1 << 46;  // elements of K of one layer: byte offsets stay in 64 bits
constexpr int64_t kMaxTokens = (int64_t)1 << 30; // tokens of a sequence, of a batch: positions stay in 32 bits
constexpr int64_t kMaxPool = (int64_t)1 << 20;   // pages and slots of a pool: one workgroup scans them

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

bool known_format(int32_t f) { return f == QBN_KV_BF16 || f == QBN_MXFP8 || f == QBN_MXFP4; }
bool known_page(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }
bool known_dim(int32_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

// Format and sizes of a cache; the number of K's elements in *elems.
int32_t check_shape(int32_t format, int64_t layers, int64_t pages, int32_t heads, int32_t page_size, int32_t head_dim,
                    int64_t *elems) {
    if (!known_format(format)) return QBN_ERR_FORMAT;
    if (!known_page(page_size)) return QBN_ERR_SHAPE;
    if (!known_dim(head_dim)) return QBN_ERR_UNSUPPORTED;
    if (layers <= 0 || pages <= 0 || heads <= 0) return QBN_ERR_SHAPE;
    if (pages > kMaxTokens || heads > (1 << 12) || layers > (1 << 20)) return QBN_ERR_SHAPE;
    const int64_t page = (int64_t)heads * page_size * head_dim;  // < 2^28, so that a page's bytes fit 32 bits
    if (pages > kMaxElems / page || layers > kMaxElems / (page * pages)) return QBN_ERR_SHAPE;
    *elems = layers * pages * page;
    return QBN_OK;
}

int32_t check_cache(const qbn_kv_cache *c) {
    if (!c) return QBN_ERR_NULL;
    int64_t elems;
    const int32_t st = check_shape(c->format, c->layers, c->pages, c->heads, c->page_size, c->head_dim, &elems);
    if (st) return st;
    if (!c->k || !c->v) return QBN_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return QBN_ERR_ALIGN;
    if (c->format != QBN_KV_BF16) {
        if (!c->k_scales || !c->v_scales) return QBN_ERR_NULL;
        if (!aligned(c->k_scales, 16) || !aligned(c->v_scales, 16)) return QBN_ERR_ALIGN;
    }
    return QBN_OK;
}

int32_t check_batch(const qbn_kv_cache *c, int64_t layer, const qbn_kv_batch *b) {
    int32_t st = check_cache(c);
    if (st) return st;
    if (!b) return QBN_ERR_NULL;
    if (layer < 0 || layer >= c->layers) return QBN_ERR_SHAPE;
    if (b->seqs < 0 || b->tokens < 0 || b->row < 0 || b->seqs > kMaxPool || b->tokens > kMaxTokens) return QBN_ERR_SHAPE;
    if (b->row > kMaxTokens / c->page_size || b->row_stride < b->row || b->row_stride > kMaxTokens) return QBN_ERR_SHAPE;
    if (!b->cu && b->tokens != b->seqs) return QBN_ERR_SHAPE;
    if (b->seqs == 0 || b->tokens == 0) return b->tokens == 0 ? QBN_OK : QBN_ERR_SHAPE;
    if (!b->lens || (b->row > 0 && !b->table)) return QBN_ERR_NULL;
    if (!aligned(b->lens, 4) || !aligned(b->table, 4) || !aligned(b->cu, 4)) return QBN_ERR_ALIGN;
    return QBN_OK;
}

// Vectors of `dim` elements of `size` bytes per (token, head): 16-byte pieces.
int32_t check_rows(const void *p, int64_t token_stride, int64_t head_stride, int64_t tokens, int64_t heads, int size) {
    if (!p) return QBN_ERR_NULL;
    if (token_stride < 0 || head_stride < 0 || token_stride > kMaxElems / tokens || head_stride > kMaxElems / heads)
        return QBN_ERR_SHAPE;
    if (!aligned(p, 16) || token_stride * size % 16 || head_stride * size % 16) return QBN_ERR_ALIGN;
    return QBN_OK;
}

int32_t check_pool(const qbn_kv_pool *p) {
    if (!p) return QBN_ERR_NULL;
    if (p->reserved != 0) return QBN_ERR_FORMAT;
    if (!known_page(p->page_size)) return QBN_ERR_SHAPE;
    if (p->seqs < 0 || p->row < 0 || p->pages < 0 || p->seqs > kMaxPool || p->pages > kMaxPool) return QBN_ERR_SHAPE;
    if (p->row > kMaxTokens / p->page_size) return QBN_ERR_SHAPE;
    if ((p->seqs > 0 && (!p->lens || (p->row > 0 && !p->table))) || (p->pages > 0 && !p->refs)) return QBN_ERR_NULL;
    if (!aligned(p->table, 4) || !aligned(p->lens, 4) || !aligned(p->refs, 4)) return QBN_ERR_ALIGN;
    return QBN_OK;
}

bool apart(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return na == 0 || nb == 0 || x + 4 * (uintptr_t)na <= y || y + 4 * (uintptr_t)nb <= x;
}

// in and out: the same tables, or tables with no byte in common.
int32_t check_pools(const qbn_kv_pool *in, const qbn_kv_pool *out, int64_t count) {
    int32_t st = check_pool(in);
    if (!st) st = check_pool(out);
    if (st) return st;
    if (in->seqs != out->seqs || in->row != out->row || in->pages != out->pages || in->page_size != out->page_size)
        return QBN_ERR_SHAPE;
    if (count < 0 || count > kMaxPool) return QBN_ERR_SHAPE;
    if (in->table == out->table && in->lens == out->lens && in->refs == out->refs) return QBN_OK;
    const void *a[3] = {in->table, in->lens, in->refs}, *b[3] = {out->table, out->lens, out->refs};
    const int64_t n[3] = {in->seqs * in->row, in->seqs, in->pages};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j)
            if (!apart(a[i], n[i], b[j], n[j])) return QBN_ERR_UNSUPPORTED;
    return QBN_OK;
}

int32_t check_workspace(const void *ws, int64_t have, int64_t need) {
    if (need < 0) return QBN_ERR_SHAPE;
    if (need == 0) return QBN_OK;
    if (!ws) return QBN_ERR_NULL;
    if (!aligned(ws, 16)) return QBN_ERR_ALIGN;
    return have < need ? QBN_ERR_SHAPE : QBN_OK;
}

int32_t check_cache_pool(const qbn_kv_cache *c, const qbn_kv_pool *p) {
    const int32_t st = check_cache(c);
    if (st) return st;
    if (!p) return QBN_ERR_NULL;
    return c->pages != p->pages || c->page_size != p->page_size ? QBN_ERR_SHAPE : QBN_OK;
}

int32_t check_attention(const qbn_kv_cache *c, int64_t layer, const qbn_kv_batch *b, int32_t q_heads, const void *q,
                        int64_t qt, int64_t qh, float scale, int32_t window, int32_t sinks, const void *out,
                        const float *lse) {
    int32_t st = check_batch(c, layer, b);
    if (st) return st;
    if (q_heads <= 0 || q_heads % c->heads || q_heads > (1 << 16)) return QBN_ERR_SHAPE;
    if (window < 0 || sinks < 0 || window > kMaxTokens || sinks > kMaxTokens) return QBN_ERR_SHAPE;
    if (!isfinite(scale * (float)M_LOG2E)) return QBN_ERR_SHAPE;  // the kernels' factor
    if (b->tokens == 0) return QBN_OK;
    if (b->tokens > kMaxTokens / q_heads) return QBN_ERR_SHAPE;
    st = check_rows(q, qt, qh, b->tokens, q_heads, 2);
    if (st) return st;
    if (!out) return QBN_ERR_NULL;
    return aligned(out, 16) && aligned(lse, 4) ? QBN_OK : QBN_ERR_ALIGN;
}

int32_t check_rotation(const qbn_rotation *r, int32_t dim) {
    if (!r) return QBN_ERR_NULL;
    if ((r->layout != QBN_ROPE_HALF && r->layout != QBN_ROPE_INTERLEAVED) || r->reserved != 0) return QBN_ERR_FORMAT;
    if (r->rot <= 0 || r->rot % 16 || r->rot > dim || !isfinite(r->factor)) return QBN_ERR_SHAPE;
    if (!r->turns) return QBN_ERR_NULL;
    return aligned(r->turns, 16) ? QBN_OK : QBN_ERR_ALIGN;
}

// The bytes from the first to the last of [tokens][heads] vectors of `dim` elements.
uintptr_t extent(int64_t token_stride, int64_t head_stride, int64_t tokens, int64_t heads, int64_t dim, int size) {
    return ((tokens - 1) * token_stride + (heads - 1) * head_stride + dim) * size;
}
bool ranges_apart(const void *a, uintptr_t na, const void *b, uintptr_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x + na <= y || y + nb <= x;
}

// Vectors to be written: as check_rows, and no two share an element.
int32_t check_rows_out(const void *p, int64_t token_stride, int64_t head_stride, int64_t tokens, int64_t heads,
                       int64_t dim, int size) {
    const int32_t st = check_rows(p, token_stride, head_stride, tokens, heads, size);
    if (st) return st;
    const int64_t t = tokens > 1 ? token_stride : INT64_MAX, h = heads > 1 ? head_stride : INT64_MAX;
    const bool heads_inner = h >= dim && (tokens == 1 || t >= (heads - 1) * head_stride + dim);
    const bool tokens_inner = t >= dim && (heads == 1 || h >= (tokens - 1) * token_stride + dim);
    return heads_inner || tokens_inner ? QBN_OK : QBN_ERR_SHAPE;
}

}  // namespace

extern "C" {

size_t qbn_rotation_struct_size(void) { return sizeof(qbn_rotation); }

int32_t qbn_rope(const qbn_rotation *rope, int64_t tokens, int32_t heads, int32_t dim, const int32_t *positions,
                 const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out, int64_t out_token_stride,
                 int64_t out_head_stride, int32_t dtype, void *stream) {
    if (dim <= 0 || dim % 16 || dim > 1024 || tokens < 0 || heads < 0 || heads > (1 << 16) || tokens > kMaxTokens)
        return QBN_ERR_SHAPE;
    int32_t st = check_rotation(rope, dim);
    if (st) return st;
    if (dtype < QBN_F32 || dtype > QBN_F16) return QBN_ERR_FORMAT;
    if (dtype == QBN_F16) return QBN_ERR_DTYPE;
    if (tokens == 0 || heads == 0) return QBN_OK;
    if (!positions) return QBN_ERR_NULL;
    if (!aligned(positions, 4)) return QBN_ERR_ALIGN;
    const int size = dtype == QBN_F32 ? 4 : 2;
    st = check_rows(x, x_token_stride, x_head_stride, tokens, heads, size);
    if (!st) st = check_rows_out(out, out_token_stride, out_head_stride, tokens, heads, dim, size);
    if (st) return st;
    const bool same = x == out && (tokens == 1 || x_token_stride == out_token_stride) &&
                      (heads == 1 || x_head_stride == out_head_stride);
    if (!same && !ranges_apart(x, extent(x_token_stride, x_head_stride, tokens, heads, dim, size), out,
                               extent(out_token_stride, out_head_stride, tokens, heads, dim, size)))
        return QBN_ERR_UNSUPPORTED;
    return hip_status(qbn::launch_rope(*rope, tokens, heads, dim, positions, {x, x_token_stride, x_head_stride},
                                       {out, out_token_stride, out_head_stride}, dtype, (hipStream_t)stream));
}

int32_t qbn_kv_append_rope(const qbn_kv_cache *cache, int64_t layer, const qbn_kv_batch *batch,
                           const qbn_rotation *rope, int32_t q_heads, const void *q, int64_t q_token_stride,
                           int64_t q_head_stride, void *q_out, int64_t out_token_stride, int64_t out_head_stride,
                           const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                           int64_t v_token_stride, int64_t v_head_stride, int32_t dtype, void *stream) {
    int32_t st = check_batch(cache, layer, batch);
    if (!st) st = check_rotation(rope, cache->head_dim);
    if (st) return st;
    if (dtype < QBN_F32 || dtype > QBN_F16) return QBN_ERR_FORMAT;
    if (dtype == QBN_F16) return QBN_ERR_DTYPE;
    if (q_heads < 0 || q_heads > (1 << 16)) return QBN_ERR_SHAPE;
    if (batch->tokens == 0) return QBN_OK;
    const int64_t tokens = batch->tokens, dim = cache->head_dim;
    const int size = dtype == QBN_F32 ? 4 : 2;
    st = check_rows(k, k_token_stride, k_head_stride, tokens, cache->heads, size);
    if (!st) st = check_rows(v, v_token_stride, v_head_stride, tokens, cache->heads, size);
    if (!st && q_heads) st = check_rows(q, q_token_stride, q_head_stride, tokens, q_heads, size);
    if (!st && q_heads) st = check_rows_out(q_out, out_token_stride, out_head_stride, tokens, q_heads, dim, 2);
    if (st) return st;
    if (q_heads) {
        const uintptr_t n = extent(out_token_stride, out_head_stride, tokens, q_heads, dim, 2);
        const bool same = q == q_out && dtype == QBN_BF16 && (tokens == 1 || q_token_stride == out_token_stride) &&
                          (q_heads == 1 || q_head_stride == out_head_stride);
        if (!same &&
            !(ranges_apart(q, extent(q_token_stride, q_head_stride, tokens, q_heads, dim, size), q_out, n) &&
              ranges_apart(k, extent(k_token_stride, k_head_stride, tokens, cache->heads, dim, size), q_out, n) &&
              ranges_apart(v, extent(v_token_stride, v_head_stride, tokens, cache->heads, dim, size), q_out, n)))
            return QBN_ERR_UNSUPPORTED;
    }
    return hip_status(qbn::launch_kv_append_rope(
        *cache, layer, *batch, *rope, q_heads, {q, q_token_stride, q_head_stride},
        {q_out, out_token_stride, out_head_stride}, {k, k_token_stride, k_head_stride},
        {v, v_token_stride, v_head_stride}, dtype, (hipStream_t)stream));
}

size_t qbn_kv_struct_size(int32_t which) {
    return which == 0 ? sizeof(qbn_kv_cache) : which == 1 ? sizeof(qbn_kv_batch) : which == 2 ? sizeof(qbn_kv_pool) : 0;
}

int64_t qbn_kv_bytes(int32_t format, int64_t layers, int64_t pages, int32_t heads, int32_t page_size, int32_t head_dim,
                     int32_t part) {
    int64_t n;
    if (part < 0 || part > 1 || check_shape(format, layers, pages, heads, page_size, head_dim, &n)) return -1;
    if (part == 1) return format == QBN_KV_BF16 ? 0 : n / 32;
    return format == QBN_KV_BF16 ? 2 * n : format == QBN_MXFP8 ? n : n / 2;
}

int32_t qbn_kv_append(const qbn_kv_cache *cache, int64_t layer, const qbn_kv_batch *batch, const void *k,
                      int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                      int64_t v_head_stride, int32_t dtype, void *stream) {
    int32_t st = check_batch(cache, layer, batch);
    if (st) return st;
    if (dtype < QBN_F32 || dtype > QBN_F16) return QBN_ERR_FORMAT;
    if (dtype == QBN_F16) return QBN_ERR_DTYPE;
    if (batch->tokens == 0 || batch->row == 0) return QBN_OK;
    const int size = dtype == QBN_F32 ? 4 : 2;
    st = check_rows(k, k_token_stride, k_head_stride, batch->tokens, cache->heads, size);
    if (!st) st = check_rows(v, v_token_stride, v_head_stride, batch->tokens, cache->heads, size);
    if (st) return st;
    return hip_status(qbn::launch_kv_append(*cache, layer, *batch, {k, k_token_stride, k_head_stride},
                                            {v, v_token_stride, v_head_stride}, dtype, (hipStream_t)stream));
}

int64_t qbn_kv_attention_workspace(const qbn_kv_cache *cache, const qbn_kv_batch *batch, int32_t q_heads,
                                   int32_t window, int32_t sinks, int32_t decode) {
    if (!cache || !batch || q_heads <= 0) return -1;
    int64_t n;
    if (check_shape(cache->format, cache->layers, cache->pages, cache->heads, cache->page_size, cache->head_dim, &n))
        return -1;
    if (q_heads % cache->heads || q_heads > (1 << 16) || batch->seqs < 0 || batch->seqs > kMaxPool || batch->row < 0 ||
        batch->row > kMaxTokens / cache->page_size || batch->tokens < 0 || batch->tokens > kMaxTokens / q_heads ||
        window < 0 || sinks < 0)
        return -1;
    return decode ? qbn::kv_decode_workspace(*cache, *batch, q_heads, window, sinks)
                  : qbn::kv_prefill_workspace(*cache, *batch, q_heads, window, sinks);
}

int32_t qbn_kv_attention_decode(const qbn_kv_cache *cache, int64_t layer, const qbn_kv_batch *batch, int32_t q_heads,
                                const void *q, int64_t q_token_stride, int64_t q_head_stride, float scale,
                                int32_t window, int32_t sinks, void *out, float *lse, void *workspace,
                                int64_t workspace_bytes, void *stream) {
    int32_t st = check_attention(cache, layer, batch, q_heads, q, q_token_stride, q_head_stride, scale, window, sinks,
                                 out, lse);
    if (st) return st;
    if (batch->cu) return QBN_ERR_UNSUPPORTED;
    if (batch->tokens == 0) return QBN_OK;
    st = check_workspace(workspace, workspace_bytes, qbn::kv_decode_workspace(*cache, *batch, q_heads, window, sinks));
    if (st) return st;
    return hip_status(qbn::launch_kv_decode(*cache, layer, *batch, q_heads, {q, q_token_stride, q_head_stride}, scale,
                                            window, sinks, out, lse, workspace, (hipStream_t)stream));
}

int32_t qbn_kv_attention_prefill(const qbn_kv_cache *cache, int64_t layer, const qbn_kv_batch *batch, int32_t q_heads,
                                 const void *q, int64_t q_token_stride, int64_t q_head_stride, float scale,
                                 int32_t window, int32_t sinks, void *out, float *lse, void *workspace,
                                 int64_t workspace_bytes, void *stream) {
    int32_t st = check_attention(cache, layer, batch, q_heads, q, q_token_stride, q_head_stride, scale, window, sinks,
                                 out, lse);
    if (st) return st;
    if (batch->tokens == 0) return QBN_OK;
    st = check_workspace(workspace, workspace_bytes, qbn::kv_prefill_workspace(*cache, *batch, q_heads, window, sinks));
    if (st) return st;
    return hip_status(qbn::launch_kv_prefill(*cache, layer, *batch, q_heads, {q, q_token_stride, q_head_stride}, scale,
                                             window, sinks, out, lse, workspace, (hipStream_t)stream));
}

int64_t qbn_kv_pool_workspace(const qbn_kv_pool *pool, int64_t count) {
    if (!pool || count < 0 || count > kMaxPool || pool->seqs < 0 || pool->seqs > kMaxPool || pool->pages < 0 ||
        pool->pages > kMaxPool)
        return -1;
    return qbn::kv_pool_workspace(*pool, count);
}

int32_t qbn_kv_reserve(const qbn_kv_pool *in, const qbn_kv_pool *out, int64_t count, const int32_t *rows,
                       const int32_t *tokens, int32_t *status, void *workspace, int64_t workspace_bytes,
                       void *stream) {
    int32_t st = check_pools(in, out, count);
    if (st) return st;
    if (!status || (count > 0 && (!rows || !tokens))) return QBN_ERR_NULL;
    if (!aligned(status, 4) || !aligned(rows, 4) || !aligned(tokens, 4)) return QBN_ERR_ALIGN;
    st = check_workspace(workspace, workspace_bytes, qbn::kv_pool_workspace(*out, count));
    if (st) return st;
    return hip_status(qbn::launch_kv_reserve(*in, *out, count, rows, tokens, status, workspace, (hipStream_t)stream));
}

int32_t qbn_kv_fork(const qbn_kv_cache *cache, const qbn_kv_pool *in, const qbn_kv_pool *out, int64_t count,
                    const int32_t *parents, const int32_t *children, int32_t *status, void *workspace,
                    int64_t workspace_bytes, void *stream) {
    int32_t st = check_pools(in, out, count);
    if (!st) st = check_cache_pool(cache, in);
    if (st) return st;
    if (!status || (count > 0 && (!parents || !children))) return QBN_ERR_NULL;
    if (!aligned(status, 4) || !aligned(parents, 4) || !aligned(children, 4)) return QBN_ERR_ALIGN;
    st = check_workspace(workspace, workspace_bytes, qbn::kv_pool_workspace(*out, count));
    if (st) return st;
    return hip_status(qbn::launch_kv_fork(*cache, *in, *out, count, parents, children, status, workspace,
                                          (hipStream_t)stream));
}

int32_t qbn_kv_free(const qbn_kv_pool *in, const qbn_kv_pool *out, int64_t count, const int32_t *rows, int32_t window,
                    int32_t sinks, void *stream) {
    const int32_t st = check_pools(in, out, count);
    if (st) return st;
    if (window < 0 || sinks < 0 || window > kMaxTokens || sinks > kMaxTokens) return QBN_ERR_SHAPE;
    if (count > 0 && !rows) return QBN_ERR_NULL;
    if (!aligned(rows, 4)) return QBN_ERR_ALIGN;
    return hip_status(qbn::launch_kv_free(*in, *out, count, rows, window, sinks, (hipStream_t)stream));
}

int32_t qbn_kv_compact(const qbn_kv_cache *cache, const qbn_kv_pool *in, const qbn_kv_pool *out, int32_t *live,
                       void *workspace, int64_t workspace_bytes, void *stream) {
    int32_t st = check_pools(in, out, 0);
    if (!st) st = check_cache_pool(cache, in);
    if (st) return st;
    if (!live) return QBN_ERR_NULL;
    if (!aligned(live, 4)) return QBN_ERR_ALIGN;
    st = check_workspace(workspace, workspace_bytes, qbn::kv_pool_workspace(*out, 0));
    if (st) return st;
    return hip_status(qbn::launch_kv_compact(*cache, *in, *out, live, workspace, (hipStream_t)stream));
}

}  // extern "C"
