// Writing new tokens into the paged key-value cache with the keys turned by their
// positions on the way, and the queries beside them.
//
// The rotation is that of rope.hip, from the source's elements in binary32, and
// the rounding that of kv_append.hip, once. What a separate rotation would cost is
// its launch, a write and a read of q and k, and a rounding to bfloat16 before the one
// to the cache's format. A wave has the same elements of every head that it comes to,
// so that a token's angles are computed once for its heads of q and once for those of
// k; a step's few tokens have their heads spread over waves instead. Keys go by eight
// elements a lane, as the blocks of the MX formats want them (four lanes a block of 32),
// with the eight that they are paired with read beside them (from the same lines);
// queries go by eight pairs a lane, which lets them be turned in their place.
//
// 32 sequences' one token, 32 and 8 heads of 128, MXFP8: 4.8 us, a chain of dependent loads (length,
// page, elements) and a launch. 4789 tokens of four prompts: 25 us, 4.4 TB/s; bound by HBM.
#include "kv_store.h"
#include "rope_device.h"
#include "rope_launch.h"

namespace qbn {
namespace {

using namespace rope;

struct Args {
    Rotation r;
    uint8_t *k, *v, *ks, *vs;
    const void *sq, *sk, *sv;
    void *oq;
    int64_t qt, qh, ot, oh, kt, kh, vt, vh;  // strides in elements
    kv::Batch b;
    int heads, q_heads, dim, page_shift, pages;
    int q_each, k_each;      // heads that a wave has at a time
    int q_slices, k_slices;  // waves of a token's q, and of its k, as many of its v
    bool keep;               // oq is sq: what does not turn is there already
};

// Where a token goes: its position (negative: it has none) and, if its place
// is a page of the cache, page and slot (else page is -1).
struct Place {
    int pos, page, slot;
};
__device__ __forceinline__ Place place_of(const Args &a, int token) {
    const kv::Batch &b = a.b;
    int seq = token;
    int64_t left = 1;
    bool has = true;
    if (b.cu) {
        if (b.seqs <= 64) {
            const int lane = threadIdx.x & 63, end = lane < b.seqs ? b.cu[lane + 1] : 0x7FFFFFFF;
            seq = __popcll(__ballot(end <= token));
        } else {
            seq = kv::count_upto(b.cu, b.seqs, token);
        }
        has = seq < b.seqs;
        seq = min(seq, b.seqs - 1);
        has = has && kv::start_of(b, seq) <= token;
        left = (int64_t)kv::start_of(b, seq + 1) - token;
    }
    const int64_t pos = kv::length_of(b, seq) - left;
    if (!has || pos < 0) return {-1, -1, 0};
    const int64_t col = pos >> a.page_shift;
    const int entry = col < b.row ? kv::table_entry(b, seq, (int)col) : -1;
    return {(int)min(pos, (int64_t)0x7FFFFFFF), (uint32_t)entry < (uint32_t)a.pages ? entry : -1,
            (int)pos & ((1 << a.page_shift) - 1)};
}

template <typename T, bool HALF>
__device__ __forceinline__ void queries(const Args &a, int token, int slice) {
    const int lane = threadIdx.x & 63, groups = a.dim / 16, group = lane % groups, sub = lane / groups;
    const Lane16 at = lane16<HALF>(group, a.r.rot);
    const T *x = (const T *)a.sq + token * a.qt;
    __bf16 *out = (__bf16 *)a.oq + token * a.ot;
    int h = slice * a.q_each + sub;
    if (sub >= a.q_each || (a.keep && !at.turns)) h = a.q_heads;
    Eight<T> p, q;
    if (h < a.q_heads) p = load8(x + h * a.qh + at.first), q = load8(x + h * a.qh + at.second);
    u32x2 turns[8];
    load_turns(a.r, at.turns ? 8 * group : 0, turns);
    const Place place = place_of(a, token);
    const bool turned = at.turns && place.pos >= 0;
    float c[8], s[8];
    spin8(turns, a.r.factor, place.pos, c, s);
    while (h < a.q_heads) {
        float v[8], w[8];
        floats(p, v);
        floats(q, w);
        const int now = h;
        h += a.q_slices * a.q_each;
        if (h < a.q_heads) p = load8(x + h * a.qh + at.first), q = load8(x + h * a.qh + at.second);
        if (turned) turn16<HALF>(v, w, c, s);
        store8(out + now * a.oh + at.first, v);
        store8(out + now * a.oh + at.second, w);
    }
}

template <int F, typename T, bool HALF>
__device__ __forceinline__ void keys(const Args &a, int token, int slice, bool is_v) {
    const int lane = threadIdx.x & 63, groups = a.dim / 8, sub = lane / groups, d = (lane % groups) * 8;
    const int half = a.r.rot / 2;
    const bool turned = !is_v && d < a.r.rot, upper = HALF && d >= half;
    const int other = !HALF || !turned ? d : upper ? d - half : d + half;  // the elements that these are paired with
    const T *x = is_v ? (const T *)a.sv + token * a.vt : (const T *)a.sk + token * a.kt;
    const int64_t xh = is_v ? a.vh : a.kh;
    int h = slice * a.k_each + sub;
    if (sub >= a.k_each) h = a.heads;
    Eight<T> p, q;
    if (h < a.heads) {
        p = load8(x + h * xh + d);
        if (HALF) q = load8(x + h * xh + other);
    }
    u32x2 turns[8];
    load_turns(a.r, !turned ? 0 : HALF ? (upper ? d - half : d) : min(d / 2, half - 8), turns);
    const Place place = place_of(a, token);
    if (place.page < 0) return;
    float c[8], s[8];
    if (!is_v) {
        if constexpr (HALF) {
            spin8(turns, a.r.factor, place.pos, c, s);
        } else {  // four pairs: the second four of those loaded at the end of what turns
            const bool late = d / 2 > half - 8;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                cos_sin(angle_of(place.pos, late ? turns[4 + i] : turns[i]), a.r.factor, c[i], s[i]);
        }
    }
    const int ps = 1 << a.page_shift;
    while (h < a.heads) {
        float v[8], w[8];
        floats(p, v);
        if (HALF) floats(q, w);
        const int now = h;
        h += a.k_slices * a.k_each;
        if (h < a.heads) {
            p = load8(x + h * xh + d);
            if (HALF) q = load8(x + h * xh + other);
        }
        if (turned) {
            if constexpr (HALF) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // one of the two of rope::turn, whose products are rounded alike in both
                    const float t = w[i] * s[i];
                    v[i] = upper ? __builtin_fmaf(v[i], c[i], t) : __builtin_fmaf(v[i], c[i], -t);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) turn(v[2 * i], v[2 * i + 1], c[i], s[i]);
            }
        }
        const int64_t head = (int64_t)place.page * a.heads + now;
        uint8_t *dst = (is_v ? a.v : a.k) + ((head * ps + place.slot) * a.dim + d) * kv::kBits<F> / 8;
        const int e = kv::put8<F>(dst, v);
        if constexpr (F != kv::BF16)
            if ((lane & 3) == 0)
                (is_v ? a.vs : a.ks)[(head * (a.dim / 32) + d / 32) * ps + place.slot] = (uint8_t)(e + 127);
    }
}

template <int F, typename T, bool HALF>
__global__ __launch_bounds__(256) void k_append_rope(Args a) {
    const int64_t waves = (int64_t)gridDim.x * 4;
    const int each = a.q_slices + 2 * a.k_slices;
    const int64_t units = (int64_t)a.b.tokens * each;
    for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < units; u += waves) {
        const int token = (int)kv::div_i64(u, each);
        int slice = (int)(u - (int64_t)token * each);
        if (slice < a.q_slices) {
            queries<T, HALF>(a, token, slice);
        } else {
            slice -= a.q_slices;
            keys<F, T, HALF>(a, token, slice < a.k_slices ? slice : slice - a.k_slices, slice >= a.k_slices);
        }
    }
}

template <int F>
hipError_t launch(const Args &a, bool half, int dtype, hipStream_t s) {
    const int64_t blocks = ((int64_t)a.b.tokens * (a.q_slices + 2 * a.k_slices) + 3) / 4;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    if (dtype == QBN_F32) (half ? k_append_rope<F, float, true> : k_append_rope<F, float, false>)<<<grid, 256, 0, s>>>(a);
    else (half ? k_append_rope<F, __bf16, true> : k_append_rope<F, __bf16, false>)<<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append_rope(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, const qbn_rotation &r,
                                 int q_heads, const KvRows &q, const KvRowsOut &out, const KvRows &k, const KvRows &v,
                                 int dtype, hipStream_t s) {
    const int64_t elems = layer * c.pages * c.heads * c.page_size * c.head_dim;
    const int bits = c.format == QBN_KV_BF16 ? 16 : c.format == QBN_MXFP8 ? 8 : 4;
    Args a;
    a.r = {r.turns, r.rot, r.factor};
    a.k = (uint8_t *)c.k + elems * bits / 8;
    a.v = (uint8_t *)c.v + elems * bits / 8;
    a.ks = (uint8_t *)c.k_scales + elems / 32;
    a.vs = (uint8_t *)c.v_scales + elems / 32;
    a.sq = q.p, a.sk = k.p, a.sv = v.p, a.oq = out.p;
    a.qt = q.token_stride, a.qh = q.head_stride, a.ot = out.token_stride, a.oh = out.head_stride;
    a.kt = k.token_stride, a.kh = k.head_stride, a.vt = v.token_stride, a.vh = v.head_stride;
    a.b = {(int)b.seqs, (int)b.tokens, (int)b.row, b.row_stride, b.table, b.lens, b.cu};
    a.heads = c.heads, a.q_heads = q_heads, a.dim = c.head_dim, a.pages = (int)c.pages;
    a.page_shift = __builtin_ctz(c.page_size);
    a.q_each = 64 / (c.head_dim / 16), a.k_each = 64 / (c.head_dim / 8);
    a.keep = out.p == q.p && dtype == QBN_BF16;
    const int qp = (q_heads + a.q_each - 1) / a.q_each, kp = (c.heads + a.k_each - 1) / a.k_each;
    // Waves that run at once (32 on each of 256 compute units) over the tokens' thirds.
    const int64_t spread = (8192 + 3 * b.tokens - 1) / (3 * b.tokens);
    a.q_slices = (int)(spread < qp ? spread : qp);
    a.k_slices = (int)(spread < kp ? spread : kp);
    const bool half = r.layout == QBN_ROPE_HALF;
    if (c.format == QBN_KV_BF16) return launch<kv::BF16>(a, half, dtype, s);
    return c.format == QBN_MXFP8 ? launch<kv::FP8>(a, half, dtype, s) : launch<kv::FP4>(a, half, dtype, s);
}

}  // namespace qbn
