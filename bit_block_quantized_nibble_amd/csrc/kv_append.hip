// Writing new tokens into the paged key-value cache.
//
// Per 32 elements of a token's head, the MX rule of quantize_mx: shared
// exponent e = floor(log2 max|x|) - emax (emax 2 for E2M1, 8 for E4M3),
// clamped to [-127, 127]; elements x * 2^-e (exact) rounded to nearest even
// and saturated by the gfx950 converts (E4M3 is clamped to +-448 first: the
// convert overflows to NaN). bfloat16 caches store the value rounded to
// nearest even.
//
// Bound by latency for a decode step and by HBM for prompts: every element
// is read once and written once. A wave takes 512 elements of K or V of one
// token, or of four where there are many, eight per lane and token, so that a
// lane's load is 16 bytes (bf16) and its store 4 (E2M1), 8 (E4M3) or 16; four lanes share a block's maximum by
// quad permutes. The token's sequence is found by one ballot, of more than 64
// by a search with 64 samples a step.
//
// Measured, 8 heads of 128: 16 tokens to MXFP8 3.4 us; 4789 tokens in four
// prompts, bf16 to bf16, MXFP8 and MXFP4 9.0, 9.5 and 8.9 us; 16384 26.9, 26.7
// and 21.5; 65536 100, 82 and 73 (4.7 to 5.4 TB/s; a copy of 2 GiB reaches
// 4.95). That is 3 us for the chain of launch, cu, length, table and store, and
// then the bytes (MXFP4 1.07 us for 1024 tokens, its floor), so that a few
// thousand tokens take nearly twice their floor.
#include "kv_launch.h"
#include "kv_store.h"

namespace qbn {
namespace {

using namespace kv;

struct AppendArgs {
    uint8_t *k, *v, *ks, *vs;
    const void *sk, *sv;
    int64_t kt, kh, vt, vh;  // strides in elements
    Batch b;
    int heads, dim, page_shift, pages, chunks;
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, u32x4 (&w)[sizeof(T) / 2]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = *reinterpret_cast<const u32x4 *>(p + 4 * i);
}
__device__ __forceinline__ void floats(const u32x4 (&w)[2], float (&x)[8]) {  // binary32
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i / 4][i % 4]);
}
__device__ __forceinline__ void floats(const u32x4 (&w)[1], float (&x)[8]) {  // bfloat16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[0][i] << 16);
        x[2 * i + 1] = __uint_as_float(w[0][i] & 0xFFFF0000u);
    }
}

// A wave takes the same 512 elements of TOK consecutive tokens, whose loads
// and lookups are in flight together.
template <int F, typename T, int TOK>
__global__ __launch_bounds__(256) void k_append(AppendArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * 4;
    const int64_t units = ((int64_t)a.b.tokens + TOK - 1) / TOK * 2 * a.chunks;
    const int ps = 1 << a.page_shift, width = a.heads * a.dim;
    for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < units; u += waves) {
        const int first = (int)div_i64(u, 2 * a.chunks) * TOK, rest = (int)(u - (int64_t)(first / TOK) * 2 * a.chunks);
        const bool is_v = rest >= a.chunks;
        const int e0 = (is_v ? rest - a.chunks : rest) * 512 + lane * 8;
        // the elements do not wait for the tokens' places
        const int at = min(e0, width - 8), h = at / a.dim, d = at - h * a.dim;
        const T *src = is_v ? (const T *)a.sv + h * a.vh + d : (const T *)a.sk + h * a.kh + d;
        u32x4 raw[TOK][sizeof(T) / 2];
#pragma unroll
        for (int t = 0; t < TOK; ++t)
            load8<T>(src + (int64_t)min(first + t, a.b.tokens - 1) * (is_v ? a.vt : a.kt), raw[t]);
        // the sequences: how many of cu[1..seqs] are <= token
        int b[TOK], left[TOK], page[TOK], slot[TOK];
        bool has[TOK];  // a row before cu[0] has no sequence, nor one that cu does not reach
#pragma unroll
        for (int t = 0; t < TOK; ++t) b[t] = first + t, left[t] = 1, has[t] = true;
        if (a.b.cu) {
            if (a.b.seqs <= 64) {
                const int end = lane < a.b.seqs ? a.b.cu[lane + 1] : 0x7FFFFFFF;
#pragma unroll
                for (int t = 0; t < TOK; ++t) b[t] = __popcll(__ballot(end <= first + t));
            } else {
                b[0] = count_upto(a.b.cu, a.b.seqs, first);
#pragma unroll
                for (int t = 1; t < TOK; ++t) {
                    const bool same = b[t - 1] < a.b.seqs && first + t < start_of(a.b, min(b[t - 1], a.b.seqs - 1) + 1);
                    b[t] = same ? b[t - 1] : count_upto(a.b.cu, a.b.seqs, first + t);
                }
            }
#pragma unroll
            for (int t = 0; t < TOK; ++t) {
                const int seq = min(b[t], a.b.seqs - 1);
                has[t] = start_of(a.b, seq) <= first + t;
                left[t] = start_of(a.b, seq + 1) - (first + t);
            }
        }
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            const bool known = has[t] && first + t < a.b.tokens && b[t] < a.b.seqs;
            const int seq = min(b[t], a.b.seqs - 1);
            const int64_t pos = (int64_t)length_of(a.b, seq) - left[t];
            const bool in = known && pos >= 0 && (pos >> a.page_shift) < a.b.row;
            page[t] = table_entry(a.b, seq, in ? (int)(pos >> a.page_shift) : 0);
            if (!in) page[t] = -1;
            slot[t] = (int)pos & (ps - 1);
        }
        int exps[TOK] = {};
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            if ((uint32_t)page[t] >= (uint32_t)a.pages || e0 >= width) continue;
            float x[8];
            floats(raw[t], x);
            const int64_t head = (int64_t)page[t] * a.heads + h;
            uint8_t *dst = (is_v ? a.v : a.k) + ((head * ps + slot[t]) * a.dim + d) * kBits<F> / 8;
            exps[t] = put8<F>(dst, x);
        }
        if constexpr (F != BF16) {
            // a lane of the block's four per token: their scales lie side by side
#pragma unroll
            for (int t0 = 0; t0 < TOK; t0 += 4) {
                int e = exps[t0], p = page[t0], i = slot[t0];
#pragma unroll
                for (int t = t0 + 1; t < TOK && t < t0 + 4; ++t)
                    if ((lane & 3) == t - t0) e = exps[t], p = page[t], i = slot[t];
                if ((lane & 3) < TOK && (uint32_t)p < (uint32_t)a.pages && e0 < width)
                    (is_v ? a.vs : a.ks)[(((int64_t)p * a.heads + h) * (a.dim / 32) + d / 32) * ps + i] = (uint8_t)(e + 127);
            }
        }
    }
}

template <int F>
hipError_t launch(const AppendArgs &a, int dtype, hipStream_t s) {
    // Four tokens a wave where the elements have scales and there are more waves
    // than run at once (32 on each of 256 compute units): the scales' stores
    // are then a quarter as many. 8 heads of 128 to MXFP4, one and four: 1024
    // tokens 3.9 and 4.3 us, 2048 5.6 and 5.6, 4789 9.4 and 8.3, 65536 101 and
    // 70; bf16 8.8 and 8.6 at 4789, 101 and 104 at 65536.
    constexpr int MOST = F == BF16 ? 1 : 4;
    const int each = (int64_t)a.b.tokens * 2 * a.chunks > 8192 ? MOST : 1;
    const int64_t units = ((int64_t)a.b.tokens + each - 1) / each * 2 * a.chunks;
    const int64_t blocks = (units + 3) / 4;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    if (dtype == QBN_F32) (each == 1 ? k_append<F, float, 1> : k_append<F, float, MOST>)<<<grid, 256, 0, s>>>(a);
    else (each == 1 ? k_append<F, __bf16, 1> : k_append<F, __bf16, MOST>)<<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const qbn_kv_cache &c, int64_t layer, const qbn_kv_batch &b, const KvRows &k,
                            const KvRows &v, int dtype, hipStream_t s) {
    const int64_t elems = layer * c.pages * c.heads * c.page_size * c.head_dim;
    const int bits = c.format == QBN_KV_BF16 ? 16 : c.format == QBN_MXFP8 ? 8 : 4;
    AppendArgs a;
    a.k = (uint8_t *)c.k + elems * bits / 8;
    a.v = (uint8_t *)c.v + elems * bits / 8;
    a.ks = (uint8_t *)c.k_scales + elems / 32;
    a.vs = (uint8_t *)c.v_scales + elems / 32;
    a.sk = k.p, a.sv = v.p;
    a.kt = k.token_stride, a.kh = k.head_stride, a.vt = v.token_stride, a.vh = v.head_stride;
    a.b = {(int)b.seqs, (int)b.tokens, (int)b.row, b.row_stride, b.table, b.lens, b.cu};
    a.heads = c.heads, a.dim = c.head_dim, a.pages = (int)c.pages;
    a.page_shift = __builtin_ctz(c.page_size);
    a.chunks = (c.heads * c.head_dim + 511) / 512;
    if (c.format == QBN_KV_BF16) return launch<BF16>(a, dtype, s);
    return c.format == QBN_MXFP8 ? launch<FP8>(a, dtype, s) : launch<FP4>(a, dtype, s);
}

}  // namespace qbn
