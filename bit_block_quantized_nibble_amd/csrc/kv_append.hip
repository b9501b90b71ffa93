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
// is read once and written once. A wave takes 512 elements of one token's K
// or V, eight per lane, so that a lane's load is 16 bytes (bf16) and its
// store 4 (E2M1), 8 (E4M3) or 16; four lanes share a block's maximum by
// quad permutes. The token's sequence is found by one ballot per 64
// sequences instead of a search.
//
// Measured: 16 tokens of 8 heads of 128 to MXFP8 3.3 us; prompts of 9700
// tokens in all, bf16 to MXFP4, 10.4 us.
#include "kv_device.h"
#include "kv_launch.h"

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
__device__ __forceinline__ void load8(const T *p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x4 t = *reinterpret_cast<const f32x4 *>(p + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = t[j];
    }
}
template <>
__device__ __forceinline__ void load8<__bf16>(const __bf16 *p, float (&x)[8]) {
    uint32_t w[4];
    load_words<16>(reinterpret_cast<const uint8_t *>(p), w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

template <int F, typename T>
__global__ __launch_bounds__(256) void k_append(AppendArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * 4;
    const int64_t units = (int64_t)a.b.tokens * 2 * a.chunks;
    const int ps = 1 << a.page_shift, width = a.heads * a.dim;
    for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < units; u += waves) {
        const int token = (int)div_i64(u, 2 * a.chunks), rest = (int)(u - (int64_t)token * 2 * a.chunks);
        const bool is_v = rest >= a.chunks;
        const int e0 = (is_v ? rest - a.chunks : rest) * 512 + lane * 8;
        // the elements do not wait for the token's place
        const int at = min(e0, width - 8), h = at / a.dim, d = at - h * a.dim;
        const T *src = is_v ? (const T *)a.sv + token * a.vt + h * a.vh + d : (const T *)a.sk + token * a.kt + h * a.kh + d;
        float x[8];
        load8<T>(src, x);
        // the sequence: how many of cu[1..seqs] are <= token
        int b = token, left = 1;
        if (a.b.cu) {
            b = 0;
            for (int i = 0; i < a.b.seqs; i += 64) {
                const bool past = i + lane < a.b.seqs && a.b.cu[i + lane + 1] <= token;
                const int n = __popcll(__ballot(past));
                b += n;
                if (n < 64) break;
            }
            if (b >= a.b.seqs) continue;  // cu does not reach this token
            left = a.b.cu[b + 1] - token;
        }
        const int64_t pos = (int64_t)a.b.lens[b] - left;
        if (pos < 0 || (pos >> a.page_shift) >= a.b.row) continue;
        const int page = a.b.table[(int64_t)b * a.b.row_stride + (pos >> a.page_shift)];
        if ((uint32_t)page >= (uint32_t)a.pages || e0 >= width) continue;
        const int slot = (int)pos & (ps - 1);
        const int64_t head = (int64_t)page * a.heads + h;
        uint8_t *dst = (is_v ? a.v : a.k) + ((head * ps + slot) * a.dim + d) * kBits<F> / 8;
        if constexpr (F == BF16) {
            *reinterpret_cast<u32x4 *>(dst) = u32x4{pack2(x[0], x[1]), pack2(x[2], x[3]),
                                                    pack2(x[4], x[5]), pack2(x[6], x[7])};
        } else {
            uint32_t top = 0;  // magnitudes as bit patterns order like the values
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
            top = max(top, dpp_u32<0xB1>(top));  // quad_perm [1,0,3,2]
            top = max(top, dpp_u32<0x4E>(top));  // quad_perm [2,3,0,1]: the four lanes of the block
            constexpr int EMAX = F == FP8 ? 8 : 2;
            int e = (int)(top >> 23) - 127 - EMAX;
            e = e < -127 ? -127 : (e > 127 ? 127 : e);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_ldexpf(x[i], -e);
            if constexpr (F == FP8) {
                typedef short v2s __attribute__((ext_vector_type(2)));
                uint32_t w[2];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __builtin_fminf(__builtin_fmaxf(x[i], -448.0f), 448.0f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    v2s p = {0, 0};
                    p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, x[4 * i], x[4 * i + 1], 1.0f, false);
                    p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, x[4 * i + 2], x[4 * i + 3], 1.0f, true);
                    w[i] = __builtin_bit_cast(uint32_t, p);
                }
                *reinterpret_cast<u32x2 *>(dst) = u32x2{w[0], w[1]};
            } else {
                uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], 1.0f, 0);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], 1.0f, 1);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], 1.0f, 2);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], 1.0f, 3);
                *reinterpret_cast<uint32_t *>(dst) = w;
            }
            if ((lane & 3) == 0) (is_v ? a.vs : a.ks)[(head * (a.dim / 32) + d / 32) * ps + slot] = (uint8_t)(e + 127);
        }
    }
}

template <int F>
hipError_t launch(const AppendArgs &a, int dtype, hipStream_t s) {
    const int64_t units = (int64_t)a.b.tokens * 2 * a.chunks;
    const int64_t blocks = (units + 3) / 4;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    if (dtype == QBN_F32) k_append<F, float><<<grid, 256, 0, s>>>(a);
    else k_append<F, __bf16><<<grid, 256, 0, s>>>(a);
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
