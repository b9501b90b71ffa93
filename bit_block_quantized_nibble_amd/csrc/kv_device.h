// Device-side helpers of the paged key-value cache kernels (gfx950 only).
#pragma once

#include "qbn_device.h"
#include "qbn_kv.h"

namespace qbn {
namespace kv {

enum Fmt { BF16 = 0, FP8 = 1, FP4 = 2 };

constexpr int64_t kGridThreads = (int64_t)1 << 32;  // a launch has fewer threads along x

template <int F>
constexpr int kBits = F == BF16 ? 16 : F == FP8 ? 8 : 4;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_huge_valf();

// A cache of one layer as the kernels see it: bases of that layer's pages.
struct Cache {
    const uint8_t *k, *v, *ks, *vs;
    int heads, page_shift;  // page_size = 1 << page_shift
    int pages;
};

struct Batch {
    int seqs, tokens, row;
    int64_t row_stride;
    const int32_t *table, *lens, *cu;
};

// The scale operand of the converts for E8M0 byte `j` of w. They take its
// exponent bits, so the byte in their place serves for all 256 values (0 stands
// for 2^-127 there, 255 gives NaN; tests pass every byte with every code through
// both attention kernels).
__device__ __forceinline__ float e8m0_operand(uint32_t w, int j = 0) {
    return __uint_as_float(((w >> (8 * j)) & 0xFFu) << 23);
}

// Entry `i` of sequence b's table row, both the same in the whole wave. A scalar
// load: it waits on its own counter, so that looking up the next pages does
// not wait for the loads of K and V that are in flight (vector loads return
// in order). No kernel that calls this writes the table.
__device__ __forceinline__ int table_entry(const Batch &b, int seq, int i) {
    typedef const int32_t __attribute__((address_space(4))) *Const;
    return ((Const)(uintptr_t)b.table)[(int64_t)seq * b.row_stride + i];
}
__device__ __forceinline__ int length_of(const Batch &b, int seq) {
    typedef const int32_t __attribute__((address_space(4))) *Const;
    return ((Const)(uintptr_t)b.lens)[seq];
}
__device__ __forceinline__ int start_of(const Batch &b, int seq) {
    typedef const int32_t __attribute__((address_space(4))) *Const;
    return ((Const)(uintptr_t)b.cu)[seq];
}

// Up to this many sequences the waves of attention find their own by scans of
// all lengths, 64 at a time; of more, a first kernel lists what stands before
// each sequence and they search the list. That kernel costs 3 us, a scan of
// 64 one or two (MXFP8, 32 / 8 heads of 128, 512 tokens, decode: 128 sequences
// 28.4 us by scans, 31.3 by the list, 256 55.5 and 52.8; of 64 tokens, 4096
// sequences 1966 and 375).
constexpr int kScanned = 192;

// How many of list[1 .. n] are <= v: the list ascends, v is the same in the
// whole wave. 64 samples a step: two dependent loads up to 4096. Any content
// gives a result in 0 .. n.
__device__ __forceinline__ int count_upto(const int32_t *list, int n, int v) {
    int at = 0, len = n;
    while (len > 0) {
        const int step = (len + 63) >> 6, lane = threadIdx.x & 63;
        const int k = __popcll(__ballot(list[at + min((lane + 1) * step, len)] <= v));
        if (k == 64) return at + len;
        at += k * step;
        len = min(step, len - k * step) - 1;
    }
    return min(at, n);
}

// Eight consecutive elements (4, 8 or 16 bytes in w) -> bf16 pairs: exact, an
// E2M1 or E4M3FN value having at most 4 significant bits, where the exponent fits
// (E4M3 from scale byte 3 to 246, E2M1 up to 252); beyond, rounded to nearest or infinite.
template <int F>
__device__ __forceinline__ void expand8(const uint32_t *w, float scale, uint32_t (&o)[4]) {
    if constexpr (F == FP4) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 3));
    } else if constexpr (F == FP8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, false));
            o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, true));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = w[i];
    }
}

// W (2, 4 or 8) consecutive elements -> W / 2 bf16 pairs.
template <int F, int W>
__device__ __forceinline__ void expand(const uint32_t *w, float scale, uint32_t (&o)[W / 2]) {
    if constexpr (W == 8) {
        expand8<F>(w, scale, o);
    } else if constexpr (F == FP4) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 0));
        if constexpr (W == 4)
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 1));
    } else if constexpr (F == FP8) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, false));
        if constexpr (W == 4)
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, true));
    } else {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) o[i] = w[i];
    }
}

// Loads of 1, 2, 4, 8 or 16 bytes into 32-bit words (zero-extended).
template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w) {
    if constexpr (BYTES == 1) {
        w[0] = *p;
    } else if constexpr (BYTES == 2) {
        w[0] = *reinterpret_cast<const uint16_t *>(p);
    } else if constexpr (BYTES == 4) {
        w[0] = ld4(p);
    } else if constexpr (BYTES == 8) {
        const u32x2 t = ld8(p);
        w[0] = t.x;
        w[1] = t.y;
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const u32x4 t = ld16(p + 16 * i);
            w[4 * i] = t.x;
            w[4 * i + 1] = t.y;
            w[4 * i + 2] = t.z;
            w[4 * i + 3] = t.w;
        }
    }
}

// Four 16-bit elements of a column from LDS: the 16 lanes of a row of lanes
// address 8 bytes each, four lanes a matrix row of 16 elements, and lane i gets
// column i of the four rows.
__device__ __forceinline__ u32x2 ld_tr16(const uint8_t *lds) {
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s *Lds;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)lds));
}

// The words of eight tokens (row j: W elements as bf16 pairs) -> for each
// element t, the eight tokens' values as four dwords: the A operand of a
// matrix product over tokens.
template <int W>
__device__ __forceinline__ u32x4 column8(const uint32_t (&c)[8][W / 2], int t) {
    const uint32_t sel = (t & 1) ? 0x07060302u : 0x05040100u;
    return u32x4{__builtin_amdgcn_perm(c[1][t / 2], c[0][t / 2], sel),
                 __builtin_amdgcn_perm(c[3][t / 2], c[2][t / 2], sel),
                 __builtin_amdgcn_perm(c[5][t / 2], c[4][t / 2], sel),
                 __builtin_amdgcn_perm(c[7][t / 2], c[6][t / 2], sel)};
}

// Two binary32 values rounded to bfloat16 (nearest even), low half first. As a
// vector conversion this is one instruction; two scalar ones put together are four.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// v_exp_f32: 2^x within one unit in the last place, 2^-inf = 0. Results below
// 2^-126 may come out as 0; a softmax term that small is 2^-126 of the row's
// largest.
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A row's running reference and the unit that its scores are taken in. A
// weight's exponent is fma(x, unit, -ref), ref being a product x unit rounded to
// binary32. What it was rounded by is common to all weights of a row and falls
// out of their quotient, but from 2^31 on it passes 64, and soon all weights
// would be 0 or infinite. There the unit is the power of two below the scale,
// whose products are exact: two scores so far out that differ at all differ by
// 128 or more, and by 64 in that unit, so that only the largest has a weight in
// either. (Rounding all products before the difference, in a branch, cost the
// prefill kernel 1 to 5 %.)
constexpr float kFar = 2147483648.0f;
struct Reference {
    float at, unit;
};
// Raises r to the score `top` if that is larger; the factor of what is summed.
__device__ __forceinline__ float raise(Reference &r, float top, float scale, float far_unit) {
    if (!(top * r.unit > r.at)) return 1.0f;
    const float unit = __builtin_fabsf(top * scale) >= kFar ? far_unit : scale, now = top * unit;
    const float f = unit == r.unit ? exp2_fast(r.at - now) : 0.0f;
    r.at = now;
    r.unit = unit;
    return f;
}
// The reference as a score times the scale.
__device__ __forceinline__ float scaled(const Reference &r, float scale) {
    return r.unit == scale ? r.at : r.at * (scale / r.unit);
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int dpp_i32(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}

// Inclusive sums over the lanes of a wave: shifts within rows of 16, then the
// last lane of row 0 (2) to row 1 (3) and of row 1 to rows 2 and 3.
__device__ __forceinline__ int wave_scan(int v) {
    v += dpp_i32<0x111>(v);
    v += dpp_i32<0x112>(v);
    v += dpp_i32<0x114>(v);
    v += dpp_i32<0x118>(v);
    v += dpp_i32<0x142, 0xA>(v);
    v += dpp_i32<0x143, 0xC>(v);
    return v;
}

// a / b for a >= 0, b > 0, the same in all lanes: the 64-bit division is 130 instructions long.
__device__ __forceinline__ int64_t div_i64(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Sums over the threads of a workgroup of NT threads; every thread gets the
// sum of all threads and the sum of those before it. `lds` holds NT / 64 + 1
// values and may be reused after the call.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *lds, int64_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t t = __shfl_up(s, d);
        if (lane >= d) s += t;
    }
    if (lane == 63) lds[wave] = s;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        if (w < wave) before += lds[w];
        total += lds[w];
    }
    __syncthreads();
    return before + s - v;
}

}  // namespace kv
}  // namespace qbn
