// The experts' layer over 4-bit weights, for a few tokens.
//
//   out_t = sum_j w_tj W2[e] (silu(Wg[e] x_t) * (Wu[e] x_t)),  e = ids[t][j]
// An assignment a = t * top_k + j is a token's j-th expert. Bound by the weights'
// bytes: each of a layer's active experts is read once, for one token or for sixty-four.
// So the weights go from memory to registers with nothing in between, are expanded
// there to bfloat16 (exactly) and multiplied on the matrix cores with the tokens as
// columns, 16 of them at the price of one.
//
// A lane's 16-byte load has 32 consecutive elements of a weight row, one MXFP4
// block or two of NVFP4, and the four 8-element words of it are the operands of four
// product steps: which k a step takes is free as long as the columns agree, and
// they have the same 8 elements each in one 16-byte load of x.
//
// First kernel: h for each assignment, 16 gate rows and the 16 up rows beside them
// per workgroup, k split over its four waves and joined in LDS. h goes on as two
// bfloat16 values, the upper bits and the rest: one alone would round it by 2^-9,
// as much as the output's own rounding. Second kernel: the same products with W2.
// Where assignments are few (64), a workgroup has 16 output rows of all of them and
// adds up the tokens' experts itself; else the assignments' results go to memory
// and a third kernel adds them.
#include <type_traits>

#include "kv_device.h"
#include "moe_launch.h"

namespace qbn {
namespace {

enum Fmt { MX = 0, NV = 1 };

constexpr int kFew = 64;  // assignments that a wave holds, one a lane

struct Args {
    const uint8_t *w13, *s13, *w2, *s2;
    const float *f13, *f2;
    const uint16_t *x;
    const int32_t *ids;
    const float *weights;
    uint16_t *out;
    int64_t xs, os;
    uint16_t *hi, *lo;  // h [assignments][inter], upper bits and rest
    float *y;           // [assignments][hidden]: results of W2, weighted (many assignments)
    const int32_t *list, *start, *active;  // many: assignments by expert, where each expert's start, the experts that have any
    int tokens, top, n, experts, hidden, inter;  // n: assignments
};

// A weight row's 32 elements and their scales.
struct Piece {
    u32x4 codes;
    uint32_t scale;
};
template <int F>
__device__ __forceinline__ Piece load_piece(const uint8_t *w, const uint8_t *s, int block) {
    Piece p;
    p.codes = ld16(w + (int64_t)block * 16);
    if constexpr (F == MX) p.scale = s[block];
    else p.scale = *reinterpret_cast<const uint16_t *>(s + 2 * block);
    return p;
}
// Word i of a piece: eight elements as bfloat16, exact.
template <int F>
__device__ __forceinline__ bf16x8 expand(const Piece &p, int i) {
    const uint32_t c = p.codes[i];
    u32x4 o;
    if constexpr (F == MX) {
        const float s = kv::e8m0_operand(p.scale);
        o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
        o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
        o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
        o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
    } else {
        const float s = e4m3fn_f32(i < 2 ? p.scale & 0xFFu : p.scale >> 8);
        const f32x2 a = e2m1x2_f32<0>(c), b = e2m1x2_f32<1>(c), d = e2m1x2_f32<2>(c), e = e2m1x2_f32<3>(c);
        o = u32x4{kv::pack2(a.x * s, a.y * s), kv::pack2(b.x * s, b.y * s), kv::pack2(d.x * s, d.y * s),
                  kv::pack2(e.x * s, e.y * s)};
    }
    return kv::as_bf16x8(o);
}

// acc[i][m] += rows i of 16 weights x columns of 16 vectors m, over the steps (of 128
// elements) from `first` on, `every` apart. w, s: this lane's row (lane % 16) of each
// tile; x, xl: its column (lane % 16) of each, upper bits and rest.
template <int F, int NT, int MT, bool LO>
__device__ __forceinline__ void products(const uint8_t *const (&w)[NT], const uint8_t *const (&s)[NT],
                                         const uint16_t *const (&x)[MT], const uint16_t *const (&xl)[MT], int k,
                                         int first, int every, f32x4 (&acc)[NT][MT]) {
    const int quarter = (threadIdx.x & 63) >> 4, blocks = k / 32, steps = (blocks + 3) / 4;
    const auto step = [&](int t, auto tail) {
        int block = 4 * t + quarter;
        const bool in = !tail || block < blocks;
        if (tail && !in) block = blocks - 1;
        Piece p[NT];
        bf16x8 v[MT][4], l[MT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) p[i] = load_piece<F>(w[i], s[i], block);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[m][j] = kv::as_bf16x8(ld16(x[m] + block * 32 + 8 * j));
                if (LO) l[m][j] = kv::as_bf16x8(ld16(xl[m] + block * 32 + 8 * j));
            }
        if (tail && !in) {  // beyond the row: nothing, whatever its last block has
#pragma unroll
            for (int i = 0; i < NT; ++i) p[i] = {u32x4{0, 0, 0, 0}, 0};
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[m][j] = l[m][j] = kv::as_bf16x8(u32x4{0, 0, 0, 0});
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const bf16x8 a = expand<F>(p[i], j);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, v[m][j], acc[i][m], 0, 0, 0);
                    if (LO) acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, l[m][j], acc[i][m], 0, 0, 0);
                }
            }
    };
    const int whole = blocks / 4;
    int t = first;
    for (; t < whole; t += every) step(t, std::false_type{});
    if (t < steps) step(t, std::true_type{});
}

// The upper bits of h, and what they leave out, both bfloat16. Cut, not rounded: the
// upper part then is no infinity where h is none.
__device__ __forceinline__ void split(float h, uint16_t &hi, uint16_t &lo) {
    const uint32_t b = __float_as_uint(h);
    if ((b & 0x7F800000u) == 0x7F800000u) {
        hi = bf16_bits_rne(h);
        lo = 0;
    } else {
        hi = (uint16_t)(b >> 16);
        lo = bf16_bits_rne(h - __uint_as_float(b & 0xFFFF0000u));
    }
}

__device__ __forceinline__ float silu(float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + kv::exp2_fast(-kv::kLog2e * g));
}

// Few assignments: the lanes that have lane `slot`'s expert (0 if it is none, or a lane
// before it has it too: then that one does the work).
__device__ __forceinline__ uint64_t same_expert(int id, bool valid, int slot, int &expert) {
    expert = __builtin_amdgcn_readlane(id, slot);
    const uint64_t m = __ballot(valid && id == expert);
    return m && __builtin_ctzll(m) == slot ? m : 0;
}

// The workgroup's expert and its assignments (in LDS or memory). False: nothing to do.
template <bool FEW>
__device__ __forceinline__ bool find(const Args &a, int slot, int *lds, int &expert, int &n, const int *&list) {
    if constexpr (FEW) {
        const int lane = threadIdx.x & 63, id = lane < a.n ? a.ids[lane] : -1;
        const bool valid = (uint32_t)id < (uint32_t)a.experts;
        const uint64_t m = same_expert(id, valid, slot, expert);
        n = __popcll(m);
        if (!m) return false;
        if (threadIdx.x < 64 && (m >> lane & 1)) lds[__popcll(m & (((uint64_t)1 << lane) - 1))] = lane;
        list = lds;
        __syncthreads();
    } else {
        expert = a.active[slot];
        if (expert < 0) return false;
        const int at = a.start[expert];
        n = a.start[expert + 1] - at;
        list = a.list + at;
    }
    return true;
}

constexpr int kWaves = 4;

// Sums of the waves' accumulators, through LDS: value (row, column) of tile (i, m).
template <int NT, int MT>
struct Joined {
    float v[kWaves][NT * MT][256];
};

template <int F, int MT>
__device__ __forceinline__ void gate_up(const Args &a, float *lds, int tile, int expert, int n, const int *list) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quarter = lane >> 4;
    const uint8_t *w[2], *s[2];
    constexpr int SB = F == MX ? 32 : 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = (int64_t)expert * 2 * a.inter + i * a.inter + tile * 16 + row;
        w[i] = a.w13 + r * (a.hidden / 2);
        s[i] = a.s13 + r * (a.hidden / SB);
    }
    const uint16_t *x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = a.x + (int64_t)(list[min(16 * m + row, n - 1)] / a.top) * a.xs;
    f32x4 acc[2][MT] = {};
    products<F, 2, MT, false>(w, s, x, x, a.hidden, wave, kWaves, acc);
    auto *joined = reinterpret_cast<Joined<2, MT> *>(lds);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)  // rows 4 quarter .. + 3 of column `row`
            *reinterpret_cast<f32x4 *>(&joined->v[wave][i * MT + m][row * 16 + quarter * 4]) = acc[i][m];
    __syncthreads();
    const float f = F == NV ? a.f13[expert] : 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int c = 16 * m + threadIdx.x / 16;
        if (c >= n) continue;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int j = 0; j < kWaves; ++j) {
            g += joined->v[j][m][threadIdx.x];
            u += joined->v[j][MT + m][threadIdx.x];
        }
        const int64_t to = (int64_t)list[c] * a.inter + tile * 16 + threadIdx.x % 16;
        split(silu(g * f) * (u * f), a.hi[to], a.lo[to]);
    }
    __syncthreads();
}

template <int F, bool FEW>
__global__ __launch_bounds__(256) void k_gate_up(Args a) {
    __shared__ __attribute__((aligned(16))) float lds[sizeof(Joined<2, 4>) / 4];
    __shared__ int list_lds[64];
    int expert, n;
    const int *list;
    if (!find<FEW>(a, blockIdx.y, list_lds, expert, n, list)) return;
    for (; n > 0; n -= 64, list += 64) {
        if (n <= 16) gate_up<F, 1>(a, lds, blockIdx.x, expert, n, list);
        else if (n <= 32) gate_up<F, 2>(a, lds, blockIdx.x, expert, n, list);
        else gate_up<F, 4>(a, lds, blockIdx.x, expert, min(n, 64), list);
    }
}

template <int F, int MT>
__device__ __forceinline__ void down(const Args &a, float *lds, int tile, int expert, int n, const int *list) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quarter = lane >> 4;
    const uint8_t *w[2], *s[2];
    constexpr int SB = F == MX ? 32 : 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = (int64_t)expert * a.hidden + tile * 32 + i * 16 + row;
        w[i] = a.w2 + r * (a.inter / 2);
        s[i] = a.s2 + r * (a.inter / SB);
    }
    const uint16_t *x[MT], *xl[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t at = (int64_t)list[min(16 * m + row, n - 1)] * a.inter;
        x[m] = a.hi + at, xl[m] = a.lo + at;
    }
    f32x4 acc[2][MT] = {};
    products<F, 2, MT, true>(w, s, x, xl, a.inter, wave, kWaves, acc);
    auto *joined = reinterpret_cast<Joined<2, MT> *>(lds);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            *reinterpret_cast<f32x4 *>(&joined->v[wave][i * MT + m][row * 16 + quarter * 4]) = acc[i][m];
    __syncthreads();
    const float f = F == NV ? a.f2[expert] : 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int c = 16 * m + threadIdx.x / 16;
        if (c >= n) continue;
        const float weight = a.weights[list[c]] * f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v = 0.0f;
#pragma unroll
            for (int j = 0; j < kWaves; ++j) v += joined->v[j][i * MT + m][threadIdx.x];
            a.y[(int64_t)list[c] * a.hidden + tile * 32 + i * 16 + threadIdx.x % 16] = v * weight;
        }
    }
    __syncthreads();
}

template <int F>
__global__ __launch_bounds__(256) void k_down(Args a) {
    __shared__ __attribute__((aligned(16))) float lds[sizeof(Joined<2, 4>) / 4];
    int expert, n;
    const int *list;
    if (!find<false>(a, blockIdx.y, nullptr, expert, n, list)) return;
    for (; n > 0; n -= 64, list += 64) {
        if (n <= 16) down<F, 1>(a, lds, blockIdx.x, expert, n, list);
        else if (n <= 32) down<F, 2>(a, lds, blockIdx.x, expert, n, list);
        else down<F, 4>(a, lds, blockIdx.x, expert, min(n, 64), list);
    }
}

// out = the sum of a token's weighted results, in the order of its experts.
__global__ __launch_bounds__(256) void k_add(Args a) {
    const int64_t pieces = (int64_t)a.tokens * (a.hidden / 8);
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < pieces; p += (int64_t)gridDim.x * 256) {
        const int t = (int)(p / (a.hidden / 8)), i = (int)(p - (int64_t)t * (a.hidden / 8)) * 8;
        float v[8] = {};
        for (int j = 0; j < a.top; ++j) {
            const int at = t * a.top + j;
            if ((uint32_t)a.ids[at] >= (uint32_t)a.experts) continue;
            const float *y = a.y + (int64_t)at * a.hidden + i;
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += y[q];
        }
        *reinterpret_cast<u32x4 *>(a.out + t * a.os + i) =
            u32x4{kv::pack2(v[0], v[1]), kv::pack2(v[2], v[3]), kv::pack2(v[4], v[5]), kv::pack2(v[6], v[7])};
    }
}

// Few assignments: 16 output rows of all of them. An item is an expert and a part of k
// (so that eight waves have work where experts are fewer); its results, weighted, go
// to LDS, one place for each (part, assignment), and are added in a fixed order.
template <int F, int MT>
__device__ __forceinline__ void down_item(const Args &a, float *part, const int *cols, int n, int expert, int first,
                                          int every) {
    const int lane = threadIdx.x & 63, row = lane & 15, quarter = lane >> 4;
    constexpr int SB = F == MX ? 32 : 16;
    const int64_t r = (int64_t)expert * a.hidden + blockIdx.x * 16 + row;
    const uint8_t *w[1] = {a.w2 + r * (a.inter / 2)}, *s[1] = {a.s2 + r * (a.inter / SB)};
    const uint16_t *x[MT], *xl[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t at = (int64_t)cols[min(16 * m + row, n - 1)] * a.inter;
        x[m] = a.hi + at, xl[m] = a.lo + at;
    }
    f32x4 acc[1][MT] = {};
    products<F, 1, MT, true>(w, s, x, xl, a.inter, first, every, acc);
    const float f = F == NV ? a.f2[expert] : 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
        if (16 * m + row < n) {
            const int at = cols[16 * m + row];
            *reinterpret_cast<f32x4 *>(part + at * 16 + quarter * 4) = acc[0][m] * (a.weights[at] * f);
        }
}

constexpr int kDownWaves = 8;

template <int F>
__global__ __launch_bounds__(kDownWaves * 64) void k_down_few(Args a) {
    __shared__ __attribute__((aligned(16))) float part[kDownWaves * kFew * 16];
    __shared__ int cols[kDownWaves][kFew];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int id = lane < a.n ? a.ids[lane] : -1;
    const bool valid = (uint32_t)id < (uint32_t)a.experts;
    int found = 0, expert;
    for (int i = 0; i < a.n; ++i) found += same_expert(id, valid, i, expert) != 0;
    const int parts = found > 0 && found < kDownWaves ? kDownWaves / found : 1;
    for (int item = wave; item < found * parts; item += kDownWaves) {
        const int p = item / found;
        int left = item - p * found, slot = -1;
        uint64_t m = 0;
        for (int i = 0; i < a.n && left >= 0; ++i)
            if ((m = same_expert(id, valid, i, expert)) != 0) --left, slot = i;
        m = same_expert(id, valid, slot, expert);
        if (m >> lane & 1) cols[wave][__popcll(m & (((uint64_t)1 << lane) - 1))] = lane;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int n = __popcll(m);
        if (n <= 16) down_item<F, 1>(a, part + p * a.n * 16, cols[wave], n, expert, p, parts);
        else down_item<F, 4>(a, part + p * a.n * 16, cols[wave], n, expert, p, parts);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * 16; i += kDownWaves * 64) {
        const int t = i / 16, row = i % 16;
        float v = 0.0f;
        for (int j = 0; j < a.top; ++j) {
            const int at = t * a.top + j;
            if ((uint32_t)a.ids[at] >= (uint32_t)a.experts) continue;
            float y = 0.0f;
            for (int p = 0; p < parts; ++p) y += part[(p * a.n + at) * 16 + row];
            v += y;
        }
        a.out[t * a.os + blockIdx.x * 16 + row] = bf16_bits_rne(v);
    }
}

// Many assignments: lists by expert, and the experts that have any (then -1). One
// workgroup. The order within an expert's list is left open: no result depends on it.
constexpr int kListThreads = 1024;
__global__ __launch_bounds__(kListThreads) void k_lists(Args a, int32_t *list, int32_t *start, int32_t *active) {
    __shared__ int count[1024], at[1024];
    __shared__ int64_t scan[kListThreads / 64 + 1];
    const int e = threadIdx.x;
    count[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kListThreads) {
        const uint32_t id = (uint32_t)a.ids[i];
        if (id < (uint32_t)a.experts) atomicAdd(&count[id], 1);
    }
    __syncthreads();
    const int mine = count[e];
    int64_t total;
    // both sums at once: assignments below, experts with any above
    const int64_t before = kv::block_scan<kListThreads>((int64_t)mine | (int64_t)(mine > 0) << 32, scan, total);
    at[e] = (int)(uint32_t)before;
    if (e < a.experts) start[e] = (int)(uint32_t)before;
    if (e == 0) start[a.experts] = (int)(uint32_t)total;
    if (mine > 0) active[before >> 32] = e;
    const int slots = min(a.n, a.experts);
    if (e < slots && e >= (int)(total >> 32)) active[e] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kListThreads) {
        const uint32_t id = (uint32_t)a.ids[i];
        if (id < (uint32_t)a.experts) list[atomicAdd(&at[id], 1)] = i;
    }
}

struct Layout {  // of the workspace, in bytes
    int64_t hi, lo, y, list, start, active, end;
};
Layout layout_of(const qbn_moe_weights &e, int64_t tokens, int top) {
    const int64_t n = (tokens < QBN_MOE_PORTION ? tokens : QBN_MOE_PORTION) * top;
    const bool few = n <= kFew;
    Layout l;
    l.hi = 0;
    l.lo = l.hi + n * e.inter * 2;
    l.y = l.lo + n * e.inter * 2;
    l.list = l.y + (few ? 0 : n * e.hidden * 4);
    l.start = l.list + (few ? 0 : n * 4);
    l.active = l.start + (few ? 0 : (e.experts + 1) * 4);
    l.end = l.active + (few ? 0 : e.experts * 4);
    return l;
}

template <int F>
hipError_t launch(const Args &a, int32_t *list, int32_t *start, int32_t *active, hipStream_t s) {
    if (a.n <= kFew) {
        k_gate_up<F, true><<<dim3(a.inter / 16, a.n), 256, 0, s>>>(a);
        k_down_few<F><<<a.hidden / 16, kDownWaves * 64, 0, s>>>(a);
    } else {
        const int slots = a.n < a.experts ? a.n : a.experts;
        k_lists<<<1, kListThreads, 0, s>>>(a, list, start, active);
        k_gate_up<F, false><<<dim3(a.inter / 16, slots), 256, 0, s>>>(a);
        k_down<F><<<dim3(a.hidden / 32, slots), 256, 0, s>>>(a);
        const int64_t blocks = ((int64_t)a.tokens * (a.hidden / 8) + 255) / 256;
        k_add<<<(unsigned)blocks, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

int64_t moe_experts_workspace(const qbn_moe_weights &e, int64_t tokens, int top_k) {
    return tokens > 0 ? layout_of(e, tokens, top_k).end : 0;
}

hipError_t launch_moe_experts(const qbn_moe_weights &e, int64_t tokens, int top_k, const void *x, int64_t x_stride,
                              const int32_t *ids, const float *weights, void *out, int64_t out_stride, void *ws,
                              hipStream_t s) {
    const Layout l = layout_of(e, tokens, top_k);
    uint8_t *b = (uint8_t *)ws;
    for (int64_t at = 0; at < tokens; at += QBN_MOE_PORTION) {
        Args a;
        a.w13 = (const uint8_t *)e.w13, a.s13 = (const uint8_t *)e.w13_scales, a.f13 = e.w13_scale2;
        a.w2 = (const uint8_t *)e.w2, a.s2 = (const uint8_t *)e.w2_scales, a.f2 = e.w2_scale2;
        a.x = (const uint16_t *)x + at * x_stride, a.xs = x_stride;
        a.out = (uint16_t *)out + at * out_stride, a.os = out_stride;
        a.ids = ids + at * top_k, a.weights = weights + at * top_k;
        a.hi = (uint16_t *)(b + l.hi), a.lo = (uint16_t *)(b + l.lo), a.y = (float *)(b + l.y);
        a.list = (int32_t *)(b + l.list), a.start = (int32_t *)(b + l.start), a.active = (int32_t *)(b + l.active);
        a.tokens = (int)(tokens - at < QBN_MOE_PORTION ? tokens - at : QBN_MOE_PORTION);
        a.top = top_k, a.n = a.tokens * top_k, a.experts = e.experts, a.hidden = e.hidden, a.inter = e.inter;
        int32_t *list = (int32_t *)(b + l.list), *start = (int32_t *)(b + l.start), *active = (int32_t *)(b + l.active);
        const hipError_t st = e.format == QBN_MXFP4 ? launch<MX>(a, list, start, active, s) : launch<NV>(a, list, start, active, s);
        if (st != hipSuccess) return st;
    }
    return hipSuccess;
}

}  // namespace qbn
